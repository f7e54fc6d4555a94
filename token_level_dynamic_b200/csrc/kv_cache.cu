// kv_cache.cu -- wide_kv_append and wide_kv_read: rows of keys and values
// into the cache, in bf16 or in 8 bits with a power-of-two scale per 32
// elements, and back.
//
// Each row is read and written once; both are bound by memory (256 B in and
// 132 B out per row of an 8-bit cache), at a decoding step's few rows by the
// launch.  16 lanes hold one row, 8 elements each, so a scale block is 4
// neighbouring lanes: its largest magnitude takes two shuffles and a row is
// one coalesced 256-byte access.  A thread has several rows in flight.  With a rotation, K's partners within a pair
// are in the same lane (interleaved) or, in the half layout, rot_dim / 16
// lanes away (rot_dim a multiple of 16), so the exchange is a shuffle too and
// K goes from its bf16 row to its code with one rounding.  A CTA takes whole
// tokens of one sequence: their angles are computed once for all heads, and
// the sequence's length and place are looked up once.
#include "host.h"
#include "kv.cuh"
#include "rope.cuh"

namespace wide {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsAtOnce = kThreads / 16;

struct KvArgs {
    const __nv_bfloat16 *k, *v;       // append: source rows
    __nv_bfloat16 *k_out, *v_out;     // read: destination rows
    void *kc, *vc;
    uint8_t *ks, *vs;
    const int32_t *start, *count, *pos;
    int64_t tokens, seq_len, cap;     // tokens <= 2^28
    int64_t kt, kh, vt, vh;           // row strides
    int n_kv, tok_per_cta, chunks;    // chunks of a sequence
    int pairs;                        // 0: no rotation
    int inter;
    int32_t *status;
};

// The tokens of a CTA: up to tok_per_cta of one sequence.
struct KvChunk {
    int64_t t0, row0;                 // first token; its cache row for head 0 (heads cap rows apart)
    int nt, start;                    // tokens in range; the first one's position in the cache
};
__device__ __forceinline__ KvChunk kv_chunk(const KvArgs &a)
{
    const uint32_t s = blockIdx.x / (uint32_t)a.chunks;
    const int i0 = (int)(blockIdx.x - s * (uint32_t)a.chunks) * a.tok_per_cta;
    const int n = a.count ? a.count[s] : (int)a.seq_len;
    const int64_t start = a.start ? a.start[s] : 0;
    KvChunk c = {};
    if (n < 0 || n > a.seq_len) {
        if (threadIdx.x == 0)
            set_status(a.status, WIDE_DEV_BAD_RANGE);
        return c;
    }
    // tokens i0 .. i1 - 1, of which lo .. hi - 1 have a place in the cache
    const int64_t i1 = min(i0 + a.tok_per_cta, n), lo = max((int64_t)i0, -start), hi = min(i1, a.cap - start);
    if (i1 > i0 && (lo > i0 || hi < i1) && threadIdx.x == 0)
        set_status(a.status, WIDE_DEV_BAD_RANGE);
    c.nt = (int)max(hi - lo, (int64_t)0);
    c.t0 = s * a.seq_len + lo;
    c.start = (int)(start + lo);
    c.row0 = (int64_t)s * a.n_kv * a.cap + c.start;
    return c;
}

// One row's 8 elements of this lane into the cache; row < 0: no row (the lane
// still takes part in its warp's shuffles).
template <int KIND>
__device__ __forceinline__ void kv_store_row(void *codes, uint8_t *scales, int64_t row, int l,
                                             const float (&x)[8], const uint4 raw, bool rotated)
{
    if constexpr (KIND == WIDE_KV_BF16) {
        if (row < 0)
            return;
        uint4 o = raw;
        if (rotated) {
            uint32_t *w = reinterpret_cast<uint32_t *>(&o);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&p);
            }
        }
        reinterpret_cast<uint4 *>(codes)[row * (kKvHD / 8) + l] = o;
    } else {
        uint32_t top = 0;             // magnitudes order like their bits, NaN above infinity
        if (rotated) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
        } else {
            const uint32_t m = __vmaxu2(__vmaxu2(raw.x & 0x7fff7fffu, raw.y & 0x7fff7fffu),
                                        __vmaxu2(raw.z & 0x7fff7fffu, raw.w & 0x7fff7fffu));
            top = max(m & 0xffff0000u, m << 16);
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        if (row < 0)
            return;
        const uint32_t b = kv_scale_byte<KIND>(top);
        reinterpret_cast<uint2 *>(codes)[row * (kKvHD / 8) + l] = kv_encode8<KIND>(x, b);
        if ((l & 3) == 0)
            scales[row * (kKvHD / kKvBlock) + (l >> 2)] = (uint8_t)b;
    }
}

// Rows that a thread of the writer has in flight (the reader: twice as many).
constexpr int kDeep = 2;

// A thread's rows, 16 apart in the CTA's nt x n_kv (heads fastest), without a
// division per row.
struct KvWalk {
    int i, j;                         // token and head
    int hop_i, hop_j, n_kv;
    __device__ __forceinline__ KvWalk(int r, int n) : n_kv(n)
    {
        i = r / n;
        j = r - i * n;
        hop_i = kRowsAtOnce / n;
        hop_j = kRowsAtOnce - hop_i * n;
    }
    __device__ __forceinline__ void next()
    {
        i += hop_i;
        j += hop_j;
        if (j >= n_kv) {
            j -= n_kv;
            ++i;
        }
    }
};

template <int KIND, bool ROPE>
__global__ void __launch_bounds__(kThreads)
    kv_append_rows(const __grid_constant__ RopeTable tab, const KvArgs a)
{
    extern __shared__ float2 cs[];                    // [tok_per_cta][pairs]
    const KvChunk c = kv_chunk(a);
    if constexpr (ROPE) {
        for (int i = threadIdx.x; i < c.nt * a.pairs; i += kThreads) {
            const int t = i / a.pairs, p = i - t * a.pairs;
            cs[i] = rope_cos_sin(tab.turns[p], a.pos ? a.pos[c.t0 + t] : c.start + t, tab.amplitude);
        }
        __syncthreads();
    }
    const int l = threadIdx.x & 15;
    const int rows = c.nt * a.n_kv;
    KvWalk at((int)threadIdx.x >> 4, a.n_kv);
    for (int r0 = 0; r0 < rows; r0 += kDeep * kRowsAtOnce) {  // whole warps stay together
        int64_t row[kDeep];
        int tl[kDeep];
        uint4 kw[kDeep], vw[kDeep];
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
            const bool in = at.i < c.nt;
            row[u] = in ? c.row0 + at.j * a.cap + at.i : -1;
            tl[u] = in ? at.i : 0;
            kw[u] = vw[u] = make_uint4(0u, 0u, 0u, 0u);
            if (in) {
                const int64_t t = c.t0 + at.i;
                kw[u] = *reinterpret_cast<const uint4 *>(a.k + t * a.kt + at.j * a.kh + l * 8);
                vw[u] = *reinterpret_cast<const uint4 *>(a.v + t * a.vt + at.j * a.vh + l * 8);
            }
            at.next();
        }
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
            float x[8];
            bf16x8_to_f32(kw[u], x);
            if constexpr (ROPE) {
                const float2 *w = cs + tl[u] * a.pairs;
                if (a.inter) {
                    const int p0 = l * 4;             // this lane's first pair
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (p0 + i < a.pairs)
                            rope_pair(x[2 * i], x[2 * i + 1], w[p0 + i]);
                } else {
                    const int half = a.pairs / 8;     // lanes of the a elements
                    const bool is_a = l < half, is_b = !is_a && l < 2 * half;
                    const int from = (threadIdx.x & 16) + (is_a ? l + half : is_b ? l - half : l);
                    const float2 *wl = w + (is_b ? l - half : is_a ? l : 0) * 8;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float y = __shfl_sync(0xffffffffu, x[e], from);
                        if (is_a)
                            rope_pair(x[e], y, wl[e]);
                        else if (is_b)
                            rope_pair(y, x[e], wl[e]);
                    }
                }
            }
            kv_store_row<KIND>(a.kc, a.ks, row[u], l, x, kw[u], ROPE);
            bf16x8_to_f32(vw[u], x);
            kv_store_row<KIND>(a.vc, a.vs, row[u], l, x, vw[u], false);
        }
    }
}

// A lane's 8 elements of a row as they are in the cache.
template <int KIND> struct KvRaw {
    uint4 w;                                          // bf16, or codes in x and y
    uint32_t scale;
    __device__ __forceinline__ void load(const void *codes, const uint8_t *scales, int64_t row, int l)
    {
        if constexpr (KIND == WIDE_KV_BF16) {
            w = reinterpret_cast<const uint4 *>(codes)[row * (kKvHD / 8) + l];
        } else {
            const uint2 c = reinterpret_cast<const uint2 *>(codes)[row * (kKvHD / 8) + l];
            w.x = c.x;
            w.y = c.y;
            scale = scales[row * (kKvHD / kKvBlock) + (l >> 2)];
        }
    }
    __device__ __forceinline__ uint4 values() const
    {
        if constexpr (KIND == WIDE_KV_BF16) {
            return w;
        } else {
            const float s = kv_scale(scale);
            float f[4], g[4];
            kv_decode4<KIND>(w.x, s, f);
            kv_decode4<KIND>(w.y, s, g);
            uint4 o;
            uint32_t *q = reinterpret_cast<uint32_t *>(&o);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                const __nv_bfloat162 r = __floats2bfloat162_rn(g[2 * i], g[2 * i + 1]);
                q[i] = *reinterpret_cast<const uint32_t *>(&p);
                q[2 + i] = *reinterpret_cast<const uint32_t *>(&r);
            }
            return o;
        }
    }
};

template <int KIND> __global__ void __launch_bounds__(kThreads) kv_read_rows(const KvArgs a)
{
    constexpr int kReadDeep = 2 * kDeep;
    const KvChunk c = kv_chunk(a);
    const int l = threadIdx.x & 15;
    KvWalk at((int)threadIdx.x >> 4, a.n_kv);
    while (at.i < c.nt) {
        KvRaw<KIND> kw[kReadDeep], vw[kReadDeep];
        const KvWalk from = at;
#pragma unroll
        for (int u = 0; u < kReadDeep; ++u) {
            if (at.i < c.nt) {
                const int64_t row = c.row0 + at.j * a.cap + at.i;
                kw[u].load(a.kc, a.ks, row, l);
                vw[u].load(a.vc, a.vs, row, l);
            }
            at.next();
        }
        KvWalk to = from;
#pragma unroll
        for (int u = 0; u < kReadDeep; ++u) {
            if (to.i < c.nt) {
                const int64_t t = c.t0 + to.i;
                *reinterpret_cast<uint4 *>(a.k_out + t * a.kt + to.j * a.kh + l * 8) = kw[u].values();
                *reinterpret_cast<uint4 *>(a.v_out + t * a.vt + to.j * a.vh + l * 8) = vw[u].values();
            }
            to.next();
        }
    }
}

// Tokens per CTA: `deep` passes of its 16 row slots, one token at least, while
// the grid still covers the GPU.
void kv_grid(KvArgs *a, int64_t n_seq, int deep)
{
    int64_t n = deep * kRowsAtOnce / a->n_kv;
    n = n < 1 ? 1 : n > a->seq_len ? a->seq_len : n;
    while (n > 1 && n_seq * ((a->seq_len + n - 1) / n) < 296)
        n = (n + 1) / 2;
    a->tok_per_cta = (int)n;
    a->chunks = (int)((a->seq_len + n - 1) / n);
}

}  // namespace

// Argument checks shared by the cache's entry points.
int kv_cache_check(const wide_kv_cache *c)
{
    if (!c || c->n_seq < 0 || c->cap <= 0 || c->n_kv <= 0 || c->head_dim <= 0 ||
        c->kind < WIDE_KV_BF16 || c->kind > WIDE_KV_I8)
        return WIDE_EINVAL;
    if (c->n_seq > 0 && (!c->k || !c->v || (c->kind != WIDE_KV_BF16 && (!c->k_scale || !c->v_scale))))
        return WIDE_EINVAL;
    if (c->head_dim != kKvHD || c->n_seq > (1 << 24) || c->n_kv > 1024 || c->cap > (1 << 30) ||
        !aligned16(c->k) || !aligned16(c->v) ||
        (c->kind != WIDE_KV_BF16 && ((reinterpret_cast<uintptr_t>(c->k_scale) & 3u) ||
                                     (reinterpret_cast<uintptr_t>(c->v_scale) & 3u))))
        return WIDE_EUNSUPPORTED;
    return WIDE_OK;
}

namespace {

int kv_args(KvArgs *a, const wide_kv_cache *cache, const int32_t *d_start, const int32_t *d_count,
            const wide_kv_rows *rows, const void *k, const void *v, bool out)
{
    if (!rows || rows->seq_len < 0)
        return WIDE_EINVAL;
    if (int rc = kv_cache_check(cache))
        return rc;
    const wide_kv_rows &r = *rows;
    if (r.k_token_stride < 0 || r.k_head_stride < 0 || r.v_token_stride < 0 || r.v_head_stride < 0)
        return WIDE_EINVAL;
    if (r.seq_len > (1 << 24) || cache->n_seq * r.seq_len > (1 << 28))
        return WIDE_EUNSUPPORTED;
    a->tokens = cache->n_seq * r.seq_len;
    if (a->tokens == 0)
        return WIDE_OK;
    if (!k || !v)
        return WIDE_EINVAL;
    const bool many_t = a->tokens > 1, many_h = cache->n_kv > 1;
    if (out &&
        (!rows_apart(a->tokens, r.k_token_stride, cache->n_kv, r.k_head_stride, kKvHD) ||
         !rows_apart(a->tokens, r.v_token_stride, cache->n_kv, r.v_head_stride, kKvHD)))
        return WIDE_EINVAL;
    a->kt = many_t ? r.k_token_stride : 0;
    a->vt = many_t ? r.v_token_stride : 0;
    a->kh = many_h ? r.k_head_stride : 0;
    a->vh = many_h ? r.v_head_stride : 0;
    if (!aligned16(k) || !aligned16(v) || a->kt % 8 || a->vt % 8 || a->kh % 8 || a->vh % 8 ||
        (reinterpret_cast<uintptr_t>(d_start) & 3u) || (reinterpret_cast<uintptr_t>(d_count) & 3u))
        return WIDE_EUNSUPPORTED;
    a->kc = cache->k;
    a->vc = cache->v;
    a->ks = cache->k_scale;
    a->vs = cache->v_scale;
    a->start = d_start;
    a->count = d_count;
    a->seq_len = r.seq_len;
    a->cap = cache->cap;
    a->n_kv = cache->n_kv;
    kv_grid(a, cache->n_seq, out ? 2 * kDeep : kDeep);
    a->status = status_ptr();
    return WIDE_OK;
}

}  // namespace
}  // namespace wide

using namespace wide;

extern "C" {

int wide_kv_append(const void *d_k, const void *d_v, const wide_kv_cache *cache,
                   const int32_t *d_start, const int32_t *d_count, const int32_t *d_positions,
                   const wide_kv_rows *rows, const wide_rope_config *rope, void *stream)
{
    RopeTable tab = {};
    if (rope && (!rope_table(rope, &tab) || rope->rot_dim > kKvHD))
        return WIDE_EINVAL;
    KvArgs a = {};
    if (int rc = kv_args(&a, cache, d_start, d_count, rows, d_k, d_v, false))
        return rc;
    if (rope && rope->layout == WIDE_ROPE_HALF && rope->rot_dim % 16)
        return WIDE_EUNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(d_positions) & 3u)
        return WIDE_EUNSUPPORTED;
    if (a.tokens == 0)
        return WIDE_OK;
    a.k = static_cast<const __nv_bfloat16 *>(d_k);
    a.v = static_cast<const __nv_bfloat16 *>(d_v);
    a.pos = d_positions;
    a.pairs = rope ? rope->rot_dim / 2 : 0;
    a.inter = rope && rope->layout == WIDE_ROPE_INTERLEAVED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)(cache->n_seq * a.chunks);
    const size_t smem = (size_t)a.tok_per_cta * a.pairs * sizeof(float2);
    LaunchScope scope(KID_KV_APPEND, s);
    const bool r = a.pairs != 0;
    if (cache->kind == WIDE_KV_BF16)
        (r ? kv_append_rows<WIDE_KV_BF16, true> : kv_append_rows<WIDE_KV_BF16, false>)<<<grid, kThreads, smem, s>>>(tab, a);
    else if (cache->kind == WIDE_KV_E4M3)
        (r ? kv_append_rows<WIDE_KV_E4M3, true> : kv_append_rows<WIDE_KV_E4M3, false>)<<<grid, kThreads, smem, s>>>(tab, a);
    else
        (r ? kv_append_rows<WIDE_KV_I8, true> : kv_append_rows<WIDE_KV_I8, false>)<<<grid, kThreads, smem, s>>>(tab, a);
    return launch_status();
}

int wide_kv_read(void *d_k, void *d_v, const wide_kv_cache *cache, const int32_t *d_start,
                 const int32_t *d_count, const wide_kv_rows *rows, void *stream)
{
    KvArgs a = {};
    if (int rc = kv_args(&a, cache, d_start, d_count, rows, d_k, d_v, true))
        return rc;
    if (a.tokens == 0)
        return WIDE_OK;
    a.k_out = static_cast<__nv_bfloat16 *>(d_k);
    a.v_out = static_cast<__nv_bfloat16 *>(d_v);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)(cache->n_seq * a.chunks);
    LaunchScope scope(KID_KV_READ, s);
    if (cache->kind == WIDE_KV_BF16)
        kv_read_rows<WIDE_KV_BF16><<<grid, kThreads, 0, s>>>(a);
    else if (cache->kind == WIDE_KV_E4M3)
        kv_read_rows<WIDE_KV_E4M3><<<grid, kThreads, 0, s>>>(a);
    else
        kv_read_rows<WIDE_KV_I8><<<grid, kThreads, 0, s>>>(a);
    return launch_status();
}

}  // extern "C"
