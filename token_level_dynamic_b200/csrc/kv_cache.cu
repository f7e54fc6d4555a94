// kv_cache.cu -- wide_kv_append and wide_kv_read: rows of keys and values
// into the cache, in bf16 or in 8 bits with a power-of-two scale per 32
// elements, and back.
//
// Each row is read and written once; both are bound by memory (256 B in and
// 132 B out per row of an 8-bit cache), at a decoding step's few rows by the
// launch.  16 lanes hold one row, 8 elements each, so a scale block is 4
// neighbouring lanes: its largest magnitude takes two shuffles and a row is
// one coalesced 256-byte access.  With a rotation, K's partners within a pair
// are in the same lane (interleaved) or, in the half layout, rot_dim / 16
// lanes away (rot_dim a multiple of 16), so the exchange is a shuffle too and
// K goes from its bf16 row to its code with one rounding.  A CTA takes whole
// tokens: their angles are computed once for all heads.
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
    int n_kv, tok_per_cta;
    int pairs;                        // 0: no rotation
    int inter;
    int32_t *status;
};

// The cache row of token t (index of its 128-element row for head 0, rows of
// the next head cap further), or -1: nothing to do.
__device__ __forceinline__ int64_t kv_slot(const KvArgs &a, int64_t t, int64_t &p)
{
    const int64_t s = (uint32_t)t / (uint32_t)a.seq_len, i = t - s * a.seq_len;
    const int64_t n = a.count ? a.count[s] : a.seq_len;
    if (n < 0 || n > a.seq_len) {
        set_status(a.status, WIDE_DEV_BAD_RANGE);
        return -1;
    }
    if (i >= n)
        return -1;
    p = (a.start ? (int64_t)a.start[s] : 0) + i;
    if (p < 0 || p >= a.cap) {
        set_status(a.status, WIDE_DEV_BAD_RANGE);
        return -1;
    }
    return s * a.n_kv * a.cap + p;
}

template <int KIND>
__device__ __forceinline__ void kv_store_row(void *codes, uint8_t *scales, int64_t row, int l,
                                             const float (&x)[8], const uint4 raw, bool rotated)
{
    // row < 0: no row; the lane still takes part in its warp's shuffles
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
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t b = kv_scale_byte<KIND>(top);
        const int base = threadIdx.x & 16;
        uint32_t w = __shfl_sync(0xffffffffu, b, base);
        w |= __shfl_sync(0xffffffffu, b, base + 4) << 8;
        w |= __shfl_sync(0xffffffffu, b, base + 8) << 16;
        w |= __shfl_sync(0xffffffffu, b, base + 12) << 24;
        if (row < 0)
            return;
        reinterpret_cast<uint2 *>(codes)[row * (kKvHD / 8) + l] = kv_encode8<KIND>(x, b);
        if (l == 0)
            reinterpret_cast<uint32_t *>(scales)[row] = w;
    }
}

template <int KIND>
__global__ void __launch_bounds__(kThreads)
    kv_append_rows(const __grid_constant__ RopeTable tab, const KvArgs a)
{
    extern __shared__ float2 cs[];                    // [tok_per_cta][pairs]
    const int64_t t0 = (int64_t)blockIdx.x * a.tok_per_cta;
    const int nt = (int)min((int64_t)a.tok_per_cta, a.tokens - t0);
    if (a.pairs) {
        for (int i = threadIdx.x; i < nt * a.pairs; i += kThreads) {
            const int t = i / a.pairs, p = i - t * a.pairs;
            int32_t at;
            if (a.pos) {
                at = a.pos[t0 + t];
            } else {
                const int64_t s = (uint32_t)(t0 + t) / (uint32_t)a.seq_len;
                at = (a.start ? a.start[s] : 0) + (int32_t)(t0 + t - s * a.seq_len);
            }
            cs[i] = rope_cos_sin(tab.turns[p], at, tab.amplitude);
        }
        __syncthreads();
    }
    const int l = threadIdx.x & 15;
    const int rows = nt * a.n_kv;
    for (int r0 = 0; r0 < rows; r0 += kRowsAtOnce) {  // whole warps stay together
        const int r = r0 + ((int)threadIdx.x >> 4);
        const int tl = min(r, rows - 1) / a.n_kv, j = min(r, rows - 1) - tl * a.n_kv;
        const int64_t t = t0 + tl;
        int64_t p = 0;
        const int64_t slot = r < rows ? kv_slot(a, t, p) : -1;
        const int64_t row = slot < 0 ? -1 : slot + j * a.cap;
        uint4 kw = make_uint4(0u, 0u, 0u, 0u), vw = kw;
        if (row >= 0) {
            kw = *reinterpret_cast<const uint4 *>(a.k + t * a.kt + j * a.kh + l * 8);
            vw = *reinterpret_cast<const uint4 *>(a.v + t * a.vt + j * a.vh + l * 8);
        }
        float x[8];
        bf16x8_to_f32(kw, x);
        if (a.pairs) {
            const float2 *w = cs + tl * a.pairs;
            if (a.inter) {
                const int p0 = l * 4;                 // this lane's first pair
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (p0 + i < a.pairs)
                        rope_pair(x[2 * i], x[2 * i + 1], w[p0 + i]);
            } else {
                const int half = a.pairs / 8;         // lanes of the a elements
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
        kv_store_row<KIND>(a.kc, a.ks, row, l, x, kw, a.pairs != 0);
        bf16x8_to_f32(vw, x);
        kv_store_row<KIND>(a.vc, a.vs, row, l, x, vw, false);
    }
}

template <int KIND>
__device__ __forceinline__ uint4 kv_load8(const void *codes, const uint8_t *scales, int64_t row,
                                          int l)
{
    if constexpr (KIND == WIDE_KV_BF16) {
        return reinterpret_cast<const uint4 *>(codes)[row * (kKvHD / 8) + l];
    } else {
        const uint2 c = reinterpret_cast<const uint2 *>(codes)[row * (kKvHD / 8) + l];
        const float s = kv_scale(scales[row * (kKvHD / kKvBlock) + (l >> 2)]);
        float f[4], g[4];
        kv_decode4<KIND>(c.x, s, f);
        kv_decode4<KIND>(c.y, s, g);
        uint4 o;
        uint32_t *w = reinterpret_cast<uint32_t *>(&o);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            const __nv_bfloat162 q = __floats2bfloat162_rn(g[2 * i], g[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&p);
            w[2 + i] = *reinterpret_cast<const uint32_t *>(&q);
        }
        return o;
    }
}

template <int KIND> __global__ void __launch_bounds__(kThreads) kv_read_rows(const KvArgs a)
{
    const int64_t t0 = (int64_t)blockIdx.x * a.tok_per_cta;
    const int nt = (int)min((int64_t)a.tok_per_cta, a.tokens - t0);
    const int l = threadIdx.x & 15;
    const int rows = nt * a.n_kv;
    for (int r = (int)threadIdx.x >> 4; r < rows; r += kRowsAtOnce) {
        const int tl = r / a.n_kv, j = r - tl * a.n_kv;
        int64_t p;
        const int64_t slot = kv_slot(a, t0 + tl, p);
        if (slot < 0)
            continue;
        const int64_t row = slot + j * a.cap, t = t0 + tl;
        const uint4 kw = kv_load8<KIND>(a.kc, a.ks, row, l);
        const uint4 vw = kv_load8<KIND>(a.vc, a.vs, row, l);
        *reinterpret_cast<uint4 *>(a.k_out + t * a.kt + j * a.kh + l * 8) = kw;
        *reinterpret_cast<uint4 *>(a.v_out + t * a.vt + j * a.vh + l * 8) = vw;
    }
}

// Tokens per CTA: about two passes of its 16 row slots, one token at least,
// while the grid still covers the GPU.
int kv_tokens_per_cta(int64_t tokens, int n_kv)
{
    int64_t n = 2 * kRowsAtOnce / n_kv;
    if (n < 1)
        n = 1;
    while (n > 1 && (tokens + n - 1) / n < 296)
        n = (n + 1) / 2;
    return (int)n;
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
    a->tok_per_cta = kv_tokens_per_cta(a->tokens, a->n_kv);
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
    const unsigned grid = (unsigned)((a.tokens + a.tok_per_cta - 1) / a.tok_per_cta);
    const size_t smem = (size_t)a.tok_per_cta * a.pairs * sizeof(float2);
    LaunchScope scope(KID_KV_APPEND, s);
    if (cache->kind == WIDE_KV_BF16)
        kv_append_rows<WIDE_KV_BF16><<<grid, kThreads, smem, s>>>(tab, a);
    else if (cache->kind == WIDE_KV_E4M3)
        kv_append_rows<WIDE_KV_E4M3><<<grid, kThreads, smem, s>>>(tab, a);
    else
        kv_append_rows<WIDE_KV_I8><<<grid, kThreads, smem, s>>>(tab, a);
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
    const unsigned grid = (unsigned)((a.tokens + a.tok_per_cta - 1) / a.tok_per_cta);
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
