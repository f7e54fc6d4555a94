// attn_tree.cuh -- what the kernels of wide_attn_tree share: the division of
// the work over the GPU, made on the device from the lengths and masks, and
// the records that join the parts of a run.
//
// A unit is a (sequence, KV head).  Its rows are the query heads of the
// tokens that keep the head group, rep per token, in token order; a run is
// `rt` of those rows over the unit's keys, in blocks of `bk` keys.  A run takes
// `rc` places for what it costs beside its blocks, then one for each block (two
// in a run of more than 128 rows).  All runs' places, unit after unit, form one line of `total`, and
// CTA c of n takes the blocks whose (first) place is in its n-th of the line: equal work for
// any mixture of lengths and masks, without a value read back by the
// host.  A CTA that holds only a part of a run (at most its first and its last
// segment) leaves the part's unnormalised output, maximum and sum in one of its
// two workspace slots, the first if the run began in an earlier CTA; the CTA
// that holds a run's first block records the run's extent, and attn_tree_join
// adds the parts in order, so results never depend on timing.
#pragma once

#include "common.cuh"

namespace wide {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTreeHD = 128;
constexpr float kTreeLag = 8.f;          // log2 units by which a row's reference is set above its maximum
constexpr int kTreeMaxUnits = 4096;
constexpr int kTreeMaxDraft = 1024;
constexpr int kTreeMaxRep = 32;          // query heads of a KV head

struct TreeArgs {
    const __nv_bfloat16 *q;            // [T][n_q][128], q_stride apart
    const void *k, *v;                 // caches
    const uint8_t *ks, *vs;
    const int32_t *cache_len, *draft_len;
    const uint32_t *tree, *heads;
    __nv_bfloat16 *out;
    int n_seq, draft, n_q, n_kv, rep, Wt, Wh;
    int64_t cap, q_stride;
    float scale_log2;
    uint32_t opaque;                   // kv_opaque of the cache's kind
    // parts: slot 2 c (a run begun in an earlier CTA than c) and 2 c + 1 (begun in c)
    float *part_o;                     // [2 n][rt][128]
    float2 *part_ml;                   // [2 n][rt] (reference in log2 units, sum)
    int4 *joins;                       // [n]: run starting in CTA c: (last CTA, first slot, rows, 0); rows 0: none
    int32_t *join_rows;                // [n][rt] output row of each row of that run
    int32_t *status;
};

// 2^x by the SFU (results below the normal range become 0, which a weight in
// bf16 next to one of at least 2^-9 loses anyway)
__device__ __forceinline__ float exp2_sfu(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16 bytes that are read once
__device__ __forceinline__ uint4 load_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// Sequence s: its earlier and new positions; both 0 if its lengths are bad.
__device__ __forceinline__ int2 tree_lens(const TreeArgs &a, int s, bool report)
{
    const int cl = a.cache_len[s], dl = a.draft_len ? a.draft_len[s] : a.draft;
    if (cl < 0 || dl < 0 || dl > a.draft || (int64_t)cl + dl > a.cap) {
        if (report)
            set_status(a.status, WIDE_DEV_BAD_RANGE);
        return make_int2(0, 0);
    }
    return make_int2(cl, dl);
}

// Places of one block of a run of `rows` rows.
__host__ __device__ __forceinline__ int tree_weight(int rows) { return rows > 128 ? 2 : 1; }
// Places of a unit of `rows` rows and nb blocks.
__device__ __forceinline__ uint32_t tree_places(int rows, int rt, int nb, int rc)
{
    const int full = rows / rt, rest = rows - full * rt;
    return nb ? (uint32_t)full * (uint32_t)(rc + tree_weight(rt) * nb) +
                    (rest ? (uint32_t)(rc + tree_weight(rest) * nb) : 0u)
              : 0u;
}
// CTAs that share `total` places: each has a block's worth at least, so every
// CTA between a run's first and last has a part of it.
__device__ __forceinline__ int tree_ctas(int grid, uint32_t total, int rt)
{
    const uint32_t most = total / (uint32_t)tree_weight(rt);
    return (int)min((uint32_t)grid, most ? most : total);
}

// cum[u] = places before unit u (u = s * n_kv + j; cum[U] = all), cnt[u] =
// tokens that keep the group; part: THREADS / 32 words of scratch, all in
// shared memory.  All threads of the CTA; ends with a barrier.
template <int THREADS>
__device__ void tree_plan(const TreeArgs &a, int rt, int bk, int rc, uint32_t *cum, uint16_t *cnt,
                          uint32_t *part)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int U = a.n_seq * a.n_kv;
#pragma unroll 1
    for (int s = warp; s < a.n_seq; s += THREADS / 32) {
        const int2 len = tree_lens(a, s, blockIdx.x == 0 && lane == 0);
        const int nb = (len.x + len.y + bk - 1) / bk;
#pragma unroll 1
        for (int w = 0; w < (a.n_kv + 31) / 32; ++w) {
            const int nj = min(32, a.n_kv - 32 * w);
            int mine = 0;              // lane j: tokens that keep group 32 w + j
            if (!a.heads) {
                mine = len.y;
            } else {
#pragma unroll 1
                for (int t0 = 0; t0 < len.y; t0 += 32) {
                    const int t = t0 + lane;
                    const uint32_t bits =
                        t < len.y ? a.heads[((size_t)s * a.draft + t) * a.Wh + w] : 0u;
#pragma unroll 1
                    for (int j = 0; j < nj; ++j) {
                        const int c = __popc(__ballot_sync(0xffffffffu, (bits >> j) & 1u));
                        mine += lane == j ? c : 0;
                    }
                }
            }
            if (lane < nj) {
                const int u = s * a.n_kv + 32 * w + lane;
                cnt[u] = (uint16_t)mine;
                cum[u + 1] = tree_places(mine * a.rep, rt, nb, rc);
            }
        }
    }
    if (tid == 0)
        cum[0] = 0;
    __syncthreads();
    // inclusive scan of cum[1..U]: each thread a stretch, then the stretches
    const int per = (U + THREADS - 1) / THREADS;
    const int lo = min(U, tid * per), hi = min(U, lo + per);
    uint32_t sum = 0;
#pragma unroll 1
    for (int i = lo; i < hi; ++i)
        sum += cum[i + 1];
    uint32_t inc = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off)
            inc += o;
    }
    if (lane == 31)
        part[warp] = inc;
    __syncthreads();
    static_assert(THREADS <= 1024, "a lane for each warp");
    uint32_t before = inc - sum + __reduce_add_sync(0xffffffffu, lane < warp ? part[lane] : 0u);
#pragma unroll 1
    for (int i = lo; i < hi; ++i) {
        before += cum[i + 1];
        cum[i + 1] = before;
    }
    __syncthreads();
}

// The unit that holds place b: the largest u with cum[u] <= b.
__device__ __forceinline__ int tree_unit(const uint32_t *cum, int U, uint32_t b)
{
    int lo = 0, hi = U;                // cum[lo] <= b < cum[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= b)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// The line's `total` places shared out to n CTAs: total % n of them get one more.
struct TreeShare {
    uint32_t each, more;               // places of a CTA; CTAs with one more
    __device__ __forceinline__ TreeShare(uint32_t total, uint32_t n) : each(total / n), more(total - n * each) {}
    __device__ __forceinline__ uint32_t first(uint32_t c) const { return c * each + min(c, more); }
    __device__ __forceinline__ int owner(uint32_t b) const
    {
        const uint32_t head = more * (each + 1);
        return (int)(b < head ? b / (each + 1) : more + (b - head) / each);
    }
};

// Tokens of the unit that keep the group, numbers [from, to) of them, into
// tok[]; by one whole warp.
template <typename T>
__device__ __forceinline__ void tree_tokens(const TreeArgs &a, int s, int j, int dl, int from,
                                            int to, T *tok)
{
    const int lane = threadIdx.x & 31;
    int seen = 0;
#pragma unroll 1
    for (int t0 = 0; t0 < dl && seen < to; t0 += 32) {
        const int t = t0 + lane;
        const bool on =
            t < dl &&
            (!a.heads ||
             ((a.heads[((size_t)s * a.draft + t) * a.Wh + (j >> 5)] >> (j & 31)) & 1u));
        const uint32_t b = __ballot_sync(0xffffffffu, on);
        const int at = seen + __popc(b & ((1u << lane) - 1u));
        if (on && at >= from && at < to)
            tok[at - from] = (T)t;
        seen += __popc(b);
    }
}

// Whether new token t of sequence s attends new token j.
__device__ __forceinline__ bool tree_sees(const TreeArgs &a, int s, int t, int j)
{
    if (!a.tree)
        return j <= t;
    return (a.tree[((size_t)s * a.draft + t) * a.Wt + (j >> 5)] >> (j & 31)) & 1u;
}

// Values that are not finite.  A weight is positive, so an infinity attended
// makes its element of the output that infinity whatever the weight rounds to,
// but a product gives 0 * inf = NaN where a weight became 0: one too small for
// its format, an output scaled down to nothing by a later maximum, a copy of a
// row that takes other keys.  So where a sum comes out as NaN and the weights'
// does not, its element is the sum of what is not finite alone: of the context's
// values, which every row attends, or of the parts' outputs.  That costs a
// comparison an element of the output; only then are the values read again.
__device__ __forceinline__ float tree_inf_or_0(float x) { return fabsf(x) <= 3.402823466e38f ? 0.f : x; }
__device__ __forceinline__ bool tree_any_nan(float x, float y, float z, float w)
{
    return !(x == x && y == y && z == z && w == w);
}
// The sum of what is not finite among 4 elements (v: those of the first row) of
// n rows of a bf16 cache; 0 where there is none.
__device__ __forceinline__ void tree_not_finite(const __nv_bfloat16 *v, int n, float (&sum)[4])
{
    sum[0] = sum[1] = sum[2] = sum[3] = 0.f;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const uint2 w = *reinterpret_cast<const uint2 *>(v + (int64_t)i * kTreeHD);
        const float x[4] = {bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y)};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            sum[e] += tree_inf_or_0(x[e]);
    }
}

// Zeros for the pairs of new token and head group that are skipped; the CTAs
// share the pairs.
template <int THREADS> __device__ void tree_zero_skipped(const TreeArgs &a)
{
    if (!a.heads)
        return;
    const int lane = threadIdx.x & 31;
    const int64_t pairs = (int64_t)a.n_seq * a.draft * a.n_kv;
    const int64_t warps = (int64_t)gridDim.x * (THREADS / 32);
#pragma unroll 1
    for (int64_t p0 = ((int64_t)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5)) * 32; p0 < pairs;
         p0 += warps * 32) {
        const int64_t p = p0 + lane;
        bool zero = false;
        if (p < pairs) {
            const int64_t t = p / a.n_kv;
            const int j = (int)(p - t * a.n_kv), s = (int)(t / a.draft);
            zero = (int)(t - (int64_t)s * a.draft) < tree_lens(a, s, false).y &&
                   !((a.heads[(size_t)t * a.Wh + (j >> 5)] >> (j & 31)) & 1u);
        }
        uint32_t todo = __ballot_sync(0xffffffffu, zero);
        while (todo) {
            const int64_t z = p0 + __ffs(todo) - 1;
            todo &= todo - 1;
            const int64_t t = z / a.n_kv;
            const int j = (int)(z - t * a.n_kv);
            uint4 *o = reinterpret_cast<uint4 *>(a.out + (t * a.n_q + (int64_t)j * a.rep) * kTreeHD);
#pragma unroll 1
            for (int i = lane; i < a.rep * (kTreeHD / 8); i += 32)
                o[i] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
}

// attn_tree_tc.cu: runs of rt = 32, 64, 128 or 256 rows, by n CTAs.
int attn_tree_tiles_launch(const TreeArgs &a, int kind, int rt, int n, cudaStream_t s);

// Waits for the kernels this launch depends on (programmatic launch).
__device__ __forceinline__ void grid_dependency_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void grid_launch_dependents()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace wide
