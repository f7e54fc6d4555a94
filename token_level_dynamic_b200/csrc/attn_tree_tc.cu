// attn_tree_tc.cu -- wide_attn_tree on the tensor cores: the rows of a run, up
// to 256, share one pass over their keys.
//
// One persistent CTA per SM, whose warps hand work over through mbarriers:
//   copy     one warp: tiles of 128 keys and of 128 values, in the order in
//            which the MMAs use them, by TMA; bf16 straight into the operands'
//            swizzled layout, 8-bit rows and their scales into a ring of raw
//            tiles
//   convert  8 warps (4 for bf16): raw tiles to bf16 operand tiles, exactly, in
//            a second ring.  A thread takes 32 codes with one scale; the bf16
//            pairs are bytes (0, 2) and (1, 3) of a word, which saves the
//            permutes (integer instructions issue at half rate): the dims of an
//            operand row are in the order 0 2 1 3 within each four, the
//            queries are written in the same order and outputs put back at the
//            end.  Values of new positions are checked: what is not finite is
//            left out of the tile (0 * NaN would reach rows that do not attend
//            it) and added to the attending rows at the end
//   MMA      one thread:  S = Q K^T  (M 128 rows, N 128 keys)  and
//            O += P V  (N 128 dims), fp32 in tensor memory; P, rounded to
//            bf16, is read from tensor memory too
//   softmax  8 warps per 128 rows: two threads to a row, each with half of the
//            keys.  A row's reference is set 8 (log2 units) above its maximum and
//            moves only when the maximum passes it, so no weight is above 1 and O
//            is rarely rescaled: the weights are computed with the reference so
//            far, and once more if any row of the tile has to move
//   plan     one warp: the next run and its tokens
// Runs of at most 128 rows have two tiles of scores and of weights in turn, so
// the scores of the next keys are ready when a softmax ends.  Larger ones have
// one per 128 rows, with the weights over the scores' first half, and the two
// halves' softmax and MMAs overlap each other.
// Rows along M: a run of at most 64 or 32 rows is repeated R = 2 or 4 times,
// and a copy takes 128 / R keys of a tile (its weights for other keys are
// zero).  The exponentials of a warp all issue in one quarter of the SM, and
// this spreads those of a few rows over the quarters.  The copies are added at
// the end.
// Tensor memory, 512 columns: scores at 0 and 128; output at 256 (and 384 with
// two halves); weights at 384 and 448.
#include "attn_tree.cuh"
#include "host.h"
#include "kv.cuh"
#include "umma.cuh"

namespace wide {
namespace {

constexpr int kBK = 128;                         // keys per tile
constexpr uint32_t kHalf = 128 * 128;            // 128 rows of 64 bf16, 128-byte swizzle
constexpr uint32_t kTile = 2 * kHalf;            // 128 x 128 bf16
constexpr uint32_t kRawCodes = kBK * kTreeHD;    // codes of a raw tile; the scales follow the ring
constexpr uint32_t kRawScales = kBK * 4;
constexpr int kRunCost = 3;                      // tiles' time that a run costs beside its tiles
constexpr int kOPitch = kTreeHD + 4;             // floats; row pitch when copies are added

// NM: row halves of a run (2: up to 256 rows)
template <int KIND, int NM> struct Cfg {
    static constexpr bool k8 = KIND != WIDE_KV_BF16;
    // warps, and registers per thread: every four warps the same number, out of
    // kLaunchRegs each (setmaxnreg); the last of the issuing four idles
    static constexpr int kSoftWarps = 8 * NM, kConvWarps = k8 ? 8 : 4;
    static constexpr int kMmaWarp = kSoftWarps + kConvWarps, kCopyWarp = kMmaWarp + 1, kPlanWarp = kMmaWarp + 2;
    static constexpr int kWarps = kMmaWarp + 4, kThreads = 32 * kWarps;
    static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
    static constexpr int kConvRegs = NM == 2 ? 48 : 72, kIssueRegs = NM == 2 ? (k8 ? 56 : 48) : 64;
    static constexpr int kSoftRegs = NM == 2 ? (k8 ? 88 : 96) : k8 ? 136 : 184;
    static_assert(kLaunchRegs * kThreads <= 65536 && kSoftRegs * kSoftWarps + kConvRegs * kConvWarps +
                                                             kIssueRegs * 4 <= kLaunchRegs * kWarps,
                  "registers");
    static constexpr int kOps = k8 ? 3 : 6 - NM;           // operand tiles
    static constexpr int kRaw = k8 ? 7 - 2 * NM : 1;       // raw tiles (bf16: unused)
    static constexpr uint32_t kOffOps = NM * kTile, kOffRaw = kOffOps + kOps * kTile;
    static constexpr uint32_t kOffScales = kOffRaw + (k8 ? kRaw * kRawCodes : 0);
    static constexpr uint32_t kOffCtl = kOffScales + (k8 ? kRaw * kRawScales : 0);
};

// One run, as far as a CTA does it.
struct Run {
    int64_t row0;                // the unit's first cache row
    int s, j, cl, dl;            // sequence, KV head, earlier and new positions
    int run, blk0, nt;           // number within the unit, first tile, tiles
    int nrows, nm, slot;         // rows, row halves in use, workspace slot
    int whole;                   // all of the run's tiles
};

template <int OPS, int RAW, int ROWS, int NM> struct __align__(16) TcCtl {
    uint64_t op_full[OPS];                       // bf16: the tile's copies have landed
    uint64_t op_ready[OPS];                      // the convert warps are done with the tile
    uint64_t op_empty[OPS];                      // the MMAs have read it
    uint64_t raw_full[RAW], raw_empty[RAW];      // raw rows landed / converted
    uint64_t q_full;                             // the run's queries are written
    // of the two tiles in turn, or the two row halves
    uint64_t s_full[2];                          // the scores are complete
    uint64_t p_full[2];                          // the weights are written (8 warps)
    uint64_t pv_done[2];                         // O += P V is complete
    uint64_t o_full[2];                          // the run's output of a row half is complete
    uint64_t all_done;                           // error path: every MMA is complete
    Run run;                                     // the current one; nt 0: there are no more
    uint32_t tmem;
    int abort, any_bad;
    int32_t at[ROWS];                            // output row of each row
    int16_t tok[ROWS], head[ROWS];               // its token (-1: no row) and query head
    int16_t list[ROWS];                          // tokens of the next run
    float pair[2][128 * NM];                     // what the two threads of a row tell each other
    uint32_t bad[kTreeMaxDraft / 32];            // new positions with a value that is not finite
};

// Waits for this thread's tensor memory loads; v, loaded by one of them, is
// not used before.
__device__ __forceinline__ void tmem_ld_wait_for(float (&v)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
                   "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]),
                   "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]),
                   "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]),
                   "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29])
                 :: "memory");
    // (an asm statement takes 30 operands at most)
    asm volatile("" : "+f"(v[30]), "+f"(v[31])::"memory");
}

// a * b + c and a + b of pairs, each element rounded as fmaf / + does
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 16 fp32 columns of this thread's lane, once they have arrived.
__device__ __forceinline__ void tmem_get16(uint32_t taddr, float (&v)[16])
{
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
                   "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                   "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                   "+r"(r[13]), "+r"(r[14])
                 :
                 : "memory");
    asm volatile("" : "+r"(r[15])::"memory");
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] = __uint_as_float(r[i]);
}

// Weights 2^(sc x - mref) of COLS scores x in tensor memory as bf16 pairs;
// returns the largest sc x and the sum of the weights.  tail: see(i) has the
// bits of the scores 32 i .. that the row attends.  CH scores at a time.
template <int COLS, int CH, class See>
__device__ __forceinline__ float2 tile_weights(uint32_t ts, float sc, float mref, uint32_t (&pw)[COLS / 2],
                                               bool tail, See &&see)
{
    const float mb = mref > -INFINITY ? -mref : 0.f;
    const float2 sc2 = make_float2(sc, sc), mb2 = make_float2(mb, mb);
    float mx[2] = {-INFINITY, -INFINITY};
    float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int i = 0; i < COLS / CH; ++i) {
        float v[CH];
        if constexpr (CH == 16) {
            tmem_get16(ts + 16 * i, v);
        } else {
            umma::tmem_ld32(ts + 32 * i, v);
            tmem_ld_wait_for(v);
        }
        if (tail) {
            const uint32_t bits = see(i * CH / 32) >> (i * CH % 32);
#pragma unroll
            for (int e = 0; e < CH; ++e)
                v[e] = (bits >> e) & 1u ? v[e] : -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < CH; e += 2) {
            mx[(e >> 1) & 1] = max3(mx[(e >> 1) & 1], v[e], v[e + 1]);
            const float2 x = fma2(make_float2(v[e], v[e + 1]), sc2, mb2);
            const float2 p = make_float2(exp2_sfu(x.x), exp2_sfu(x.y));
            ls[(e >> 1) & 1] = add2(ls[(e >> 1) & 1], p);
            pw[(i * CH + e) / 2] = pack_bf16(p.x, p.y);
        }
    }
    ls[0] = add2(ls[0], ls[1]);
    return make_float2(fmaxf(mx[0], mx[1]) * sc, ls[0].x + ls[0].y);
}

// Position in a ring of N slots.
template <int N> struct Ring {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next()
    {
        phase ^= slot == N - 1 ? 1u : 0u;
        slot = slot == N - 1 ? 0 : slot + 1;
    }
    __device__ __forceinline__ void back()
    {
        phase ^= slot == 0 ? 1u : 0u;
        slot = slot == 0 ? N - 1 : slot - 1;
    }
};

// A bounded wait: gives up after kWaitLimitNs, or when another warp has.  The
// time is read every 1024 polls only.
__device__ __forceinline__ bool tc_wait(uint64_t *bar, uint32_t parity, int *abort, int32_t *status)
{
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n) {
        if (n & 1023u)
            continue;
        if (*(volatile int *)abort)
            return false;
        const uint64_t now = globaltimer();
        if (t0 == 0)
            t0 = now;
        if (now - t0 > kWaitLimitNs) {
            set_status(status, WIDE_DEV_TIMEOUT);
            *(volatile int *)abort = 1;
            return false;
        }
    }
    return true;
}

// D[tmem] (+)= A[tmem] * B[smem]: A's rows are lanes, two bf16 per column.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Barrier of the 8 softmax warps of row half m; true if any thread says so.
__device__ __forceinline__ bool softmax_or(int m, bool say)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %2, 0;\n\t"
                 "barrier.cta.red.or.pred p, %1, 256, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r)
                 : "r"(m + 1), "r"((uint32_t)say)
                 : "memory");
    return r != 0;
}

// True in one thread of a whole warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

template <int N> __device__ __forceinline__ void more_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void fewer_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 16 words to 16 columns of this thread's lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *w)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]),
        "r"(w[8]), "r"(w[9]), "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15])
        : "memory");
}

// As tmem_st16, 8 words.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *w)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// 4 bytes, or zeros if !in (src must still be a valid address).
__device__ __forceinline__ void cp_async4_zfill(uint32_t dst, const void *src, bool in)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
                 "r"(in ? 4 : 0)
                 : "memory");
}

// Takes what is not finite out of 8 bf16; whether there was any.
__device__ __forceinline__ bool drop_not_finite(uint4 &w)
{
    uint32_t *x = reinterpret_cast<uint32_t *>(&w);
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if ((x[e] & 0x7f80u) == 0x7f80u) {
            x[e] &= 0xffff0000u;
            bad = true;
        }
        if ((x[e] & 0x7f800000u) == 0x7f800000u) {
            x[e] &= 0x0000ffffu;
            bad = true;
        }
    }
    return bad;
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}
__device__ __forceinline__ void st_shared16(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}

// 32 codes with one scale byte as bf16 to 64 bytes of a swizzled operand row;
// dst: address of the first 16 (the next ones differ in bits 4 and 5).
template <int KIND>
__device__ __forceinline__ void convert32(uint32_t dst, const uint4 c0, const uint4 c1, uint32_t sc, uint32_t opaque)
{
    const uint32_t m = kv_mult<KIND>(sc) * 0x00010001u;
    uint32_t o[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t x = word(e < 4 ? c0 : c1, e & 3);
        kv_pairs_0213<KIND>(x, m, opaque, o[2 * e], o[2 * e + 1]);
    }
    if (KIND == WIDE_KV_E4M3 && sc > 134u && sc < 255u) {
        const uint32_t mh = kv_mult_high(sc) * 0x00010001u;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            o[e] = mul_bf16x2(o[e], mh);
    }
#pragma unroll
    for (int g = 0; g < 4; ++g)
        st_shared16(dst ^ (uint32_t)(g << 4), o[4 * g], o[4 * g + 1], o[4 * g + 2], o[4 * g + 3]);
}

// The bits of row `t` for the 32 positions from kb on: earlier positions all,
// new ones as the tree says, none past the end.
__device__ __forceinline__ uint32_t seen_bits(const TreeArgs &a, int s, int t, int kb, int cl, int dl)
{
    auto low = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
    const uint32_t ctx = low(cl - kb), end = low(cl + dl - kb);
    uint32_t tree;
    if (t < 0) {
        tree = 0u;
    } else if (!a.tree) {
        tree = low(cl + t + 1 - kb);
    } else {
        const uint32_t *w = a.tree + ((size_t)s * a.draft + t) * a.Wt;
        const int j0 = kb - cl;                   // new position of bit 0
        const int i0 = j0 >> 5, sh = j0 & 31;     // floor division
        const uint32_t lo = i0 >= 0 && i0 < a.Wt ? w[i0] : 0u;
        const uint32_t hi = i0 + 1 >= 0 && i0 + 1 < a.Wt ? w[i0 + 1] : 0u;
        tree = __funnelshift_r(lo, hi, sh);
    }
    return (ctx | tree) & end;
}

template <int KIND, int NM, int R>
__global__ void __launch_bounds__(Cfg<KIND, NM>::kThreads, 1)
    attn_tree_tiles(const TreeArgs a, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v)
{
    using C = Cfg<KIND, NM>;
    constexpr int kThreads = C::kThreads, kMmaWarp = C::kMmaWarp, kCopyWarp = C::kCopyWarp, kPlanWarp = C::kPlanWarp;
    constexpr int rt = NM == 2 ? 256 : 128 / R;       // rows of a run
    constexpr int kMine = 64 / R;                     // keys of a tile per softmax thread
    using Ctl = TcCtl<C::kOps, C::kRaw, rt, NM>;
    static_assert(C::kOffCtl + sizeof(Ctl) <= 227 * 1024, "shared memory");
    static_assert(128 * (kOPitch * 4 + 8) <= C::kOps * kTile, "the copies' outputs fit in the ring");
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int me = (int)blockIdx.x, U = a.n_seq * a.n_kv;
    if (smem_u32(smem) & 1023u) {
        if (tid == 0) {
            set_status(a.status, WIDE_DEV_LAYOUT);
            a.joins[me] = make_int4(0, 0, 0, 0);
        }
        return;
    }
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + C::kOffCtl);
    uint8_t *ops = smem + C::kOffOps, *raw = smem + C::kOffRaw;

    // (before the plan, whose loads other warps wait for meanwhile)
    if (tid == 32 * kCopyWarp) {
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
        ctl->abort = 0;
        for (int i = 0; i < C::kOps; ++i) {
            mbar_init(&ctl->op_full[i], 1);
            mbar_init(&ctl->op_ready[i], C::kConvWarps);
            mbar_init(&ctl->op_empty[i], 1);
        }
        for (int i = 0; i < C::kRaw; ++i) {
            mbar_init(&ctl->raw_full[i], 33);
            mbar_init(&ctl->raw_empty[i], C::kConvWarps);
        }
        mbar_init(&ctl->q_full, C::kConvWarps);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->s_full[i], 1);
            mbar_init(&ctl->p_full[i], 8);
            mbar_init(&ctl->pv_done[i], 1);
            mbar_init(&ctl->o_full[i], 1);
        }
        mbar_init(&ctl->all_done, 1);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        umma::tmem_alloc(&ctl->tmem, 512);
        umma::tmem_relinquish();
    }

    // ---- the plan, in the ring of operand tiles
    uint32_t *cum = reinterpret_cast<uint32_t *>(ops);
    uint16_t *cnt = reinterpret_cast<uint16_t *>(cum + kTreeMaxUnits + 1);
    static_assert((kTreeMaxUnits + 1) * 4 + (kTreeMaxUnits + 2) * 2 + C::kWarps * 4 <= C::kOps * kTile,
                  "the plan fits in the ring");
    tree_plan<kThreads>(a, rt, kBK, kRunCost, cum, cnt, reinterpret_cast<uint32_t *>(cnt + kTreeMaxUnits + 2));
    const uint32_t total = cum[U];
    const int n_cta = tree_ctas((int)gridDim.x, total, rt);
    // (a CTA past them has no places, and no work but the zeros at the end)
    const TreeShare share(total, max(n_cta, 1));
    const uint32_t first = me < n_cta ? share.first(me) : 0u, end = me < n_cta ? share.first(me + 1) : 0u;
    // of the plan warp: the 32 units from u0 on; lane i holds the places before
    // unit u0 + i + 1, and the tokens of unit u0 + i
    int u0 = 0, mine = 0;
    uint32_t base = 0, upto = 0;
    if (warp == kPlanWarp) {
        u0 = tree_unit(cum, U, first);
        base = cum[u0];
        upto = cum[min(u0 + lane + 1, U)];
        mine = u0 + lane < U ? cnt[u0 + lane] : 0;
    }
    fence_proxy_async_smem();                         // the ring is written by copies next
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = ctl->tmem;

    // ring positions and parities that a role carries from run to run
    Ring<C::kRaw> raw_at;
    Ring<C::kOps> op_at;
    uint32_t runs = 0;                                // so far
    // bit b: parity of the tiles that scores b have held so far, and with it of
    // the completions of s_full[b], p_full[b] and pv_done[b]
    uint32_t held = 0;
    uint32_t o_phase = 0;                             // bit m: parity of the runs of row half m
    bool ok = true;
    int *abort = &ctl->abort;

    // The runs of this CTA's places, one after another: each role calls it with
    // its part of the work.  All threads meet before and after a run.
    const Run &x = ctl->run;
    auto each_run = [&](auto &&work) {
        for (;;) {
            __syncthreads();
            const int nt = x.nt;
            if (nt == 0)
                break;
            work();
            held ^= x.nm == 2 ? (nt & 1) * 3u : (((nt + 1) >> 1) & 1u) | ((nt >> 1) & 1u) << 1;
            ++runs;
            o_phase ^= x.nm == 2 ? 3u : 1u;
            if (__syncthreads_or(!ok))
                break;
        }
        umma::fence_before_sync();
        __syncthreads();
    };

    // -------------------------------------------------------------- plan
    // One warp finds the next run and its tokens while the others work on the
    // current one.
    auto plan_role = [&] {
        uint32_t b = first;
        int lo = 0;                                   // the next run's first token among those that keep the group
        int4 join = make_int4(0, 0, 0, 0);
        auto window = [&] {                           // of the 32 units from u0 on, `base` places before them
            const int u = u0 + lane, s = (int)((uint32_t)min(u, U - 1) / (uint32_t)a.n_kv), j = u - s * a.n_kv;
            const int2 len = u < U ? tree_lens(a, s, false) : make_int2(0, 0);
            mine = a.heads ? 0 : len.y;
            if (a.heads)
#pragma unroll 4
                for (int t = 0; t < len.y; ++t)
                    mine += (a.heads[((size_t)s * a.draft + t) * a.Wh + (j >> 5)] >> (j & 31)) & 1u;
            upto = tree_places(mine * a.rep, rt, (len.x + len.y + kBK - 1) / kBK, kRunCost);
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, upto, off);
                upto += lane >= off ? o : 0u;
            }
            upto += base;
        };
        auto next = [&](Run &r) {                     // false: none left
            for (;;) {
                r.nt = 0;
                if (b >= end)
                    return false;
                uint32_t past = __ballot_sync(0xffffffffu, upto <= b);
                while (past == 0xffffffffu) {
                    base = __shfl_sync(0xffffffffu, upto, 31);
                    u0 += 32;
                    window();
                    past = __ballot_sync(0xffffffffu, upto <= b);
                }
                const int i = __popc(past), u = u0 + i;    // upto rises with the lane
                const uint32_t prev = __shfl_sync(0xffffffffu, upto, max(i - 1, 0)), before = i ? prev : base;
                r.s = (int)((uint32_t)u / (uint32_t)a.n_kv);
                r.j = u - r.s * a.n_kv;
                const int2 len = tree_lens(a, r.s, false);
                r.cl = len.x;
                r.dl = len.y;
                const int nb = (r.cl + r.dl + kBK - 1) / kBK, per = kRunCost + tree_weight(rt) * nb;
                const int rows = __shfl_sync(0xffffffffu, mine, i) * a.rep;
                r.run = min((int)((b - before) / (uint32_t)per), (rows - 1) / rt);
                const uint32_t run0 = before + (uint32_t)r.run * per;   // the run's first place
                r.nrows = min(rt, rows - r.run * rt);
                const int w = tree_weight(r.nrows), pos = (int)(b - run0);
                const int stop = (int)min((uint32_t)(kRunCost + w * nb), (uint32_t)pos + (end - b));
                b += (uint32_t)(stop - pos);
                r.blk0 = (max(pos - kRunCost, 0) + w - 1) / w;
                r.nt = (max(stop - kRunCost, 0) + w - 1) / w - r.blk0;
                if (r.nt == 0)
                    continue;
                r.nm = NM == 2 ? w : 1;
                r.whole = r.nt == nb;
                r.slot = 2 * me + (r.blk0 == 0);
                r.row0 = (int64_t)u * a.cap;
                if (!r.whole && r.blk0 == 0)          // the run starts here: record its extent
                    join = make_int4(share.owner(run0 + (uint32_t)(kRunCost + w * (nb - 1))),
                                     r.slot, r.nrows, 0);
                lo = (int)((uint32_t)(r.run * rt) / (uint32_t)a.rep);
                tree_tokens(a, r.s, r.j, r.dl, lo, (int)((uint32_t)(r.run * rt + r.nrows - 1) / (uint32_t)a.rep) + 1,
                            ctl->list);
                __syncwarp();
                return true;
            }
        };
        Run r;
        for (bool current = false;;) {                // a run of which the others work on
            const bool more = next(r);
            if (current && __syncthreads_or(0)) {
                join = make_int4(0, 0, 0, 0);
                break;
            }
            current = more;
            if (lane == 0) {
                ctl->run = r;
                ctl->any_bad = 0;
            }
            ctl->bad[lane] = 0;
            if (more) {
#pragma unroll 1
                for (int i = lane; i < rt; i += 32) {
                    const int t = (int)((uint32_t)(r.run * rt + i) / (uint32_t)a.rep), h = r.run * rt + i - t * a.rep;
                    const int tok = i < r.nrows ? ctl->list[t - lo] : -1;
                    ctl->tok[i] = (int16_t)tok;
                    ctl->head[i] = (int16_t)(r.j * a.rep + h);
                    ctl->at[i] = (r.s * a.draft + tok) * a.n_q + r.j * a.rep + h;
                }
            }
            __syncthreads();
            if (!more)
                break;
        }
        if (lane == 0)
            a.joins[me] = join;
        umma::fence_before_sync();
        __syncthreads();
    };

    // Operand tile i of a run, in the order of use: K of the first tile, then of
    // each next tile before V of the one before it.  Returns the tile; values?
    auto item = [](int i, int nt, bool &values) {
        values = i > 0 && ((i & 1) == 0 || i == 2 * nt - 1);
        return i == 0 ? 0 : i == 2 * nt - 1 ? nt - 1 : (i & 1) ? (i + 1) >> 1 : (i >> 1) - 1;
    };

    // -------------------------------------------------------------- copy
    auto copy_role = [&] {
        const int blk0 = x.blk0, nt = x.nt, nkeys = x.cl + x.dl;
        const int64_t row0 = x.row0;
        uint32_t issued = 0;
#pragma unroll 1
        for (int i = 0; i < 2 * nt; ++i, ++issued) {
            bool values;
            const int p0 = (blk0 + item(i, nt, values)) * kBK;
            const CUtensorMap *map = values ? &map_v : &map_k;
            const int32_t y = (int32_t)(row0 + p0);
            if constexpr (C::k8) {
                ok = __all_sync(0xffffffffu, tc_wait(&ctl->raw_empty[raw_at.slot], raw_at.phase ^ 1u,
                                                     abort, a.status));
                if (!ok)
                    break;
                uint64_t *bar = &ctl->raw_full[raw_at.slot];
                if (lane == 0) {
                    // (rows past the unit's end may hold anything: finite with scale 0)
                    mbar_arrive_expect_tx(bar, kRawCodes);
                    tma_load_2d(raw + raw_at.slot * kRawCodes, map, 0, y, bar);
                }
                const uint8_t *scales = (values ? a.vs : a.ks) + (row0 + p0) * 4;
                const uint32_t dst = smem_u32(smem + C::kOffScales + raw_at.slot * kRawScales);
#pragma unroll
                for (int r = lane; r < kBK; r += 32) {
                    const bool in = p0 + r < nkeys;
                    cp_async4_zfill(dst + r * 4, scales + (in ? r * 4 : 0), in);
                }
                cp_async_arrive_noinc(bar);
                raw_at.next();
            } else {
                ok = __all_sync(0xffffffffu, tc_wait(&ctl->op_empty[op_at.slot], op_at.phase ^ 1u, abort,
                                                     a.status));
                if (!ok)
                    break;
                if (lane == 0) {
                    uint64_t *bar = &ctl->op_full[op_at.slot];
                    uint8_t *dst = ops + op_at.slot * kTile;
                    mbar_arrive_expect_tx(bar, kTile);
                    tma_load_2d(dst, map, 0, y, bar);
                    tma_load_2d(dst + kHalf, map, 64, y, bar);
                }
                op_at.next();
            }
        }
        if (!ok) {                                    // copies in flight land before shared memory goes
            if constexpr (C::k8) {
                cp_async_wait_all();
#pragma unroll 1
                for (uint32_t i = 0; i < min(issued, (uint32_t)C::kRaw); ++i) {
                    raw_at.back();
                    mbar_wait(&ctl->raw_full[raw_at.slot], raw_at.phase);
                }
            } else {
#pragma unroll 1
                for (uint32_t i = 0; i < min(issued, (uint32_t)C::kOps); ++i) {
                    op_at.back();
                    mbar_wait(&ctl->op_full[op_at.slot], op_at.phase);
                }
            }
        }
    };

    // ----------------------------------------------------------- convert
    auto convert_role = [&] {
        const int cl = x.cl, dl = x.dl, blk0 = x.blk0, nt = x.nt;
        constexpr int kConv = 32 * C::kConvWarps;
        const int ct = tid - 32 * C::kSoftWarps;
        // (8 bits) this thread's row of a tile, its swizzle pattern, and its first block of 32
        const int row = ct & 127, blk = ct >> 7;
        const uint32_t row_swz = swz128(row, 0);
        // the queries first, several loads at a time
        constexpr int kAtOnce = NM == 2 ? 4 : 8;
        const __nv_bfloat16 *q_seq = a.q + (int64_t)x.s * a.draft * a.q_stride;
#pragma unroll 1
        for (int i0 = ct; i0 < x.nm * 128 * 16; i0 += kAtOnce * kConv) {
            uint4 w[kAtOnce];
#pragma unroll
            for (int n = 0; n < kAtOnce; ++n) {
                const int i = i0 + n * kConv, r = i >> 4, c = i & 15;
                const int q_row = NM == 2 ? r : r & (rt - 1), tok = ctl->tok[q_row];
                w[n] = make_uint4(0u, 0u, 0u, 0u);
                if (tok >= 0)
                    w[n] = *reinterpret_cast<const uint4 *>(q_seq + (int64_t)tok * a.q_stride +
                                                            ctl->head[q_row] * kTreeHD + c * 8);
            }
#pragma unroll
            for (int n = 0; n < kAtOnce; ++n) {
                const int i = i0 + n * kConv, r = i >> 4, c = i & 15;
                if (C::k8)                            // dims in the operand order 0 2 1 3
                    w[n] = make_uint4(__byte_perm(w[n].x, w[n].y, 0x5410), __byte_perm(w[n].x, w[n].y, 0x7632),
                                      __byte_perm(w[n].z, w[n].w, 0x5410), __byte_perm(w[n].z, w[n].w, 0x7632));
                *reinterpret_cast<uint4 *>(smem + (r >> 7) * kTile + (c >> 3) * kHalf +
                                           swz128(r & 127, c & 7)) = w[n];
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&ctl->q_full);
        auto note_bad = [&](int jj) {
            if (jj < dl) {
                atomicOr(&ctl->bad[jj >> 5], 1u << (jj & 31));
                ctl->any_bad = 1;
            }
        };
#pragma unroll 1
        for (int i = 0; i < 2 * nt && ok; ++i) {
            bool values;
            const int p0 = (blk0 + item(i, nt, values)) * kBK;
            const bool fresh = values && p0 + kBK > cl;         // values with new positions
            if constexpr (C::k8) {
                constexpr int kN = kBK * 4 / kConv;             // blocks of 32 codes of a thread
                ok = tc_wait(&ctl->raw_full[raw_at.slot], raw_at.phase, abort, a.status) &&
                     tc_wait(&ctl->op_empty[op_at.slot], op_at.phase ^ 1u, abort, a.status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                uint32_t sb4 = reinterpret_cast<const uint32_t *>(smem + C::kOffScales + raw_at.slot * kRawScales)[row];
                if (fresh && p0 + row >= cl && __vcmpeq4(sb4, ~0u)) {   // their codes are zeros
                    note_bad(p0 + row - cl);
                    sb4 &= ~__vcmpeq4(sb4, ~0u);
                }
                const uint32_t from = smem_u32(raw) + raw_at.slot * kRawCodes + row_swz;
                const uint32_t to = smem_u32(ops) + op_at.slot * kTile + row_swz;
#pragma unroll
                for (int n = 0; n < kN; ++n) {
                    const int bk = blk + n * (kConv / 128);     // pieces 2 bk, 2 bk + 1 of the codes' row
                    const uint32_t f = from ^ (uint32_t)(bk << 5);
                    convert32<KIND>((to ^ (uint32_t)((bk & 1) << 6)) + (uint32_t)(bk >> 1) * kHalf,
                                    ld_shared16(f), ld_shared16(f ^ 16u), (sb4 >> (8 * bk)) & 255u, a.opaque);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&ctl->raw_empty[raw_at.slot]);
                    mbar_arrive(&ctl->op_ready[op_at.slot]);
                }
                raw_at.next();
            } else {
                ok = __all_sync(0xffffffffu, tc_wait(&ctl->op_full[op_at.slot], op_at.phase, abort, a.status));
                if (!ok)
                    break;
                if (fresh) {
                    // rows of new positions, and rows past the end, which may hold anything
                    uint8_t *tile = ops + op_at.slot * kTile;
#pragma unroll 1
                    for (int e = max(cl - p0, 0) * 16 + ct; e < kBK * 16; e += kConv) {
                        const int r = e >> 4, c = e & 15;
                        uint4 *at = reinterpret_cast<uint4 *>(tile + (c >> 3) * kHalf + swz128(r, c & 7));
                        uint4 w = *at;
                        if (drop_not_finite(w)) {
                            *at = w;
                            note_bad(p0 + r - cl);
                        }
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&ctl->op_ready[op_at.slot]);
            }
            op_at.next();
        }
    };

    // --------------------------------------------------------------- MMA
    // The whole warp walks through the tiles and one thread issues: with values
    // that are the same in all lanes the operands stay in uniform registers.
    // (Issued from a branch of one lane, eight MMAs took 700 clocks.)
    auto mma_role = [&] {
        const int nt = __shfl_sync(0xffffffffu, x.nt, 0);
        const bool two = NM == 2 && __shfl_sync(0xffffffffu, x.nm, 0) == 2;
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        constexpr uint32_t idesc_s = umma::idesc_bf16_f32(128, 128);
        constexpr uint32_t idesc_pv = umma::idesc_bf16_f32_bmn(128, 128);
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xffffffffu, tc_wait(bar, parity, abort, a.status));
        };
        auto ready = [&](const Ring<C::kOps> &at) {
            return (C::k8 || wait(&ctl->op_full[at.slot], at.phase)) && wait(&ctl->op_ready[at.slot], at.phase);
        };
        // scores b = row half m of Q times the tile at `at`; the last to read the tile frees it
        auto scores = [&](const Ring<C::kOps> &at, int b, int m, bool last) {
            const uint64_t q0 = umma::desc_kmajor_sw128(smem_u32(smem) + (uint32_t)m * kTile);
            const uint64_t k0 = umma::desc_kmajor_sw128(smem_u32(ops) + at.slot * kTile);
            umma::fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kTreeHD / 16; ++k) {
                    const uint32_t off = ((uint32_t)(k >> 2) * kHalf + (uint32_t)(k & 3) * 32u) >> 4;
                    umma::mma_bf16(tm + (uint32_t)b * 128u, q0 + off, k0 + off, idesc_s, k != 0);
                }
                umma::commit(&ctl->s_full[b]);
                if (last)
                    umma::commit(&ctl->op_empty[at.slot]);
            }
            __syncwarp();
        };
        // output of row half m (+)= weights b times the tile at `at`; end: the run's last
        auto product = [&](const Ring<C::kOps> &at, int b, int m, bool add, bool last, bool end) {
            const uint64_t v0 = umma::desc_mnmajor_sw128(smem_u32(ops) + at.slot * kTile, kHalf);
            const uint32_t p0 = NM == 2 ? tm + (uint32_t)b * 128u : tm + 384u + (uint32_t)b * 64u;
            umma::fence_after_sync();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kBK / 16; ++k)
                    mma_bf16_ta(tm + 256u + (uint32_t)m * 128u, p0 + (uint32_t)k * 8u,
                                v0 + (uint32_t)k * (16u * 128u >> 4), idesc_pv, add || k != 0);
                umma::commit(&ctl->pv_done[b]);
                if (end)
                    umma::commit(&ctl->o_full[m]);
                if (last)
                    umma::commit(&ctl->op_empty[at.slot]);
            }
            __syncwarp();
        };
        auto weights_ready = [&](int b, int i) {      // the i-th of this run in b
            return wait(&ctl->p_full[b], ((held >> b) + (uint32_t)i) & 1u);
        };
        ok = wait(&ctl->q_full, runs & 1u);
        if (two) {
            // scores of a half's next tile come after the product that reads its
            // weights, which lie over the scores: MMAs complete in order
            Ring<C::kOps> v_at = op_at;
#pragma unroll 1
            for (int t = -1; t < nt && ok; ++t) {
                const bool more = t + 1 < nt;
                const Ring<C::kOps> k_at = op_at;               // K of the next tile, then V of this one
                if (more)
                    op_at.next();
#pragma unroll 1
                for (int m = 0; m < 2 && ok; ++m) {
                    if (t >= 0) {
                        ok = weights_ready(m, t) && (m || ready(v_at = op_at));
                        if (!ok)
                            break;
                        product(v_at, m, m, t > 0, m == 1, !more);
                    }
                    if (more) {
                        ok = m || ready(k_at);
                        if (ok)
                            scores(k_at, m, m, m == 1);
                    }
                }
                if (t >= 0)
                    op_at.next();
            }
        } else {
            // S(0)  S(1) PV(0)  S(2) PV(1) ...: scores t + 1 go where the softmax of t - 1 has read
#pragma unroll 1
            for (int t = -1; t < nt && ok; ++t) {
                if (t + 1 < nt) {
                    ok = ready(op_at);
                    if (!ok)
                        break;
                    scores(op_at, (t + 1) & 1, 0, true);
                    op_at.next();
                }
                if (t >= 0) {
                    ok = weights_ready(t & 1, t >> 1) && ready(op_at);
                    if (!ok)
                        break;
                    product(op_at, t & 1, 0, t > 0, true, t + 1 == nt);
                    op_at.next();
                }
            }
        }
        if (!ok) {
            // every MMA issued so far completes before tensor memory is freed
            if (elect_one())
                umma::commit(&ctl->all_done);
            __syncwarp();
            mbar_wait(&ctl->all_done, 0);
        }
    };

    // ----------------------------------------------------------- softmax
    auto softmax_role = [&] {
        // (references: loaded from shared memory where they are used, not held in registers)
        const int &s = x.s, &dl = x.dl, &nrows = x.nrows, &slot = x.slot, &whole = x.whole;
        const int64_t &row0 = x.row0;
        const int m = NM == 2 ? warp >> 3 : 0, part = (warp >> 2) & 1;    // row half; half of the keys
        if (m >= x.nm)
            return;
        const int cl = x.cl, blk0 = x.blk0, nt = x.nt;
        const bool two = NM == 2 && x.nm == 2;
        const int quad = warp & 3, tl = 32 * quad + lane;     // this thread's lane of tensor memory
        const int r = R == 1 ? 128 * m + tl : tl & (rt - 1);  // row of the run
        const int c0 = tl / (128 / R) * (2 * kMine) + part * kMine;       // first key of the tile
        const uint32_t lanes = (uint32_t)quad << 21;
        const uint32_t to = tmem + 256u + (uint32_t)m * 128u + lanes;
        const int tok = ctl->tok[r];
        const bool any = (r & ~31) < nrows;                   // a live row in this warp
        const float sc = a.scale_log2;
        float *pair = &ctl->pair[part][128 * m + tl], *other = &ctl->pair[part ^ 1][128 * m + tl];
        float mref = -INFINITY, l = 0.f;
#pragma unroll 1
        for (int t = 0; t < nt; ++t) {
            const int b = two ? m : t & 1;
            ok = __all_sync(0xffffffffu, tc_wait(&ctl->s_full[b], ((held >> b) + (uint32_t)(two ? t : t >> 1)) & 1u,
                                                 abort, a.status));
            umma::fence_after_sync();
            const uint32_t ts = tmem + (uint32_t)b * 128u + lanes;
            const int k0 = (blk0 + t) * kBK + c0;
            const auto see = [&](int g) {
                // (kMine 16: the words are those of 32 keys, from an even multiple of 16 on)
                return kMine < 32 ? seen_bits(a, s, tok, k0 & ~31, cl, dl) >> (k0 & 31)
                                  : seen_bits(a, s, tok, k0 + 32 * g, cl, dl);
            };
            constexpr int kCh = NM == 2 || kMine < 32 ? 16 : 32;
            uint32_t pw[kMine / 2];
            float2 w = make_float2(-INFINITY, 0.f);
            float alpha = 1.f;
#pragma unroll 1
            for (bool again = false;; again = true) {
                if (any && ok)
                    w = tile_weights<kMine, kCh>(ts + (uint32_t)c0, sc, mref, pw, k0 + kMine > cl, see);
                // Every thread of the half says whether its reference has to move (or that it
                // gives up); it has read its scores then, so weights may be stored over them.
                if (!softmax_or(m, !ok || (!again && w.x > mref)))
                    break;
                if (softmax_or(m, !ok)) {
                    ok = false;
                    break;
                }
                *pair = w.x;
                softmax_or(m, false);
                const float top = fmaxf(w.x, *other);
                if (top > mref) {
                    // a whole number (of log2 units), so that scaling by the step is exact
                    const float m1 = ceilf(top) + kTreeLag;
                    alpha = m1 - mref <= 126.f ? exp2i((int)(mref - m1)) : 0.f;
                    mref = m1;
                }
                if (t > 0) {
                    // the output so far, half of its columns by each thread of a row
                    if (!two)                          // (two halves: it came before these scores)
                        ok = tc_wait(&ctl->pv_done[b ^ 1], ((held >> (b ^ 1)) + (uint32_t)((t - 1) >> 1)) & 1u,
                                     abort, a.status);
                    ok = __all_sync(0xffffffffu, ok);
                    umma::fence_after_sync();
                    if (ok && __any_sync(0xffffffffu, alpha != 1.f))
#pragma unroll 1
                        for (int g = 2 * part; g < 2 * part + 2; ++g) {
                            float o[32];
                            umma::tmem_ld32(to + 32 * g, o);
                            tmem_ld_wait_for(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] *= alpha;
                            umma::tmem_st32(to + 32 * g, o);
                        }
                }
            }
            if (!ok)
                break;
            l = l * alpha + w.y;
            if (any) {
                const uint32_t tp = (NM == 2 ? ts : tmem + 384u + (uint32_t)b * 64u + lanes) + (uint32_t)(c0 / 2);
                if constexpr (kMine == 16) {
                    tmem_st8(tp, pw);
                } else {
#pragma unroll
                    for (int g = 0; g < kMine / 32; ++g)
                        tmem_st16(tp + 16 * g, pw + 16 * g);
                }
                umma::tmem_st_wait();
            }
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&ctl->p_full[b]);
        }
        if (ok)
            ok = __all_sync(0xffffffffu, tc_wait(&ctl->o_full[m], (o_phase >> m) & 1u, abort, a.status));
        // the row's sum: both threads' parts
        *pair = l;
        ok = !softmax_or(m, !ok);
        if (!ok)
            return;
        l += *other;
        umma::fence_after_sync();
        // what is not finite in the new positions that the row of token row_tok attends, added
        // to its elements d ..
        auto add_bad = [&](int row_tok, int d, auto &o) {
            constexpr int kE = sizeof(o) / sizeof(o[0]);
            if (!*(volatile int *)&ctl->any_bad)
                return;
#pragma unroll 1
            for (int jj = 0; jj < dl; ++jj) {
                if (!((ctl->bad[jj >> 5] >> (jj & 31)) & 1u) || !tree_sees(a, s, row_tok, jj))
                    continue;
                const int64_t p = row0 + cl + jj;
                if constexpr (C::k8) {
                    const float y = a.vs[p * 4 + d / 32] == 255 ? __uint_as_float(0x7fffffffu) : 0.f;
#pragma unroll
                    for (int e = 0; e < kE; ++e)
                        o[e] += y;
                } else {
                    const uint2 *vr = reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(a.v) +
                                                                      p * kTreeHD + d);
#pragma unroll
                    for (int e = 0; e < kE; e += 4) {
                        const uint2 w = vr[e / 4];
                        const float y[4] = {bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y)};
#pragma unroll
                        for (int f = 0; f < 4; ++f)
                            o[e + f] += fabsf(y[f]) <= 3.4e38f ? 0.f : y[f];
                    }
                }
            }
        };
        // (bf16) what is not finite in dims d .. of the run's earlier positions
        bool lost = false;                                    // elements to be made up for, see tree_not_finite
        const auto not_finite = [&](int d, float (&y)[4]) {
            tree_not_finite(static_cast<const __nv_bfloat16 *>(a.v) + (row0 + (int64_t)x.blk0 * kBK) * kTreeHD + d,
                            min((x.blk0 + x.nt) * kBK, x.cl) - x.blk0 * kBK, y);
        };
        const bool live = r < nrows;
        const int64_t at = max(ctl->at[r], 0);
        const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
        float *so = reinterpret_cast<float *>(ops);           // the ring, at rest: [128][kOPitch]
        float2 *sml = reinterpret_cast<float2 *>(so + 128 * kOPitch);   // maximum and sum
        if (any)
#pragma unroll 1
            for (int g = 2 * part; g < 2 * part + 2; ++g) {
                float o[32];
                umma::tmem_ld32(to + 32 * g, o);
                tmem_ld_wait_for(o);
                if (C::k8)                                    // dims back in order
#pragma unroll
                    for (int e = 1; e < 32; e += 4) {
                        const float y = o[e];
                        o[e] = o[e + 1];
                        o[e + 1] = y;
                    }
                if constexpr (R > 1) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4 *>(so + tl * kOPitch + 32 * g + e) =
                            make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                } else if (live) {
                    add_bad(tok, 32 * g, o);
                    if constexpr (!C::k8)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            lost |= o[e] != o[e];
                    if (whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(a.out + at * kTreeHD + g * 32);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            dst[e] = make_uint4(pack_bf16(o[8 * e] * inv, o[8 * e + 1] * inv),
                                                pack_bf16(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                                                pack_bf16(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                                                pack_bf16(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
                    } else {
                        float4 *dst = reinterpret_cast<float4 *>(a.part_o + ((int64_t)slot * rt + r) * kTreeHD +
                                                                 g * 32);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                }
            }
        if (R == 1 && !C::k8 && lost && l > 0.f)
#pragma unroll 1
            for (int d = 64 * part; d < 64 * part + 64; d += 4) {
                float y[4], z[4];
                not_finite(d, y);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    z[e] = y[e];
                add_bad(tok, d, z);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (y[e] != 0.f) {
                        if (whole)
                            a.out[at * kTreeHD + d + e] = __float2bfloat16_rn(z[e] * inv);
                        else
                            a.part_o[((int64_t)slot * rt + r) * kTreeHD + d + e] = z[e];
                    }
            }
        if (R == 1 && live && !whole && part == 0) {
            a.part_ml[(int64_t)slot * rt + r] = make_float2(mref, l);
            if (blk0 == 0)
                a.join_rows[(int64_t)me * rt + r] = (int32_t)at;
        }
        if constexpr (R > 1) {                                // add the copies
            if (part == 0)
                sml[tl] = make_float2(mref, l);
            softmax_or(m, false);
#pragma unroll 1
            for (int row = warp; row < nrows; row += 8) {
                float M = -INFINITY;
#pragma unroll
                for (int c = 0; c < R; ++c)
                    M = fmaxf(M, sml[c * rt + row].x);
                float L = 0.f;
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < R; ++c) {
                    const float2 ml = sml[c * rt + row];
                    const float f = ml.x > -INFINITY ? exp2f(ml.x - M) : (ml.y == 0.f ? 0.f : 1.f);
                    const float4 y = *reinterpret_cast<const float4 *>(so + (c * rt + row) * kOPitch + lane * 4);
                    L += f * ml.y;
                    acc[0] = fmaf(f, y.x, acc[0]);
                    acc[1] = fmaf(f, y.y, acc[1]);
                    acc[2] = fmaf(f, y.z, acc[2]);
                    acc[3] = fmaf(f, y.w, acc[3]);
                }
                if constexpr (!C::k8) {
                    if (L > 0.f && tree_any_nan(acc[0], acc[1], acc[2], acc[3])) {
                        float y[4];
                        not_finite(lane * 4, y);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[e] = y[e] != 0.f ? y[e] : acc[e];
                    }
                }
                add_bad(ctl->tok[row], lane * 4, acc);
                const int64_t row_at = ctl->at[row];
                if (whole) {
                    const float scale = L == 0.f ? 0.f : 1.f / L;
                    reinterpret_cast<uint2 *>(a.out + row_at * kTreeHD)[lane] =
                        make_uint2(pack_bf16(acc[0] * scale, acc[1] * scale),
                                   pack_bf16(acc[2] * scale, acc[3] * scale));
                } else {
                    reinterpret_cast<float4 *>(a.part_o + ((int64_t)slot * rt + row) * kTreeHD)[lane] =
                        make_float4(acc[0], acc[1], acc[2], acc[3]);
                    if (lane == 0) {
                        a.part_ml[(int64_t)slot * rt + row] = make_float2(M, L);
                        if (blk0 == 0)
                            a.join_rows[(int64_t)me * rt + row] = (int32_t)row_at;
                    }
                }
            }
            fence_proxy_async_smem();                         // the ring is written by copies next
        }
        umma::fence_before_sync();
    };

    if (warp >= kMmaWarp) {
        fewer_registers<C::kIssueRegs>();
        if (warp == kMmaWarp) {
            each_run(mma_role);
            umma::fence_after_sync();
            umma::tmem_dealloc(tmem, 512);
        } else if (warp == kCopyWarp) {
            each_run(copy_role);
        } else if (warp == kPlanWarp) {
            plan_role();
        } else {
            each_run([] {});
        }
    } else if (warp >= C::kSoftWarps) {
        fewer_registers<C::kConvRegs>();
        each_run(convert_role);
    } else {
        more_registers<C::kSoftRegs>();
        if (R > 1) {                                  // the weights of a copy for other copies' keys: zero for good
            const uint32_t zero[16] = {};
            if (warp < 4)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    tmem_st16(tmem + 384u + ((uint32_t)warp << 21) + 16 * i, zero);
            umma::tmem_st_wait();
            softmax_or(0, false);
        }
        each_run(softmax_role);
        // zeros of the pairs that are skipped: last, when the CTAs wait for the slowest
        if (warp < 8)
            tree_zero_skipped<256>(a);
    }
    grid_launch_dependents();
}

template <int KIND, int NM, int R>
int tiles_launch(const TreeArgs &a, int n, cudaStream_t s)
{
    using C = Cfg<KIND, NM>;
    constexpr int rt = NM == 2 ? 256 : 128 / R;
    constexpr size_t smem = C::kOffCtl + sizeof(TcCtl<C::kOps, C::kRaw, rt, NM>);
    auto kernel = attn_tree_tiles<KIND, NM, R>;
    CUtensorMap map_k = {}, map_v = {};
    // boxes of 128 rows x 128 bytes: half a bf16 row, or a row of codes (as 64 pairs)
    const uint64_t rows = (uint64_t)a.n_seq * a.n_kv * (uint64_t)a.cap;
    constexpr uint32_t cols = KIND == WIDE_KV_BF16 ? kTreeHD : kTreeHD / 2;
    if (!make_tmap_2d_swz(&map_k, a.k, rows, cols, cols, kBK, 64, 128) ||
        !make_tmap_2d_swz(&map_v, a.v, rows, cols, cols, kBK, 64, 128))
        return WIDE_EUNSUPPORTED;
    if (!raise_smem_limit(reinterpret_cast<const void *>(kernel), smem))
        return WIDE_CUDA_FAIL();
    // the roles' registers come out of what the block is launched with
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, kernel) != cudaSuccess)
        return WIDE_CUDA_FAIL();
    if (attr.numRegs != C::kLaunchRegs)
        return WIDE_EUNSUPPORTED;
    LaunchScope scope(KID_ATTN_TREE_TC, s);
    kernel<<<n, C::kThreads, smem, s>>>(a, map_k, map_v);
    return launch_status();
}

template <int KIND> int tiles_launch_rows(const TreeArgs &a, int rt, int n, cudaStream_t s)
{
    return rt == 32    ? tiles_launch<KIND, 1, 4>(a, n, s)
           : rt == 64  ? tiles_launch<KIND, 1, 2>(a, n, s)
           : rt == 128 ? tiles_launch<KIND, 1, 1>(a, n, s)
                       : tiles_launch<KIND, 2, 1>(a, n, s);
}

}  // namespace

int attn_tree_tiles_launch(const TreeArgs &a, int kind, int rt, int n, cudaStream_t s)
{
    return kind == WIDE_KV_BF16   ? tiles_launch_rows<WIDE_KV_BF16>(a, rt, n, s)
           : kind == WIDE_KV_E4M3 ? tiles_launch_rows<WIDE_KV_E4M3>(a, rt, n, s)
                                  : tiles_launch_rows<WIDE_KV_I8>(a, rt, n, s);
}

}  // namespace wide
