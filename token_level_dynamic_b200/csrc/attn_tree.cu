// attn_tree.cu -- wide_attn_tree: attention of several new tokens per
// sequence over the KV cache, in bf16 or 8 bits (formula in wide.h).
//
// With few rows the kernel is bound by reading the cache once: 512 B per key
// and head group in bf16, 264 B in 8 bits.  attn_tree_rows takes 16 rows at a
// time on mma.sync: every warp owns its own keys, loads them from global
// memory straight into the matrix instructions' operand registers and keeps
// its own running maximum, sum and output, so the loop has no barrier and a
// warp always has its next keys and values in flight.
//   S = Q K^T   m16n8k16.  The order of the 128 dims along k is free as long
//               as Q and K agree, so a lane's 16-byte loads are its operands:
//               lane (g = lane / 4, c = lane % 4) reads 16 bytes of key row g
//               per four (bf16) or eight (8-bit) of its operand registers.
//   O += P V    the order of the output dims over the n index is free too:
//               lane (g, c) reads 16 bytes of the value rows 2c, 2c + 1,
//               2c + 8, 2c + 9 and pairs the rows up by byte permutes.
// 8-bit codes become bf16 in registers, exactly: two or three integer and two
// half-rate float operations per two elements, the scale's multiplication among
// them.
#include "attn_tree.cuh"
#include "host.h"
#include "kv.cuh"

namespace wide {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kRows = 16;              // rows of a run
constexpr int kRunCost = 2;            // blocks' time that a run costs beside its blocks
constexpr int kOPitch = kTreeHD + 4;   // floats; row pitch of the warps' outputs when merged

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int KIND> struct TreeCfg {
    static constexpr bool k8 = KIND != WIDE_KV_BF16;
    static constexpr int kPW = k8 ? 32 : 16;          // keys of a warp per step
    static constexpr int kBK = kWarps * kPW;          // keys of a block
    static constexpr int kNT = kPW / 8, kNG = kPW / 16;
    static constexpr int kKC = k8 ? 2 : 4;            // 16-byte pieces of a key row per lane
    static constexpr int kVC = k8 ? 1 : 2;            // ... of a value row
    static constexpr int kRowB = kTreeHD * (k8 ? 1 : 2);
};

// A warp's next keys and values, as loaded.
template <int KIND> struct TreeTile {
    using C = TreeCfg<KIND>;
    uint4 k[C::kNT][C::kKC];
    uint4 v[C::kNG][4][C::kVC];
    uint32_t ks[C::k8 ? C::kNT : 1];                  // the rows' four scale bytes
    uint32_t vs[C::k8 ? C::kNG : 1];                  // scale bytes of the four rows' piece

    __device__ void load_k(const uint8_t *base, const uint8_t *scales, int p0, int last, int lane)
    {
        const int g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int n = 0; n < C::kNT; ++n) {
            const int64_t p = min(p0 + n * 8 + g, last);
            const uint8_t *r = base + p * C::kRowB + c * 16;
#pragma unroll
            for (int i = 0; i < C::kKC; ++i)
                k[n][i] = load_stream(r + i * 64);
            if constexpr (C::k8)
                ks[n] = __ldg(reinterpret_cast<const uint32_t *>(scales) + p);
        }
    }
    __device__ void load_v(const uint8_t *base, const uint8_t *scales, int p0, int last, int lane)
    {
        const int g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int n = 0; n < C::kNG; ++n) {
            uint32_t w = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t p = min(p0 + n * 16 + 2 * c + (i & 1) + 8 * (i >> 1), last);
                const uint8_t *r = base + p * C::kRowB + g * 16;
#pragma unroll
                for (int h = 0; h < C::kVC; ++h)
                    v[n][i][h] = load_stream(r + h * 128);
                if constexpr (C::k8)
                    w |= (uint32_t)__ldg(scales + p * 4 + (g >> 1)) << (8 * i);
            }
            if constexpr (C::k8)
                vs[n] = w;
        }
    }
};

template <int KIND>
__global__ void __launch_bounds__(kThreads, 2) attn_tree_rows(const TreeArgs a)
{
    using C = TreeCfg<KIND>;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;
    const int U = a.n_seq * a.n_kv;
    float *so = reinterpret_cast<float *>(smem);                       // [kWarps][kRows][kOPitch]
    uint32_t *cum = reinterpret_cast<uint32_t *>(so + kWarps * kRows * kOPitch);
    uint16_t *cnt = reinterpret_cast<uint16_t *>(cum + U + 1);
    __shared__ float2 sml[kWarps][kRows];
    __shared__ int32_t stok[kRows];                                    // token of each row, -1: none
    __shared__ int32_t slist[kRows];
    __shared__ uint32_t sbad[kTreeMaxDraft / 32];                      // new positions with a value that is not finite
    __shared__ int s_any_bad;
    __shared__ uint32_t spart[kWarps];

    tree_zero_skipped<kThreads>(a);
    tree_plan<kThreads>(a, kRows, C::kBK, kRunCost, cum, cnt, spart);
    const uint32_t total = cum[U];
    const int n_cta = (int)min((uint32_t)gridDim.x, total);
    const int me = (int)blockIdx.x;
    if (me >= n_cta) {
        if (tid == 0)
            a.joins[me] = make_int4(0, 0, 0, 0);
        return;
    }
    const TreeShare share(total, (uint32_t)n_cta);
    const uint32_t first = share.first(me), end = share.first(me + 1);
    bool joined = false;
    const float sc = a.scale_log2;
    // (int8) this lane's scale byte of a key row's first 16-byte piece, in both halves
    const uint32_t k_sel = 0x4040u + 0x0101u * (uint32_t)(c >> 1);

    for (uint32_t b = first; b < end;) {
        const int u = tree_unit(cum, U, b);
        const int s = u / a.n_kv, j = u - s * a.n_kv;
        const int2 len = tree_lens(a, s, false);
        const int nkeys = len.x + len.y;
        const int nb = (nkeys + C::kBK - 1) / C::kBK, per = nb + kRunCost;
        const int run = (int)(b - cum[u]) / per;
        const int pos = (int)(b - cum[u]) - run * per;
        const int stop = (int)min((uint32_t)per, (uint32_t)pos + (end - b));
        b += (uint32_t)(stop - pos);
        const int blk0 = max(pos - kRunCost, 0), blk1 = max(stop - kRunCost, 0);
        if (blk0 == blk1)
            continue;
        const int nrows = min(kRows, (int)cnt[u] * a.rep - run * kRows);

        // rows of the run: their tokens
        const int t_lo = run * kRows / a.rep, t_hi = (run * kRows + nrows - 1) / a.rep + 1;
        __syncthreads();                       // the last segment's shared memory is read
        if (warp == 0)
            tree_tokens(a, s, j, len.y, t_lo, t_hi, slist);
        if (tid < kTreeMaxDraft / 32)
            sbad[tid] = 0;
        if (tid == 0)
            s_any_bad = 0;
        __syncthreads();
        if (tid < kRows)
            stok[tid] = tid < nrows ? slist[(run * kRows + tid) / a.rep - t_lo] : -1;
        __syncthreads();

        // Q operands: rows g and g + 8
        uint32_t qf[8][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = g + 8 * h, tok = stok[r];
            const int head = j * a.rep + (run * kRows + r) % a.rep;
            const __nv_bfloat16 *qr = a.q + ((int64_t)s * a.draft + max(tok, 0)) * a.q_stride +
                                      (int64_t)head * kTreeHD;
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // 8 elements: two k steps (bf16 order) or half a piece (8-bit order)
                const int d = C::k8 ? (i >> 1) * 64 + c * 16 + (i & 1) * 8 : i * 32 + c * 8;
                const uint4 w = tok >= 0 ? *reinterpret_cast<const uint4 *>(qr + d) : zero;
                // 8 bits: elements 0 2 and 1 3 of each four together, as the codes come
                qf[2 * i][h] = C::k8 ? __byte_perm(w.x, w.y, 0x5410) : w.x;
                qf[2 * i][2 + h] = C::k8 ? __byte_perm(w.x, w.y, 0x7632) : w.y;
                qf[2 * i + 1][h] = C::k8 ? __byte_perm(w.z, w.w, 0x5410) : w.z;
                qf[2 * i + 1][2 + h] = C::k8 ? __byte_perm(w.z, w.w, 0x7632) : w.w;
            }
        }
        const int tok0 = stok[g], tok1 = stok[g + 8];

        const int64_t row0 = ((int64_t)s * a.n_kv + j) * a.cap;
        const uint8_t *kb = static_cast<const uint8_t *>(a.k) + row0 * C::kRowB;
        const uint8_t *vb = static_cast<const uint8_t *>(a.v) + row0 * C::kRowB;
        const uint8_t *ksb = C::k8 ? a.ks + row0 * 4 : nullptr;
        const uint8_t *vsb = C::k8 ? a.vs + row0 * 4 : nullptr;

        float o[16][4];
#pragma unroll
        for (int n = 0; n < 16; ++n)
            o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

        TreeTile<KIND> t;
        int p0 = blk0 * C::kBK + warp * C::kPW;        // this warp's keys of the block
        if (p0 < nkeys) {
            t.load_k(kb, ksb, p0, nkeys - 1, lane);
            t.load_v(vb, vsb, p0, nkeys - 1, lane);
        }
        for (int blk = blk0; blk < blk1 && p0 < nkeys; ++blk, p0 += C::kBK) {
            const bool more = blk + 1 < blk1 && p0 + C::kBK < nkeys;
            // ---- scores
            float sv[C::kNT][4];
#pragma unroll
            for (int n = 0; n < C::kNT; ++n) {
                sv[n][0] = sv[n][1] = sv[n][2] = sv[n][3] = 0.f;
                if constexpr (C::k8) {
                    const bool big = KIND == WIDE_KV_E4M3 &&
                                     __any_sync(0xffffffffu, __vmaxu4(t.ks[n], 0x86868686u) != 0x86868686u);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t sb = (t.ks[n] >> (16 * i + 8 * (c >> 1))) & 255u;
                        const uint32_t m = KIND == WIDE_KV_I8
                                               ? kv_mult2<KIND>(__byte_perm(t.ks[n], 0u, k_sel + 0x0202u * i))
                                               : kv_mult<KIND>(sb) * 0x00010001u;
                        const uint32_t mh = kv_mult_high(sb) * 0x00010001u;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t w = word(t.k[n][i], e);
                            uint32_t b0, b1;
                            kv_pairs_0213<KIND>(w, m, a.opaque, b0, b1);
                            if (KIND == WIDE_KV_E4M3 && big) {
                                b0 = mul_bf16x2(b0, mh);
                                b1 = mul_bf16x2(b1, mh);
                            }
                            mma16816(sv[n], qf[4 * i + e], b0, b1);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        mma16816(sv[n], qf[2 * i], t.k[n][i].x, t.k[n][i].y);
                        mma16816(sv[n], qf[2 * i + 1], t.k[n][i].z, t.k[n][i].w);
                    }
                }
            }
            if (more)
                t.load_k(kb, ksb, p0 + C::kBK, nkeys - 1, lane);

            // ---- masks: only blocks that reach the new tokens or the end
            const bool tail = p0 + C::kPW > len.x;
            if (tail) {
#pragma unroll
                for (int n = 0; n < C::kNT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int jj = p0 + n * 8 + 2 * c + (e & 1) - len.x;
                        const int tok = e < 2 ? tok0 : tok1;
                        if (jj >= 0 && (jj >= len.y || tok < 0 || !tree_sees(a, s, tok, jj)))
                            sv[n][e] = -INFINITY;
                    }
                // values of new positions that are not finite leave the product
                // (0 * NaN would reach rows that do not attend them) and are
                // added to the rows that do at the end
#pragma unroll
                for (int n = 0; n < C::kNG; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int jj = p0 + n * 16 + 2 * c + (i & 1) + 8 * (i >> 1) - len.x;
                        if (jj < 0)
                            continue;
                        bool bad = false;
                        if constexpr (C::k8) {
                            if (((t.vs[n] >> (8 * i)) & 255u) == 255u) {
                                bad = true;
                                t.vs[n] &= ~(255u << (8 * i));       // zero codes, scale 0
                            }
                        } else {
#pragma unroll
                            for (int h = 0; h < C::kVC; ++h) {
                                uint32_t *w = reinterpret_cast<uint32_t *>(&t.v[n][i][h]);
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    if ((w[e] & 0x7f80u) == 0x7f80u) {
                                        w[e] &= 0xffff0000u;
                                        bad = true;
                                    }
                                    if ((w[e] & 0x7f800000u) == 0x7f800000u) {
                                        w[e] &= 0x0000ffffu;
                                        bad = true;
                                    }
                                }
                            }
                        }
                        if (bad && jj < len.y) {
                            atomicOr(&sbad[jj >> 5], 1u << (jj & 31));
                            s_any_bad = 1;
                        }
                    }
            }

            // ---- reference of the weights (log2 units): 8 above the maximum when it
            // moves, which it does only when the maximum passes it, so rescaling is
            // rare and no weight is above 1
            float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
            for (int n = 0; n < C::kNT; ++n) {
                x0 = fmaxf(x0, fmaxf(sv[n][0], sv[n][1]));
                x1 = fmaxf(x1, fmaxf(sv[n][2], sv[n][3]));
            }
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2)) * sc;
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2)) * sc;
            if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
                float a0 = 1.f, a1 = 1.f;
                if (x0 > m0) {
                    x0 += kTreeLag;
                    a0 = exp2f(m0 - x0);
                    m0 = x0;
                }
                if (x1 > m1) {
                    x1 += kTreeLag;
                    a1 = exp2f(m1 - x1);
                    m1 = x1;
                }
                l0 *= a0;
                l1 *= a1;
#pragma unroll
                for (int n = 0; n < 16; ++n) {
                    o[n][0] *= a0;
                    o[n][1] *= a0;
                    o[n][2] *= a1;
                    o[n][3] *= a1;
                }
            }
            const float mb0 = m0 > -INFINITY ? m0 : 0.f, mb1 = m1 > -INFINITY ? m1 : 0.f;
            uint32_t pf[C::kNG][4];
#pragma unroll
            for (int n = 0; n < C::kNT; ++n) {
                const float e0 = exp2_sfu(fmaf(sv[n][0], sc, -mb0)),
                            e1 = exp2_sfu(fmaf(sv[n][1], sc, -mb0)),
                            e2 = exp2_sfu(fmaf(sv[n][2], sc, -mb1)),
                            e3 = exp2_sfu(fmaf(sv[n][3], sc, -mb1));
                l0 += e0 + e1;
                l1 += e2 + e3;
                pf[n >> 1][2 * (n & 1)] = pack_bf16(e0, e1);
                pf[n >> 1][2 * (n & 1) + 1] = pack_bf16(e2, e3);
            }

            // ---- O += P V
#pragma unroll
            for (int n = 0; n < C::kNG; ++n) {
                if constexpr (C::k8) {
                    const uint32_t m01 = kv_mult2<KIND>(__byte_perm(t.vs[n], 0u, 0x4140));
                    const uint32_t m23 = kv_mult2<KIND>(__byte_perm(t.vs[n], 0u, 0x4342));
                    const bool big = KIND == WIDE_KV_E4M3 &&
                                     __any_sync(0xffffffffu, __vmaxu4(t.vs[n], 0x86868686u) != 0x86868686u);
                    const uint32_t h01 = kv_mult_high(t.vs[n] & 255u) |
                                         kv_mult_high((t.vs[n] >> 8) & 255u) << 16;
                    const uint32_t h23 = kv_mult_high((t.vs[n] >> 16) & 255u) |
                                         kv_mult_high(t.vs[n] >> 24) << 16;
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        // byte e of the four rows; e4m3 wants it high in each half, i8 low
                        const int q = e & 3;
                        const uint32_t sel = KIND == WIDE_KV_E4M3 ? (uint32_t)((4 + q) << 12 | q << 4)
                                                                  : (uint32_t)((4 + q) << 8 | q);
                        uint32_t b0 = kv_pair<KIND>(__byte_perm(word(t.v[n][0][0], e >> 2),
                                                                word(t.v[n][1][0], e >> 2), sel), m01, a.opaque);
                        uint32_t b1 = kv_pair<KIND>(__byte_perm(word(t.v[n][2][0], e >> 2),
                                                                word(t.v[n][3][0], e >> 2), sel), m23, a.opaque);
                        if (big) {
                            b0 = mul_bf16x2(b0, h01);
                            b1 = mul_bf16x2(b1, h23);
                        }
                        mma16816(o[e], pf[n], b0, b1);
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint32_t sel = e & 1 ? 0x7632 : 0x5410;
                            const uint32_t b0 = __byte_perm(word(t.v[n][0][h], e >> 1),
                                                            word(t.v[n][1][h], e >> 1), sel);
                            const uint32_t b1 = __byte_perm(word(t.v[n][2][h], e >> 1),
                                                            word(t.v[n][3][h], e >> 1), sel);
                            mma16816(o[8 * h + e], pf[n], b0, b1);
                        }
                }
            }
            if (more)
                t.load_v(vb, vsb, p0 + C::kBK, nkeys - 1, lane);
        }

        // ---- merge the warps' outputs
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        if (c == 0) {
            sml[warp][g] = make_float2(m0, l0);
            sml[warp][g + 8] = make_float2(m1, l1);
        }
        // dims of o[n][e]: bf16 64 (n / 8) + 8 (2c + e % 2) + n % 8, 8-bit 16 (2c + e % 2) + n
#pragma unroll
        for (int n = 0; n < 16; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = C::k8 ? 16 * (2 * c + (e & 1)) + n
                                    : 64 * (n >> 3) + 8 * (2 * c + (e & 1)) + (n & 7);
                so[(warp * kRows + g + 8 * (e >> 1)) * kOPitch + d] = o[n][e];
            }
        __syncthreads();
        const bool whole = blk0 == 0 && blk1 == nb;
        const int slot = 2 * me + (blk0 == 0);
        if (!whole && blk0 == 0) {              // the run starts here: record its extent
            joined = true;
            if (tid == 0)
                a.joins[me] = make_int4(
                    share.owner(cum[u] + (uint32_t)(run + 1) * per - 1), slot, nrows, 0);
            if (tid < nrows)
                a.join_rows[me * kRows + tid] = (int32_t)(((int64_t)s * a.draft + stok[tid]) * a.n_q +
                                                          j * a.rep + (run * kRows + tid) % a.rep);
        }
        for (int r = warp; r < nrows; r += kWarps) {
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                M = fmaxf(M, sml[w][r].x);
            float L = 0.f, f[kWarps];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 ml = sml[w][r];
                f[w] = ml.x > -INFINITY ? exp2f(ml.x - M) : (ml.y == 0.f ? 0.f : 1.f);
                L += f[w] * ml.y;
            }
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 x = *reinterpret_cast<const float4 *>(
                    so + (w * kRows + r) * kOPitch + lane * 4);
                acc.x = fmaf(f[w], x.x, acc.x);
                acc.y = fmaf(f[w], x.y, acc.y);
                acc.z = fmaf(f[w], x.z, acc.z);
                acc.w = fmaf(f[w], x.w, acc.w);
            }
            const int tok = stok[r];
            if constexpr (!C::k8) {
                if (L > 0.f && tree_any_nan(acc.x, acc.y, acc.z, acc.w)) {
                    const int from = blk0 * C::kBK, n = min(blk1 * C::kBK, len.x) - from;
                    float y[4];
                    tree_not_finite(reinterpret_cast<const __nv_bfloat16 *>(vb + (int64_t)from * C::kRowB) + lane * 4,
                                    n, y);
                    acc.x = y[0] != 0.f ? y[0] : acc.x;
                    acc.y = y[1] != 0.f ? y[1] : acc.y;
                    acc.z = y[2] != 0.f ? y[2] : acc.z;
                    acc.w = y[3] != 0.f ? y[3] : acc.w;
                }
            }
            if (s_any_bad) {
                // infinities and NaNs of the new positions this row attends
                for (int jj = 0; jj < len.y; ++jj) {
                    if (!((sbad[jj >> 5] >> (jj & 31)) & 1u) || !tree_sees(a, s, tok, jj))
                        continue;
                    const int64_t p = len.x + jj;
                    float v[4];
                    if constexpr (C::k8) {
                        v[0] = v[1] = v[2] = v[3] =
                            vsb[p * 4 + (lane >> 3)] == 255 ? __uint_as_float(0x7fffffffu) : 0.f;
                    } else {
                        const __nv_bfloat16 *vr =
                            reinterpret_cast<const __nv_bfloat16 *>(vb + p * C::kRowB) + lane * 4;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = __bfloat162float(vr[e]);
                            v[e] = fabsf(x) <= 3.4e38f ? 0.f : x;
                        }
                    }
                    acc.x += v[0];
                    acc.y += v[1];
                    acc.z += v[2];
                    acc.w += v[3];
                }
            }
            if (whole) {
                const float inv = L == 0.f ? 0.f : 1.f / L;
                const int64_t at = ((int64_t)s * a.draft + tok) * a.n_q + j * a.rep +
                                   (run * kRows + r) % a.rep;
                reinterpret_cast<uint2 *>(a.out + at * kTreeHD)[lane] =
                    make_uint2(pack_bf16(acc.x * inv, acc.y * inv),
                               pack_bf16(acc.z * inv, acc.w * inv));
            } else {
                reinterpret_cast<float4 *>(a.part_o + ((int64_t)slot * kRows + r) * kTreeHD)[lane] = acc;
                if (lane == 0)
                    a.part_ml[(int64_t)slot * kRows + r] = make_float2(M, L);
            }
        }
    }
    if (!joined && tid == 0)
        a.joins[me] = make_int4(0, 0, 0, 0);
    grid_launch_dependents();
}

// Adds the parts of the run that starts in CTA blockIdx.x.  Bound by the
// latency of its few reads (rows * parts * 512 bytes, most of them in L2), so a
// row's parts are shared out to several warps where there are few rows; always
// in the same order.
template <int ROWS> struct JoinCfg {
    static constexpr int kPer = ROWS >= 256 ? 1 : ROWS >= 128 ? 2 : 4;   // warps of a row
    static constexpr int kRowsPerBlock = 8 / kPer;
    // Registers for this many blocks on an SM, 32 and 40.  With the 56 that the
    // compiler takes for its unrolled loop the calls of 8 trees of 61 in bf16
    // are 69.2 instead of 68.4 us, of 16 trees of 8 in e4m3 43.7 instead of 42.8,
    // of 29 ragged ones in int8 83.3 instead of 82.3; one token over 2048 bf16
    // keys is 10.0 instead of 11.2.
    static constexpr int kBlocksPerSm = ROWS >= 256 ? 7 : 6;
};
template <int ROWS>
__global__ void __launch_bounds__(256, JoinCfg<ROWS>::kBlocksPerSm)
    attn_tree_join(const float *part_o, const float2 *part_ml, const int4 *joins,
                   const int32_t *join_rows, __nv_bfloat16 *out)
{
    using C = JoinCfg<ROWS>;
    __shared__ float4 sacc[8][32];
    grid_dependency_wait();
    const int c0 = (int)blockIdx.x, lane = threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
    const int4 jn = joins[c0];
    const int r0 = (int)blockIdx.y * C::kRowsPerBlock;
    if (r0 >= jn.z)
        return;
    const int r = min(r0 + warp / C::kPer, jn.z - 1), sub = warp % C::kPer;
    const int parts = jn.x - c0 + 1;
    // part 0 is in its CTA's second slot, the others in their CTAs' first
    auto at_of = [&](int i) { return (int64_t)(i ? 2 * (c0 + i) : jn.y) * ROWS + r; };
    float M = -INFINITY;
    for (int i = lane; i < parts; i += 32)
        M = fmaxf(M, part_ml[at_of(i)].x);
#pragma unroll
    for (int off = 16; off; off >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    auto scale_of = [&](float2 ml) { return ml.x > -INFINITY ? exp2f(ml.x - M) : (ml.y == 0.f ? 0.f : 1.f); };
    float L = 0.f;
    for (int i = lane; i < parts; i += 32) {
        const float2 ml = part_ml[at_of(i)];
        L += scale_of(ml) * ml.y;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1)
        L += __shfl_xor_sync(0xffffffffu, L, off);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = sub; i < parts; i += C::kPer) {
        const float4 x = reinterpret_cast<const float4 *>(part_o + at_of(i) * kTreeHD)[lane];
        const float f = scale_of(part_ml[at_of(i)]);
        acc.x = fmaf(f, x.x, acc.x);
        acc.y = fmaf(f, x.y, acc.y);
        acc.z = fmaf(f, x.z, acc.z);
        acc.w = fmaf(f, x.w, acc.w);
    }
    if constexpr (C::kPer > 1) {
        sacc[warp][lane] = acc;
        __syncthreads();
        if (sub)
            return;
        for (int i = 1; i < C::kPer; ++i) {
            const float4 x = sacc[warp + i][lane];
            acc.x += x.x;
            acc.y += x.y;
            acc.z += x.z;
            acc.w += x.w;
        }
    }
    if (r0 + warp / C::kPer >= jn.z)
        return;
    if (L > 0.f && tree_any_nan(acc.x, acc.y, acc.z, acc.w)) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int i = 0; i < parts; ++i) {
            const float4 x = reinterpret_cast<const float4 *>(part_o + at_of(i) * kTreeHD)[lane];
            y.x += tree_inf_or_0(x.x);
            y.y += tree_inf_or_0(x.y);
            y.z += tree_inf_or_0(x.z);
            y.w += tree_inf_or_0(x.w);
        }
        acc.x = y.x != 0.f ? y.x : acc.x;
        acc.y = y.y != 0.f ? y.y : acc.y;
        acc.z = y.z != 0.f ? y.z : acc.z;
        acc.w = y.w != 0.f ? y.w : acc.w;
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    reinterpret_cast<uint2 *>(out + (int64_t)join_rows[c0 * ROWS + r] * kTreeHD)[lane] =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
}

// ------------------------------------------------------------------- host

struct TreeWs {
    float *part_o;
    float2 *part_ml;
    int4 *joins;
    int32_t *join_rows;
    size_t total;
};

TreeWs tree_ws(int n, int rows, void *base)
{
    TreeWs w = {};
    char *p = static_cast<char *>(base);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char *at = p ? p + off : nullptr;
        off += align_up(bytes, 256);
        return at;
    };
    w.part_o = reinterpret_cast<float *>(take((size_t)2 * n * rows * kTreeHD * 4));
    w.part_ml = reinterpret_cast<float2 *>(take((size_t)2 * n * rows * 8));
    w.joins = reinterpret_cast<int4 *>(take((size_t)n * 16));
    w.join_rows = reinterpret_cast<int32_t *>(take((size_t)n * rows * 4));
    w.total = off;
    return w;
}

// The GPU's SM count (workspace sizes depend on it; without a GPU, B200's).
int sm_count()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        n = 148;
    }
    return n;
}

constexpr int kCtasPerSm = 2;          // of attn_tree_rows

// Which kernel takes the call: rows of a run and CTAs.  attn_tree_rows starts
// faster, attn_tree_tiles reads and converts the cache once for up to 256 rows.
// Measured (us; rows kernel against tiles kernel; units x keys, bf16; int8 differs
// by up to 16% and in no choice but that of 64 rows over 32 x 512, where both take 19):
//   up to 16 rows: one token over 8 x 2048 keys 14 against 18, 29 ragged
//     sequences in int8 80 against 100;
//   32 rows: 8 x 512 keys 12 against 15, 32 x 2000 20 against 20, 32 x 8000 50
//     against 36; 64 rows: 32 x 512 18 against 19, 32 x 2000 28 against 25;
//   128 rows: 32 x 128 16 against 20, 32 x 512 24 against 22; 256 rows: 8 x 512
//     19 against 29, 32 x 512 37 against 31, 128 x 8000 1227 against 214.
// So the rows kernel takes up to 16 rows, and where its blocks of 16 rows and
// 128 keys (with every sequence as long as the cache, the lengths being on the
// device) are few: up to 256, and 5 more for each row of a run of the other.
struct TreeChoice {
    int rt, n;
};
TreeChoice tree_choice(const wide_kv_cache *c, const wide_attn_tree_dims *d)
{
    const int64_t rows = d->draft * (d->n_q / c->n_kv);
    const int rt = rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 256;
    const int64_t blocks = c->n_seq * c->n_kv * ((rows + kRows - 1) / kRows) * ((c->cap + 127) / 128);
    if (rows <= kRows || blocks <= 256 + 5 * rt)
        return {kRows, kCtasPerSm * sm_count()};
    return {rt, sm_count()};
}

int tree_check(const wide_kv_cache *c, const wide_attn_tree_dims *d)
{
    // (the kernels multiply by scale * log2(e))
    if (!d || d->draft < 1 || d->n_q <= 0 || d->q_token_stride < 0 || !(d->scale > 0.f) ||
        !isfinite(d->scale * kLog2e))
        return WIDE_EINVAL;
    if (int rc = kv_cache_check(c))
        return rc;
    if (d->n_q % c->n_kv != 0)
        return WIDE_EINVAL;
    if (d->draft > kTreeMaxDraft || d->n_q / c->n_kv > kTreeMaxRep ||
        c->n_seq * c->n_kv > kTreeMaxUnits || d->q_token_stride % 8 != 0)
        return WIDE_EUNSUPPORTED;
    static_assert((int64_t)kTreeMaxUnits * kTreeMaxRep * kTreeMaxDraft <= 0x7fffffff, "output rows are counted in 32 bits");
    const int64_t rows = d->draft * (d->n_q / c->n_kv);
    if (// a cache row is a 32-bit coordinate of a copy
        c->n_seq * c->n_kv * c->cap > (int64_t)0x7fffffff ||
        // the work's places are counted in 32 bits
        c->n_seq * c->n_kv * ((rows + kRows - 1) / kRows) * (c->cap / 32 + 3) > (int64_t)0x7fffffff)
        return WIDE_EUNSUPPORTED;
    return WIDE_OK;
}

template <int KIND>
int tree_rows_launch(const TreeArgs &a, int n, cudaStream_t s)
{
    const int U = a.n_seq * a.n_kv;
    const size_t smem = (size_t)kWarps * kRows * kOPitch * 4 + (size_t)(U + 1) * 4 + (size_t)U * 2;
    if (!raise_smem_limit(reinterpret_cast<const void *>(attn_tree_rows<KIND>), smem))
        return WIDE_CUDA_FAIL();
    LaunchScope scope(KID_ATTN_TREE, s);
    attn_tree_rows<KIND><<<n, kThreads, smem, s>>>(a);
    return launch_status();
}

template <int ROWS> int tree_join_launch(const TreeArgs &a, int n, cudaStream_t s)
{
    // launched while the attention still runs; it waits for it on the device
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n, (ROWS + JoinCfg<ROWS>::kRowsPerBlock - 1) / JoinCfg<ROWS>::kRowsPerBlock);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    LaunchScope scope(KID_ATTN_TREE_JOIN, s);
    if (cudaLaunchKernelEx(&cfg, attn_tree_join<ROWS>, (const float *)a.part_o,
                           (const float2 *)a.part_ml, (const int4 *)a.joins,
                           (const int32_t *)a.join_rows, a.out) != cudaSuccess)
        return WIDE_CUDA_FAIL();
    return WIDE_OK;
}

}  // namespace
}  // namespace wide

using namespace wide;

extern "C" {

size_t wide_attn_tree_workspace_bytes(const wide_kv_cache *cache, const wide_attn_tree_dims *d)
{
    if (tree_check(cache, d) != WIDE_OK)
        return 0;
    const TreeChoice ch = tree_choice(cache, d);
    return tree_ws(ch.n, ch.rt, nullptr).total;
}

int wide_attn_tree(const void *d_q, const wide_kv_cache *cache, const int32_t *d_cache_len,
                   const int32_t *d_draft_len, const uint32_t *d_tree_mask,
                   const uint32_t *d_head_mask, void *d_out, const wide_attn_tree_dims *d,
                   void *d_workspace, size_t workspace_bytes, void *stream)
{
    if (int rc = tree_check(cache, d))
        return rc;
    if (cache->n_seq == 0)
        return WIDE_OK;
    if (!d_q || !d_cache_len || !d_out || !d_workspace)
        return WIDE_EINVAL;
    if (d->q_token_stride < (int64_t)d->n_q * kTreeHD && cache->n_seq * d->draft > 1)
        return WIDE_EINVAL;
    const void *al4[] = {d_cache_len, d_draft_len, d_tree_mask, d_head_mask};
    for (const void *p : al4)
        if (reinterpret_cast<uintptr_t>(p) & 3u)
            return WIDE_EUNSUPPORTED;
    if (!aligned16(d_q) || !aligned16(d_out) || (reinterpret_cast<uintptr_t>(d_workspace) & 255u))
        return WIDE_EUNSUPPORTED;
    const TreeChoice ch = tree_choice(cache, d);
    const TreeWs w = tree_ws(ch.n, ch.rt, d_workspace);
    if (workspace_bytes < w.total)
        return WIDE_EWORKSPACE;
    TreeArgs a = {};
    a.q = static_cast<const __nv_bfloat16 *>(d_q);
    a.k = cache->k;
    a.v = cache->v;
    a.ks = cache->k_scale;
    a.vs = cache->v_scale;
    a.cache_len = d_cache_len;
    a.draft_len = d_draft_len;
    a.tree = d_tree_mask;
    a.heads = d_head_mask;
    a.out = static_cast<__nv_bfloat16 *>(d_out);
    a.n_seq = (int)cache->n_seq;
    a.draft = (int)d->draft;
    a.n_q = d->n_q;
    a.n_kv = cache->n_kv;
    a.rep = d->n_q / cache->n_kv;
    a.Wt = (a.draft + 31) / 32;
    a.Wh = (a.n_kv + 31) / 32;
    a.cap = cache->cap;
    a.q_stride = d->q_token_stride;
    a.scale_log2 = d->scale * kLog2e;
    a.opaque = kv_opaque(cache->kind);
    a.part_o = w.part_o;
    a.part_ml = w.part_ml;
    a.joins = w.joins;
    a.join_rows = w.join_rows;
    a.status = status_ptr();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (ch.rt != kRows) {
        if (int rc = attn_tree_tiles_launch(a, cache->kind, ch.rt, ch.n, s))
            return rc;
        return ch.rt == 32    ? tree_join_launch<32>(a, ch.n, s)
               : ch.rt == 64  ? tree_join_launch<64>(a, ch.n, s)
               : ch.rt == 128 ? tree_join_launch<128>(a, ch.n, s)
                              : tree_join_launch<256>(a, ch.n, s);
    }
    const int rc = cache->kind == WIDE_KV_BF16   ? tree_rows_launch<WIDE_KV_BF16>(a, ch.n, s)
                   : cache->kind == WIDE_KV_E4M3 ? tree_rows_launch<WIDE_KV_E4M3>(a, ch.n, s)
                                                 : tree_rows_launch<WIDE_KV_I8>(a, ch.n, s);
    if (rc)
        return rc;
    return tree_join_launch<kRows>(a, ch.n, s);
}

}  // extern "C"
