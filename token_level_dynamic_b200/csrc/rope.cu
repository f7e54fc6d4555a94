// rope.cu -- wide_rope: the rotation of the first rot_dim elements of every
// head by its token's position (formula in wide.h).
//
// Each element is read and written once, so the kernel is bound by memory
// (at small token counts by its launch).  A CTA takes a few tokens: its
// threads first compute the tokens' (cos, sin) pairs into shared memory, each
// once for all heads (the double product and the reduction to one turn cost
// more than rotating a pair, and a token of 40 heads uses every angle 40
// times), then rotate.  rope_pieces, for rows made of aligned 16-byte pieces:
// a thread keeps its place within a head (16 bytes of the a elements and 16 of
// the b elements, 16 of whole pairs, or 16 to copy) and walks through the rows,
// two at a time, without a division; the angles lie so that neighbouring
// threads read neighbouring 16 bytes (read as pairs of a thread, 64 bytes
// apart, they met in the same banks and bounded the kernel: 37 us against 29
// for 8192 tokens of 40 heads of 128 in bf16, 168 MB).  rope_rows takes all
// other rows one pair at a time.
#include "host.h"
#include "rope.cuh"

#include <math.h>

namespace wide {

bool rope_table(const wide_rope_config *c, RopeTable *t)
{
    if (!c || c->rot_dim < 2 || c->rot_dim > 2 * kRopeMaxPairs || (c->rot_dim & 1) ||
        (c->layout != WIDE_ROPE_HALF && c->layout != WIDE_ROPE_INTERLEAVED) ||
        !(c->theta > 0.0) || !isfinite(c->theta) || !(c->factor > 0.0) || !isfinite(c->factor) ||
        !((float)c->amplitude > 0.f) || !isfinite((float)c->amplitude) || c->original_len < 0)
        return false;
    const bool ramp = c->factor != 1.0 && c->original_len > 0;
    if (ramp && (!(c->low_freq >= 0.0) || !(c->high_freq > c->low_freq) || !isfinite(c->high_freq)))
        return false;
    // theta^(-2 i / rot_dim) for i = 8 a + b as a product of two powers: 24
    // calls of pow instead of 128, off by 3 units of 2^-53 (relative)
    const double two_pi = 6.283185307179586476925286766559;
    const int pairs = c->rot_dim / 2;
    double low[8], high = 1.0;
    for (int i = 0; i < 8; ++i)
        low[i] = pow(c->theta, -2.0 * i / c->rot_dim);
    for (int i = 0; i < pairs; ++i) {
        if (i % 8 == 0)
            high = pow(c->theta, -2.0 * i / c->rot_dim);
        double f = high * low[i % 8];
        if (ramp) {
            const double r = (double)c->original_len * f / two_pi;
            double g = (r - c->low_freq) / (c->high_freq - c->low_freq);
            g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
            f *= g + (1.0 - g) / c->factor;
        } else {
            f /= c->factor;
        }
        t->turns[i] = f / two_pi;
        if (!isfinite(t->turns[i] * 2147483648.0))   // at the farthest position
            return false;
    }
    for (int i = pairs; i < kRopeMaxPairs; ++i)
        t->turns[i] = 0.0;
    t->amplitude = (float)c->amplitude;
    return true;
}

namespace {

constexpr int kThreads = 256;

struct RopeArgs {
    const void *x;
    const int32_t *pos;
    void *out;
    int64_t xt, xh, ot, oh;        // token and head strides, elements
    int64_t tokens;
    int heads, head_dim, pairs;    // pairs = rot_dim / 2
    int tok_per_cta, heads_per_cta;
    int rest;                      // elements past the rotated part to copy (0 in place)
};

template <typename T, int VEC> struct Piece;    // VEC elements, moved as one access
template <> struct Piece<__nv_bfloat16, 8> {
    uint4 w;
    __device__ void get(float (&f)[8]) const { bf16x8_to_f32(w, f); }
    __device__ void set(const float (&f)[8])
    {
        uint32_t *o = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            o[i] = *reinterpret_cast<const uint32_t *>(&p);
        }
    }
};
template <> struct Piece<float, 4> {
    float4 w;
    __device__ void get(float (&f)[4]) const { f[0] = w.x, f[1] = w.y, f[2] = w.z, f[3] = w.w; }
    __device__ void set(const float (&f)[4]) { w = make_float4(f[0], f[1], f[2], f[3]); }
};
// 16-byte pieces.  Angles in shared memory: [token][i][piece] float4, the two
// pairs 2 i and 2 i + 1 of a piece.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kThreads)
    rope_pieces(const __grid_constant__ RopeTable tab, const RopeArgs a)
{
    constexpr int VEC = 16 / (int)sizeof(T);
    constexpr int kPer = INTER ? VEC / 2 : VEC;     // pairs of a piece
    constexpr int kRowsAtOnce = 2;
    using P = Piece<T, VEC>;
    extern __shared__ float4 cs4[];
    float2 *cs = reinterpret_cast<float2 *>(cs4);
    const int64_t t0 = (int64_t)blockIdx.x * a.tok_per_cta;
    const int nt = (int)min((int64_t)a.tok_per_cta, a.tokens - t0);
    const int h0 = (int)blockIdx.y * a.heads_per_cta;
    const int nh = min(a.heads_per_cta, a.heads - h0);
    const int steps = a.pairs / kPer;
    for (int i = threadIdx.x; i < nt * a.pairs; i += kThreads) {
        const int t = i / a.pairs, p = i - t * a.pairs;
        const int piece = p / kPer, q = p - piece * kPer;
        cs[((t * (kPer / 2) + (q >> 1)) * steps + piece) * 2 + (q & 1)] =
            rope_cos_sin(tab.turns[p], a.pos[t0 + t], tab.amplitude);
    }
    __syncthreads();
    const int per_row = steps + a.rest / VEC;
    const int lanes = kThreads / per_row;           // rows side by side
    const int lane = threadIdx.x / per_row, c = threadIdx.x - lane * per_row;
    if (lane >= lanes)
        return;
    const bool copy = c >= steps;
    const int e0 = copy ? 2 * a.pairs + (c - steps) * VEC : c * VEC;
    const bool half = !INTER && !copy;              // a second piece, the b elements
    const T *x = static_cast<const T *>(a.x) + t0 * a.xt + (int64_t)h0 * a.xh + e0;
    T *out = static_cast<T *>(a.out) + t0 * a.ot + (int64_t)h0 * a.oh + e0;
    int t = lane / nh, h = lane - t * nh;           // this thread's row
    const int hop_t = lanes / nh, hop_h = lanes - hop_t * nh;
    while (t < nt) {
        P pa[kRowsAtOnce], pb[kRowsAtOnce];
        int rt[kRowsAtOnce], rh[kRowsAtOnce];
#pragma unroll
        for (int u = 0; u < kRowsAtOnce; ++u) {
            rt[u] = t;
            rh[u] = h;
            if (t < nt) {
                const T *r = x + (int64_t)t * a.xt + (int64_t)h * a.xh;
                pa[u] = *reinterpret_cast<const P *>(r);
                if (half)
                    pb[u] = *reinterpret_cast<const P *>(r + a.pairs);
            }
            t += hop_t;
            h += hop_h;
            if (h >= nh) {
                h -= nh;
                ++t;
            }
        }
#pragma unroll
        for (int u = 0; u < kRowsAtOnce; ++u) {
            if (rt[u] >= nt)
                break;
            T *r = out + (int64_t)rt[u] * a.ot + (int64_t)rh[u] * a.oh;
            if (!copy) {
                const float4 *w = cs4 + rt[u] * (kPer / 2) * steps + c;
                float va[VEC], vb[VEC];
                pa[u].get(va);
                if constexpr (!INTER)
                    pb[u].get(vb);
#pragma unroll
                for (int k = 0; k < kPer; k += 2) {
                    const float4 cs2 = w[(k / 2) * steps];
                    if constexpr (INTER) {
                        rope_pair(va[2 * k], va[2 * k + 1], make_float2(cs2.x, cs2.y));
                        rope_pair(va[2 * k + 2], va[2 * k + 3], make_float2(cs2.z, cs2.w));
                    } else {
                        rope_pair(va[k], vb[k], make_float2(cs2.x, cs2.y));
                        rope_pair(va[k + 1], vb[k + 1], make_float2(cs2.z, cs2.w));
                    }
                }
                pa[u].set(va);
                if constexpr (!INTER) {
                    pb[u].set(vb);
                    *reinterpret_cast<P *>(r + a.pairs) = pb[u];
                }
            }
            *reinterpret_cast<P *>(r) = pa[u];
        }
    }
}

// One pair, or one element to copy, at a time.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kThreads)
    rope_rows(const __grid_constant__ RopeTable tab, const RopeArgs a)
{
    extern __shared__ float2 cs[];          // [tok_per_cta][pairs]
    const int64_t t0 = (int64_t)blockIdx.x * a.tok_per_cta;
    const int nt = (int)min((int64_t)a.tok_per_cta, a.tokens - t0);
    const int h0 = (int)blockIdx.y * a.heads_per_cta;
    const int nh = min(a.heads_per_cta, a.heads - h0);
    for (int i = threadIdx.x; i < nt * a.pairs; i += kThreads) {
        const int t = i / a.pairs, p = i - t * a.pairs;
        cs[i] = rope_cos_sin(tab.turns[p], a.pos[t0 + t], tab.amplitude);
    }
    __syncthreads();
    const int per_row = a.pairs + a.rest;
    const int items = nt * nh * per_row;
    const T *x = static_cast<const T *>(a.x);
    T *out = static_cast<T *>(a.out);
    for (int i = threadIdx.x; i < items; i += kThreads) {
        const int row = i / per_row, c = i - row * per_row;
        const int t = row / nh, h = row - t * nh;
        const T *xr = x + (t0 + t) * a.xt + (int64_t)(h0 + h) * a.xh;
        T *orow = out + (t0 + t) * a.ot + (int64_t)(h0 + h) * a.oh;
        if (c >= a.pairs) {
            orow[a.pairs + c] = xr[a.pairs + c];
            continue;
        }
        const int ia = INTER ? 2 * c : c, ib = INTER ? 2 * c + 1 : c + a.pairs;
        float va = to_f32(xr[ia]), vb = to_f32(xr[ib]);
        rope_pair(va, vb, cs[t * a.pairs + c]);
        orow[ia] = from_f32<T>(va);
        orow[ib] = from_f32<T>(vb);
    }
}

template <typename T>
int rope_launch(RopeArgs a, const RopeTable &tab, bool inter, cudaStream_t s)
{
    constexpr int V = 16 / (int)sizeof(T);
    const bool vec = (a.pairs * (inter ? 2 : 1)) % V == 0 && a.head_dim % V == 0 && a.xt % V == 0 &&
                     a.xh % V == 0 && a.ot % V == 0 && a.oh % V == 0 && aligned16(a.x) &&
                     aligned16(a.out) && (2 * a.pairs) % V == 0;
    // tokens: enough angles to occupy the CTA, but a grid of several CTAs per
    // SM; heads: split until the grid covers the GPU (few tokens), down to
    // about one step per thread
    a.tok_per_cta = a.pairs >= kThreads ? 1 : kThreads / a.pairs;
    while (a.tok_per_cta > 1 && (a.tokens + a.tok_per_cta - 1) / a.tok_per_cta < 1184)
        a.tok_per_cta = (a.tok_per_cta + 1) / 2;
    const int64_t bx = (a.tokens + a.tok_per_cta - 1) / a.tok_per_cta;
    const int steps = vec ? (a.pairs * (inter ? 2 : 1)) / V : a.pairs;
    a.heads_per_cta = a.heads;
    while (a.heads_per_cta > 1 && bx * ((a.heads + a.heads_per_cta - 1) / a.heads_per_cta) < 296 &&
           a.tok_per_cta * a.heads_per_cta * steps > kThreads)
        a.heads_per_cta = (a.heads_per_cta + 1) / 2;
    const dim3 grid((unsigned)bx, (unsigned)((a.heads + a.heads_per_cta - 1) / a.heads_per_cta));
    const size_t smem = (size_t)a.tok_per_cta * a.pairs * sizeof(float2);
    LaunchScope scope(KID_ROPE, s);
    if (vec)
        (inter ? rope_pieces<T, true> : rope_pieces<T, false>)<<<grid, kThreads, smem, s>>>(tab, a);
    else
        (inter ? rope_rows<T, true> : rope_rows<T, false>)<<<grid, kThreads, smem, s>>>(tab, a);
    return launch_status();
}

}  // namespace
}  // namespace wide

using namespace wide;

extern "C" int wide_rope(const void *d_x, const int32_t *d_positions, void *d_out,
                         const wide_rope_dims *d, const wide_rope_config *rope, void *stream)
{
    RopeTable tab;
    if (!d || d->tokens < 0 || d->heads <= 0 || d->head_dim <= 0 ||
        (d->dtype != WIDE_BF16 && d->dtype != WIDE_F32) || !rope_table(rope, &tab) ||
        rope->rot_dim > d->head_dim || d->x_token_stride < 0 || d->x_head_stride < 0 ||
        (d->tokens > 0 && !rows_apart(d->tokens, d->out_token_stride, d->heads,
                                      d->out_head_stride, d->head_dim)))
        return WIDE_EINVAL;
    if (d->tokens == 0)
        return WIDE_OK;
    if (!d_x || !d_positions || !d_out)
        return WIDE_EINVAL;
    const uintptr_t es = d->dtype == WIDE_BF16 ? 2 : 4;
    if (d->head_dim > 1024 || d->head_dim % 2 || d->tokens > (1 << 28) || d->heads > 65535 || (int64_t)d->heads * d->head_dim > (1 << 20) ||
        reinterpret_cast<uintptr_t>(d_x) % es || reinterpret_cast<uintptr_t>(d_out) % es ||
        (reinterpret_cast<uintptr_t>(d_positions) & 3u))
        return WIDE_EUNSUPPORTED;
    RopeArgs a = {};
    a.x = d_x;
    a.pos = d_positions;
    a.out = d_out;
    // a stride of a dimension of one element is never used: make it neutral
    a.xt = d->tokens > 1 ? d->x_token_stride : 0;
    a.xh = d->heads > 1 ? d->x_head_stride : 0;
    a.ot = d->tokens > 1 ? d->out_token_stride : 0;
    a.oh = d->heads > 1 ? d->out_head_stride : 0;
    a.tokens = d->tokens;
    a.heads = d->heads;
    a.head_dim = d->head_dim;
    a.pairs = rope->rot_dim / 2;
    a.rest = d_out == d_x ? 0 : d->head_dim - rope->rot_dim;
    if (d_out == d_x && (a.xt != a.ot || a.xh != a.oh))
        return WIDE_EINVAL;
    const bool inter = rope->layout == WIDE_ROPE_INTERLEAVED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return d->dtype == WIDE_BF16 ? rope_launch<__nv_bfloat16>(a, tab, inter, s)
                                 : rope_launch<float>(a, tab, inter, s);
}
