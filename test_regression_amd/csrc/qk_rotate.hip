// qk_rotate.hip -- per-head RMS norm of queries and keys and the rotation of their
// pairs of features by the token's position, in one pass, and the gradients (gfx950).
//
// Per token at position p and head, x a row of d features, w the weights:
//   n = x rsqrt(mean(x^2) + eps) w        (n = x without the norm)
//   y_a = m (n_a cos(p f_i) - n_b sin(p f_i)),   y_b = m (n_b cos(p f_i) + n_a sin(p f_i))
// for the pairs i < rot / 2: (a, b) = (2 i, 2 i + 1) interleaved, (i, i + rot / 2) by
// halves; features rot and up stay n.  Gradients, with g the transposed rotation of dy:
//   dw = sum of g x rsqrt(..),   dx = rsqrt(..) (w g - u mean(w g u)),  u = x rsqrt(..)
//
// Angles: p f in quarter turns is formed as the sum of two float64 values, so that positions
// keep their place in the turn (one value leaves 2^-16 of a turn at 2^37 turns), reduced
// to the nearest whole number, up to 2^51 of them, and the rest, at most pi / 4, goes
// through the Taylor polynomials of sine and cosine in float32 (to theta^9 and theta^10:
// 2e-9).  The second value shows only where a lane forms its angles for one head: 64 x
// 8192 tokens, d 128, bfloat16: 106 us without it, 110 us with it.
//
// HBM-bound: rows are read once and written once.  A row takes d / 8 lanes of eight
// features; a lane forms the cosines and sines of its features once a token and
// uses them for all heads that it takes of the token.  16 + 4 heads of 8 x 4096
// tokens, d 128, bfloat16: 56-70 us forward (4.8-6.0 TB/s; the next head's row on its way,
// without it 74 us), 82-87 us backward (5.9 TB/s) and 4 us for the weights' sums.
#include <algorithm>

#include "io8.h"
#include "mesa_kernels.h"

namespace mesa {

template <int L>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// The angle p f less its nearest whole number of quarter turns, and that number mod 4:
// the low bits of a sum whose last place is one.
__device__ __forceinline__ float rest_of_quarters(double p, double f, int* k) {
// a product's rounding is what the fma after it forms: no merging of the two
#pragma clang fp contract(off)
    constexpr double per = 0x1.45f306dc9c883p-1, per_rest = -0x1.6b01ec5417056p-55;   // quarter turns in one: 2 / pi
    constexpr double ones = 0x1.8p52;
    const double one = f * per, one_rest = fma(f, per_rest, fma(f, per, -one));      // of one position
    const double all = p * one, rest = fma(p, one_rest, fma(p, one, -all));
    const double sum = all + ones;
    *k = (int)__builtin_bit_cast(uint64_t, sum) & 3;
    // positions past those that have an angle left get some turn, nothing larger
    return __builtin_amdgcn_fmed3f((float)(((all - (sum - ones)) + rest) * 1.5707963267948966), -1.6f, 1.6f);
}
// cos and sin of the angle p f, times m.
__device__ __forceinline__ void turn_cos_sin(double p, double f, float m, float* c, float* s) {
    int k;
    const float th = rest_of_quarters(p, f, &k);
    const float q = th * th;
    const float sn = th * (1.0f + q * (-1.0f / 6 + q * (1.0f / 120 + q * (-1.0f / 5040 + q * (1.0f / 362880)))));
    const float cs = 1.0f + q * (-0.5f + q * (1.0f / 24 + q * (-1.0f / 720 + q * (1.0f / 40320 - q * (1.0f / 3628800)))));
    const float a = k & 1 ? sn : cs, b = k & 1 ? cs : sn;   // cos, sin up to signs
    *c = m * (k == 1 || k == 2 ? -a : a);
    *s = m * (k & 2 ? -b : b);
}

// The cosines and sines of a lane's eight features at one position (1 and 0 where
// turned() does not use them).
template <bool INTER>
struct Turns {
    static constexpr int n = INTER ? 4 : 8;
    float c[n], s[n];
    __device__ __forceinline__ void at(const RotateArgs& a, long b, long t, int d0) {
        const double p = (double)(a.positions ? a.positions[b * a.pos_stride + t] : a.position0 + t);
        const int half = a.rot / 2;
#pragma unroll
        for (int e = 0; e < n; ++e) {
            c[e] = 1.0f;
            s[e] = 0.0f;
            if (d0 < a.rot) {
                const int i = INTER ? d0 / 2 + e : (d0 < half ? d0 : d0 - half) + e;
                turn_cos_sin(p, a.freqs[i], a.amplitude, &c[e], &s[e]);
            }
        }
    }
};

// The eight features that stand opposite to a lane's in their pairs (by halves):
// d0 + rot / 2 for the first half's lanes, d0 - rot / 2 for the second's.  All lanes
// of a row take part.
__device__ __forceinline__ int partner_lane(int lane, int d0, int rot) {
    const int half = rot / 2;
    return d0 < half ? lane + half / 8 : d0 < rot ? lane - half / 8 : lane;
}
__device__ __forceinline__ f32x8 from_lane(const f32x8& x, int lane) {
    f32x8 r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e] = __shfl(x.v[e], lane, 64);
    return r;
}

// y = the rotation of x (SIGN 1) or its transpose (-1), o the opposite features; x
// itself past the rotated ones.
template <bool INTER, int SIGN>
__device__ __forceinline__ f32x8 turned(const f32x8& x, const Turns<INTER>& r, int partner, int d0, int rot) {
    f32x8 y;
    if constexpr (INTER) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y.v[2 * e] = x.v[2 * e] * r.c[e] - SIGN * x.v[2 * e + 1] * r.s[e];
            y.v[2 * e + 1] = x.v[2 * e + 1] * r.c[e] + SIGN * x.v[2 * e] * r.s[e];
        }
    } else {
        const f32x8 o = from_lane(x, partner);
        const float sign = d0 < rot / 2 ? -SIGN : SIGN;
#pragma unroll
        for (int e = 0; e < 8; ++e) y.v[e] = x.v[e] * r.c[e] + sign * o.v[e] * r.s[e];
    }
    // not by a product with 0, which an infinity would turn into a NaN
#pragma unroll
    for (int e = 0; e < 8; ++e) y.v[e] = d0 < rot ? y.v[e] : x.v[e];
    return y;
}

// Row of head h of the queries or keys at token t, and its place in the contiguous
// outputs [B, heads, T, d].
template <bool KEY, typename In>
__device__ __forceinline__ const In* row_in(const RotateArgs& a, int h, long b, long t) {
    const RowStrides& s = KEY ? a.ks : a.qs;
    return static_cast<const In*>(KEY ? a.k : a.q) + b * s.batch + h * s.head + t * s.token;
}
template <bool KEY>
__device__ __forceinline__ long row_out(const RotateArgs& a, int h, long b, long t, int d) {
    return ((b * (KEY ? a.Hk : a.Hq) + h) * (long)a.T + t) * d;
}

// The queries' or keys' rows of one token that a row of lanes takes.
template <bool KEY, int d, bool INTER, typename In>
__device__ __forceinline__ void rotate_heads(const RotateArgs& a, const Turns<INTER>& r, int partner, int slot, int d0, long b,
                                             long t) {
    const float* w = KEY ? a.wk : a.wq;
    f32x8 wv;
#pragma unroll
    for (int e = 0; e < 8; ++e) wv.v[e] = 1.0f;
    if (w) wv = load8_upto<true>(w + d0, 8);
    const int heads = KEY ? a.Hk : a.Hq;
    Held8<In> held;   // the next head's row, on its way
    if (slot < heads) held.load(row_in<KEY, In>(a, slot, b, t) + d0);
    for (int h = slot; h < heads; h += a.slots) {
        f32x8 x = held.get();
        if (h + a.slots < heads) held.load(row_in<KEY, In>(a, h + a.slots, b, t) + d0);
        if (a.norm) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss += x.v[e] * x.v[e];
            const float rs = rsqrtf(row_sum<d / 8>(ss) * (1.0f / d) + a.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) x.v[e] *= rs * wv.v[e];
        }
        const f32x8 y = turned<INTER, 1>(x, r, partner, d0, a.rot);
        store8_upto<true>(static_cast<In*>(KEY ? a.yk : a.yq) + row_out<KEY>(a, h, b, t, d) + d0, y, 8);
    }
}
template <bool KEY, int d, bool INTER, typename In>
__device__ __forceinline__ void rotate_heads_bwd(const RotateBwdArgs& g, const Turns<INTER>& r, int partner, int slot, int d0,
                                                 long b, long t, f32x8& dw) {
    const RotateArgs& a = g.f;
    const RowStrides& gs = KEY ? g.gks : g.gqs;
    const float* w = KEY ? a.wk : a.wq;
    f32x8 wv;
#pragma unroll
    for (int e = 0; e < 8; ++e) wv.v[e] = 1.0f;
    if (w) wv = load8_upto<true>(w + d0, 8);
    for (int h = slot; h < (KEY ? a.Hk : a.Hq); h += a.slots) {
        f32x8 y = load8_upto<true>(static_cast<const In*>(KEY ? g.grad_yk : g.grad_yq) + row_out<KEY>(a, h, b, t, d) + d0, 8);
        f32x8 x{};
        if (a.norm) x = load8_upto<true>(row_in<KEY, In>(a, h, b, t) + d0, 8);
        y = turned<INTER, -1>(y, r, partner, d0, a.rot);
        if (a.norm) {
            float ss = 0.f, gx = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss += x.v[e] * x.v[e];
                gx += x.v[e] * (y.v[e] * wv.v[e]);
            }
            const float rs = rsqrtf(row_sum<d / 8>(ss) * (1.0f / d) + a.eps);
            const float mean = row_sum<d / 8>(gx) * (1.0f / d) * rs * rs;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dw.v[e] += y.v[e] * (x.v[e] * rs);
                y.v[e] = rs * (y.v[e] * wv.v[e] - x.v[e] * mean);
            }
        }
        store8_upto<true>(static_cast<In*>(KEY ? g.grad_k : g.grad_q) + b * gs.batch + h * gs.head + t * gs.token + d0, y, 8);
    }
}

// `slots` rows of a token go side by side, rows / slots tokens a workgroup.
template <int d, bool INTER, typename In>
__global__ __launch_bounds__(256) void qk_rotate_kernel(RotateArgs a) {
    constexpr int L = d / 8, rows = 256 / L;
    const int lane = threadIdx.x % L, row = threadIdx.x / L, d0 = 8 * lane;
    const int slot = row % a.slots;
    const long at = (long)blockIdx.x * (rows / a.slots) + row / a.slots, b = at / a.T, t = at - b * a.T;
    if (b >= a.B) return;   // whole rows of lanes
    Turns<INTER> r;
    r.at(a, b, t, d0);
    const int partner = partner_lane(threadIdx.x % 64, d0, a.rot);
    rotate_heads<false, d, INTER, In>(a, r, partner, slot, d0, b, t);
    rotate_heads<true, d, INTER, In>(a, r, partner, slot, d0, b, t);
}

// The weights' gradients of a lane's features are added in float32 over kRotateAdd tokens
// and these in float64, in the lane's own places in LDS, so that a sum's error does not
// grow with the tokens (16 + 4 heads of 8 x 4096 tokens, d 128, bfloat16: 81 us with one
// float32 sum, 82 us so).
constexpr int kRotateAdd = 16;
template <int d, bool INTER, typename In>
__global__ __launch_bounds__(256) void qk_rotate_bwd_kernel(RotateBwdArgs g) {
    constexpr int L = d / 8, rows = 256 / L;
    __shared__ double red[2][rows][d + 2];
    const RotateArgs& a = g.f;
    const int lane = threadIdx.x % L, row = threadIdx.x / L, d0 = 8 * lane;
    const int slot = row % a.slots;
    const int partner = partner_lane(threadIdx.x % 64, d0, a.rot);
    f32x8 dw[2] = {};
    bool first = true;
    auto put = [&] {
        if (!g.partial) return;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) red[k][row][d0 + e] = (first ? 0.0 : red[k][row][d0 + e]) + dw[k].v[e];
        dw[0] = dw[1] = f32x8{};
        first = false;
    };
    const long step = rows / a.slots, all = (long)a.B * a.T;
    int held = 0;
    for (long at = (long)blockIdx.x * step + row / a.slots; at < all; at += (long)gridDim.x * step) {
        const long b = at / a.T, t = at - b * a.T;
        Turns<INTER> r;
        r.at(a, b, t, d0);
        rotate_heads_bwd<false, d, INTER, In>(g, r, partner, slot, d0, b, t, dw[0]);
        rotate_heads_bwd<true, d, INTER, In>(g, r, partner, slot, d0, b, t, dw[1]);
        if (++held == kRotateAdd) {
            put();
            held = 0;
        }
    }
    if (!g.partial) return;
    put();
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * d; c += 256) {
        double s = 0.0;
        for (int i = 0; i < rows; ++i) s += red[c / d][i][c % d];
        g.partial[(long)blockIdx.x * 2 * d + c] = (float)s;
    }
}

// grad_wq and grad_wk over the workgroups' parts: eight columns a workgroup, 32 runs of
// parts side by side.
__global__ __launch_bounds__(256) void rotate_sums_kernel(const float* partial, long parts, int d, float* gq, float* gk) {
    __shared__ double red[32][8];
    const int col = blockIdx.x * 8 + threadIdx.x % 8, slot = threadIdx.x / 8;
    red[slot][threadIdx.x % 8] = strided_sum(partial + col, slot, parts, 32, 2L * d);
    __syncthreads();
    if (slot != 0) return;
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
    float* to = col < d ? gq : gk;
    if (to) to[col % d] = (float)s;
}

// Rows of a token side by side: as few as still fill the card (a lane's cosines
// then serve the most heads), at most a workgroup's.
static int rotate_slots(const RotateArgs& a) {
    const int rows = 256 / (a.d / 8), heads = a.Hq + a.Hk;
    const long tokens = (long)a.B * a.T;
    int s = 1;
    while (s < rows && s < heads && tokens * s < 256L * 4 * rows) s *= 2;
    return s;
}

template <int d, typename In>
static void rotate_go(const RotateArgs& a, unsigned blocks, hipStream_t s) {
    if (a.interleaved) hipLaunchKernelGGL((qk_rotate_kernel<d, true, In>), dim3(blocks), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((qk_rotate_kernel<d, false, In>), dim3(blocks), dim3(256), 0, s, a);
}
template <int d, typename In>
static void rotate_go(const RotateBwdArgs& a, unsigned blocks, hipStream_t s) {
    if (a.f.interleaved) hipLaunchKernelGGL((qk_rotate_bwd_kernel<d, true, In>), dim3(blocks), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((qk_rotate_bwd_kernel<d, false, In>), dim3(blocks), dim3(256), 0, s, a);
}
template <typename Args>
static hipError_t rotate_sized(const Args& a, int d, bool bf16, unsigned blocks, hipStream_t s) {
    switch (d) {
        case 16: bf16 ? rotate_go<16, bf16_t>(a, blocks, s) : rotate_go<16, float>(a, blocks, s); break;
        case 32: bf16 ? rotate_go<32, bf16_t>(a, blocks, s) : rotate_go<32, float>(a, blocks, s); break;
        case 64: bf16 ? rotate_go<64, bf16_t>(a, blocks, s) : rotate_go<64, float>(a, blocks, s); break;
        case 128: bf16 ? rotate_go<128, bf16_t>(a, blocks, s) : rotate_go<128, float>(a, blocks, s); break;
        case 256: bf16 ? rotate_go<256, bf16_t>(a, blocks, s) : rotate_go<256, float>(a, blocks, s); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

hipError_t launch_qk_rotate(RotateArgs a, hipStream_t s) {
    a.slots = rotate_slots(a);
    const long tokens = 256 / (a.d / 8) / a.slots;   // of a workgroup
    return rotate_sized(a, a.d, a.bf16, (unsigned)(((long)a.B * a.T + tokens - 1) / tokens), s);
}

hipError_t launch_qk_rotate_bwd(RotateBwdArgs a, hipStream_t s) {
    a.f.slots = rotate_slots(a.f);
    const long tokens = 256 / (a.f.d / 8) / a.f.slots, groups = ((long)a.f.B * a.f.T + tokens - 1) / tokens;
    const unsigned blocks = (unsigned)std::min(groups, (long)kRotateParts);
    if (!a.f.norm || (!a.grad_wq && !a.grad_wk)) a.partial = nullptr;
    const hipError_t e = rotate_sized(a, a.f.d, a.f.bf16, blocks, s);
    if (e != hipSuccess || !a.partial) return e;
    hipLaunchKernelGGL(rotate_sums_kernel, dim3((unsigned)(2 * a.f.d / 8)), dim3(256), 0, s, a.partial, (long)blocks, a.f.d,
                       a.grad_wq, a.grad_wk);
    return hipGetLastError();
}

}  // namespace mesa
