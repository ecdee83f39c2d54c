// block_norms.hip -- the norms around a layer and their gradients (gfx950).
//
// Gate norm, per token and head (x a layer's output row of d features, g its
// gate row, w the head's weights):
//   u = x rsqrt(mean(x^2) + eps),   y = u w silu(g),   silu(g) = g sigmoid(g)
// with x in the layers' [B, H, T, d] order and g, y in the projections'
// [B, T, H, d] order.  Gradients, with d_u = dy w silu(g):
//   dx = rsqrt(..) (d_u - u mean(d_u u)),   dw = sum over tokens of dy u silu(g)
//   dg = dy u w sigmoid(g) (1 + g (1 - sigmoid(g)))
//
// Residual norm, per row of D features:
//   z = h + s y,   n = z rsqrt(mean(z^2) + eps) w
// Gradients, with u = z rsqrt(..), d_u = dn w and dh' the gradient of z as
// the residual's next value:
//   dz = rsqrt(..) (d_u - u mean(d_u u)) + dh',   dh = dz,  dy = s dz
//   dw = sum over rows of dn u,   ds = sum over rows of dz y
//
// All of them are HBM-bound: each input element is read once and each output
// element written once, and a row stays in registers between its sums and
// its outputs.  The arithmetic is float32; outputs are rounded once.  The
// parameter gradients are summed in registers over the rows that a thread
// sees, then over the workgroup in LDS, then over the workgroups by a second
// small kernel (4-5 us), all in a fixed order (no atomics).
//
// Measured (times of whole calls; a large copy reaches 5.5 TB/s):
//   gate norm 8x16x4096x128 bf16         79 us  5.1 TB/s; gradients 136 us  4.9 TB/s
//   residual norm 32768x2048 f32 + bf16 144 us  5.6 TB/s; gradients with the
//     residual's 216 us 5.6 TB/s, without 178 us 5.3 TB/s
//   4099x1237 f32: 16 us, gradients with the residual's 32 us, without 28; a row
//     or 256: 3 to 5 us in the kernel
#include <algorithm>

#include "io8.h"
#include "mesa_kernels.h"

namespace mesa {

// Sum over groups of L consecutive lanes (L a power of two up to 64).
template <int L>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// The fast exponential rounds its exponent and is off by |g| 2^-24: little beside
// a bf16 output's rounding, but 64 of a float one's at g = -64.  For bf16 rows the exact one takes 218 us and not 201 (forward and
// gradients of 8x16x4096x128); float rows move twice the bytes and hide it.
template <typename G>
__device__ __forceinline__ float sigmoid(float g) {
    return 1.0f / (1.0f + (sizeof(G) == 2 ? __expf(-g) : expf(-g)));
}

// ---------------------------------------------------------------- gate norm

constexpr int kGateThreads = 256;
constexpr int kGateTokens = 8;   // consecutive tokens of a head that neighbouring rows of a workgroup take

// A row takes d / 8 lanes.  Rows go by as [b][block of 8 tokens][h][token]:
// a workgroup's rows are then runs of 8 tokens in x and runs of heads in the
// gate, so both sides use whole cache lines.  y goes out in streaming stores.
template <int d, typename X, typename G>
__global__ __launch_bounds__(kGateThreads) void gate_norm_kernel(GateNormArgs a) {
    constexpr int L = d / 8, rows = kGateThreads / L;
    const int lane = threadIdx.x % L;
    const long tb = (a.T + kGateTokens - 1) / kGateTokens;
    const long r = (long)blockIdx.x * rows + threadIdx.x / L;
    const int ti = (int)(r % kGateTokens);
    const long r1 = r / kGateTokens;
    const int h = (int)(r1 % a.H);
    const long r2 = r1 / a.H;
    const long t = (r2 % tb) * kGateTokens + ti, b = r2 / tb;
    const bool live = b < a.B && t < a.T;
    const size_t xo = (((size_t)b * a.H + h) * a.T + t) * d + 8 * lane;
    const size_t go = (((size_t)b * a.T + t) * a.H + h) * d + 8 * lane;
    f32x8 x{}, g{};
    if (live) {
        x = load8(static_cast<const X*>(a.x) + xo);
        if (a.gate) g = load8(static_cast<const G*>(a.gate) + go);
    }
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss += x.v[e] * x.v[e];
    const float rs = rsqrtf(lane_sum<L>(ss) * (1.0f / d) + a.eps);
    if (!live) return;
    const f32x8 w = load8(a.w + (size_t)h * d + 8 * lane);
    f32x8 y;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float act = a.gate ? g.v[e] * sigmoid<G>(g.v[e]) : 1.0f;
        y.v[e] = x.v[e] * rs * w.v[e] * act;
    }
    store8_upto<true>(static_cast<G*>(a.y) + go, y, 8);
}

// A workgroup takes one head and a run of its (b, t) rows, so that a thread
// keeps the same eight columns of dw in registers throughout.
template <int d, typename X, typename G>
__global__ __launch_bounds__(kGateThreads) void gate_norm_bwd_kernel(GateNormBwdArgs a) {
    constexpr int L = d / 8, rows = kGateThreads / L;
    __shared__ float red[rows][d + 4];
    const int lane = threadIdx.x % L, slot = threadIdx.x / L;
    const int h = blockIdx.x % a.H;
    const int part = blockIdx.x / a.H;
    const long BT = (long)a.B * a.T;
    const f32x8 w = load8(a.w + (size_t)h * d + 8 * lane);
    float dw[8] = {};
    const long end = min(BT, (long)(part + 1) * a.rows_per_part);
    struct Row { f32x8 x, g, dy; };
    auto offset = [&](long r, bool gate_side) {
        const long b = r / a.T, t = r % a.T;
        return (gate_side ? ((size_t)b * a.T + t) * a.H + h : ((size_t)b * a.H + h) * a.T + t) * d + 8 * lane;
    };
    auto load = [&](long r) {
        Row v{};
        if (r < end) {
            v.x = load8(static_cast<const X*>(a.x) + offset(r, false));
            if (a.gate) v.g = load8(static_cast<const G*>(a.gate) + offset(r, true));
            v.dy = load8(static_cast<const G*>(a.grad_y) + offset(r, true));
        }
        return v;
    };
    // every lane of a wave runs the same number of rounds: the row sums cross
    // lanes.  The next round's rows are in flight meanwhile.
    Row next = load((long)part * a.rows_per_part + slot);
    for (long r0 = (long)part * a.rows_per_part; r0 < end; r0 += rows) {
        const long r = r0 + slot;
        const Row v = next;
        next = load(r + rows);
        float ss = 0.f, c = 0.f, act[8], sg[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            sg[e] = sigmoid<G>(v.g.v[e]);
            act[e] = a.gate ? v.g.v[e] * sg[e] : 1.0f;
            ss += v.x.v[e] * v.x.v[e];
            c += v.dy.v[e] * w.v[e] * act[e] * v.x.v[e];
        }
        const float rs = rsqrtf(lane_sum<L>(ss) * (1.0f / d) + a.eps);
        const float m = lane_sum<L>(c) * rs * rs * (1.0f / d);   // mean(d_u u) rs
        f32x8 dx, dg;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float u = v.x.v[e] * rs;
            dx.v[e] = rs * (v.dy.v[e] * w.v[e] * act[e]) - u * m;
            dg.v[e] = v.dy.v[e] * u * w.v[e] * sg[e] * (1.0f + v.g.v[e] * (1.0f - sg[e]));
            dw[e] += v.dy.v[e] * u * act[e];
        }
        if (r < end) {
            store8_upto<true>(static_cast<X*>(a.grad_x) + offset(r, false), dx, 8);
            if (a.gate) store8_upto<true>(static_cast<G*>(a.grad_gate) + offset(r, true), dg, 8);
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) red[slot][8 * lane + e] = dw[e];
    __syncthreads();
    for (int f = threadIdx.x; f < d; f += kGateThreads) {
        float s = 0.f;
        for (int i = 0; i < rows; ++i) s += red[i][f];
        a.partial[((size_t)part * a.H + h) * d + f] = s;
    }
}

// out[f] = sum over the parts of partial[part][f] for f < n, and out2[f - n2] from
// column n2 on where out2 is given: 64 columns a workgroup, its sixteen waves
// taking every sixteenth part.
__global__ __launch_bounds__(1024) void sum_parts_kernel(const float* partial, size_t pitch, int parts, long n, float* out,
                                                         long n2, float* out2) {
    __shared__ float red[16][64];
    const long f = (long)blockIdx.x * 64 + threadIdx.x % 64;
    const int q = threadIdx.x / 64;
    float s[4] = {};
    if (f < n) {
        const float* p = partial + f;
        int i = q;
        for (; i + 48 < parts; i += 64)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] += p[(size_t)(i + 16 * k) * pitch];
        for (; i < parts; i += 16) s[0] += p[(size_t)i * pitch];
    }
    red[q][threadIdx.x % 64] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    if (q == 0 && f < n) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) t += red[k][threadIdx.x];
        if (out2 && f >= n2) out2[f - n2] = t;
        else out[f] = t;
    }
}

hipError_t launch_sum_parts(const float* partial, size_t pitch, int parts, long n, float* out, long n2, float* out2,
                            hipStream_t s) {
    hipLaunchKernelGGL(sum_parts_kernel, dim3((unsigned)((n + 63) / 64)), dim3(1024), 0, s, partial, pitch, parts, n, out,
                       n2, out2);
    return hipGetLastError();
}

template <int d, typename X, typename G>
hipError_t gate_norm_go(const GateNormArgs& a, hipStream_t s) {
    constexpr int rows = kGateThreads / (d / 8);
    const long n = (long)a.B * ((a.T + kGateTokens - 1) / kGateTokens) * a.H * kGateTokens;
    hipLaunchKernelGGL((gate_norm_kernel<d, X, G>), dim3((unsigned)((n + rows - 1) / rows)), dim3(kGateThreads), 0, s, a);
    return hipGetLastError();
}
template <int d, typename X, typename G>
hipError_t gate_norm_bwd_go(const GateNormBwdArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((gate_norm_bwd_kernel<d, X, G>), dim3((unsigned)(a.parts * a.H)), dim3(kGateThreads), 0, s, a);
    return hipGetLastError();
}

#define MESA_GATE_DISPATCH(go)                                                         \
    template <int d, typename A>                                                       \
    hipError_t go##_t(const A& a, hipStream_t s) {                                     \
        if (a.x_bf16) return a.g_bf16 ? go<d, bf16_t, bf16_t>(a, s) : go<d, bf16_t, float>(a, s); \
        return a.g_bf16 ? go<d, float, bf16_t>(a, s) : go<d, float, float>(a, s);      \
    }                                                                                  \
    template <typename A>                                                              \
    hipError_t go##_d(const A& a, hipStream_t s) {                                     \
        switch (a.d) {                                                                 \
            case 16: return go##_t<16>(a, s);                                          \
            case 32: return go##_t<32>(a, s);                                          \
            case 64: return go##_t<64>(a, s);                                          \
            case 128: return go##_t<128>(a, s);                                        \
            case 256: return go##_t<256>(a, s);                                        \
        }                                                                              \
        return hipErrorInvalidValue;                                                   \
    }
MESA_GATE_DISPATCH(gate_norm_go)
MESA_GATE_DISPATCH(gate_norm_bwd_go)

hipError_t launch_gate_norm(const GateNormArgs& a, hipStream_t s) { return gate_norm_go_d(a, s); }
hipError_t launch_gate_norm_bwd(const GateNormBwdArgs& a, hipStream_t s) {
    const hipError_t e = gate_norm_bwd_go_d(a, s);
    if (e != hipSuccess) return e;
    const long n = (long)a.H * a.d;
    return launch_sum_parts(a.partial, (size_t)n, a.parts, n, a.grad_w, n, nullptr, s);
}

// ------------------------------------------------------------ residual norm

// W waves share a row (W = 1: each of a workgroup's four waves has its own);
// a thread holds N pieces of 8 elements, piece j of thread t at column
// 8 (t + 64 W j).  Rows need no more than their elements' alignment; rows of a
// multiple of 8 elements (WHOLE) leave out the tests for a cut last piece
// (403 us and not 467 for 32768 x 2048 and its gradients).
//
// One piece a thread moves the most: with a wave and four pieces a row, 32768 x
// 2048 takes 159 us forward and 216 back, with four waves and one piece 145 and
// 177; at 8192 x 8192 four waves and four pieces 162 and 225, sixteen and one
// 141 forward, eight and two 189 back (sixteen waves leave a thread 128
// registers: 223).  Gradients of up to 1024 columns keep a wave a row, its four
// rows a workgroup in flight together: 88 us at 32768 x 1024, and 114 with two
// waves.  A few rows cost the same in every layout.
template <int W> struct RowGroup {
    static constexpr int threads = W == 1 ? 256 : 64 * W;
    static constexpr int rows = W == 1 ? 4 : 1;   // rows of a workgroup at a time
    static __device__ int tid() { return W == 1 ? threadIdx.x % 64 : threadIdx.x; }
    // sums of two values over a row's threads; `red` holds 2 W floats a round
    static __device__ void sum2(float& x, float& y, float (&red)[2][2][16], int& flip) {
        x = lane_sum<64>(x);
        y = lane_sum<64>(y);
        if constexpr (W > 1) {
            const int w = threadIdx.x / 64;
            // two buffers in turn: a wave may write its next row's sums
            // while another still reads this row's
            if (threadIdx.x % 64 == 0) { red[flip][0][w] = x; red[flip][1][w] = y; }
            __syncthreads();
            x = y = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) { x += red[flip][0][i]; y += red[flip][1][i]; }
            flip ^= 1;
        }
    }
};

template <int W, int N, bool WHOLE, typename Hh, typename Y>
__global__ __launch_bounds__(RowGroup<W>::threads) void residual_norm_kernel(ResidualNormArgs a) {
    using RG = RowGroup<W>;
    __shared__ float red[2][2][16];
    int flip = 0;
    const int t = RG::tid();
    const long r = (long)blockIdx.x * RG::rows + (W == 1 ? threadIdx.x / 64 : 0);
    if (r >= a.R) return;   // a whole wave (W = 1), or never
    const size_t ro = (size_t)r * a.D;
    f32x8 z[N];
    float ss = 0.f, none = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int f = 8 * (t + 64 * W * j), left = a.D - f;
        z[j] = f32x8{};
        if (left > 0) {
            z[j] = load8_upto<WHOLE>(static_cast<const Hh*>(a.h) + ro + f, left);
            if (a.y) {
                const f32x8 y = load8_upto<WHOLE>(static_cast<const Y*>(a.y) + ro + f, left);
                if (a.scale) {
                    const f32x8 s = load8_upto<WHOLE>(a.scale + f, left);
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[j].v[e] += s.v[e] * y.v[e];
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[j].v[e] += y.v[e];
                }
                store8_upto<WHOLE>(static_cast<Hh*>(a.h_out) + ro + f, z[j], left);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += z[j].v[e] * z[j].v[e];
    }
    RG::sum2(ss, none, red, flip);
    const float rs = rsqrtf(ss / (float)a.D + a.eps);
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int f = 8 * (t + 64 * W * j), left = a.D - f;
        if (left > 0) {
            f32x8 w = load8_upto<WHOLE>(a.w + f, left);
#pragma unroll
            for (int e = 0; e < 8; ++e) w.v[e] *= z[j].v[e] * rs;
            store8_upto<WHOLE>(static_cast<Y*>(a.n) + ro + f, w, left);
        }
    }
}

// Workgroup i takes row groups i, i + gridDim.x, ...; its sums of dw and ds go
// to partial[i][0..D) and partial[i][D..2D).  With one piece a thread the next
// row is in flight while a row's sums are joined.
template <int W, int N, bool WHOLE, typename Hh, typename Y>
__global__ __launch_bounds__(RowGroup<W>::threads) void residual_norm_bwd_kernel(ResidualNormBwdArgs a) {
    using RG = RowGroup<W>;
    // the next row on its way; w, scale and dh' kept from the sums to the outputs
    // (a thread of sixteen waves has half the registers)
    constexpr bool AHEAD = N == 1, KEEP = W < 16;
    __shared__ float red[2][2][16];
    __shared__ float own[W == 1 ? 4 : 1][W == 1 ? 64 * 8 * N : 1];
    int flip = 0;
    const int t = RG::tid(), wave = threadIdx.x / 64;
    float dw[N][8] = {}, ds[N][8] = {};
    const float inv_D = 1.0f / (float)a.D;
    struct Row { f32x8 z[N], y[N], d[N], g[N]; };
    auto load = [&](Row& x, long r) {
        const size_t ro = (size_t)r * a.D;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int f = 8 * (t + 64 * W * j), left = a.D - f;
            x.z[j] = x.y[j] = x.d[j] = x.g[j] = f32x8{};
            if (left > 0) {
                x.z[j] = load8_upto<WHOLE>(static_cast<const Hh*>(a.h) + ro + f, left);
                x.d[j] = load8_upto<WHOLE>(static_cast<const Y*>(a.grad_n) + ro + f, left);
                if (a.y) x.y[j] = load8_upto<WHOLE>(static_cast<const Y*>(a.y) + ro + f, left);
                if (KEEP && a.grad_h_out) x.g[j] = load8_upto<WHOLE>(static_cast<const Hh*>(a.grad_h_out) + ro + f, left);
            }
        }
    };
    struct Weights { f32x8 w, s; };
    auto weights = [&](int j) {
        const int f = 8 * (t + 64 * W * j), left = a.D - f;
        Weights x{};
#pragma unroll
        for (int e = 0; e < 8; ++e) x.s.v[e] = 1.f;
        if (left > 0) {
            x.w = load8_upto<WHOLE>(a.w + f, left);
            if (a.scale) x.s = load8_upto<WHOLE>(a.scale + f, left);
        }
        return x;
    };
    Weights kept[KEEP ? N : 1];
    if constexpr (KEEP)
#pragma unroll
        for (int j = 0; j < N; ++j) kept[j] = weights(j);
    Row next;
    const long step = (long)gridDim.x * RG::rows;
    long r = (long)blockIdx.x * RG::rows + (W == 1 ? wave : 0);
    if (AHEAD && r < a.R) load(next, r);
    for (; r < a.R; r += step) {
        const size_t ro = (size_t)r * a.D;
        Row x;
        if constexpr (AHEAD) {
            x = next;
            if (r + step < a.R) load(next, r + step);
        } else {
            load(x, r);
        }
        float ss = 0.f, c = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const Weights p = KEEP ? kept[KEEP ? j : 0] : weights(j);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x.z[j].v[e] += p.s.v[e] * x.y[j].v[e];
                ss += x.z[j].v[e] * x.z[j].v[e];
                c += x.d[j].v[e] * p.w.v[e] * x.z[j].v[e];
            }
        }
        RG::sum2(ss, c, red, flip);
        const float rs = rsqrtf(ss * inv_D + a.eps);
        const float m = c * rs * rs * inv_D;   // mean(d_u u) rs
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int f = 8 * (t + 64 * W * j), left = a.D - f;
            if (left > 0) {
                const Weights p = KEEP ? kept[KEEP ? j : 0] : weights(j);
                if (!KEEP && a.grad_h_out) x.g[j] = load8_upto<WHOLE>(static_cast<const Hh*>(a.grad_h_out) + ro + f, left);
                f32x8 dz;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float u = x.z[j].v[e] * rs;
                    dz.v[e] = rs * (x.d[j].v[e] * p.w.v[e]) - u * m + x.g[j].v[e];
                    dw[j][e] += x.d[j].v[e] * u;
                    ds[j][e] += dz.v[e] * x.y[j].v[e];
                }
                store8_upto<WHOLE>(static_cast<Hh*>(a.grad_h) + ro + f, dz, left);
                if (a.grad_y) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) dz.v[e] *= p.s.v[e];
                    store8_upto<WHOLE>(static_cast<Y*>(a.grad_y) + ro + f, dz, left);
                }
            }
        }
    }
    float* out = a.partial + (size_t)blockIdx.x * 2 * a.D;
    if constexpr (W > 1) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int f = 8 * (t + 64 * W * j);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (f + e < a.D) {
                    out[f + e] = dw[j][e];
                    if (a.grad_scale) out[a.D + f + e] = ds[j][e];
                }
        }
    } else {
        for (int k = 0; k < (a.grad_scale ? 2 : 1); ++k) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) own[wave][8 * (t + 64 * j) + e] = k ? ds[j][e] : dw[j][e];
            __syncthreads();
            for (int f = threadIdx.x; f < a.D; f += 256)
                out[(size_t)k * a.D + f] = (own[0][f] + own[1][f]) + (own[2][f] + own[3][f]);
        }
    }
}

template <int W, int N, bool WHOLE> struct FwdGo {
    template <typename Hh, typename Y>
    static hipError_t one(const ResidualNormArgs& a, hipStream_t s) {
        using RG = RowGroup<W>;
        hipLaunchKernelGGL((residual_norm_kernel<W, N, WHOLE, Hh, Y>), dim3((unsigned)((a.R + RG::rows - 1) / RG::rows)),
                           dim3(RG::threads), 0, s, a);
        return hipGetLastError();
    }
    static hipError_t go(const ResidualNormArgs& a, hipStream_t s) {
        if (a.h_bf16) return a.y_bf16 ? one<bf16_t, bf16_t>(a, s) : one<bf16_t, float>(a, s);
        return a.y_bf16 ? one<float, bf16_t>(a, s) : one<float, float>(a, s);
    }
};
template <int W, int N, bool WHOLE> struct BwdGo {
    template <typename Hh, typename Y>
    static hipError_t one(const ResidualNormBwdArgs& a, hipStream_t s) {
        hipLaunchKernelGGL((residual_norm_bwd_kernel<W, N, WHOLE, Hh, Y>), dim3((unsigned)a.parts),
                           dim3(RowGroup<W>::threads), 0, s, a);
        return hipGetLastError();
    }
    static hipError_t go(const ResidualNormBwdArgs& a, hipStream_t s) {
        if (a.h_bf16) return a.y_bf16 ? one<bf16_t, bf16_t>(a, s) : one<bf16_t, float>(a, s);
        return a.y_bf16 ? one<float, bf16_t>(a, s) : one<float, float>(a, s);
    }
};

template <bool WHOLE>
hipError_t residual_fwd(const ResidualNormArgs& a, hipStream_t s) {
    if (a.D <= 512) return FwdGo<1, 1, WHOLE>::go(a, s);
    if (a.D <= 1024) return FwdGo<2, 1, WHOLE>::go(a, s);
    if (a.D <= 2048) return FwdGo<4, 1, WHOLE>::go(a, s);
    if (a.D <= 4096) return FwdGo<8, 1, WHOLE>::go(a, s);
    return a.D <= 8192 ? FwdGo<16, 1, WHOLE>::go(a, s) : FwdGo<16, 2, WHOLE>::go(a, s);
}
template <bool WHOLE>
hipError_t residual_bwd(const ResidualNormBwdArgs& a, hipStream_t s) {
    if (a.D <= 512) return BwdGo<1, 1, WHOLE>::go(a, s);
    if (a.D <= 1024) return BwdGo<1, 2, WHOLE>::go(a, s);
    if (a.D <= 2048) return BwdGo<4, 1, WHOLE>::go(a, s);
    if (a.D <= 4096) return BwdGo<8, 1, WHOLE>::go(a, s);
    return a.D <= 8192 ? BwdGo<8, 2, WHOLE>::go(a, s) : BwdGo<16, 2, WHOLE>::go(a, s);
}

hipError_t launch_residual_norm(const ResidualNormArgs& a, hipStream_t s) {
    return a.D % 8 == 0 ? residual_fwd<true>(a, s) : residual_fwd<false>(a, s);
}
hipError_t launch_residual_norm_bwd(const ResidualNormBwdArgs& a, hipStream_t s) {
    const hipError_t e = a.D % 8 == 0 ? residual_bwd<true>(a, s) : residual_bwd<false>(a, s);
    if (e != hipSuccess) return e;
    return launch_sum_parts(a.partial, 2 * (size_t)a.D, a.parts, a.grad_scale ? 2L * a.D : a.D, a.grad_w, a.D, a.grad_scale,
                            s);
}

}  // namespace mesa
