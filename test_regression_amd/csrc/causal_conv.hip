// causal_conv.hip -- the short causal convolution over the rows of an input
// projection, and its gradients (gfx950).
//
// Per channel, with x_t = hist before t = 0 and n the row's length:
//   z_t = bias + sum_{j<W} w_j x_{t-j},   y_t = silu(z_t) = z_t sigmoid(z_t)   (t < n)
// Gradients, with dz_t = dy_t sigmoid(z_t) (1 + z_t (1 - sigmoid(z_t))) for t < n, else 0:
//   dx_t = sum_j w_j dz_{t+j},   dw_j = sum_{b,t} dz_t x_{t-j},   dbias = sum_{b,t} dz_t
// Without the activation y = z and dz = dy.
//
// HBM-bound: each input element is read once (but for the W - 1 rows around a
// thread's run of tokens) and each output element written once.  A thread takes
// eight neighbouring channels of a run of tokens and keeps the last rows in
// registers.  Sums are float32; outputs are rounded once.
#include <algorithm>

#include "io8.h"
#include "mesa_kernels.h"

namespace mesa {

__device__ __forceinline__ float conv_sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }
__device__ __forceinline__ float conv_sigmoid_exact(float z) { return 1.0f / (1.0f + expf(-z)); }
// bf16 outputs take the fast exponential (off by |z| 2^-24, little beside their rounding).
template <typename In>
__device__ __forceinline__ float conv_act(float z) { return sizeof(In) == 2 ? conv_sigmoid(z) : conv_sigmoid_exact(z); }

__device__ __forceinline__ int conv_length(const int32_t* lens, long b, int T) {
    return lens ? min(max(lens[b], 0), T) : T;
}

// Token t of the history followed by x (t >= -(W - 1)); zeros where there is none.
template <int W, bool WHOLE, typename In>
__device__ __forceinline__ f32x8 conv_row(const In* x, long ts, const In* hist, int t, int n, int D, int left) {
    if (t >= 0) return t < n ? load8_upto<WHOLE>(x + t * ts, left) : f32x8{};
    return hist ? load8_upto<WHOLE>(hist + (long)(t + W - 1) * D, left) : f32x8{};
}

// A thread's place: eight channels, a run of tokens, a batch row.
struct ConvPlace { int d0, left, t0; long b; };
__device__ __forceinline__ bool conv_place(long i, int D, int segs, int run, long B, ConvPlace* p) {
    const int pieces = (D + 7) / 8;
    const long r = i / pieces;
    p->d0 = 8 * (int)(i - r * pieces);
    p->left = D - p->d0;
    p->b = r / segs;
    p->t0 = (int)(r - p->b * segs) * run;
    return p->b < B;
}

template <int W, bool WHOLE, typename In>
__global__ __launch_bounds__(256) void causal_conv_kernel(ConvArgs a) {
    ConvPlace p;
    if (!conv_place((long)blockIdx.x * 256 + threadIdx.x, a.D, a.segs, a.run, a.B, &p)) return;
    const int n = conv_length(a.lens, p.b, a.T), D = a.D;
    const In* x = static_cast<const In*>(a.x) + p.b * a.xb + p.d0;
    const In* hist = a.hist ? static_cast<const In*>(a.hist) + p.b * (W - 1) * D + p.d0 : nullptr;
    In* y = static_cast<In*>(a.y) + p.b * (long)a.T * D + p.d0;
    f32x8 w[W], bias{}, last[W];   // last[j]: the row j tokens back
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = load8_upto<WHOLE>(a.w + (long)j * D + p.d0, p.left);
    if (a.bias) bias = load8_upto<WHOLE>(a.bias + p.d0, p.left);
#pragma unroll
    for (int j = 1; j < W; ++j) last[j - 1] = conv_row<W, WHOLE>(x, a.xt, hist, p.t0 - j, n, D, p.left);
    const int end = min(p.t0 + a.run, a.T);
    // the rows after this piece's last token, by the one thread that has read the
    // history: hist_out may be hist itself
    if (W > 1 && a.hist_out && p.t0 == 0) {
        f32x8 keep[W];
#pragma unroll
        for (int j = 1; j < W; ++j) keep[j - 1] = conv_row<W, WHOLE>(x, a.xt, hist, n - j, n, D, p.left);
        In* ho = static_cast<In*>(a.hist_out) + p.b * (W - 1) * D + p.d0;
#pragma unroll
        for (int j = 1; j < W; ++j) store8_upto<WHOLE>(ho + (long)(W - 1 - j) * D, keep[j - 1], p.left);
    }
    for (int t = p.t0; t < end; t += 4) {
        f32x8 in[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) in[i] = t + i < min(n, end) ? load8_upto<WHOLE>(x + (long)(t + i) * a.xt, p.left) : f32x8{};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (t + i >= end) break;
            f32x8 o{};
            if (t + i < n)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float z = bias.v[e] + w[0].v[e] * in[i].v[e];
#pragma unroll
                    for (int j = 1; j < W; ++j) z += w[j].v[e] * last[j - 1].v[e];
                    o.v[e] = a.silu ? z * conv_act<In>(z) : z;
                }
            store8_upto<WHOLE>(y + (long)(t + i) * D, o, p.left);
#pragma unroll
            for (int j = W - 1; j > 1; --j) last[j - 1] = last[j - 2];
            if (W > 1) last[0] = in[i];
        }
    }
}

// A workgroup takes 32 pieces of eight channels and eight runs of tokens of one
// batch row, so that the weights' gradients are summed in LDS over the runs and
// written once a workgroup: partial[part][W + 1][D].
constexpr int kConvPieces = 32, kConvRuns = 8;
template <int W, bool WHOLE, typename In>
__global__ __launch_bounds__(256) void causal_conv_bwd_kernel(ConvBwdArgs a) {
    __shared__ float red[kConvRuns][kConvPieces * 8 + 4];
    const int piece = threadIdx.x % kConvPieces, slot = threadIdx.x / kConvPieces, D = a.f.D;
    const int groups = (D + 8 * kConvPieces - 1) / (8 * kConvPieces);
    const long part = blockIdx.x / groups;
    const int d0 = 8 * ((int)(blockIdx.x - part * groups) * kConvPieces + piece), left = D - d0;
    const long b = part / a.f.segs;
    const int run = a.f.run, t0 = ((int)(part - b * a.f.segs) * kConvRuns + slot) * run;
    const bool live = left > 0 && t0 < a.f.T;
    f32x8 dw[W + 1] = {};   // the weights', then the bias's
    if (live) {
        const int n = conv_length(a.f.lens, b, a.f.T), end = min(t0 + run, a.f.T);
        const In* x = static_cast<const In*>(a.f.x) + b * a.f.xb + d0;
        const In* dy = static_cast<const In*>(a.grad_y) + b * (long)a.f.T * D + d0;
        const In* hist = a.f.hist ? static_cast<const In*>(a.f.hist) + b * (W - 1) * D + d0 : nullptr;
        In* dx = static_cast<In*>(a.grad_x) + b * a.gxb + d0;
        f32x8 w[W], bias{}, last[W], dz[W];   // last[j]: x of j + 1 tokens back; dz[j]: of j tokens back
#pragma unroll
        for (int j = 0; j < W; ++j) w[j] = load8_upto<WHOLE>(a.f.w + (long)j * D + d0, left);
        if (a.f.bias) bias = load8_upto<WHOLE>(a.f.bias + d0, left);
#pragma unroll
        for (int j = 1; j < W; ++j) last[j - 1] = conv_row<W, WHOLE>(x, a.f.xt, hist, t0 - j, n, D, left);
#pragma unroll
        for (int j = 0; j < W; ++j) dz[j] = f32x8{};
        // dx of a token is complete W - 1 tokens later; the last of them are the next run's
        const int stop = end + W - 1;
        for (int t = t0; t < stop; t += 4) {
            f32x8 in[4], g[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool on = t + i < min(n, stop);
                in[i] = on ? load8_upto<WHOLE>(x + (long)(t + i) * a.f.xt, left) : f32x8{};
                g[i] = on ? load8_upto<WHOLE>(dy + (long)(t + i) * D, left) : f32x8{};
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = t + i;
                if (at >= stop) break;
                f32x8 cur{};
                if (at < n)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float z = bias.v[e] + w[0].v[e] * in[i].v[e];
#pragma unroll
                        for (int j = 1; j < W; ++j) z += w[j].v[e] * last[j - 1].v[e];
                        const float s = a.f.silu ? conv_act<In>(z) : 1.0f;
                        cur.v[e] = a.f.silu ? g[i].v[e] * s * (1.0f + z * (1.0f - s)) : g[i].v[e];
                    }
                if (at < end)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        dw[0].v[e] += cur.v[e] * in[i].v[e];
#pragma unroll
                        for (int j = 1; j < W; ++j) dw[j].v[e] += cur.v[e] * last[j - 1].v[e];
                        dw[W].v[e] += cur.v[e];
                    }
#pragma unroll
                for (int j = W - 1; j > 0; --j) dz[j] = dz[j - 1];
                dz[0] = cur;
                const int to = at - (W - 1);
                if (to >= t0 && to < end) {
                    f32x8 o{};
#pragma unroll
                    for (int e = 0; e < 8; ++e)
#pragma unroll
                        for (int j = 0; j < W; ++j) o.v[e] += w[j].v[e] * dz[W - 1 - j].v[e];
                    store8_upto<WHOLE>(dx + (long)to * a.gxt, o, left);
                }
                // the history's rows see the first W - 1 tokens only: row i (token i - (W - 1))
                // takes w_j dz_{i - (W - 1) + j}, all of which are known after token i
                if (W > 1 && t0 == 0 && a.grad_hist && at < W - 1) {
                    f32x8 o{};
#pragma unroll
                    for (int e = 0; e < 8; ++e)
#pragma unroll
                        for (int j = 1; j < W; ++j)
                            if (W - 1 - j <= at) o.v[e] += w[j].v[e] * dz[W - 1 - j].v[e];
                    store8_upto<WHOLE>(static_cast<In*>(a.grad_hist) + (b * (W - 1) + at) * D + d0, o, left);
                }
#pragma unroll
                for (int j = W - 1; j > 1; --j) last[j - 1] = last[j - 2];
                if (W > 1) last[0] = in[i];
            }
        }
    }
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        __syncthreads();
        *reinterpret_cast<f32x4*>(&red[slot][8 * piece]) = f32x4{dw[j].v[0], dw[j].v[1], dw[j].v[2], dw[j].v[3]};
        *reinterpret_cast<f32x4*>(&red[slot][8 * piece + 4]) = f32x4{dw[j].v[4], dw[j].v[5], dw[j].v[6], dw[j].v[7]};
        __syncthreads();
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < kConvRuns; ++r) sum += red[r][threadIdx.x];
        const int d = d0 - 8 * piece + (int)threadIdx.x;
        if (d < D) a.partial[(part * (W + 1) + j) * D + d] = sum;
    }
}

// grad_w [W][D] and grad_bias [D] over the parts: 64 columns of the partial rows a
// workgroup, four runs of parts side by side.
__global__ __launch_bounds__(256) void conv_sums_kernel(const float* partial, long parts, int W, int D, float* grad_w,
                                                        float* grad_bias) {
    __shared__ float red[4][64];
    const long col = (long)blockIdx.x * 64 + threadIdx.x % 64, cols = (long)(W + 1) * D;
    const int slot = threadIdx.x / 64;
    float s = 0.f;
    if (col < cols)
        for (long p = slot; p < parts; p += 4) s += partial[p * cols + col];
    red[slot][threadIdx.x % 64] = s;
    __syncthreads();
    if (slot != 0 || col >= cols) return;
    s = (red[0][threadIdx.x] + red[1][threadIdx.x]) + (red[2][threadIdx.x] + red[3][threadIdx.x]);
    if (col < (long)W * D) grad_w[col] = s;
    else if (grad_bias) grad_bias[col - (long)W * D] = s;
}

template <int W, typename In>
static void conv_go(const ConvArgs& a, unsigned blocks, hipStream_t s) {
    if (a.D % 8 == 0) hipLaunchKernelGGL((causal_conv_kernel<W, true, In>), dim3(blocks), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((causal_conv_kernel<W, false, In>), dim3(blocks), dim3(256), 0, s, a);
}
template <int W>
static void conv_dtype(const ConvArgs& a, unsigned blocks, hipStream_t s) {
    if (a.bf16) conv_go<W, bf16_t>(a, blocks, s);
    else conv_go<W, float>(a, blocks, s);
}

hipError_t launch_causal_conv(ConvArgs a, hipStream_t s) {
    a.run = kConvRun;
    a.segs = std::max(1, (a.T + a.run - 1) / a.run);   // without a token the history still moves on
    const unsigned blocks = (unsigned)(((long)a.B * a.segs * ((a.D + 7) / 8) + 255) / 256);
    switch (a.W) {
        case 1: conv_dtype<1>(a, blocks, s); break;
        case 2: conv_dtype<2>(a, blocks, s); break;
        case 3: conv_dtype<3>(a, blocks, s); break;
        case 4: conv_dtype<4>(a, blocks, s); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

template <int W, typename In>
static void conv_bwd_go(const ConvBwdArgs& a, unsigned blocks, hipStream_t s) {
    if (a.f.D % 8 == 0) hipLaunchKernelGGL((causal_conv_bwd_kernel<W, true, In>), dim3(blocks), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((causal_conv_bwd_kernel<W, false, In>), dim3(blocks), dim3(256), 0, s, a);
}
template <int W>
static void conv_bwd_dtype(const ConvBwdArgs& a, unsigned blocks, hipStream_t s) {
    if (a.f.bf16) conv_bwd_go<W, bf16_t>(a, blocks, s);
    else conv_bwd_go<W, float>(a, blocks, s);
}

long conv_bwd_parts(long B, int T) { return B * ((T + (long)kConvRun * kConvRuns - 1) / ((long)kConvRun * kConvRuns)); }

hipError_t launch_causal_conv_bwd(ConvBwdArgs a, hipStream_t s) {
    a.f.run = kConvRun;
    a.f.segs = (int)((a.f.T + (long)kConvRun * kConvRuns - 1) / ((long)kConvRun * kConvRuns));
    const long parts = conv_bwd_parts(a.f.B, a.f.T);
    const unsigned blocks = (unsigned)(parts * ((a.f.D + 8 * kConvPieces - 1) / (8 * kConvPieces)));
    switch (a.f.W) {
        case 1: conv_bwd_dtype<1>(a, blocks, s); break;
        case 2: conv_bwd_dtype<2>(a, blocks, s); break;
        case 3: conv_bwd_dtype<3>(a, blocks, s); break;
        case 4: conv_bwd_dtype<4>(a, blocks, s); break;
        default: return hipErrorInvalidValue;
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const long cols = (long)(a.f.W + 1) * a.f.D;
    hipLaunchKernelGGL(conv_sums_kernel, dim3((unsigned)((cols + 63) / 64)), dim3(256), 0, s, a.partial, parts, a.f.W, a.f.D,
                       a.grad_w, a.grad_bias);
    return hipGetLastError();
}

}  // namespace mesa
