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
// thread's run of tokens) and each output element written once.  A thread takes four
// neighbouring channels of a run of tokens, keeps the last rows in registers and has
// the next ones on their way; eight channels a thread left half as many waves and no
// registers to load ahead with.  Sums are float32; outputs are rounded once.  8 x 4096
// tokens, 2304 channels, W 4, bfloat16: 64 us (4.7 TB/s), with eight channels 83 us;
// the gradients 97-100 us (4.6 TB/s) and 4 us for the parts' sums, with eight channels 204
// and 10 us, with four and no loads ahead 129 us.
#include <algorithm>

#include "io8.h"
#include "mesa_kernels.h"

namespace mesa {

__device__ __forceinline__ float conv_sigmoid_exact(float z) { return 1.0f / (1.0f + expf(-z)); }
// Outputs in bfloat16 take the fast exponential (off by |z| 2^-24, little beside their
// rounding).
template <typename In>
__device__ __forceinline__ float conv_act(float z) {
    return sizeof(In) == 2 ? __builtin_amdgcn_rcpf(1.0f + __expf(-z)) : conv_sigmoid_exact(z);
}
// The weights' gradients are float32 for bfloat16 rows too: what the power's rounding left
// of z is put back to first order (beyond 88, where float32 ends, as at 88).  64 x 8192
// tokens, 1024 channels: 656 us without it, 675 us with it, 710 us with expf.
template <typename In>
__device__ __forceinline__ float conv_act_bwd(float z) {
    if constexpr (sizeof(In) == 4) return conv_sigmoid_exact(z);
    const float x = __builtin_amdgcn_fmed3f(z, -88.0f, 88.0f), power = x * -1.442695041f, e = __builtin_amdgcn_exp2f(power);
    return __builtin_amdgcn_rcpf(1.0f + fmaf(e, fmaf(power, -0.6931471806f, -x), e));
}

__device__ __forceinline__ int conv_length(const int32_t* lens, long b, int T) {
    return lens ? min(max(lens[b], 0), T) : T;
}

// Token t of the history followed by x (t >= -(W - 1)); zeros where there is none.
template <int W, bool WHOLE, typename In>
__device__ __forceinline__ f32x4 conv_row(const In* x, long ts, const In* hist, int t, int n, int D, int left) {
    if (t >= 0) return t < n ? load4_upto<WHOLE>(x + t * ts, left) : f32x4{};
    return hist ? load4_upto<WHOLE>(hist + (long)(t + W - 1) * D, left) : f32x4{};
}

constexpr int kConvChannels = 4;   // of a thread

// A thread's place: kConvChannels channels, a run of tokens, a batch row.
struct ConvPlace { int d0, left, t0; long b; };
__device__ __forceinline__ bool conv_place(long i, int D, int segs, int run, long B, ConvPlace* p) {
    const int pieces = (D + kConvChannels - 1) / kConvChannels;
    const long r = i / pieces;
    p->d0 = kConvChannels * (int)(i - r * pieces);
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
    f32x4 w[W], bias{}, last[W];   // last[j]: the row j tokens back
#pragma unroll
    for (int j = 0; j < W; ++j) w[j] = load4_upto<WHOLE>(a.w + (long)j * D + p.d0, p.left);
    if (a.bias) bias = load4_upto<WHOLE>(a.bias + p.d0, p.left);
#pragma unroll
    for (int j = 1; j < W; ++j) last[j - 1] = conv_row<W, WHOLE>(x, a.xt, hist, p.t0 - j, n, D, p.left);
    const int end = min(p.t0 + a.run, a.T);
    // the rows after this piece's last token, by the one thread that has read the
    // history: hist_out may be hist itself
    if (W > 1 && a.hist_out && p.t0 == 0) {
        f32x4 keep[W];
#pragma unroll
        for (int j = 1; j < W; ++j) keep[j - 1] = conv_row<W, WHOLE>(x, a.xt, hist, n - j, n, D, p.left);
        In* ho = static_cast<In*>(a.hist_out) + p.b * (W - 1) * D + p.d0;
#pragma unroll
        for (int j = 1; j < W; ++j) store4_upto<WHOLE>(ho + (long)(W - 1 - j) * D, keep[j - 1], p.left);
    }
    Held4<WHOLE, In> held[4];   // the next four rows, on their way
    auto fetch = [&](int t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            held[i].clear();
            if (t + i < min(n, end)) held[i].load(x + (long)(t + i) * a.xt, p.left);
        }
    };
    fetch(p.t0);
    for (int t = p.t0; t < end; t += 4) {
        f32x4 in[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) in[i] = held[i].get();
        fetch(t + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (t + i >= end) break;
            f32x4 o{};
            if (t + i < n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float z = bias[e] + w[0][e] * in[i][e];
#pragma unroll
                    for (int j = 1; j < W; ++j) z += w[j][e] * last[j - 1][e];
                    o[e] = a.silu ? z * conv_act<In>(z) : z;
                }
            store4_upto<WHOLE>(y + (long)(t + i) * D, o, p.left);
#pragma unroll
            for (int j = W - 1; j > 1; --j) last[j - 1] = last[j - 2];
            if (W > 1) last[0] = in[i];
        }
    }
}

// A workgroup takes 64 pieces of four channels and eight runs of tokens of one
// batch row, so that the weights' gradients are summed in LDS over the runs and
// written once a workgroup: partial[part][W + 1][D].  A thread adds its run's tokens in
// float32, kConvMost at most, so that a sum's error does not grow with the length; the
// parts are joined in float64.
constexpr int kConvMost = 256;
constexpr int kConvPieces = 64, kConvRuns = 8, kConvThreads = kConvPieces * kConvRuns, kConvColumns = kConvPieces * kConvChannels;
template <int W, bool WHOLE, typename In>
__global__ __launch_bounds__(kConvThreads) void causal_conv_bwd_kernel(ConvBwdArgs a) {
    constexpr int R = WHOLE && sizeof(In) == 2 ? 4 : 2;   // as many rows ahead as 128 registers hold
    __shared__ float red[kConvRuns][kConvPieces * kConvChannels + 4];
    // a wave's lanes are the pieces of one run
    const int piece = threadIdx.x % kConvPieces, slot = __builtin_amdgcn_readfirstlane(threadIdx.x / kConvPieces), D = a.f.D;
    const int groups = (D + kConvColumns - 1) / kConvColumns;
    const long part = blockIdx.x / groups;
    const int d0 = kConvChannels * ((int)(blockIdx.x - part * groups) * kConvPieces + piece), left = D - d0;
    const long b = part / a.f.segs;
    const int run = a.f.run, t0 = ((int)(part - b * a.f.segs) * kConvRuns + slot) * run;
    const bool live = left > 0 && t0 < a.f.T;
    f32x4 dw[W + 1] = {};   // the weights', then the bias's
    if (live) {
        const int n = conv_length(a.f.lens, b, a.f.T), end = min(t0 + run, a.f.T);
        const In* x = static_cast<const In*>(a.f.x) + b * a.f.xb + d0;
        const In* dy = static_cast<const In*>(a.grad_y) + b * (long)a.f.T * D + d0;
        const In* hist = a.f.hist ? static_cast<const In*>(a.f.hist) + b * (W - 1) * D + d0 : nullptr;
        In* dx = static_cast<In*>(a.grad_x) + b * a.gxb + d0;
        f32x4 w[W], bias{}, last[W], dz[W];   // last[j]: x of j + 1 tokens back; dz[j]: of j tokens back
#pragma unroll
        for (int j = 0; j < W; ++j) w[j] = load4_upto<WHOLE>(a.f.w + (long)j * D + d0, left);
        if (a.f.bias) bias = load4_upto<WHOLE>(a.f.bias + d0, left);
#pragma unroll
        for (int j = 1; j < W; ++j) last[j - 1] = conv_row<W, WHOLE>(x, a.f.xt, hist, t0 - j, n, D, left);
#pragma unroll
        for (int j = 0; j < W; ++j) dz[j] = f32x4{};
        // dx of a token is complete W - 1 tokens later; the last of them are the next run's
        const int stop = end + W - 1;
        Held4<WHOLE, In> hx[R], hg[R];   // the next rows, on their way
        auto fetch = [&](int t) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                hx[i].clear();
                hg[i].clear();
                if (t + i >= min(n, stop)) continue;
                hx[i].load(x + (long)(t + i) * a.f.xt, left);
                hg[i].load(dy + (long)(t + i) * D, left);
            }
        };
        fetch(t0);
        for (int t = t0; t < stop; t += R) {
            f32x4 in[R], g[R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                in[i] = hx[i].get();
                g[i] = hg[i].get();
            }
            fetch(t + R);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int at = t + i;
                if (at >= stop) break;
                f32x4 cur{};
                if (at < n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float z = bias[e] + w[0][e] * in[i][e];
#pragma unroll
                        for (int j = 1; j < W; ++j) z += w[j][e] * last[j - 1][e];
                        const float s = a.f.silu ? conv_act_bwd<In>(z) : 1.0f;
                        cur[e] = a.f.silu ? g[i][e] * s * (1.0f + z * (1.0f - s)) : g[i][e];
                    }
                if (at < end)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        dw[0][e] += cur[e] * in[i][e];
#pragma unroll
                        for (int j = 1; j < W; ++j) dw[j][e] += cur[e] * last[j - 1][e];
                        dw[W][e] += cur[e];
                    }
#pragma unroll
                for (int j = W - 1; j > 0; --j) dz[j] = dz[j - 1];
                dz[0] = cur;
                const int to = at - (W - 1);
                if (to >= t0 && to < end) {
                    f32x4 o{};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int j = 0; j < W; ++j) o[e] += w[j][e] * dz[W - 1 - j][e];
                    store4_upto<WHOLE>(dx + (long)to * a.gxt, o, left);
                }
                // the history's rows see the first W - 1 tokens only: row i (token i - (W - 1))
                // takes w_j dz_{i - (W - 1) + j}, all of which are known after token i
                if (W > 1 && t0 == 0 && a.grad_hist && at < W - 1) {
                    f32x4 o{};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int j = 1; j < W; ++j)
                            if (W - 1 - j <= at) o[e] += w[j][e] * dz[W - 1 - j][e];
                    store4_upto<WHOLE>(static_cast<In*>(a.grad_hist) + (b * (W - 1) + at) * D + d0, o, left);
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
        *reinterpret_cast<f32x4*>(&red[slot][kConvChannels * piece]) = dw[j];
        __syncthreads();
        if (threadIdx.x >= kConvColumns) continue;
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < kConvRuns; ++r) sum += red[r][threadIdx.x];
        const int d = d0 - kConvChannels * piece + (int)threadIdx.x;
        if (d < D) a.partial[(part * (W + 1) + j) * D + d] = sum;
    }
}

// grad_w [W][D] and grad_bias [D] over the parts: 32 columns of the partial rows a
// workgroup, eight runs of parts side by side.
__global__ __launch_bounds__(256) void conv_sums_kernel(const float* partial, long parts, int W, int D, float* grad_w,
                                                        float* grad_bias) {
    __shared__ double red[8][32];
    const long col = (long)blockIdx.x * 32 + threadIdx.x % 32, cols = (long)(W + 1) * D;
    const int slot = threadIdx.x / 32;
    red[slot][threadIdx.x % 32] = col < cols ? strided_sum(partial + col, slot, parts, 8, cols) : 0.0;
    __syncthreads();
    if (slot != 0 || col >= cols) return;
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += red[i][threadIdx.x];
    if (col < (long)W * D) grad_w[col] = (float)s;
    else if (grad_bias) grad_bias[col - (long)W * D] = (float)s;
}

template <int W, typename In>
static void conv_go(const ConvArgs& a, unsigned blocks, hipStream_t s) {
    if (a.D % kConvChannels == 0) hipLaunchKernelGGL((causal_conv_kernel<W, true, In>), dim3(blocks), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((causal_conv_kernel<W, false, In>), dim3(blocks), dim3(256), 0, s, a);
}
template <int W>
static void conv_dtype(const ConvArgs& a, unsigned blocks, hipStream_t s) {
    if (a.bf16) conv_go<W, bf16_t>(a, blocks, s);
    else conv_go<W, float>(a, blocks, s);
}

// Tokens a thread.  Workgroups that one more round over the card would be needed for
// cost as much as a full round, and the rows around a run are read again: of the runs
// that make one to six rounds the one with the fewest rows to go over, if a run of
// `side` threads over T tokens makes `blocks` workgroups and `slots` of them fit; no run
// of more than `most`.  The slots are those of W = 4 (seven workgroups a CU in bfloat16,
// five otherwise); narrower windows fit up to eight, and their own counts gain 2.5 % at
// 64 x 8192 x 1024 in bfloat16 and lose 4 % at 8 x 4096 x 2304 in float32.
static int conv_run(int T, double blocks, int slots, int side, int W, int most) {
    int best = 1;
    double least = 0.0;
    for (int k = 1; k <= 6; ++k) {
        const long splits = std::max(1L, (long)(k * slots / blocks));
        const int run = (int)std::min<long>(most, std::max<long>(std::min(T, kConvLeast), (T + splits * side - 1) / (splits * side)));
        if (run < 1) return 1;   // no tokens
        const double groups = (T + (long)run * side - 1) / ((long)run * side) * blocks;
        const double rows = (double)(long)((groups + slots - 1) / slots) * (run + 2 * (W - 1));
        if (k == 1 || rows < least) {
            best = run;
            least = rows;
        }
    }
    return best;
}

hipError_t launch_causal_conv(ConvArgs a, hipStream_t s) {
    const long pieces = (a.D + kConvChannels - 1) / kConvChannels;
    a.run = conv_run(a.T, (double)a.B * pieces / 256, 256 * (a.bf16 && a.D % kConvChannels == 0 ? 7 : 5), 1, a.W, std::max(a.T, 1));
    a.segs = std::max(1, (a.T + a.run - 1) / a.run);   // without a token the history still moves on
    const unsigned blocks = (unsigned)(((long)a.B * a.segs * pieces + 255) / 256);
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
    if (a.f.D % kConvChannels == 0) hipLaunchKernelGGL((causal_conv_bwd_kernel<W, true, In>), dim3(blocks), dim3(kConvThreads), 0, s, a);
    else hipLaunchKernelGGL((causal_conv_bwd_kernel<W, false, In>), dim3(blocks), dim3(kConvThreads), 0, s, a);
}
template <int W>
static void conv_bwd_dtype(const ConvBwdArgs& a, unsigned blocks, hipStream_t s) {
    if (a.f.bf16) conv_bwd_go<W, bf16_t>(a, blocks, s);
    else conv_bwd_go<W, float>(a, blocks, s);
}

long conv_bwd_parts(long B, int T) { return B * ((T + (long)kConvLeast * kConvRuns - 1) / ((long)kConvLeast * kConvRuns)); }

hipError_t launch_causal_conv_bwd(ConvBwdArgs a, hipStream_t s) {
    const long groups = (a.f.D + kConvColumns - 1) / kConvColumns;
    a.f.run = conv_run(a.f.T, (double)a.f.B * groups, 256 * 2, kConvRuns, a.f.W, kConvMost);
    a.f.segs = (int)((a.f.T + (long)a.f.run * kConvRuns - 1) / ((long)a.f.run * kConvRuns));
    const long parts = (long)a.f.B * a.f.segs;
    const unsigned blocks = (unsigned)(parts * groups);
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
    hipLaunchKernelGGL(conv_sums_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(256), 0, s, a.partial, parts, a.f.W, a.f.D,
                       a.grad_w, a.grad_bias);
    return hipGetLastError();
}

}  // namespace mesa
