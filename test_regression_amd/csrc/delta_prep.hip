// delta_prep.hip -- the state-free matrices of every chunk of the gated delta
// rule (gfx950): M = (I + A diag(b))^-1 and P (delta_core.h), with the scales
// and gate factors the passes over the chunks use.
//
// One workgroup of four waves per chunk and head.  The decays are formed as
// exp(L_i - L_j) from the chunk's prefix sums L of ln g in double: in float the
// sums' rounding alone would put 1e-5 on the decays of a strongly gated chunk.
// Wave w forms the 16-row block w of K K^T and Q K^T (all four column blocks,
// those above the diagonal being dropped: an accumulator that only some waves
// use was kept in registers that the next MFMAs' inputs reuse too early).  M comes block by block in float: the four 16 x 16 diagonal
// blocks by forward substitution, one a wave with a column a lane, then the
// blocks below by diagonals, M_ij = -M_ii sum_{j<=k<i} (A diag b)_ik M_kj, on
// float MFMAs whose accumulator order is the next product's operand order.
// M is kept to 22 bits (its errors reach the state); P to 11 for bf16
// outputs, whose own rounding is 8 times coarser, and to 22 for float ones and
// for the gradients (those of the gates are float32 sums over P).
#include "delta_core.h"

namespace mesa {

template <int DKP, int NP>
struct alignas(16) PrepLds {
    static constexpr int KW = delta_row_words(DKP);
    uint32_t K[NP][kDC * KW];
    union {
        uint32_t Q[NP][kDC * KW];
        float M[kDC * kDF];
    };
    float N[kDC * kDF];   // A diag(b); after the inverse, P
    double L[kDC];
    float beta[kDC], ks[kDC], qs[kDC], mi[kDC], pi[kDC];
};

// Rows of a float matrix in LDS as fp16 planes of perm32 rows in memory, each
// row scaled by a power of two whose inverse goes to inv[row].
template <int PLANES>
__device__ __forceinline__ void planes_out(const float* F, uint16_t* img, float* inv) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int unit = threadIdx.x + 256 * h, row = unit / 8, q = unit % 8, b = q / 4, g = q % 4;
        const f32x4 x = *reinterpret_cast<const f32x4*>(F + row * kDF + 32 * b + 4 * g);
        const f32x4 y = *reinterpret_cast<const f32x4*>(F + row * kDF + 32 * b + 16 + 4 * g);
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) m = fmaxf(m, fmaxf(fabsf(x[e]), fabsf(y[e])));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
        const int E = h2_exp(m);
        f16x8 hi, lo;
        h2_split(x, y, pow2(E), hi, lo);
        *reinterpret_cast<f16x8*>(img + row * kDC + 8 * q) = hi;
        if constexpr (PLANES == 2) *reinterpret_cast<f16x8*>(img + kDC * kDC + row * kDC + 8 * q) = lo;
        if (q == 0) inv[row] = pow2(-E);
    }
}

template <int DKP, typename In, int PP>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaArgs a) {
    constexpr int NP = delta_planes<In>(), NJ = DKP / 32, KW = delta_row_words(DKP);
    __shared__ PrepLds<DKP, NP> L;
    const int lane = threadIdx.x % 64, w = threadIdx.x / 64, n = lane & 15, g = lane >> 4;
    const int c = (int)(blockIdx.x % a.nc);
    const long bh = blockIdx.x / a.nc;
    const long bk = (bh / a.H) * a.Hk + (bh % a.H) / (a.H / a.Hk);
    const int valid = min(kDC, a.T - c * kDC);
    const size_t tok = (size_t)bh * a.T + (size_t)c * kDC;
    const size_t ktok = ((size_t)bk * a.T + (size_t)c * kDC) * a.dk;
    using Units = RowUnits<DKP, In>;
    {
        Units k, q;
        k.load(static_cast<const In*>(a.k) + ktok, a.dk, valid);
        q.load(static_cast<const In*>(a.q) + ktok, a.dk, valid);
        if (w == 0) {
            // a gate of 0 (a reset) counts as e^-200, which is 0 in float
            double x = lane < valid ? fmax(log((double)a.gamma[tok + lane]), -200.0) : 0.0;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const double t = __shfl_up(x, o, 64);
                if (lane >= o) x += t;
            }
            L.L[lane] = x;
            L.beta[lane] = lane < valid ? a.beta[tok + lane] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < Units::n; ++i) {
            float mk = k.absmax(i), mq = q.absmax(i);
#pragma unroll
            for (int o = 1; o < Units::per_row; o <<= 1) {
                mk = fmaxf(mk, __shfl_xor(mk, o, 64));
                mq = fmaxf(mq, __shfl_xor(mq, o, 64));
            }
            const float sk = pow2(h2_exp(mk)), sq = pow2(h2_exp(mq));
            k.template store<NP>(L.K, i, sk);
            q.template store<NP>(L.Q, i, sq);
            if (Units::col(i) == 0) {
                L.ks[Units::row(i)] = sk;
                L.qs[Units::row(i)] = sq;
            }
        }
    }
    __syncthreads();
    // ---- rows 16 w .. 16 w + 15 of K K^T and Q K^T ----
    const f32x4 zero{0.f, 0.f, 0.f, 0.f};
    f32x4 P[4];
    {
        f32x4 A[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) A[j] = P[j] = zero;
#pragma unroll
        for (int s = 0; s < NJ; ++s) {
            const f16x8 kh = row_operand(L.K[0], KW, w, s, n, g), qh = row_operand(L.Q[0], KW, w, s, n, g);
            f16x8 kl = kh, ql = qh;
            if constexpr (NP == 2) {
                kl = row_operand(L.K[1], KW, w, s, n, g);
                ql = row_operand(L.Q[1], KW, w, s, n, g);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f16x8 bh_ = row_operand(L.K[0], KW, j, s, n, g);
                A[j] = mfma_f16x32(kh, bh_, A[j]);
                P[j] = mfma_f16x32(qh, bh_, P[j]);
                if constexpr (NP == 2) {
                    const f16x8 bl = row_operand(L.K[1], KW, j, s, n, g);
                    A[j] = mfma_f16x32(kl, bh_, A[j]);
                    P[j] = mfma_f16x32(ql, bh_, P[j]);
                    A[j] = mfma_f16x32(kh, bl, A[j]);
                    P[j] = mfma_f16x32(qh, bl, P[j]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = 16 * j + n;
            const double Lj = L.L[col];
            const float kj = 1.0f / L.ks[col], bj = L.beta[col];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * w + 4 * g + r;
                const float D = row >= col ? expf((float)(L.L[row] - Lj)) : 0.f;
                const float ki = 1.0f / L.ks[row], qi = 1.0f / L.qs[row];
                P[j][r] = row >= col ? P[j][r] * kj * qi * D : 0.f;
                L.N[row * kDF + col] = row > col ? A[j][r] * kj * ki * D * bj : 0.f;
            }
        }
    }
    __syncthreads();   // Q is read: M takes its place
    // ---- M's diagonal blocks; zeros above the diagonal ----
    {
        const float* Nd = L.N + 16 * w * kDF + 16 * w;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s0 = i == n ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
            for (int j4 = 0; j4 < (i + 3) / 4; ++j4) {
                const f32x4 r = *reinterpret_cast<const f32x4*>(Nd + i * kDF + 4 * j4);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = 4 * j4 + e;
                    if (j >= i) continue;
                    if (j & 1) s1 -= r[e] * x[j]; else s0 -= r[e] * x[j];
                }
            }
            x[i] = s0 + s1;
        }
        if (g == 0)
#pragma unroll
            for (int i = 0; i < 16; ++i) L.M[(16 * w + i) * kDF + 16 * w + n] = x[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j <= w) continue;
#pragma unroll
            for (int r = 0; r < 4; ++r) L.M[(16 * w + 4 * g + r) * kDF + 16 * j + n] = 0.f;
        }
    }
    __syncthreads();
    // ---- the blocks below, diagonal by diagonal ----
#pragma unroll
    for (int d = 1; d < 4; ++d) {
        if (w >= d) {
            const int j = w - d;
            f32x4 t = zero;
#pragma unroll
            for (int o = 0; o < d; ++o) {
                const int kb = j + o;
                const f32x4 x = *reinterpret_cast<const f32x4*>(L.N + (16 * w + n) * kDF + 16 * kb + 4 * g);
#pragma unroll
                for (int s = 0; s < 4; ++s) t = mfma4(x[s], L.M[(16 * kb + 4 * g + s) * kDF + 16 * j + n], t);
            }
            const f32x4 y = *reinterpret_cast<const f32x4*>(L.M + (16 * w + n) * kDF + 16 * w + 4 * g);
            f32x4 u = zero;
#pragma unroll
            for (int s = 0; s < 4; ++s) u = mfma4(y[s], t[s], u);
#pragma unroll
            for (int r = 0; r < 4; ++r) L.M[(16 * w + 4 * g + r) * kDF + 16 * j + n] = -u[r];
        }
        __syncthreads();
    }
    // ---- out: planes of M and P, scalars ----
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) L.N[(16 * w + 4 * g + r) * kDF + 16 * j + n] = P[j][r];
    uint16_t* img = a.img + (size_t)blockIdx.x * ((2 + PP) * kDC * kDC);
    planes_out<2>(L.M, img, L.mi);
    __syncthreads();
    planes_out<PP>(L.N, img + 2 * kDC * kDC, L.pi);
    __syncthreads();
    if (threadIdx.x < kDC) {
        const int t = threadIdx.x;
        float* sc = a.scal + (size_t)blockIdx.x * kScal;
        const double Lt = L.L[t], Lc = L.L[kDC - 1];
        const float G = expf((float)Lt), ki = 1.0f / L.ks[t];
        sc[kKs + t] = L.ks[t];
        sc[kQs + t] = L.qs[t];
        sc[kGk + t] = G * ki;
        sc[kGq + t] = G / L.qs[t];
        sc[kMi + t] = L.mi[t];
        sc[kPi + t] = L.pi[t];
        sc[kDc + t] = expf((float)(Lc - Lt)) * ki;
        sc[kBe + t] = L.beta[t];
        if (t == kDC - 1) sc[kGc] = G;
    }
}

template <int DKP>
hipError_t prep_go(const DeltaArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.BH * a.nc));
    if (!a.bf16) hipLaunchKernelGGL((delta_prep_kernel<DKP, float, 2>), grid, dim3(256), 0, s, a);
    else if (a.p_planes == 2) hipLaunchKernelGGL((delta_prep_kernel<DKP, bf16_t, 2>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((delta_prep_kernel<DKP, bf16_t, 1>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_delta_prep(const DeltaArgs& a, hipStream_t s) {
    return a.dk <= 32 ? prep_go<32>(a, s) : a.dk == 64 ? prep_go<64>(a, s) : prep_go<128>(a, s);
}

}  // namespace mesa
