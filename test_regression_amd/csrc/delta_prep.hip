// delta_prep.hip -- the state-free matrices of every chunk of the gated delta
// rule (gfx950): M = (I + A diag(b))^-1 and P diag(b) (delta_core.h), with the
// scales and gate factors the passes over the chunks use.
//
// One workgroup of four waves per chunk and head.  The decays are
// 2^(L_i - L_j) from the chunk's prefix sums L of log2 g in double: in float
// the sums' rounding alone would put 1e-5 on the decays of a strongly gated
// chunk.  A 16 x 16 block below the diagonal takes them as 2^(L_i - m)
// 2^(m - L_j) with m at the end of the block's columns (both factors are at
// most 1), so that a lane evaluates five exponentials and not sixteen.
// Wave w forms the 16-row block w of K K^T and Q K^T (all four column blocks,
// those above the diagonal being dropped: an accumulator that only some waves
// use was kept in registers that the next MFMAs' inputs reuse too early).
// M comes block by block in float: the four 16 x 16 diagonal
// blocks by forward substitution, one a wave with a column a lane, then the
// blocks below by diagonals, M_ij = -M_ii sum_{j<=k<i} (A diag b)_ik M_kj, on
// float MFMAs whose accumulator order is the next product's operand order.
// M is kept to 22 bits (its errors reach the state), and so is P for float
// outputs and for the gradients (those of the gates are float32 sums over P).
// For bf16 outputs P's second part is rounded to a byte, the upper half of its
// fp16 pattern: P is then off by at most 2^-11 2^-3 = 2^-14 of an element, a
// 32nd of the outputs' own smallest half step, for three quarters of the memory.
//
// 8x16x4096, dk = 128, bf16: 102-125 us for 273 MB of keys, queries and gates in
// and 189 MB of planes out, 3.7-4.5 TB/s; vector instructions take 59 % of the cycles.
#include "delta_core.h"

namespace mesa {

template <int DKP, int NP>
struct alignas(16) PrepLds {
    static constexpr int KW = delta_row_words(DKP);
    union {
        uint32_t K[NP][kDC * KW];
        float N[kDC * kDF];   // A diag(b); after the inverse, P diag(b)
    };
    union {
        uint32_t Q[NP][kDC * KW];
        float M[kDC * kDF];
    };
    double L[kDC];
    float beta[kDC], ks[kDC], qs[kDC];
    float rowf[4][kDC];   // 2^(L_i - L_{16j+15}) for row i below column block j
    float colf[kDC];      // 2^(L_{16j+15} - L_col) in its own block j
    float redm[4], redp[4];
};

// 1 / x for a power of two from 2^-126 to 2^126.
__device__ __forceinline__ float inverse_pow2(float x) { return __uint_as_float(0x7f000000u - __float_as_uint(x)); }

// The units of a 64 x 64 float matrix in LDS, scaled by s, as fp16 planes in memory.
template <bool BYTES>
__device__ __forceinline__ void planes_out(const float* F, uint16_t* img, float s) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int u = threadIdx.x + 256 * i;
        if (i == 1 && u >= kPlaneUnits) break;
        const int row = unit_row(u), q = unit_col(u);
        const float* p = F + row * kDF + 32 * (q / 4) + 4 * (q % 4);
        f16x8 hi, lo;
        h2_split_mix(load4(p), load4(p + 16), s, hi, lo);
        *reinterpret_cast<f16x8*>(img + 8 * u) = hi;
        if constexpr (BYTES) {
            // each half's upper byte, rounded to nearest
            u32x4 w = __builtin_bit_cast(u32x4, lo) + 0x00800080u;
            *reinterpret_cast<uint2*>(img + 8 * kPlaneUnits + 4 * u) =
                make_uint2(__builtin_amdgcn_perm(w[1], w[0], 0x07050301), __builtin_amdgcn_perm(w[3], w[2], 0x07050301));
        } else {
            *reinterpret_cast<f16x8*>(img + 8 * (kPlaneUnits + u)) = lo;
        }
    }
}

template <int DKP, typename In, bool PBYTES>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaArgs a) {
    constexpr int NP = delta_planes<In>(), NJ = DKP / 32, KW = delta_row_words(DKP);
    __shared__ PrepLds<DKP, NP> L;
    const int lane = threadIdx.x % 64, w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), n = lane & 15, g = lane >> 4;
    const int c = (int)(blockIdx.x % a.nc);
    const int bh = blockIdx.x / a.nc;
    const int bk = (bh / a.H) * a.Hk + (bh % a.H) / (a.H / a.Hk);
    const int valid = min(kDC, a.T - c * kDC);
    const size_t tok = (size_t)bh * a.T + (size_t)c * kDC;
    const size_t ktok = ((size_t)bk * a.T + (size_t)c * kDC) * a.dk;
    using Units = RowUnits<DKP, In>;
    {
        Units k, q;
        k.load(static_cast<const In*>(a.k) + ktok, a.dk, valid);
        q.load(static_cast<const In*>(a.q) + ktok, a.dk, valid);
        if (w == 0) {
            const int t = min(lane, valid - 1);
            const float ga = a.gamma[tok + t], be = a.beta[tok + t];
            double x = lane < valid ? log2_gate(ga) : 0.0;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const double t2 = __shfl_up(x, o, 64);
                if (lane >= o) x += t2;
            }
            L.L[lane] = x;
            L.beta[lane] = lane < valid ? be : 0.f;
        }
#pragma unroll
        for (int i = 0; i < Units::n; ++i) {
            const float sk = pow2(h2_exp(Units::row_max(k.absmax(i)))), sq = pow2(h2_exp(Units::row_max(q.absmax(i))));
            k.template store<NP>(L.K, i, sk);
            q.template store<NP>(L.Q, i, sq);
            if (Units::col(i) == 0) {
                L.ks[Units::row(i)] = sk;
                L.qs[Units::row(i)] = sq;
            }
        }
    }
    __syncthreads();
    {
        // lane (n, g) of wave w: row 16 w + n against column block g
        const double x = L.L[16 * w + n], m = L.L[16 * min(g, w) + 15];
        const float f = __builtin_amdgcn_exp2f((float)(g < w ? x - m : m - x));
        if (g < w) L.rowf[g][16 * w + n] = f;
        else if (g == w) L.colf[16 * w + n] = f;
    }
    // ---- rows 16 w .. 16 w + 15 of K K^T and Q K^T ----
    const f32x4 zero{0.f, 0.f, 0.f, 0.f};
    f32x4 P[4], A[4];
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
    __syncthreads();   // the decay factors are written, K and Q are read: N and M take their places
    // P keeps the scale 2^EQ of its rows, which bounds it next to the queries
    {
        const int r0 = 16 * w + 4 * g;
        const f32x4 ks = load4(L.ks + r0);
        f32x4 ki;
#pragma unroll
        for (int r = 0; r < 4; ++r) ki[r] = inverse_pow2(ks[r]);
        float mp = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = 16 * j + n;
            const float f = L.beta[col] * inverse_pow2(L.ks[col]);
            f32x4 D;
            if (j < w) {
                const f32x4 rf = load4(L.rowf[j] + r0);
                const float cf = L.colf[col] * f;
#pragma unroll
                for (int r = 0; r < 4; ++r) D[r] = rf[r] * cf;
            } else if (j == w) {
                const double Lc = L.L[col];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    D[r] = r0 + r >= col ? __builtin_amdgcn_exp2f((float)(L.L[r0 + r] - Lc)) * f : 0.f;
            } else {
                D = zero;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                P[j][r] *= D[r];
                mp = fmaxf(mp, fabsf(P[j][r]));
                L.N[(r0 + r) * kDF + col] = r0 + r > col ? A[j][r] * ki[r] * D[r] : 0.f;
            }
        }
        mp = wave_max(mp);
        if (lane == 0) L.redp[w] = mp;
    }
    __syncthreads();
    // ---- M's diagonal blocks; zeros above the diagonal ----
    float mm = 0.f;
    {
        const float* Nd = L.N + 16 * w * kDF + 16 * w;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s0 = i == n ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
            for (int j4 = 0; j4 < (i + 3) / 4; ++j4) {
                const f32x4 r = load4(Nd + i * kDF + 4 * j4);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = 4 * j4 + e;
                    if (j >= i) continue;
                    if (j & 1) s1 -= r[e] * x[j]; else s0 -= r[e] * x[j];
                }
            }
            x[i] = s0 + s1;
            mm = fmaxf(mm, fabsf(x[i]));
        }
        if (g == 0)
#pragma unroll
            for (int i = 0; i < 16; ++i) L.M[(16 * w + i) * kDF + 16 * w + n] = x[i];
        if (w == 0 || w == 2)   // the one block above the diagonal that a stored row reaches
#pragma unroll
            for (int r = 0; r < 4; ++r) L.M[(16 * w + 4 * g + r) * kDF + 16 * (w + 1) + n] = 0.f;
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
                const f32x4 x = load4(L.N + (16 * w + n) * kDF + 16 * kb + 4 * g);
#pragma unroll
                for (int s = 0; s < 4; ++s) t = mfma4(x[s], L.M[(16 * kb + 4 * g + s) * kDF + 16 * j + n], t);
            }
            const f32x4 y = load4(L.M + (16 * w + n) * kDF + 16 * w + 4 * g);
            f32x4 u = zero;
#pragma unroll
            for (int s = 0; s < 4; ++s) u = mfma4(y[s], t[s], u);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                L.M[(16 * w + 4 * g + r) * kDF + 16 * j + n] = -u[r];
                mm = fmaxf(mm, fabsf(u[r]));
            }
        }
        if (d < 3) __syncthreads();
    }
    mm = wave_max(mm);
    if (lane == 0) L.redm[w] = mm;
    __syncthreads();   // M is whole, N is read: P takes its place
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j / 2 <= w / 2)
#pragma unroll
            for (int r = 0; r < 4; ++r) L.N[(16 * w + 4 * g + r) * kDF + 16 * j + n] = P[j][r];
    uint16_t* img = a.img + (size_t)blockIdx.x * delta_image_words(PBYTES);
    const int EM = h2_exp(fmaxf(fmaxf(L.redm[0], L.redm[1]), fmaxf(L.redm[2], L.redm[3])));
    const int EP = h2_exp(fmaxf(fmaxf(L.redp[0], L.redp[1]), fmaxf(L.redp[2], L.redp[3])));
    planes_out<false>(L.M, img, pow2(EM));
    __syncthreads();
    planes_out<PBYTES>(L.N, img + 2 * kPlaneUnits * 8, pow2(EP));
    if (threadIdx.x < kDC) {
        const int t = threadIdx.x;
        float* sc = a.scal + (size_t)blockIdx.x * kScal;
        const double Lt = L.L[t];
        const float G = __builtin_amdgcn_exp2f((float)Lt), ki = inverse_pow2(L.ks[t]), qi = inverse_pow2(L.qs[t]), be = L.beta[t];
        sc[kKs + t] = L.ks[t];
        sc[kQs + t] = L.qs[t];
        sc[kGk + t] = G * ki;
        sc[kGq + t] = G * qi;
        sc[kQi + t] = qi;
        sc[kDb + t] = __builtin_amdgcn_exp2f((float)(L.L[kDC - 1] - Lt)) * be * ki;
        if (t == kDC - 1) {
            sc[kGc] = G;
            sc[kMi] = pow2(-EM);
            sc[kPi] = pow2(-EP);
        }
    }
}

template <int DKP>
hipError_t prep_go(const DeltaArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.BH * a.nc));
    if (!a.bf16) hipLaunchKernelGGL((delta_prep_kernel<DKP, float, false>), grid, dim3(256), 0, s, a);
    else if (!a.p_bytes) hipLaunchKernelGGL((delta_prep_kernel<DKP, bf16_t, false>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((delta_prep_kernel<DKP, bf16_t, true>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_delta_prep(const DeltaArgs& a, hipStream_t s) {
    return a.dk <= 32 ? prep_go<32>(a, s) : a.dk == 64 ? prep_go<64>(a, s) : prep_go<128>(a, s);
}

}  // namespace mesa
