// delta_grads.hip -- the gated delta rule's gradients per chunk (gfx950).
//
// With a chunk's start state S, the gradient dS' of its end state, E and dV
// from the two passes over the chunks (delta_core.h's notation, all 64 x dv,
// dv x dk or dk x dv as their products need):
//   Y = dO E^T,  Z = dV E^T            (64 x 64, contracted over dv)
//   oS = dO S^T, rS = dV S^T, W = E dS'^T   (64 x dk)
//   dQ = G oS + (D.Y b) K
//   dK = D_C b W - G rS + (D.Y b)^T Q - (D.Z b) K - (D.Z b)^T K
//   db_j = D_Cj k_j.W_j + sum_i (P_ij Y_ij - A_ij Z_ij)
// where D is cut to j <= i with Y and to j < i with Z, and b scales columns.
// The gate of token t scales every product of a token j < t with one i >= t,
// and the state that crosses t:
//   dg_t g_t = sum_{i >= t > j} b_j (P_ij Y_ij - A_ij Z_ij)
//              + sum_{i >= t} G_i (q_i.oS_i - k_i.rS_i)
//              + sum_{j < t} b_j D_Cj k_j.W_j + G_C <S, dS'>
// summed over the pairs that cross t, not as a difference of row and column
// sums, which would cancel.  Below kTinyGate the products that hold g_t leave
// float's range: there the same sums are taken of products without it, g_t in
// D_ij, G_i, D_Cj and G_C being left out (a wave-wide sum for each such gate).
//
// One workgroup of four waves per chunk and head; wave w owns tokens
// 16 w .. 16 w + 15 as rows.  First the products over dv, 32 columns of dv at a
// time through LDS (token rows scaled each, states per block); then, with K, Q
// and the decayed Y, Z in LDS, the products over the chunk's tokens.  All
// operands are 22-bit splits (bf16 rows are exact in one part).
//
// 2x16x4096, dk = dv = 128, bf16: 169-179 us for 0.52 GB in and 68 MB out, 3.3
// TB/s; vector instructions take 40 % of the cycles and matrix ones 16 %, at two
// waves a SIMD, which is what 128 accumulators a thread leave room for.  Eight
// waves with half of the columns each spill and take 310-365 us; the next block's
// rows in flight during the products take 186-195.
#include "delta_core.h"

namespace mesa {

constexpr int kVW = 24;   // words per LDS row of 32 dv columns
constexpr float kTinyGate = 0x1p-64f;

template <int DKP, int NP>
struct alignas(16) GradsLds {
    static constexpr int KW = delta_row_words(DKP);
    union {
        struct {
            uint32_t V[3][2][kDC * kVW];   // dO, dV, E rows
            uint32_t S[2][2][32 * KW];     // S, dS' rows (dv)
        };
        struct {
            uint32_t K[NP][kDC * KW];
            uint32_t Q[NP][kDC * KW];
            uint32_t Y[2 * kCPlane];
            uint32_t Z[2 * kCPlane];
        };
    };
    double L[kDC];
    float beta[kDC], G[kDC], end[kDC];
    union {
        float vs[3][kDC];      // 2^-E of the token rows
        float tcross[4][kDC];  // per wave the pairs' sums across the tiny gates
    };
    float read[kDC], write[kDC];   // rows' dots, without their decays
    float col[4][kDC], cross[4][kDC + 1];
    unsigned long long tiny;   // tokens with a gate below kTinyGate
    float red[8][4];           // per-wave maxima and sums
};

// Eight elements of a 64 x 32 block of rows, scaled by the row's
// own power of two into fp16 planes.
__device__ __forceinline__ void stage_row8(const f32x8& x, uint32_t (&P)[2][kDC * kVW], float* inv) {
    const int row = threadIdx.x / 4, q = threadIdx.x % 4;
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x.v[e]));
    m = fmaxf(m, dpp_f32<0xb1>(m));
    m = fmaxf(m, dpp_f32<0x4e>(m));
    const int E = h2_exp(m);
    if (q == 0) inv[row] = pow2(-E);
    f16x8 hi, lo;
    h2_split_mix(f32x4{x.v[0], x.v[1], x.v[2], x.v[3]}, f32x4{x.v[4], x.v[5], x.v[6], x.v[7]}, pow2(E), hi, lo);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int at = row * kVW + perm32(8 * q + 4 * half) / 2;
        *reinterpret_cast<f16x4*>(&P[0][at]) = f16x4{hi[4 * half], hi[4 * half + 1], hi[4 * half + 2], hi[4 * half + 3]};
        *reinterpret_cast<f16x4*>(&P[1][at]) = f16x4{lo[4 * half], lo[4 * half + 1], lo[4 * half + 2], lo[4 * half + 3]};
    }
}

// t (+)= A B as hi lo + lo hi + hi hi; AP, BP: whether A, B have a lo part.
template <bool FIRST, bool AP, bool BP>
__device__ __forceinline__ void product(f32x4& t, f16x8 ah, f16x8 al, f16x8 bh, f16x8 bl) {
    if constexpr (BP) {
        if constexpr (FIRST) mfma_first(t, ah, bl);
        else mfma_acc(t, ah, bl);
    }
    if constexpr (AP) {
        if constexpr (FIRST && !BP) mfma_first(t, al, bh);
        else mfma_acc(t, al, bh);
    }
    if constexpr (FIRST && !AP && !BP) mfma_first(t, ah, bh);
    else mfma_acc(t, ah, bh);
}

// A buffer of n elements: stores past its end are dropped.
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(T* p, int n) {
    return __builtin_amdgcn_make_buffer_rsrc(p, (short)0, n * (int)sizeof(T), 0x00020000);
}
template <typename T>
__device__ __forceinline__ void put1(__amdgpu_buffer_rsrc_t r, uint32_t i, float x) {
    if constexpr (sizeof(T) == 4) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, x), r, i * 4, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)x), r, i * 2, 0, 0);
}

template <int DKP, typename In>
__global__ __launch_bounds__(256, DKP == 128 && sizeof(In) == 4 ? 1 : 2) void delta_grads_kernel(DeltaBwdArgs b) {
    constexpr int NP = delta_planes<In>(), NJ = DKP / 32, NS = DKP / 16, KW = delta_row_words(DKP);
    constexpr bool F = NP == 2;   // rows stored as float: two parts
    __shared__ GradsLds<DKP, NP> L;
    const DeltaArgs& a = b.f;
    const int lane = threadIdx.x % 64, w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), n = lane & 15, g = lane >> 4;
    const int c = (int)(blockIdx.x % a.nc);
    const long bh = blockIdx.x / a.nc;
    const long bk = (bh / a.H) * a.Hk + (bh % a.H) / (a.H / a.Hk);
    const int valid = min(kDC, a.T - c * kDC);
    const size_t tok = (size_t)bh * a.T + (size_t)c * kDC;
    const size_t ktok = ((size_t)bk * a.T + (size_t)c * kDC) * a.dk;
    const size_t vo = (size_t)blockIdx.x * kDC * a.dv, so = (size_t)blockIdx.x * a.dv * a.dk;
    const f32x4 zero{0.f, 0.f, 0.f, 0.f};
    float gate = 1.f;
    if (w == 0) {
        gate = lane < valid ? a.gamma[tok + lane] : 1.f;
        double x = log2_gate(gate);
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double t = __shfl_up(x, o, 64);
            if (lane >= o) x += t;
        }
        L.L[lane] = x;
        L.beta[lane] = lane < valid ? a.beta[tok + lane] : 0.f;
        L.G[lane] = __builtin_amdgcn_exp2f((float)x);
        L.end[lane] = __builtin_amdgcn_exp2f((float)(__shfl(x, 63, 64) - x));
        const unsigned long long tiny = __ballot(gate > 0.f && gate < kTinyGate);
        if (lane == 0) L.tiny = tiny;
    }
    // ---- products over dv ----
    f32x4 Y[4], Z[4], oS[NS], rS[NS], W[NS];
#pragma unroll
    for (int j = 0; j < 4; ++j) Y[j] = Z[j] = zero;
#pragma unroll
    for (int m = 0; m < NS; ++m) oS[m] = rS[m] = W[m] = zero;
    float carry = 0.f;   // this thread's share of <S, dS'>
    for (int v0 = 0; v0 < a.dv; v0 += 32) {
        {
            const int row = threadIdx.x / 4, vc = v0 + 8 * (threadIdx.x % 4);
            f32x8 o{}, r{}, e{};
            if (vc < a.dv) {
                if (row < valid) o = load8(static_cast<const In*>(b.grad_out) + (tok + row) * a.dv + vc);
                r = load8(b.dR + vo + (size_t)row * a.dv + vc);
                e = load8(a.E + vo + (size_t)row * a.dv + vc);
            }
            constexpr int per_row = DKP / 8, units = 32 * per_row, SU = (units + 255) / 256;
            f32x8 s[SU], d[SU];
            float ms = 0.f, md = 0.f;
#pragma unroll
            for (int i = 0; i < SU; ++i) {
                const int u = threadIdx.x + 256 * i, vr = v0 + u / per_row, kc = 8 * (u % per_row);
                s[i] = d[i] = f32x8{};
                if (u < units && vr < a.dv && kc < a.dk) {
                    s[i] = load8(a.S + so + (size_t)vr * a.dk + kc);
                    d[i] = load8(b.dS + so + (size_t)vr * a.dk + kc);
                }
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    ms = fmaxf(ms, fabsf(s[i].v[x]));
                    md = fmaxf(md, fabsf(d[i].v[x]));
                    carry += s[i].v[x] * d[i].v[x];
                }
            }
            ms = wave_max(ms);
            md = wave_max(md);
            __syncthreads();   // the previous block is read (and the first time L.L.. are written)
            if (lane == 0) { L.red[0][w] = ms; L.red[1][w] = md; }
            stage_row8(o, L.V[0], L.vs[0]);
            stage_row8(r, L.V[1], L.vs[1]);
            stage_row8(e, L.V[2], L.vs[2]);
            __syncthreads();
            ms = fmaxf(fmaxf(L.red[0][0], L.red[0][1]), fmaxf(L.red[0][2], L.red[0][3]));
            md = fmaxf(fmaxf(L.red[1][0], L.red[1][1]), fmaxf(L.red[1][2], L.red[1][3]));
            const float ss = pow2(h2_exp(ms)), sd = pow2(h2_exp(md));
#pragma unroll
            for (int i = 0; i < SU; ++i) {
                const int u = threadIdx.x + 256 * i, kc = 8 * (u % per_row);
                if (u >= units) break;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const f32x8& x = t ? d[i] : s[i];
                    f16x8 hi, lo;
                    h2_split_mix(f32x4{x.v[0], x.v[1], x.v[2], x.v[3]}, f32x4{x.v[4], x.v[5], x.v[6], x.v[7]}, t ? sd : ss, hi, lo);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int at = (u / per_row) * KW + perm32(kc + 4 * half) / 2;
                        *reinterpret_cast<f16x4*>(&L.S[t][0][at]) = f16x4{hi[4 * half], hi[4 * half + 1], hi[4 * half + 2], hi[4 * half + 3]};
                        *reinterpret_cast<f16x4*>(&L.S[t][1][at]) = f16x4{lo[4 * half], lo[4 * half + 1], lo[4 * half + 2], lo[4 * half + 3]};
                    }
                }
            }
        }
        __syncthreads();
        const float is = pow2(-h2_exp(fmaxf(fmaxf(L.red[0][0], L.red[0][1]), fmaxf(L.red[0][2], L.red[0][3]))));
        const float id = pow2(-h2_exp(fmaxf(fmaxf(L.red[1][0], L.red[1][1]), fmaxf(L.red[1][2], L.red[1][3]))));
        const f16x8 oh = row_operand(L.V[0][0], kVW, w, 0, n, g), ol = row_operand(L.V[0][1], kVW, w, 0, n, g);
        const f16x8 rh = row_operand(L.V[1][0], kVW, w, 0, n, g), rl = row_operand(L.V[1][1], kVW, w, 0, n, g);
        const f16x8 eh = row_operand(L.V[2][0], kVW, w, 0, n, g), el = row_operand(L.V[2][1], kVW, w, 0, n, g);
        const f32x4 so4 = row4(L.vs[0], w, g), sr4 = row4(L.vs[1], w, g), se4 = row4(L.vs[2], w, g);
        {
            f32x4 y[4], z[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f16x8 bh_ = row_operand(L.V[2][0], kVW, j, 0, n, g), bl = row_operand(L.V[2][1], kVW, j, 0, n, g);
                product<true, F, true>(y[j], oh, ol, bh_, bl);
                product<true, true, true>(z[j], rh, rl, bh_, bl);
            }
            mfma_done(y);
            mfma_done(z);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float se = L.vs[2][16 * j + n];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    Y[j][r] += y[j][r] * (so4[r] * se);
                    Z[j][r] += z[j][r] * (sr4[r] * se);
                }
            }
        }
        const f32x4 os4 = so4 * is, rs4 = sr4 * is, es4 = se4 * id;
#pragma unroll
        for (int m0 = 0; m0 < NS; m0 += 2) {
            f32x4 x[2], y[2], z[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int m = m0 + k;
                const f16x8 sh = col_operand(L.S[0][0], KW, m, 0, n, g), sl = col_operand(L.S[0][1], KW, m, 0, n, g);
                const f16x8 dh = col_operand(L.S[1][0], KW, m, 0, n, g), dl = col_operand(L.S[1][1], KW, m, 0, n, g);
                product<true, F, true>(x[k], oh, ol, sh, sl);
                product<true, true, true>(y[k], rh, rl, sh, sl);
                product<true, true, true>(z[k], eh, el, dh, dl);
            }
            mfma_done(x);
            mfma_done(y);
            mfma_done(z);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                oS[m0 + k] += x[k] * os4;
                rS[m0 + k] += y[k] * rs4;
                W[m0 + k] += z[k] * es4;
            }
        }
    }
    // ---- K and Q, one scale each for the chunk ----
    carry = wavesum(carry);
    float ek, eq;   // 2^-EK, 2^-EQ
    {
        using Units = RowUnits<DKP, In>;
        Units k, q;
        k.load(static_cast<const In*>(a.k) + ktok, a.dk, valid);
        q.load(static_cast<const In*>(a.q) + ktok, a.dk, valid);
        float mk = 0.f, mq = 0.f;
#pragma unroll
        for (int i = 0; i < Units::n; ++i) {
            mk = fmaxf(mk, k.absmax(i));
            mq = fmaxf(mq, q.absmax(i));
        }
        mk = wave_max(mk);
        mq = wave_max(mq);
        if (lane == 0) { L.red[2][w] = mk; L.red[3][w] = mq; L.red[4][w] = carry; }
        __syncthreads();   // maxima written, the dv blocks read
        mk = fmaxf(fmaxf(L.red[2][0], L.red[2][1]), fmaxf(L.red[2][2], L.red[2][3]));
        mq = fmaxf(fmaxf(L.red[3][0], L.red[3][1]), fmaxf(L.red[3][2], L.red[3][3]));
        L.tcross[w][lane] = 0.f;
        const int EK = h2_exp(mk), EQ = h2_exp(mq);
        ek = pow2(-EK);
        eq = pow2(-EQ);
#pragma unroll
        for (int i = 0; i < Units::n; ++i) {
            k.template store<NP>(L.K, i, pow2(EK));
            q.template store<NP>(L.Q, i, pow2(EQ));
        }
    }
    __syncthreads();
    // ---- A and P; what crosses; the decayed Y and Z ----
    {
        // X_ij = b_j (P_ij Y_ij - A_ij Z_ij) crosses the gates j + 1 .. i: along a
        // row its sums up to column j, taken within 16 lanes and on top of the
        // blocks before, are summed over the rows below
        float before[4] = {};
        if (lane == 0) L.cross[w][0] = 0.f;
        const unsigned long long tiny = L.tiny;
        f16x8 kh[NJ], kl[NJ], qh[NJ], ql[NJ];
        auto rows = [&] {
#pragma unroll
            for (int s = 0; s < NJ; ++s) {
                kh[s] = row_operand(L.K[0], KW, w, s, n, g);
                kl[s] = row_operand(L.K[NP - 1], KW, w, s, n, g);
                qh[s] = row_operand(L.Q[0], KW, w, s, n, g);
                ql[s] = row_operand(L.Q[NP - 1], KW, w, s, n, g);
            }
        };
        // read again for each block where they would be kept in accumulator
        // registers, from which they would come too late for the MFMAs in asm
        constexpr bool KEEP = !(F && DKP == 128);
        if constexpr (KEEP) rows();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (!KEEP) {
                rows();
                __builtin_amdgcn_sched_barrier(0);
            }
            f32x4 AP[2];   // the blocks of A and P
#pragma unroll
            for (int s = 0; s < NJ; ++s) {
                const f16x8 bh_ = row_operand(L.K[0], KW, j, s, n, g), bl = row_operand(L.K[NP - 1], KW, j, s, n, g);
                if (s == 0) {
                    product<true, F, F>(AP[0], kh[s], kl[s], bh_, bl);
                    product<true, F, F>(AP[1], qh[s], ql[s], bh_, bl);
                } else {
                    product<false, F, F>(AP[0], kh[s], kl[s], bh_, bl);
                    product<false, F, F>(AP[1], qh[s], ql[s], bh_, bl);
                }
            }
            mfma_done(AP);
            const f32x4 A = AP[0], P = AP[1];
            const int cj = 16 * j + n;
            const double Lj = L.L[cj];
            const float bj = L.beta[cj];
            for (unsigned long long left = tiny; left; left &= left - 1) {
                const int t = __builtin_ctzll(left);
                float s = 0.f;
                if (t > cj) {
                    const float before = __builtin_amdgcn_exp2f((float)(L.L[t - 1] - Lj)) * bj;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int row = 16 * w + 4 * g + r;
                        if (row >= t)
                            s += __builtin_amdgcn_exp2f((float)(L.L[row] - L.L[t])) * before *
                                 (P[r] * (ek * eq) * Y[j][r] - A[r] * (ek * ek) * Z[j][r]);
                    }
                }
                s = wavesum(s);
                if (lane == 0) L.tcross[w][t] += s;
            }
            float sum = 0.f, cross = 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * w + 4 * g + r;
                const float D = row >= cj ? __builtin_amdgcn_exp2f((float)(L.L[row] - Lj)) : 0.f;
                const float Ds = row > cj ? D : 0.f;
                const float py = P[r] * (ek * eq) * D * Y[j][r], az = A[r] * (ek * ek) * Ds * Z[j][r];
                sum += py - az;
                float x = row > cj ? bj * (py - az) : 0.f;
                x += dpp_f32<0x111>(x);   // row_shr:1, 2, 4, 8
                x += dpp_f32<0x112>(x);
                x += dpp_f32<0x114>(x);
                x += dpp_f32<0x118>(x);
                x += before[r];
                before[r] = dpp_f32<0x15f>(x);   // the last lane's
                cross += row > cj ? x : 0.f;
                Y[j][r] *= D * bj;
                Z[j][r] *= Ds * bj;
            }
            sum = kslot_sum(sum);
            cross = kslot_sum(cross);
            if (g == 0) {
                L.col[w][cj] = sum;
                L.cross[w][cj + 1] = cross;
            }
        }
    }
    // row dots with the keys and queries
    {
        f32x4 qo = zero, kr = zero, kw = zero;
        const _Float16* Kh = reinterpret_cast<const _Float16*>(L.K[0]);
        const _Float16* Qh = reinterpret_cast<const _Float16*>(L.Q[0]);
        const _Float16* Kl = reinterpret_cast<const _Float16*>(L.K[NP - 1]);
        const _Float16* Ql = reinterpret_cast<const _Float16*>(L.Q[NP - 1]);
#pragma unroll
        for (int m = 0; m < NS; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int at = (16 * w + 4 * g + r) * 2 * KW + perm32(16 * m + n);
                float k = (float)Kh[at], q = (float)Qh[at];
                if constexpr (F) { k += (float)Kl[at]; q += (float)Ql[at]; }
                qo[r] += q * oS[m][r];
                kr[r] += k * rS[m][r];
                kw[r] += k * W[m][r];
            }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float q1 = rowsum16(qo[r]) * eq, k1 = rowsum16(kr[r]) * ek, k2 = rowsum16(kw[r]) * ek;
            if (n == 0) {
                L.read[16 * w + 4 * g + r] = q1 - k1;
                L.write[16 * w + 4 * g + r] = k2;
            }
        }
    }
    const float my = wave_max(absmax(Y)), mz = wave_max(absmax(Z));
    if (lane == 0) { L.red[5][w] = my; L.red[6][w] = mz; }
    __syncthreads();
    if (w == 0) {
        const float wr = L.end[lane] * L.write[lane];
        float rd = L.G[lane] * L.read[lane], before = L.beta[lane] * wr;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const float t = __shfl_down(rd, o, 64), u = __shfl_up(before, o, 64);
            if (lane + o < 64) rd += t;
            if (lane >= o) before += u;
        }
        before = __shfl_up(before, 1, 64);
        if (lane == 0) before = 0.f;
        const float carried = (L.red[4][0] + L.red[4][1]) + (L.red[4][2] + L.red[4][3]);
        const float state = L.G[kDC - 1] * carried;
        const float cross = (L.cross[0][lane] + L.cross[1][lane]) + (L.cross[2][lane] + L.cross[3][lane]);
        const float cols = (L.col[0][lane] + L.col[1][lane]) + (L.col[2][lane] + L.col[3][lane]);
        float dg = gate == 0.f ? 0.f : (cross + rd + before + state) / gate;
        for (unsigned long long left = L.tiny; left; left &= left - 1) {
            const int t = __builtin_ctzll(left);
            const double Lb = t ? L.L[t - 1] : 0.0, Lt = L.L[t], Li = L.L[lane];
            const float G = __builtin_amdgcn_exp2f((float)Lb), D = __builtin_amdgcn_exp2f((float)(L.L[kDC - 1] - Lt));
            float s = lane >= t ? __builtin_amdgcn_exp2f((float)(Li - Lt)) * G * L.read[lane]
                                : __builtin_amdgcn_exp2f((float)(Lb - Li)) * D * L.beta[lane] * L.write[lane];
            s = wavesum(s) + G * D * carried + ((L.tcross[0][t] + L.tcross[1][t]) + (L.tcross[2][t] + L.tcross[3][t]));
            if (lane == t) dg = s;
        }
        if (lane < valid) {
            b.grad_beta[tok + lane] = wr + cols;
            b.grad_gamma[tok + lane] = dg;
        }
    }
    float ey, ez;
    {
        const int EY = h2_exp(fmaxf(fmaxf(L.red[5][0], L.red[5][1]), fmaxf(L.red[5][2], L.red[5][3])));
        const int EZ = h2_exp(fmaxf(fmaxf(L.red[6][0], L.red[6][1]), fmaxf(L.red[6][2], L.red[6][3])));
        ey = pow2(-EY);
        ez = pow2(-EZ);
        const float sy = pow2(EY), sz = pow2(EZ);
        // compact planes (delta_core.h): rows below 32 have no columns from 32 on
        const int r0 = 16 * w + 4 * g, base = w < 2 ? r0 * 2 * kCP : 2 * kCU + (r0 - 32) * 2 * kDP, pitch = 2 * (w < 2 ? kCP : kDP);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j / 2 > w / 2) continue;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int at = base + r * pitch + perm32(16 * j + n);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const float x = t ? Z[j][r] * sz : Y[j][r] * sy;
                    const _Float16 hi = (_Float16)x;
                    _Float16* D = reinterpret_cast<_Float16*>(t ? L.Z : L.Y) + at;
                    D[0] = hi;
                    D[2 * kCPlane] = (_Float16)(x - (float)hi);
                }
            }
        }
    }
    __syncthreads();
    // ---- products over the tokens ----
    f16x8 yh[2], yl[2], zh[2], zl[2], yth[2], ytl[2], zth[2], ztl[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        // blocks above the diagonal are not there
        yh[j] = yl[j] = zh[j] = zl[j] = yth[j] = ytl[j] = zth[j] = ztl[j] = f16x8{};
        if (j <= w / 2) {
            yh[j] = compact_row_operand(L.Y, w, j, n, g);
            yl[j] = compact_row_operand(L.Y + kCPlane, w, j, n, g);
            zh[j] = compact_row_operand(L.Z, w, j, n, g);
            zl[j] = compact_row_operand(L.Z + kCPlane, w, j, n, g);
        }
        if (j >= w / 2) {
            yth[j] = compact_col_operand(L.Y, w, j, n, g);
            ytl[j] = compact_col_operand(L.Y + kCPlane, w, j, n, g);
            zth[j] = compact_col_operand(L.Z, w, j, n, g);
            ztl[j] = compact_col_operand(L.Z + kCPlane, w, j, n, g);
        }
    }
    const f32x4 G = row4(L.G, w, g), end = row4(L.end, w, g), be = row4(L.beta, w, g);
    // rows behind the last token fall off the end of the buffers
    const uint32_t ro = (uint32_t)(16 * w + 4 * g) * a.dk + n;
    const int elems = valid * a.dk;
    const auto rq = b.part ? row_buffer(b.part + tok * a.dk, elems) : row_buffer(static_cast<In*>(b.grad_q) + ktok, elems);
    const auto rk = b.part ? row_buffer(b.part + ((size_t)a.BH * a.T + tok) * a.dk, elems)
                           : row_buffer(static_cast<In*>(b.grad_k) + ktok, elems);
#pragma unroll
    for (int m = 0; m < NS; ++m) {
        f32x4 t[3];   // (D.Y b) K, (D.Y b)^T Q, (D.Z b) K + (D.Z b)^T K
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const f16x8 kh = col_operand(L.K[0], KW, m, j, n, g), qh = col_operand(L.Q[0], KW, m, j, n, g);
            f16x8 kl = kh, ql = qh;
            if constexpr (F) {
                kl = col_operand(L.K[1], KW, m, j, n, g);
                ql = col_operand(L.Q[1], KW, m, j, n, g);
            }
            if (j == 0) {
                product<true, true, F>(t[0], yh[j], yl[j], kh, kl);
                product<true, true, F>(t[1], yth[j], ytl[j], qh, ql);
                product<true, true, F>(t[2], zh[j], zl[j], kh, kl);
            } else {
                product<false, true, F>(t[0], yh[j], yl[j], kh, kl);
                product<false, true, F>(t[1], yth[j], ytl[j], qh, ql);
                product<false, true, F>(t[2], zh[j], zl[j], kh, kl);
            }
            product<false, true, F>(t[2], zth[j], ztl[j], kh, kl);
        }
        mfma_done(t);
        const f32x4 tq = t[0], tk = t[1], tz = t[2];
        if (DKP == 32 && 16 * m >= a.dk) continue;
        const f32x4 dq = G * oS[m] + tq * (ey * ek), dk = end * be * W[m] - G * rS[m] + tk * (ey * eq) - tz * (ez * ek);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint32_t at = ro + r * a.dk + 16 * m;
            if (b.part) {
                put1<float>(rq, at, dq[r]);
                put1<float>(rk, at, dk[r]);
            } else {
                put1<In>(rq, at, dq[r]);
                put1<In>(rk, at, dk[r]);
            }
        }
    }
}

// grad_q and grad_k of a key head: the sum over its value heads, in order.
// A thread takes four consecutive features.
template <typename In>
__global__ __launch_bounds__(256) void delta_head_sum_kernel(DeltaBwdArgs b, long quads) {
    const DeltaArgs& a = b.f;
    const long i = (long)blockIdx.x * 256 + threadIdx.x;
    if (i >= quads) return;
    const long per = (long)a.T * a.dk / 4;   // of a head
    const long head = i / per, at = i % per;
    const int rep = a.H / a.Hk;
    const float* p = b.part + 4 * ((head / a.Hk * a.H + head % a.Hk * rep) * per + at);
    f32x4 q{0.f, 0.f, 0.f, 0.f}, k = q;
    for (int r = 0; r < rep; ++r) {
        q += load4(p + 4 * r * per);
        k += load4(p + 4 * (r * per + a.BH * per));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        store1(static_cast<In*>(b.grad_q) + 4 * i + e, q[e]);
        store1(static_cast<In*>(b.grad_k) + 4 * i + e, k[e]);
    }
}

template <int DKP>
hipError_t grads_go(const DeltaBwdArgs& b, hipStream_t s) {
    const dim3 grid((unsigned)(b.f.BH * b.f.nc));
    if (b.f.bf16) hipLaunchKernelGGL((delta_grads_kernel<DKP, bf16_t>), grid, dim3(256), 0, s, b);
    else hipLaunchKernelGGL((delta_grads_kernel<DKP, float>), grid, dim3(256), 0, s, b);
    return hipGetLastError();
}

hipError_t launch_delta_grads(const DeltaBwdArgs& b, hipStream_t s) {
    hipError_t e = b.f.dk <= 32 ? grads_go<32>(b, s) : b.f.dk == 64 ? grads_go<64>(b, s) : grads_go<128>(b, s);
    if (e != hipSuccess || !b.part) return e;
    const long quads = b.f.BH / b.f.H * b.f.Hk * b.f.T * b.f.dk / 4;
    const dim3 grid((unsigned)((quads + 255) / 256));
    if (b.f.bf16) hipLaunchKernelGGL(delta_head_sum_kernel<bf16_t>, grid, dim3(256), 0, s, b, quads);
    else hipLaunchKernelGGL(delta_head_sum_kernel<float>, grid, dim3(256), 0, s, b, quads);
    return hipGetLastError();
}

}  // namespace mesa
