// delta_scan.hip -- the gated delta rule's pass over the chunks (gfx950).
//
// A wave owns 16 of the state's dv columns for the whole sequence: they never
// meet the other columns.  Its part of S (dk x 16) stays in registers in MFMA
// accumulator order, which is also the operand order of the next product
// (cg_h2.h's perm32), so the chunk's chain
//   X = K S,  R = V - G X,  E = M R,  O = G Q S + P (b E),
//   S' = G_C S + K^T (D_C b E)
// runs without exchanging anything between lanes but the column maxima that
// scale the fp16 operands.  A workgroup of four waves (64 columns) shares the
// chunk's K, Q, M and P in LDS; the next chunk's rows are in flight in
// registers meanwhile.
//
// Precision: S, R and b E enter the products that feed the state as hi + lo
// (22 bits).  For bf16 outputs the two products that only feed O take the hi
// parts alone (11 bits: 2^-12 a term against the output's own 2^-8).
#include "delta_core.h"

namespace mesa {

template <int DKP, int NP>
struct alignas(16) ScanLds {
    static constexpr int KW = delta_row_words(DKP);
    uint32_t K[NP][kDC * KW];
    uint32_t Q[NP][kDC * KW];
    uint32_t M[2][kDC * kDP];
    uint32_t P[NP][kDC * kDP];
    float sc[kScal];
};

// OUT: write O.  SAVE: write each chunk's start state and E (the backward's
// recomputation).
template <int DKP, typename In, bool OUT, bool SAVE>
__global__ __launch_bounds__(256) void delta_scan_kernel(DeltaArgs a) {
    constexpr int NP = delta_planes<In>(), NJ = DKP / 32, NS = DKP / 16, KW = delta_row_words(DKP);
    __shared__ ScanLds<DKP, NP> L;
    const int lane = threadIdx.x % 64, w = threadIdx.x / 64, n = lane & 15, g = lane >> 4;
    // the column groups of a head on one XCD (workgroups go to the 8 XCDs in turn)
    const int cgs = (a.dv + 63) / 64;
    const long bh = (long)(blockIdx.x / (8 * cgs)) * 8 + blockIdx.x % 8;
    if (bh >= a.BH) return;
    const int col = 64 * (int)(blockIdx.x / 8 % cgs) + 16 * w + n;
    const bool live = col - n < a.dv;   // a whole wave
    const long bk = (bh / a.H) * a.Hk + (bh % a.H) / (a.H / a.Hk);
    const In* Kp = static_cast<const In*>(a.k) + (size_t)bk * a.T * a.dk;
    const In* Qp = static_cast<const In*>(a.q) + (size_t)bk * a.T * a.dk;
    const In* Vp = static_cast<const In*>(a.v) + (size_t)bh * a.T * a.dv + col;
    In* Op = OUT ? static_cast<In*>(a.out) + (size_t)bh * a.T * a.dv + col : nullptr;
    const size_t image = (size_t)(2 + a.p_planes) * kDC * kDC;
    const uint16_t* img = a.img + (size_t)bh * a.nc * image;
    const float* scal = a.scal + (size_t)bh * a.nc * kScal;
    const size_t so = ((size_t)bh * a.dv + col) * a.dk + 4 * g;   // this lane's row of the (dv x dk) state
    const f32x4 zero{0.f, 0.f, 0.f, 0.f};

    f32x4 S[NS];
#pragma unroll
    for (int m = 0; m < NS; ++m)
        S[m] = a.state0 && live && 16 * m < a.dk ? load4(a.state0 + so + 16 * m) : zero;

    using Units = RowUnits<DKP, In>;
    Units kr, qr;
    PlaneUnits<2> mr;
    PlaneUnits<NP> pr;
    In vr[16];
    float ksr[Units::n], qsr[Units::n];
    f32x4 scr = zero;
    auto fetch = [&](int c) {
        const int valid = min(kDC, a.T - c * kDC);
        kr.load(Kp + (size_t)c * kDC * a.dk, a.dk, valid);
        if constexpr (OUT) qr.load(Qp + (size_t)c * kDC * a.dk, a.dk, valid);
        const float* sc = scal + (size_t)c * kScal;
#pragma unroll
        for (int i = 0; i < Units::n; ++i) {
            ksr[i] = sc[kKs + Units::row(i)];
            if constexpr (OUT) qsr[i] = sc[kQs + Units::row(i)];
        }
        mr.load(img + c * image);
        if constexpr (OUT) pr.load(img + c * image + 2 * kDC * kDC);
        if (threadIdx.x < kScal / 4) scr = load4(sc + 4 * threadIdx.x);
        const In* vp = Vp + (size_t)c * kDC * a.dv;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int t = 16 * (i / 4) + 4 * g + i % 4;
            vr[i] = live && t < valid ? vp[(size_t)t * a.dv] : In{};
        }
    };
    fetch(0);
    for (int c = 0; c < a.nc; ++c) {
        __syncthreads();   // the previous chunk's tiles are read
        f32x4 V[4];
#pragma unroll
        for (int i = 0; i < Units::n; ++i) {
            kr.template store<NP>(L.K, i, ksr[i]);
            if constexpr (OUT) qr.template store<NP>(L.Q, i, qsr[i]);
        }
        mr.store(L.M);
        if constexpr (OUT) pr.store(L.P);
        if (threadIdx.x < kScal / 4) *reinterpret_cast<f32x4*>(L.sc + 4 * threadIdx.x) = scr;
#pragma unroll
        for (int i = 0; i < 16; ++i) V[i / 4][i % 4] = to_f32(vr[i]);
        __syncthreads();
        if (c + 1 < a.nc) fetch(c + 1);
        if (!live) continue;

        if constexpr (SAVE) {
            float* sp = a.S + (size_t)c * a.dv * a.dk + ((size_t)bh * a.nc * a.dv + col) * a.dk + 4 * g;
#pragma unroll
            for (int m = 0; m < NS; ++m)
                if (16 * m < a.dk) *reinterpret_cast<f32x4*>(sp + 16 * m) = S[m];
        }
        // ---- K S and Q S ----
        f16x8 Sh[NJ], Sl[NJ];
        const float is = column_operands(S, Sh, Sl);
        f32x4 X[4], Y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            X[i] = Y[i] = zero;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const f16x8 kh = row_operand(L.K[0], KW, i, j, n, g);
                X[i] = mfma_f16x32(kh, Sl[j], X[i]);
                if constexpr (NP == 2) X[i] = mfma_f16x32(row_operand(L.K[1], KW, i, j, n, g), Sh[j], X[i]);
                X[i] = mfma_f16x32(kh, Sh[j], X[i]);
                if constexpr (OUT) {
                    const f16x8 qh = row_operand(L.Q[0], KW, i, j, n, g);
                    if constexpr (NP == 2) {
                        Y[i] = mfma_f16x32(qh, Sl[j], Y[i]);
                        Y[i] = mfma_f16x32(row_operand(L.Q[1], KW, i, j, n, g), Sh[j], Y[i]);
                    }
                    Y[i] = mfma_f16x32(qh, Sh[j], Y[i]);
                }
            }
        }
        // ---- E = M (V - G K S) ----
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 gk = row4(L.sc + kGk, i, g);
#pragma unroll
            for (int r = 0; r < 4; ++r) X[i][r] = V[i][r] - (gk[r] * is) * X[i][r];
        }
        f16x8 Bh[2], Bl[2];
        const float ir = column_operands(X, Bh, Bl);
        f32x4 U[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            U[i] = zero;
#pragma unroll
            for (int j = 0; j <= i / 2; ++j) {
                const f16x8 mh = row_operand(L.M[0], kDP, i, j, n, g);
                U[i] = mfma_f16x32(mh, Bl[j], U[i]);
                U[i] = mfma_f16x32(row_operand(L.M[1], kDP, i, j, n, g), Bh[j], U[i]);
                U[i] = mfma_f16x32(mh, Bh[j], U[i]);
            }
            const f32x4 mi = row4(L.sc + kMi, i, g), be = row4(L.sc + kBe, i, g);
#pragma unroll
            for (int r = 0; r < 4; ++r) U[i][r] *= mi[r] * ir;
            if constexpr (SAVE) {
                float* ep = a.E + ((size_t)(bh * a.nc + c) * kDC + 16 * i + 4 * g) * a.dv + col;
#pragma unroll
                for (int r = 0; r < 4; ++r) ep[(size_t)r * a.dv] = U[i][r];
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) U[i][r] *= be[r];
        }
        // ---- O = G Q S + P b E ----
        if constexpr (OUT) {
            const float iu = column_operands(U, Bh, Bl);
            const int valid = min(kDC, a.T - c * kDC);
            In* op = Op + (size_t)c * kDC * a.dv;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f32x4 Z = zero;
#pragma unroll
                for (int j = 0; j <= i / 2; ++j) {
                    const f16x8 ph = row_operand(L.P[0], kDP, i, j, n, g);
                    if constexpr (NP == 2) {
                        Z = mfma_f16x32(ph, Bl[j], Z);
                        Z = mfma_f16x32(row_operand(L.P[1], kDP, i, j, n, g), Bh[j], Z);
                    }
                    Z = mfma_f16x32(ph, Bh[j], Z);
                }
                const f32x4 gq = row4(L.sc + kGq, i, g), pi = row4(L.sc + kPi, i, g);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = 16 * i + 4 * g + r;
                    const float o = (gq[r] * is) * Y[i][r] + (pi[r] * iu) * Z[r];
                    if (t < valid) store1(op + (size_t)t * a.dv, o);
                }
            }
        }
        // ---- S' = G_C S + K^T (D_C b E) ----
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 dc = row4(L.sc + kDc, i, g);
#pragma unroll
            for (int r = 0; r < 4; ++r) U[i][r] *= dc[r];
        }
        const float iw = column_operands(U, Bh, Bl);
        const float gc = L.sc[kGc];
#pragma unroll
        for (int m = 0; m < NS; ++m) {
            f32x4 t = zero;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const f16x8 kh = col_operand(L.K[0], KW, m, j, n, g);
                t = mfma_f16x32(kh, Bl[j], t);
                if constexpr (NP == 2) t = mfma_f16x32(col_operand(L.K[1], KW, m, j, n, g), Bh[j], t);
                t = mfma_f16x32(kh, Bh[j], t);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) S[m][r] = gc * S[m][r] + iw * t[r];
        }
    }
    if (a.final_state && live)
#pragma unroll
        for (int m = 0; m < NS; ++m)
            if (16 * m < a.dk) *reinterpret_cast<f32x4*>(a.final_state + so + 16 * m) = S[m];
}

template <int DKP, bool OUT, bool SAVE>
hipError_t scan_go(const DeltaArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.BH + 7) / 8 * 8 * ((a.dv + 63) / 64)));
    if (a.bf16) hipLaunchKernelGGL((delta_scan_kernel<DKP, bf16_t, OUT, SAVE>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((delta_scan_kernel<DKP, float, OUT, SAVE>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}
template <bool OUT, bool SAVE>
hipError_t scan_dk(const DeltaArgs& a, hipStream_t s) {
    return a.dk <= 32 ? scan_go<32, OUT, SAVE>(a, s)
                      : a.dk == 64 ? scan_go<64, OUT, SAVE>(a, s) : scan_go<128, OUT, SAVE>(a, s);
}

hipError_t launch_delta_scan(const DeltaArgs& a, hipStream_t s) { return scan_dk<true, false>(a, s); }
hipError_t launch_delta_states(const DeltaArgs& a, hipStream_t s) { return scan_dk<false, true>(a, s); }

}  // namespace mesa
