// delta_scan.hip -- the gated delta rule's pass over the chunks (gfx950).
//
// A wave owns 16 of the state's dv columns for the whole sequence: they never
// meet the other columns.  Its part of S (dk x 16) stays in registers in MFMA
// accumulator order, which is also the operand order of the next product
// (cg_h2.h's perm32), so the chunk's chain
//   X = K S,  R = V - G X,  E = M R,  O = G Q S + (P diag(b)) E,
//   S' = G_C S + K^T (D_C b E)
// runs without exchanging anything between lanes but the column maxima that
// scale the fp16 operands.  S is kept scaled by a power of two per column, so
// that the update's MFMAs add onto it directly.  A workgroup of four waves
// stages the chunk's K, Q, M and P in LDS for its columns; the next chunk's
// rows are in flight in registers meanwhile.
//
// The pass is bound by the instructions a wave issues for a chunk (4 cycles
// each, a wave a SIMD) and by the chain's latencies, not by memory.  Few heads
// leave compute units idle: then a workgroup takes 32 or 16 columns and its
// other waves only stage.  Only float rows of 128 features come here, whose
// planes delta_scan_split.h's kernel has no LDS for: a forward of 8x16x4096, dv =
// 128, takes 691 us of which this is 80 %, one of 2x16x4096 497 us.
//
// Precision: every operand is hi + lo (22 bits).
#include "delta_core.h"

namespace mesa {

struct alignas(16) ScanLds {
    static constexpr int KW = delta_row_words(128);
    uint32_t K[2][kDC * KW];
    uint32_t Q[2][kDC * KW];
    uint32_t M[2][kDC * kDP];
    uint32_t P[2][kDC * kDP];
    float sc[kScal];
};

// OUT: write O.  Else the backward's recomputation: write each chunk's start
// state and E.
template <bool OUT>
__global__ __launch_bounds__(256) void delta_scan_kernel(DeltaArgs a, int waves) {
    constexpr int DK = 128, NJ = DK / 32, NS = DK / 16, KW = ScanLds::KW;
    __shared__ ScanLds L;
    const int lane = threadIdx.x % 64, w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), n = lane & 15, g = lane >> 4;
    // the column groups of a head on one XCD (workgroups go to the 8 XCDs in turn)
    const int cgs = (a.dv + 16 * waves - 1) / (16 * waves);
    const int bh = (int)(blockIdx.x / (8 * cgs)) * 8 + blockIdx.x % 8;
    if (bh >= a.BH) return;
    const int col0 = 16 * (waves * (int)(blockIdx.x / 8 % cgs) + w);   // the wave's first column
    const bool live = w < waves && col0 < a.dv;
    const int bk = (bh / a.H) * a.Hk + (bh % a.H) / (a.H / a.Hk);
    const float* Kp = static_cast<const float*>(a.k) + (size_t)bk * a.T * DK;
    const float* Qp = static_cast<const float*>(a.q) + (size_t)bk * a.T * DK;
    const float* Vp = static_cast<const float*>(a.v) + (size_t)bh * a.T * a.dv + col0;
    float* Op = OUT ? static_cast<float*>(a.out) + (size_t)bh * a.T * a.dv + col0 : nullptr;
    constexpr size_t image = delta_image_words(false);
    const uint16_t* img = a.img + (size_t)bh * a.nc * image;
    const float* scal = a.scal + (size_t)bh * a.nc * kScal;
    const size_t so = ((size_t)bh * a.dv + col0 + n) * DK + 4 * g;   // this lane's row of the (dv x dk) state
    const uint32_t lv = (4 * g * a.dv + n) * 4;               // this lane's bytes in a 16-row tile of v
    const f32x4 zero{0.f, 0.f, 0.f, 0.f};

    f32x4 S[NS];   // the state times 2^cs
    int cs = 0;
#pragma unroll
    for (int m = 0; m < NS; ++m)
        S[m] = a.state0 && live ? load4(a.state0 + so + 16 * m) : zero;

    using Units = RowUnits<DK, float>;
    using Planes = PlaneUnits<OUT ? 4 : 2>;
    Units kr, qr;
    Planes pr;
    float vr[16];
    float ksr[Units::n], qsr[Units::n];
    f32x4 scr = zero;
    auto fetch = [&](int chunk) {
        const int c = opaque(chunk);
        const int valid = min(kDC, a.T - c * kDC);
        kr.load(Kp + (size_t)c * kDC * DK, DK, valid);
        if constexpr (OUT) qr.load(Qp + (size_t)c * kDC * DK, DK, valid);
        const float* sc = scal + (size_t)c * kScal;
#pragma unroll
        for (int i = 0; i < Units::n; ++i) {
            ksr[i] = *lane_at(sc + kKs, 4 * Units::row(i));
            if constexpr (OUT) qsr[i] = *lane_at(sc + kQs, 4 * Units::row(i));
        }
        pr.load(img + c * image);
        if (threadIdx.x < kScal / 4) scr = load4(lane_at(sc, 16 * threadIdx.x));
        if (!live) return;
        const float* vp = Vp + (size_t)c * kDC * a.dv;
        each_value(lv, fresh(a.dv * 4, c), [&](uint32_t o, int i) {   // zeros behind the end
            vr[i] = valid == kDC || 16 * (i / 4) + 4 * g + i % 4 < valid ? *lane_at(vp, o) : 0.f;
        });
    };
    fetch(0);
    for (int chunk = 0; chunk < a.nc; ++chunk) {
        const int c = opaque(chunk);
        __syncthreads();   // the previous chunk's tiles are read
        f32x4 V[4];
#pragma unroll
        for (int i = 0; i < Units::n; ++i) {
            kr.template store<2>(L.K, i, ksr[i]);
            if constexpr (OUT) qr.template store<2>(L.Q, i, qsr[i]);
        }
        pr.store(L.M[0]);   // P's planes follow M's
        if (threadIdx.x < kScal / 4) *reinterpret_cast<f32x4*>(L.sc + 4 * threadIdx.x) = scr;
#pragma unroll
        for (int i = 0; i < 16; ++i) V[i / 4][i % 4] = vr[i];
        __syncthreads();
        if (chunk + 1 < a.nc) fetch(chunk + 1);
        if (!live) continue;

        if constexpr (!OUT) {
            const float s = pow2(-cs);
            float* sp = a.S + ((size_t)bh * a.nc + c) * a.dv * DK + (size_t)(col0 + n) * DK + 4 * g;
#pragma unroll
            for (int m = 0; m < NS; ++m) *reinterpret_cast<f32x4*>(sp + 16 * m) = S[m] * s;
        }
        // ---- K S and Q S ----
        f16x8 Sh[NJ], Sl[NJ];
        const float smax = column_max(S);
        const int es = h2_exp(smax);
        column_split(S, es, Sh, Sl);
        const float is = pow2(-es - cs);
        f32x4 X[4], Y[4];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            f16x8 kh[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) kh[i] = row_operand(L.K[0], KW, i, j, n, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) j ? mfma_acc(X[i], kh[i], Sl[j]) : mfma_first(X[i], kh[i], Sl[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) mfma_acc(X[i], row_operand(L.K[1], KW, i, j, n, g), Sh[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) mfma_acc(X[i], kh[i], Sh[j]);
        }
        mfma_done(X);
        if constexpr (OUT) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                f16x8 qh[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) qh[i] = row_operand(L.Q[0], KW, i, j, n, g);
#pragma unroll
                for (int i = 0; i < 4; ++i) j ? mfma_acc(Y[i], qh[i], Sl[j]) : mfma_first(Y[i], qh[i], Sl[j]);
#pragma unroll
                for (int i = 0; i < 4; ++i) mfma_acc(Y[i], row_operand(L.Q[1], KW, i, j, n, g), Sh[j]);
#pragma unroll
                for (int i = 0; i < 4; ++i) mfma_acc(Y[i], qh[i], Sh[j]);
            }
            mfma_done(Y);
        }
        // ---- E = M (V - G K S) ----
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 gk = row4(L.sc + kGk, i, g);
#pragma unroll
            for (int r = 0; r < 4; ++r) X[i][r] = V[i][r] - (gk[r] * is) * X[i][r];
        }
        f16x8 Bh[2], Bl[2];
        const int er = column_exp(X);
        column_split(X, er, Bh, Bl);
        f32x4 U[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {   // row tiles 2 j and up reach column block j
            f16x8 mh[4], ml[4];
#pragma unroll
            for (int i = 2 * j; i < 4; ++i) {
                mh[i] = row_operand(L.M[0], kDP, i, j, n, g);
                ml[i] = row_operand(L.M[1], kDP, i, j, n, g);
            }
#pragma unroll
            for (int i = 2 * j; i < 4; ++i) j ? mfma_acc(U[i], mh[i], Bl[j]) : mfma_first(U[i], mh[i], Bl[j]);
#pragma unroll
            for (int i = 2 * j; i < 4; ++i) mfma_acc(U[i], ml[i], Bh[j]);
#pragma unroll
            for (int i = 2 * j; i < 4; ++i) mfma_acc(U[i], mh[i], Bh[j]);
        }
        mfma_done(U);
        const float ir = L.sc[kMi] * pow2(-er);
#pragma unroll
        for (int i = 0; i < 4; ++i) U[i] *= ir;
        if constexpr (!OUT) {
            float* ep = a.E + ((size_t)bh * a.nc + c) * kDC * a.dv + col0;
            each_value(lv, fresh(a.dv * 4, c), [&](uint32_t o, int i) { *lane_at(ep, o) = U[i / 4][i % 4]; });
        }
        // ---- O = G Q S + P diag(b) E ----
        if constexpr (OUT) {
            const int eu = column_exp(U);
            column_split(U, eu, Bh, Bl);
            const float iu = L.sc[kPi] * pow2(-eu);
            f32x4 Z[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                f16x8 ph[4];
#pragma unroll
                for (int i = 2 * j; i < 4; ++i) ph[i] = row_operand(L.P[0], kDP, i, j, n, g);
#pragma unroll
                for (int i = 2 * j; i < 4; ++i) j ? mfma_acc(Z[i], ph[i], Bl[j]) : mfma_first(Z[i], ph[i], Bl[j]);
#pragma unroll
                for (int i = 2 * j; i < 4; ++i) mfma_acc(Z[i], row_operand(L.P[1], kDP, i, j, n, g), Bh[j]);
#pragma unroll
                for (int i = 2 * j; i < 4; ++i) mfma_acc(Z[i], ph[i], Bh[j]);
            }
            mfma_done(Z);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 gq = row4(L.sc + kGq, i, g), qi = row4(L.sc + kQi, i, g);
#pragma unroll
                for (int r = 0; r < 4; ++r) Y[i][r] = (gq[r] * is) * Y[i][r] + (qi[r] * iu) * Z[i][r];
            }
            const int valid = min(kDC, a.T - c * kDC);
            float* op = Op + (size_t)c * kDC * a.dv;
            each_value(lv, fresh(a.dv * 4, c), [&](uint32_t o, int i) {
                if (valid == kDC || 16 * (i / 4) + 4 * g + i % 4 < valid) *lane_at(op, o) = Y[i / 4][i % 4];
            });
        }
        // ---- S' = G_C S + K^T (D_C b E) ----
#pragma unroll
        for (int i = 0; i < 4; ++i) U[i] *= row4(L.sc + kDb, i, g);
        const int ew = min(column_exp(U), add_exp_cap(smax, es, cs, L.sc[kGc]));
        column_split(U, ew, Bh, Bl);
        const float gs = __builtin_amdgcn_ldexpf(L.sc[kGc], ew - cs);
        cs = ew;
#pragma unroll
        for (int m = 0; m < NS; ++m) S[m] *= gs;
        mfma_ready(S);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            f16x8 kh[NS];
#pragma unroll
            for (int m = 0; m < NS; ++m) kh[m] = col_operand(L.K[0], KW, m, j, n, g);
#pragma unroll
            for (int m = 0; m < NS; ++m) mfma_acc(S[m], kh[m], Bl[j]);
#pragma unroll
            for (int m = 0; m < NS; ++m) mfma_acc(S[m], col_operand(L.K[1], KW, m, j, n, g), Bh[j]);
#pragma unroll
            for (int m = 0; m < NS; ++m) mfma_acc(S[m], kh[m], Bh[j]);
        }
        mfma_done(S);
    }
    if (a.final_state && live) {
        const float s = pow2(-cs);
#pragma unroll
        for (int m = 0; m < NS; ++m) *reinterpret_cast<f32x4*>(a.final_state + so + 16 * m) = S[m] * s;
    }
}

template <bool OUT>
hipError_t scan_go(const DeltaArgs& a, hipStream_t s) {
    const int waves = scan_waves(a.BH, a.dv);
    hipLaunchKernelGGL((delta_scan_kernel<OUT>), dim3(scan_blocks(a.BH, a.dv, waves)), dim3(256), 0, s, a, waves);
    return hipGetLastError();
}

// Float rows of 128 features need two planes of K twice in the split kernel's
// LDS, which does not hold them; everything else takes that kernel.
hipError_t launch_delta_scan(const DeltaArgs& a, hipStream_t s) {
    if (!a.bf16 && a.dk == 128) return scan_go<true>(a, s);
    const hipError_t e = launch_delta_segments(a, s);
    return e != hipSuccess ? e : launch_delta_scan_split(a, s);
}
hipError_t launch_delta_states(const DeltaArgs& a, hipStream_t s) { return scan_go<false>(a, s); }

}  // namespace mesa
