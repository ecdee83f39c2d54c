// delta_bwd_scan.hip -- the gated delta rule's backward pass over the chunks
// (gfx950): the gradients of the chunks' states and of the values.
//
// With dS' the gradient of a chunk's end state and dO that of its outputs
// (delta_core.h's notation):
//   dE = diag(D_C b) K dS' + (P diag(b))^T dO
//   dV = M^T dE                       (the gradient of V - G K S too)
//   dS = G_C dS' + Q^T (G dO) - K^T (G dV)
// from the last chunk to the first.  Like the forward's pass (delta_scan.hip) a
// wave owns 16 of the dv columns and keeps its part of dS in registers; the
// transposes P^T, M^T, Q^T, K^T come from the same LDS planes through
// transposed reads.  Row scales of a transposed plane run along the
// contraction and are folded into the other operand.  Every operand is held
// to 22 bits: the gate gradients are float32 sums of these results.
//
// For float rows of 128 features (the others take delta_bwd_split.hip): the
// gradients of 2x16x4096, dv = 128, take 1098 us in all, bound by this chain and
// the forward's.
#include "delta_core.h"

namespace mesa {

struct alignas(16) BwdScanLds {
    static constexpr int KW = delta_row_words(128);
    uint32_t K[2][kDC * KW];
    uint32_t Q[2][kDC * KW];
    uint32_t M[2][kDC * kDP];
    uint32_t P[2][kDC * kDP];
    float sc[kScal];
};

__global__ __launch_bounds__(256) void delta_bwd_scan_kernel(DeltaBwdArgs b, int waves) {
    constexpr int DK = 128, NJ = DK / 32, NS = DK / 16, KW = BwdScanLds::KW;
    __shared__ BwdScanLds L;
    const DeltaArgs& a = b.f;
    const int lane = threadIdx.x % 64, w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), n = lane & 15, g = lane >> 4;
    const int cgs = (a.dv + 16 * waves - 1) / (16 * waves);
    const int bh = (int)(blockIdx.x / (8 * cgs)) * 8 + blockIdx.x % 8;
    if (bh >= a.BH) return;
    const int col0 = 16 * (waves * (int)(blockIdx.x / 8 % cgs) + w);   // the wave's first column
    const bool live = w < waves && col0 < a.dv;
    const int bk = (bh / a.H) * a.Hk + (bh % a.H) / (a.H / a.Hk);
    const float* Kp = static_cast<const float*>(a.k) + (size_t)bk * a.T * DK;
    const float* Qp = static_cast<const float*>(a.q) + (size_t)bk * a.T * DK;
    const float* Op = static_cast<const float*>(b.grad_out) + (size_t)bh * a.T * a.dv + col0;
    float* Vp = static_cast<float*>(b.grad_v) + (size_t)bh * a.T * a.dv + col0;
    constexpr size_t image = delta_image_words(false);
    const uint16_t* img = a.img + (size_t)bh * a.nc * image;
    const float* scal = a.scal + (size_t)bh * a.nc * kScal;
    const size_t so = ((size_t)bh * a.dv + col0 + n) * DK + 4 * g;
    const uint32_t lv = (4 * g * a.dv + n) * 4;   // this lane's bytes in a 16-row tile of v
    const f32x4 zero{0.f, 0.f, 0.f, 0.f};

    f32x4 S[NS];   // the gradient of the state times 2^cs
    int cs = 0;
#pragma unroll
    for (int m = 0; m < NS; ++m)
        S[m] = b.grad_final && live ? load4(b.grad_final + so + 16 * m) : zero;

    using Units = RowUnits<DK, float>;
    Units kr, qr;
    PlaneUnits<4> pr;
    float vr[16];
    float ksr[Units::n], qsr[Units::n];
    f32x4 scr = zero;
    auto fetch = [&](int chunk) {
        const int c = opaque(chunk);
        const int valid = min(kDC, a.T - c * kDC);
        kr.load(Kp + (size_t)c * kDC * DK, DK, valid);
        qr.load(Qp + (size_t)c * kDC * DK, DK, valid);
        const float* sc = scal + (size_t)c * kScal;
#pragma unroll
        for (int i = 0; i < Units::n; ++i) {
            ksr[i] = *lane_at(sc + kKs, 4 * Units::row(i));
            qsr[i] = *lane_at(sc + kQs, 4 * Units::row(i));
        }
        pr.load(img + c * image);
        if (threadIdx.x < kScal / 4) scr = load4(lane_at(sc, 16 * threadIdx.x));
        const float* op = Op + (size_t)c * kDC * a.dv;
        if (!live) return;
        each_value(lv, fresh(a.dv * 4, c), [&](uint32_t o, int i) {   // zeros behind the end
            vr[i] = valid == kDC || 16 * (i / 4) + 4 * g + i % 4 < valid ? *lane_at(op, o) : 0.f;
        });
    };
    fetch(a.nc - 1);
    for (int chunk = a.nc - 1; chunk >= 0; --chunk) {
        const int c = opaque(chunk);
        __syncthreads();   // the previous chunk's tiles are read
        f32x4 dO[4];
#pragma unroll
        for (int i = 0; i < Units::n; ++i) {
            kr.template store<2>(L.K, i, ksr[i]);
            qr.template store<2>(L.Q, i, qsr[i]);
        }
        pr.store(L.M[0]);   // P's planes follow M's
        if (threadIdx.x < kScal / 4) *reinterpret_cast<f32x4*>(L.sc + 4 * threadIdx.x) = scr;
#pragma unroll
        for (int i = 0; i < 16; ++i) dO[i / 4][i % 4] = vr[i];
        __syncthreads();
        if (chunk > 0) fetch(chunk - 1);
        if (!live) continue;

        {
            const float s = pow2(-cs);
            float* sp = b.dS + ((size_t)bh * a.nc + c) * a.dv * DK + (size_t)(col0 + n) * DK + 4 * g;
#pragma unroll
            for (int m = 0; m < NS; ++m) *reinterpret_cast<f32x4*>(sp + 16 * m) = S[m] * s;
        }
        // ---- dE = D_C b K dS' + (P diag(b))^T dO ----
        f16x8 Sh[NJ], Sl[NJ];
        const float smax = column_max(S);
        const int es = h2_exp(smax);
        column_split(S, es, Sh, Sl);
        const float is = pow2(-es - cs);
        f32x4 X[4], B[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 qi = row4(L.sc + kQi, i, g);
#pragma unroll
            for (int r = 0; r < 4; ++r) B[i][r] = dO[i][r] * qi[r];
        }
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
        f16x8 Bh[2], Bl[2];
        const int eb = column_exp(B);
        column_split(B, eb, Bh, Bl);
        const float ip = L.sc[kPi] * pow2(-eb);
        f32x4 t[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {   // column tiles up to 2 j + 1 reach row block j
            f16x8 ph[4], pl[4];
#pragma unroll
            for (int i = 0; i < 2 * j + 2; ++i) {
                ph[i] = col_operand(L.P[0], kDP, i, j, n, g);
                pl[i] = col_operand(L.P[1], kDP, i, j, n, g);
            }
#pragma unroll
            for (int i = 0; i < 2 * j + 2; ++i) i / 2 < j ? mfma_acc(t[i], ph[i], Bl[j]) : mfma_first(t[i], ph[i], Bl[j]);
#pragma unroll
            for (int i = 0; i < 2 * j + 2; ++i) mfma_acc(t[i], pl[i], Bh[j]);
#pragma unroll
            for (int i = 0; i < 2 * j + 2; ++i) mfma_acc(t[i], ph[i], Bh[j]);
        }
        mfma_done(t);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 db = row4(L.sc + kDb, i, g);
#pragma unroll
            for (int r = 0; r < 4; ++r) X[i][r] = X[i][r] * (db[r] * is) + t[i][r] * ip;
        }
        // ---- dV = M^T dE ----
        const int ex = column_exp(X);
        column_split(X, ex, Bh, Bl);
        const float ix = L.sc[kMi] * pow2(-ex);
        const int valid = min(kDC, a.T - c * kDC);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            f16x8 mh[4], ml[4];
#pragma unroll
            for (int i = 0; i < 2 * j + 2; ++i) {
                mh[i] = col_operand(L.M[0], kDP, i, j, n, g);
                ml[i] = col_operand(L.M[1], kDP, i, j, n, g);
            }
#pragma unroll
            for (int i = 0; i < 2 * j + 2; ++i) i / 2 < j ? mfma_acc(t[i], mh[i], Bl[j]) : mfma_first(t[i], mh[i], Bl[j]);
#pragma unroll
            for (int i = 0; i < 2 * j + 2; ++i) mfma_acc(t[i], ml[i], Bh[j]);
#pragma unroll
            for (int i = 0; i < 2 * j + 2; ++i) mfma_acc(t[i], mh[i], Bh[j]);
        }
        mfma_done(t);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x4 gk = row4(L.sc + kGk, i, g), gq = row4(L.sc + kGq, i, g);
            t[i] *= ix;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                X[i][r] = -gk[r] * t[i][r];
                B[i][r] = gq[r] * dO[i][r];
            }
        }
        {
            float* rp = b.dR + ((size_t)bh * a.nc + c) * kDC * a.dv + col0;
            float* vp = Vp + (size_t)c * kDC * a.dv;
            each_value(lv, fresh(a.dv * 4, c), [&](uint32_t o, int i) { *lane_at(rp, o) = t[i / 4][i % 4]; });
            each_value(lv, fresh(a.dv * 4, c), [&](uint32_t o, int i) {
                if (valid == kDC || 16 * (i / 4) + 4 * g + i % 4 < valid) *lane_at(vp, o) = t[i / 4][i % 4];
            });
        }
        // ---- dS = G_C dS' + Q^T (G dO) - K^T (G dV), dS kept scaled as the forward's S ----
        const int ew = min(h2_exp(kslot_max(fmaxf(absmax(X), absmax(B)))), add_exp_cap(smax, es, cs, L.sc[kGc]));
        const float gs = __builtin_amdgcn_ldexpf(L.sc[kGc], ew - cs);
        cs = ew;
        f16x8 Xh[2], Xl[2];
        column_split(X, ew, Xh, Xl);
        column_split(B, ew, Bh, Bl);
#pragma unroll
        for (int m = 0; m < NS; ++m) S[m] *= gs;
        mfma_ready(S);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int t2 = 0; t2 < 2; ++t2) {   // K with the values' gradients, Q with the outputs'
                const uint32_t* hi = t2 ? L.Q[0] : L.K[0];
                const uint32_t* lo = t2 ? L.Q[1] : L.K[1];
                const f16x8 h = t2 ? Bh[j] : Xh[j], l = t2 ? Bl[j] : Xl[j];
                f16x8 rows[NS];
#pragma unroll
                for (int m = 0; m < NS; ++m) rows[m] = col_operand(hi, KW, m, j, n, g);
#pragma unroll
                for (int m = 0; m < NS; ++m) mfma_acc(S[m], rows[m], l);
#pragma unroll
                for (int m = 0; m < NS; ++m) mfma_acc(S[m], col_operand(lo, KW, m, j, n, g), h);
#pragma unroll
                for (int m = 0; m < NS; ++m) mfma_acc(S[m], rows[m], h);
            }
        }
        mfma_done(S);
    }
    if (b.grad_state && live) {
        const float s = pow2(-cs);
#pragma unroll
        for (int m = 0; m < NS; ++m) *reinterpret_cast<f32x4*>(b.grad_state + so + 16 * m) = S[m] * s;
    }
}

// Float rows of 128 features: two planes of K, twice, do not fit the split
// kernels' LDS; everything else takes those.
hipError_t launch_delta_passes(const DeltaBwdArgs& b, hipStream_t s) {
    if (b.f.bf16 || b.f.dk < 128) return launch_delta_passes_split(b, s);
    const hipError_t e = launch_delta_states(b.f, s);
    if (e != hipSuccess) return e;
    const int waves = scan_waves(b.f.BH, b.f.dv);
    hipLaunchKernelGGL(delta_bwd_scan_kernel, dim3(scan_blocks(b.f.BH, b.f.dv, waves)), dim3(256), 0, s, b, waves);
    return hipGetLastError();
}

}  // namespace mesa
