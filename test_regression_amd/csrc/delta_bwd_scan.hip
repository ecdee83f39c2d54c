// delta_bwd_scan.hip -- the gated delta rule's backward pass over the chunks
// (gfx950): the gradients of the chunks' states and of the values.
//
// With dS' the gradient of a chunk's end state and dO that of its outputs
// (delta_core.h's notation; pE = b E is what the chunk writes):
//   d(bE) = diag(D_C) K dS' + P^T dO
//   dV    = M^T (b d(bE))                       (the gradient of V - G K S too)
//   dS    = G_C dS' + Q^T (G dO) - K^T (G dV)
// from the last chunk to the first.  Like the forward's pass (delta_scan.hip) a
// wave owns 16 of the dv columns and keeps its part of dS in registers; the
// transposes P^T, M^T, Q^T, K^T come from the same LDS planes through
// transposed reads.  Row scales of a transposed plane run along the
// contraction and are folded into the other operand.  Every operand is held
// to 22 bits: the gate gradients are float32 sums of these results.
#include "delta_core.h"

namespace mesa {

template <int DKP, int NP>
struct alignas(16) BwdScanLds {
    static constexpr int KW = delta_row_words(DKP);
    uint32_t K[NP][kDC * KW];
    uint32_t Q[NP][kDC * KW];
    uint32_t M[2][kDC * kDP];
    uint32_t P[2][kDC * kDP];
    float sc[kScal];
};

template <int DKP, typename In>
__global__ __launch_bounds__(256) void delta_bwd_scan_kernel(DeltaBwdArgs b) {
    constexpr int NP = delta_planes<In>(), NJ = DKP / 32, NS = DKP / 16, KW = delta_row_words(DKP);
    __shared__ BwdScanLds<DKP, NP> L;
    const DeltaArgs& a = b.f;
    const int lane = threadIdx.x % 64, w = threadIdx.x / 64, n = lane & 15, g = lane >> 4;
    const int cgs = (a.dv + 63) / 64;
    const long bh = (long)(blockIdx.x / (8 * cgs)) * 8 + blockIdx.x % 8;
    if (bh >= a.BH) return;
    const int col = 64 * (int)(blockIdx.x / 8 % cgs) + 16 * w + n;
    const bool live = col - n < a.dv;   // a whole wave
    const long bk = (bh / a.H) * a.Hk + (bh % a.H) / (a.H / a.Hk);
    const In* Kp = static_cast<const In*>(a.k) + (size_t)bk * a.T * a.dk;
    const In* Qp = static_cast<const In*>(a.q) + (size_t)bk * a.T * a.dk;
    const In* Op = static_cast<const In*>(b.grad_out) + (size_t)bh * a.T * a.dv + col;
    In* Vp = static_cast<In*>(b.grad_v) + (size_t)bh * a.T * a.dv + col;
    constexpr size_t image = (size_t)4 * kDC * kDC;
    const uint16_t* img = a.img + (size_t)bh * a.nc * image;
    const float* scal = a.scal + (size_t)bh * a.nc * kScal;
    const size_t so = ((size_t)bh * a.dv + col) * a.dk + 4 * g;
    const f32x4 zero{0.f, 0.f, 0.f, 0.f};

    f32x4 S[NS];   // the gradient of the state
#pragma unroll
    for (int m = 0; m < NS; ++m)
        S[m] = b.grad_final && live && 16 * m < a.dk ? load4(b.grad_final + so + 16 * m) : zero;

    using Units = RowUnits<DKP, In>;
    Units kr, qr;
    PlaneUnits<2> mr, pr;
    In vr[16];
    float ksr[Units::n], qsr[Units::n];
    f32x4 scr = zero;
    auto fetch = [&](int c) {
        const int valid = min(kDC, a.T - c * kDC);
        kr.load(Kp + (size_t)c * kDC * a.dk, a.dk, valid);
        qr.load(Qp + (size_t)c * kDC * a.dk, a.dk, valid);
        const float* sc = scal + (size_t)c * kScal;
#pragma unroll
        for (int i = 0; i < Units::n; ++i) {
            ksr[i] = sc[kKs + Units::row(i)];
            qsr[i] = sc[kQs + Units::row(i)];
        }
        mr.load(img + c * image);
        pr.load(img + c * image + 2 * kDC * kDC);
        if (threadIdx.x < kScal / 4) scr = load4(sc + 4 * threadIdx.x);
        const In* op = Op + (size_t)c * kDC * a.dv;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int t = 16 * (i / 4) + 4 * g + i % 4;
            vr[i] = live && t < valid ? op[(size_t)t * a.dv] : In{};
        }
    };
    fetch(a.nc - 1);
    for (int c = a.nc - 1; c >= 0; --c) {
        __syncthreads();   // the previous chunk's tiles are read
        f32x4 dO[4];
#pragma unroll
        for (int i = 0; i < Units::n; ++i) {
            kr.template store<NP>(L.K, i, ksr[i]);
            qr.template store<NP>(L.Q, i, qsr[i]);
        }
        mr.store(L.M);
        pr.store(L.P);
        if (threadIdx.x < kScal / 4) *reinterpret_cast<f32x4*>(L.sc + 4 * threadIdx.x) = scr;
#pragma unroll
        for (int i = 0; i < 16; ++i) dO[i / 4][i % 4] = to_f32(vr[i]);
        __syncthreads();
        if (c > 0) fetch(c - 1);
        if (!live) continue;

        {
            float* sp = b.dS + (((size_t)bh * a.nc + c) * a.dv + col) * a.dk + 4 * g;
#pragma unroll
            for (int m = 0; m < NS; ++m)
                if (16 * m < a.dk) *reinterpret_cast<f32x4*>(sp + 16 * m) = S[m];
        }
        // ---- d(bE) = D_C K dS' + P^T dO ----
        f16x8 Sh[NJ], Sl[NJ];
        const float is = column_operands(S, Sh, Sl);
        f32x4 X[4], B[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            X[i] = zero;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const f16x8 kh = row_operand(L.K[0], KW, i, j, n, g);
                X[i] = mfma_f16x32(kh, Sl[j], X[i]);
                if constexpr (NP == 2) X[i] = mfma_f16x32(row_operand(L.K[1], KW, i, j, n, g), Sh[j], X[i]);
                X[i] = mfma_f16x32(kh, Sh[j], X[i]);
            }
            const f32x4 pi = row4(L.sc + kPi, i, g);
#pragma unroll
            for (int r = 0; r < 4; ++r) B[i][r] = dO[i][r] * pi[r];
        }
        f16x8 Bh[2], Bl[2];
        const float ip = column_operands(B, Bh, Bl);   // bf16 gradients are exact in the hi part
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x4 t = zero;
#pragma unroll
            for (int j = i / 2; j < 2; ++j) {
                const f16x8 ph = col_operand(L.P[0], kDP, i, j, n, g);
                if constexpr (NP == 2) t = mfma_f16x32(ph, Bl[j], t);
                t = mfma_f16x32(col_operand(L.P[1], kDP, i, j, n, g), Bh[j], t);
                t = mfma_f16x32(ph, Bh[j], t);
            }
            const f32x4 dc = row4(L.sc + kDc, i, g), mi = row4(L.sc + kMi, i, g), be = row4(L.sc + kBe, i, g);
#pragma unroll
            for (int r = 0; r < 4; ++r) X[i][r] = (X[i][r] * (dc[r] * is) + t[r] * ip) * (be[r] * mi[r]);
        }
        // ---- dV = M^T (b d(bE)) ----
        const float ix = column_operands(X, Bh, Bl);
        const int valid = min(kDC, a.T - c * kDC);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x4 t = zero;
#pragma unroll
            for (int j = i / 2; j < 2; ++j) {
                const f16x8 mh = col_operand(L.M[0], kDP, i, j, n, g);
                t = mfma_f16x32(mh, Bl[j], t);
                t = mfma_f16x32(col_operand(L.M[1], kDP, i, j, n, g), Bh[j], t);
                t = mfma_f16x32(mh, Bh[j], t);
            }
            float* rp = b.dR + ((size_t)(bh * a.nc + c) * kDC + 16 * i + 4 * g) * a.dv + col;
            In* vp = Vp + (size_t)c * kDC * a.dv;
            const f32x4 gk = row4(L.sc + kGk, i, g), gq = row4(L.sc + kGq, i, g);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float d = t[r] * ix;
                rp[(size_t)r * a.dv] = d;
                const int tok = 16 * i + 4 * g + r;
                if (tok < valid) store1(vp + (size_t)tok * a.dv, d);
                X[i][r] = -gk[r] * d;
                B[i][r] = gq[r] * dO[i][r];
            }
        }
        // ---- dS = G_C dS' + Q^T (G dO) - K^T (G dV) ----
        const int E = h2_exp(kslot_max(fmaxf(absmax(X), absmax(B))));
        const float s = pow2(E), iw = pow2(-E), gc = L.sc[kGc];
        f16x8 Xh[2], Xl[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            h2_split(X[2 * j], X[2 * j + 1], s, Xh[j], Xl[j]);
            h2_split(B[2 * j], B[2 * j + 1], s, Bh[j], Bl[j]);
        }
#pragma unroll
        for (int m = 0; m < NS; ++m) {
            f32x4 t = zero;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const f16x8 kh = col_operand(L.K[0], KW, m, j, n, g), qh = col_operand(L.Q[0], KW, m, j, n, g);
                t = mfma_f16x32(kh, Xl[j], t);
                t = mfma_f16x32(qh, Bl[j], t);
                if constexpr (NP == 2) {
                    t = mfma_f16x32(col_operand(L.K[1], KW, m, j, n, g), Xh[j], t);
                    t = mfma_f16x32(col_operand(L.Q[1], KW, m, j, n, g), Bh[j], t);
                }
                t = mfma_f16x32(kh, Xh[j], t);
                t = mfma_f16x32(qh, Bh[j], t);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) S[m][r] = gc * S[m][r] + iw * t[r];
        }
    }
    if (b.grad_state && live)
#pragma unroll
        for (int m = 0; m < NS; ++m)
            if (16 * m < a.dk) *reinterpret_cast<f32x4*>(b.grad_state + so + 16 * m) = S[m];
}

template <int DKP>
hipError_t bwd_scan_go(const DeltaBwdArgs& b, hipStream_t s) {
    const dim3 grid((unsigned)((b.f.BH + 7) / 8 * 8 * ((b.f.dv + 63) / 64)));
    if (b.f.bf16) hipLaunchKernelGGL((delta_bwd_scan_kernel<DKP, bf16_t>), grid, dim3(256), 0, s, b);
    else hipLaunchKernelGGL((delta_bwd_scan_kernel<DKP, float>), grid, dim3(256), 0, s, b);
    return hipGetLastError();
}

hipError_t launch_delta_bwd_scan(const DeltaBwdArgs& b, hipStream_t s) {
    return b.f.dk <= 32 ? bwd_scan_go<32>(b, s) : b.f.dk == 64 ? bwd_scan_go<64>(b, s) : bwd_scan_go<128>(b, s);
}

}  // namespace mesa
