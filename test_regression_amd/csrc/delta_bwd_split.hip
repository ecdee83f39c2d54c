// delta_bwd_split.hip -- the gated delta rule's backward pass over the chunks
// with the state's chain and everything beside it on different waves (gfx950).
//
// delta_bwd_scan.hip's pass, split over twelve waves as delta_scan_split.hip
// splits the forward's.  Waves 0..3 run, for 16 dv columns each and from the
// last chunk to the first, what the next chunk waits for:
//   dE = D_C b K dS' + T,  dV = M^T dE,  dS = G_C dS' + N - K^T (G dV)
// Waves 4..7 form T = (P diag(b))^T dO and N = Q^T (G dO), which need no state,
// ahead of them, and write dV out.  Waves 8..11 stage the chunks.  Two barriers
// a chunk; between them:
//   first half of c    split, K dS', dE    N of c, dV of c + 1 out    M of c, P of c - 1 in
//   second half of c   dV, update          T of c - 1                 K, Q of c - 1 in
// K is held twice in LDS.
//
// The pass needs nothing of the forward's recomputation (the chunks' start
// states and E, delta_scan_split.h), nor that of it, so one launch holds the
// workgroups of both: with few heads they fill the GPU together.
//
// Bound, like the forward's pass, by the chain: 2x16x4096, dk = dv = 128, bf16
// (256 column tiles each way) takes 244-255 us, 3.8-4.0 us a chunk, for 0.67 GB of
// traffic; all of the gradients took 590 us with a launch for each pass and 447
// with one (428 today).  2x8x1023 float with dk = 64, dv = 128: 51-52 us.
#include "delta_scan_split.h"

namespace mesa {

template <int DKP, typename In>
struct alignas(16) BwdSplitLds {
    static constexpr int NP = delta_planes<In>(), KW = delta_row_words(DKP), NS = DKP / 16;
    uint32_t K[2][NP][kDC * KW];
    uint32_t M[2 * kCPlane];
    uint32_t Q[NP][kDC * KW];
    uint32_t P[2 * kCPlane];
    f32x4 T[4][4][64], N[4][NS][64], dV[4][4 * kTileSlots];
    int ne[4][64];   // the cap that N's column sets to the scale of what it is added to
    float sc[2][kScal];
};

template <int DKP, typename In>
__device__ __forceinline__ void bwd_split(BwdSplitLds<DKP, In>& L, const DeltaBwdArgs& b, int waves, unsigned block) {
    using Lds = BwdSplitLds<DKP, In>;
    constexpr int NP = Lds::NP, NJ = DKP / 32, NS = Lds::NS, KW = Lds::KW;
    const DeltaArgs& a = b.f;
    const int lane = threadIdx.x % 64, w12 = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), w = w12 % 4;
    const int n = lane & 15, g = lane >> 4;
    const int cols = 16 * waves, cgs = (a.dv + cols - 1) / cols;
    const int bh = (int)(block / (8 * cgs)) * 8 + block % 8;
    if (bh >= a.BH) return;
    const int col0 = cols * (int)(block / 8 % cgs) + 16 * w;
    const bool live = w < waves && col0 < a.dv;
    const size_t so = ((size_t)bh * a.dv + col0 + n) * a.dk + 4 * g;

    if (w12 < 4) {
        // ---------------- the state's chain ----------------
        f32x4 S[NS];   // the gradient of the state times 2^cs
        int cs = 0;
#pragma unroll
        for (int m = 0; m < NS; ++m)
            S[m] = b.grad_final && live && 16 * m < a.dk ? load4(b.grad_final + so + 16 * m) : f32x4{0.f, 0.f, 0.f, 0.f};
        __syncthreads();   // P of the last chunk
        for (int chunk = a.nc - 1; chunk >= 0; --chunk) {
            const int c = opaque(chunk);
            __syncthreads();
            const float* sc = L.sc[c & 1];
            const auto& K = L.K[c & 1];
            f16x8 Bh[2], Bl[2];
            float smax = 0.f;
            int es = 0, ex = 0;
            if (live) {
                {
                    const float s = pow2(-cs);
                    float* sp = b.dS + ((size_t)bh * a.nc + c) * a.dv * a.dk + (size_t)(col0 + n) * a.dk + 4 * g;
#pragma unroll
                    for (int m = 0; m < NS; ++m)
                        if (16 * m < a.dk) *reinterpret_cast<f32x4*>(sp + 16 * m) = S[m] * s;
                }
                // ---- dE = D_C b K dS' + T ----
                f16x8 Sh[NJ], Sl[NJ];
                smax = column_max(S);
                es = h2_exp(smax);
                column_split(S, es, Sh, Sl);
                const float is = pow2(-es - cs);
                f32x4 X[4];
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    f16x8 kh[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) kh[i] = row_operand(K[0], KW, i, j, n, g);
#pragma unroll
                    for (int i = 0; i < 4; ++i) j ? mfma_acc(X[i], kh[i], Sl[j]) : mfma_first(X[i], kh[i], Sl[j]);
                    if constexpr (NP == 2)
#pragma unroll
                        for (int i = 0; i < 4; ++i) mfma_acc(X[i], row_operand(K[NP - 1], KW, i, j, n, g), Sh[j]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) mfma_acc(X[i], kh[i], Sh[j]);
                }
                mfma_done(X);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 db = row4(sc + kDb, i, g), t = L.T[w][i][lane];
#pragma unroll
                    for (int r = 0; r < 4; ++r) X[i][r] = X[i][r] * (db[r] * is) + t[r];
                }
                ex = column_exp(X);
                column_split(X, ex, Bh, Bl);
            }
            __syncthreads();
            if (!live) continue;
            // ---- dV = M^T dE ----
            f32x4 U[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {   // column tiles up to 2 j + 1 reach row block j
                f16x8 mh[4], ml[4];
#pragma unroll
                for (int i = 0; i < 2 * j + 2; ++i) {
                    mh[i] = compact_col_operand(L.M, i, j, n, g);
                    ml[i] = compact_col_operand(L.M + kCPlane, i, j, n, g);
                }
#pragma unroll
                for (int i = 0; i < 2 * j + 2; ++i) i / 2 < j ? mfma_acc(U[i], mh[i], Bl[j]) : mfma_first(U[i], mh[i], Bl[j]);
#pragma unroll
                for (int i = 0; i < 2 * j + 2; ++i) mfma_acc(U[i], ml[i], Bh[j]);
#pragma unroll
                for (int i = 0; i < 2 * j + 2; ++i) mfma_acc(U[i], mh[i], Bh[j]);
            }
            mfma_done(U);
            const float ix = sc[kMi] * pow2(-ex);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                U[i] *= ix;
                L.dV[w][tile_slot(i, n, g)] = U[i];
                const f32x4 gk = row4(sc + kGk, i, g);
#pragma unroll
                for (int r = 0; r < 4; ++r) U[i][r] *= -gk[r];
            }
            // ---- dS = G_C dS' + N - K^T (G dV) ----
            const int ew = min(column_exp(U), min(add_exp_cap(smax, es, cs, sc[kGc]), L.ne[w][lane]));
            column_split(U, ew, Bh, Bl);
            const float gs = __builtin_amdgcn_ldexpf(sc[kGc], ew - cs), ns = pow2(ew);
            cs = ew;
#pragma unroll
            for (int m = 0; m < NS; ++m) {
                const f32x4 t = L.N[w][m][lane];
#pragma unroll
                for (int r = 0; r < 4; ++r) S[m][r] = S[m][r] * gs + t[r] * ns;
            }
            mfma_ready(S);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                f16x8 kh[NS];
#pragma unroll
                for (int m = 0; m < NS; ++m) kh[m] = col_operand(K[0], KW, m, j, n, g);
#pragma unroll
                for (int m = 0; m < NS; ++m) mfma_acc(S[m], kh[m], Bl[j]);
                if constexpr (NP == 2)
#pragma unroll
                    for (int m = 0; m < NS; ++m) mfma_acc(S[m], col_operand(K[NP - 1], KW, m, j, n, g), Bh[j]);
#pragma unroll
                for (int m = 0; m < NS; ++m) mfma_acc(S[m], kh[m], Bh[j]);
            }
            mfma_done(S);
        }
        __syncthreads();
        if (b.grad_state && live) {
            const float s = pow2(-cs);
#pragma unroll
            for (int m = 0; m < NS; ++m)
                if (16 * m < a.dk) *reinterpret_cast<f32x4*>(b.grad_state + so + 16 * m) = S[m] * s;
        }
    } else if (w12 < 8) {
        // ---------------- T and N; dV out ----------------
        const In* Op = static_cast<const In*>(b.grad_out) + (size_t)bh * a.T * a.dv + col0;
        In* Vp = static_cast<In*>(b.grad_v) + (size_t)bh * a.T * a.dv + col0;
        const uint32_t lv = (4 * g * a.dv + n) * sizeof(In);   // this lane's bytes in a 16-row tile of v
        In nr[16];     // dO of the next chunk
        f32x4 dO[4];   // and of this one
        auto fetch_o = [&](int chunk) {
            if (!live) return;
            const int c = opaque(chunk), valid = min(kDC, a.T - c * kDC);
            const In* op = Op + (size_t)c * kDC * a.dv;
            each_value(lv, fresh(a.dv * sizeof(In), c), [&](uint32_t o, int i) {   // zeros behind the end
                nr[i] = valid == kDC || 16 * (i / 4) + 4 * g + i % 4 < valid ? *lane_at(op, o) : In{};
            });
        };
        // T of chunk c, whose P and scalars are in LDS; its dO becomes the current one
        auto form_t = [&](int c) {
            if (!live) return;
            const float* sc = L.sc[c & 1];
            f32x4 B[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 qi = row4(sc + kQi, i, g);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    dO[i][r] = to_f32(nr[4 * i + r]);
                    B[i][r] = dO[i][r] * qi[r];
                }
            }
            f16x8 Bh[2], Bl[2];
            const int eb = column_exp(B);
            // bf16 gradients are exact in the hi part
            if constexpr (NP == 2) column_split(B, eb, Bh, Bl);
            else column_hi(B, eb, Bh);
            f32x4 t[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                f16x8 ph[4], pl[4];
#pragma unroll
                for (int i = 0; i < 2 * j + 2; ++i) {
                    ph[i] = compact_col_operand(L.P, i, j, n, g);
                    pl[i] = compact_col_operand(L.P + kCPlane, i, j, n, g);
                }
#pragma unroll
                for (int i = 0; i < 2 * j + 2; ++i) i / 2 < j ? mfma_acc(t[i], pl[i], Bh[j]) : mfma_first(t[i], pl[i], Bh[j]);
                if constexpr (NP == 2)
#pragma unroll
                    for (int i = 0; i < 2 * j + 2; ++i) mfma_acc(t[i], ph[i], Bl[j]);
#pragma unroll
                for (int i = 0; i < 2 * j + 2; ++i) mfma_acc(t[i], ph[i], Bh[j]);
            }
            mfma_done(t);
            const float ip = sc[kPi] * pow2(-eb);
#pragma unroll
            for (int i = 0; i < 4; ++i) L.T[w][i][lane] = t[i] * ip;
        };
        auto form_n = [&](int c) {
            if (!live) return;
            const float* sc = L.sc[c & 1];
            f32x4 B[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) B[i] = dO[i] * row4(sc + kGq, i, g);
            f16x8 Bh[2], Bl[2];
            const int eb = column_exp(B);
            column_split(B, eb, Bh, Bl);
            f32x4 t[NS];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                f16x8 qh[NS];
#pragma unroll
                for (int m = 0; m < NS; ++m) qh[m] = col_operand(L.Q[0], KW, m, j, n, g);
#pragma unroll
                for (int m = 0; m < NS; ++m) j ? mfma_acc(t[m], qh[m], Bl[j]) : mfma_first(t[m], qh[m], Bl[j]);
                if constexpr (NP == 2)
#pragma unroll
                    for (int m = 0; m < NS; ++m) mfma_acc(t[m], col_operand(L.Q[NP - 1], KW, m, j, n, g), Bh[j]);
#pragma unroll
                for (int m = 0; m < NS; ++m) mfma_acc(t[m], qh[m], Bh[j]);
                __builtin_amdgcn_sched_barrier(0);   // the next operands are not read ahead: registers
            }
            mfma_done(t);
            const float ib = pow2(-eb);
#pragma unroll
            for (int m = 0; m < NS; ++m) {
                t[m] *= ib;
                L.N[w][m][lane] = t[m];
            }
            const float nmax = column_max(t);
            L.ne[w][lane] = add_exp_cap(nmax, h2_exp(nmax), 0, 1.f);
        };
        auto values_out = [&](int c) {
            if (!live) return;
            const int valid = min(kDC, a.T - c * kDC);
            float* rp = b.dR + ((size_t)bh * a.nc + c) * kDC * a.dv + col0;
            In* vp = Vp + (size_t)c * kDC * a.dv;
            const uint32_t lo = lane / 4 * a.dv + lane % 4 * 4, pitch = fresh(16 * a.dv, c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 v = tile_row(L.dV[w], i, lane);
                store4(lane_at(rp, 4 * (lo + i * pitch)), v);
                if (16 * i + lane / 4 < valid) store4(lane_at(vp, (uint32_t)sizeof(In) * (lo + i * pitch)), v);
            }
        };
        fetch_o(a.nc - 1);
        __syncthreads();
        form_t(a.nc - 1);
        if (a.nc > 1) fetch_o(a.nc - 2);
        for (int chunk = a.nc - 1; chunk >= 0; --chunk) {
            const int c = opaque(chunk);
            __syncthreads();
            form_n(c);
            if (chunk + 1 < a.nc) values_out(c + 1);
            __syncthreads();
            if (chunk > 0) {
                form_t(c - 1);
                if (chunk > 1) fetch_o(chunk - 2);
            }
        }
        __syncthreads();
        values_out(0);
    } else {
        // ---------------- staging ----------------
        const int tid = threadIdx.x - 512;
        const int bk = (bh / a.H) * a.Hk + (bh % a.H) / (a.H / a.Hk);
        const In* Kp = static_cast<const In*>(a.k) + (size_t)bk * a.T * a.dk;
        const In* Qp = static_cast<const In*>(a.q) + (size_t)bk * a.T * a.dk;
        constexpr size_t image = delta_image_words(false);
        const uint16_t* img = a.img + (size_t)bh * a.nc * image;
        const float* scal = a.scal + (size_t)bh * a.nc * kScal;
        using Units = RowUnits<DKP, In>;
        using Planes = PlaneUnits<2>;
        Units kr, qr;
        Planes mr, pr;
        float ksr[Units::n], qsr[Units::n];
        f32x4 scr{0.f, 0.f, 0.f, 0.f};
        auto fetch_kq = [&](int chunk) {
            const int c = opaque(chunk), valid = min(kDC, a.T - c * kDC);
            kr.load(Kp + (size_t)c * kDC * a.dk, a.dk, valid);
            qr.load(Qp + (size_t)c * kDC * a.dk, a.dk, valid);
            const float* sc = scal + (size_t)c * kScal;
#pragma unroll
            for (int i = 0; i < Units::n; ++i) {
                ksr[i] = *lane_at(sc + kKs, 4 * Units::row(i));
                qsr[i] = *lane_at(sc + kQs, 4 * Units::row(i));
            }
        };
        auto put_kq = [&](int c) {
#pragma unroll
            for (int i = 0; i < Units::n; ++i) {
                kr.template store<NP>(L.K[c & 1], i, ksr[i]);
                qr.template store<NP>(L.Q, i, qsr[i]);
            }
        };
        auto fetch_m = [&](int chunk) { mr.load(img + opaque(chunk) * image); };
        auto fetch_p = [&](int chunk) {
            const int c = opaque(chunk);
            pr.load(img + c * image + 2 * kPlaneUnits * 8);
            if (tid < kScal / 4) scr = load4(lane_at(scal + (size_t)c * kScal, 16 * tid));
        };
        auto put = [&](uint32_t* D, const Planes& u) {
#pragma unroll
            for (int i = 0; i < Planes::n; ++i)
                if (Planes::has(i)) *reinterpret_cast<u32x4*>(compact_unit(D, tid + 256 * i)) = u.raw[i];
        };
        auto put_p = [&](int c) {
            put(L.P, pr);
            if (tid < kScal / 4) *reinterpret_cast<f32x4*>(L.sc[c & 1] + 4 * tid) = scr;
        };
        // a chunk's rows are fetched a chunk ahead of their store
        fetch_p(a.nc - 1);
        fetch_kq(a.nc - 1);
        fetch_m(a.nc - 1);
        put_p(a.nc - 1);
        if (a.nc > 1) fetch_p(a.nc - 2);
        __syncthreads();
        put_kq(a.nc - 1);
        if (a.nc > 1) fetch_kq(a.nc - 2);
        for (int chunk = a.nc - 1; chunk >= 0; --chunk) {
            const int c = opaque(chunk);
            __syncthreads();
            put(L.M, mr);
            if (chunk > 0) {
                put_p(c - 1);
                fetch_m(chunk - 1);
                if (chunk > 1) fetch_p(chunk - 2);
            }
            __syncthreads();
            if (chunk > 0) {
                put_kq(c - 1);
                if (chunk > 1) fetch_kq(chunk - 2);
            }
        }
        __syncthreads();
    }
}

template <int DKP, typename In>
__global__ __launch_bounds__(768) void delta_passes_kernel(DeltaBwdArgs b, int waves, unsigned bwd_blocks) {
    __shared__ union {
        BwdSplitLds<DKP, In> b;
        ScanSplitLds<DKP, In, false> f;
    } L;
    // the longer pass first
    if (blockIdx.x < bwd_blocks) bwd_split<DKP, In>(L.b, b, waves, blockIdx.x);
    else scan_split<DKP, In, false, true>(L.f, b.f, waves, blockIdx.x - bwd_blocks);
}

template <int DKP, typename In>
hipError_t passes_go(const DeltaBwdArgs& b, hipStream_t s) {
    const DeltaArgs& a = b.f;
    const int waves = scan_waves(a.BH * (1 + a.nseg), a.dv);
    const unsigned bwd = scan_blocks(a.BH, a.dv, waves), fwd = scan_blocks(a.BH * a.nseg, a.dv, waves);
    hipLaunchKernelGGL((delta_passes_kernel<DKP, In>), dim3(bwd + fwd), dim3(768), 0, s, b, waves, bwd);
    return hipGetLastError();
}

hipError_t launch_delta_passes_split(const DeltaBwdArgs& b, hipStream_t s) {
    if (!b.f.bf16) return b.f.dk <= 32 ? passes_go<32, float>(b, s) : passes_go<64, float>(b, s);
    return b.f.dk <= 32 ? passes_go<32, bf16_t>(b, s)
                        : b.f.dk == 64 ? passes_go<64, bf16_t>(b, s) : passes_go<128, bf16_t>(b, s);
}

}  // namespace mesa
