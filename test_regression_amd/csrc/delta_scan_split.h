// delta_scan_split.h -- the gated delta rule's pass over the chunks with the
// state's chain and everything beside it on different waves (gfx950).
//
// The chain of delta_scan.hip, split over the twelve waves of a workgroup, three
// a SIMD.  Waves 0..3 each own 16 dv columns of the state and run what the
// next chunk waits for:
//   X = K S,  E = M (V - G X),  S' = G_C S + K^T (D_C b E)
// Waves 4..7 form the outputs of the chunk before, O = G Q S + (P diag(b)) E,
// from the fp16 parts of S and E that the state waves leave in LDS (in the
// backward's recomputation they write E out).  Waves 8..11 stage the chunks.
// Two barriers a chunk; between them:
//   first half    split S, X, R    Q S of chunk c - 1    M of c, K of c + 1 in
//   second half   E, update        P E, O out            Q, P of c, V of c + 1 in
// so K is held twice in LDS and everything else once.  What the output waves
// need of P and E is in their registers by the second half; O is turned around
// in LDS of its own, for which float rows leave no room (these finish O in the
// first half, in S's and E's place).
//
// S and E enter the outputs as hi + lo too, bf16 outputs among them.  With their
// hi parts and P's alone (11 bits), a bf16 output in which the terms cancel is
// off by up to 2^-11 of the terms; the second parts make the pass 234 us and not
// 215 for 8x16x4096 (dk = dv = 128), 28 and not 26 for 4x8x4096 (dk = dv = 64).
//
// With few heads the sequence is cut into segments that are passed over at once
// (delta_segments.hip): first each segment but the last from a zero state (ENDS:
// nothing but the end state is written) and, for its transition, from the dk
// unit states with no values; then all from their joined start states.
//
// A wave alone on its SIMD issues one vector instruction in 5 cycles (9 for
// the mixed-precision ones of the splits) while the SIMD could take one in
// 1.3 from several waves (measured); the pass is bound by the state waves' own
// instructions and latencies, which is why nothing else is left to them (2500 and
// 3600 cycles in a chunk's halves; matrix instructions take 28 %), and where every
// compute unit has a workgroup by the staging waves' wait for memory as well (2900
// and 3800).  8x16x4096, dk = dv = 128, bf16: 230-285 us, 3.6-4.5 us a chunk (with
// all of a column's work on one wave, delta_scan.hip's way, 358 us); with all loads
// from the caches 205.  1x16x16384 in eight segments: 151-158 us for the ends, 16 to
// join them and 118-123 for the pass; 302 us in all, 690 in one piece.
#pragma once
#include "delta_core.h"

namespace mesa {

template <int DKP, typename In, bool OUT>
struct alignas(16) ScanSplitLds {
    static constexpr int NP = delta_planes<In>(), KW = delta_row_words(DKP), NJ = DKP / 32;
    static constexpr int VW = sizeof(In) == 2 ? 8 : 20;   // words of a row of 16 values
    static constexpr int parts = OUT ? 2 * (NJ + 2) : 1;  // operands of S and of E that the outputs take
    uint32_t K[2][NP][kDC * KW];
    uint32_t M[2 * kCPlane];
    uint32_t V[4][kDC * VW];
    uint32_t Q[OUT ? NP : 1][OUT ? kDC * KW : 4];
    uint32_t P[OUT ? 2 * kCPlane : 4];
    union {
        f16x8 ex[4][parts][64];             // for the outputs (hi parts of S, then E; the same, lo)
        f32x4 E[4][4 * kTileSlots];         // for the recomputation
    };
    float is[4][64], iu[4][64];
    float sc[2][kScal];
    // where the output waves turn O around: apart for bf16 rows, so that it can
    // wait for a chunk's second half, else in their part of ex
    static constexpr bool APART = OUT && NP == 1;
    uint2 O[APART ? 4 : 1][APART ? 4 * kTileSlots : 1];
};

// The units of a chunk's rows of v (16 `waves` columns) on their way into LDS.
template <typename In>
struct ValueUnits {
    static constexpr int per = 16 / sizeof(In), n = 64 * 64 / per / 256;   // values of a unit; units a thread at most
    u32x4 raw[n];
    __device__ __forceinline__ void load(const In* p, int dv, int cols, int left, int valid, int tid) {
        const int row_units = cols / per;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const int u = tid + 256 * i, row = u / row_units, c = u % row_units * per;
            raw[i] = u32x4{0u, 0u, 0u, 0u};
            if (row < kDC && c < left) raw[i] = *reinterpret_cast<const u32x4*>(lane_at(p, ((uint32_t)min(row, valid - 1) * dv + c) * sizeof(In)));
        }
    }
    template <int W>
    __device__ __forceinline__ void store(uint32_t (&V)[4][kDC * W], int cols, int tid) const {
        const int row_units = cols / per;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const int u = tid + 256 * i, row = u / row_units, c = u % row_units * per;
            if (row < kDC) *reinterpret_cast<u32x4*>(&V[c / 16][row * W + c % 16 * sizeof(In) / 4]) = raw[i];
        }
    }
};

// The work of workgroup `block`.  OUT: write O.  SAVE: write each chunk's start
// state and E (the backward's recomputation).  Neither: the segments' ends.
template <int DKP, typename In, bool OUT, bool SAVE>
__device__ __forceinline__ void scan_split(ScanSplitLds<DKP, In, OUT>& L, const DeltaArgs& a, int waves, unsigned block) {
    using Lds = ScanSplitLds<DKP, In, OUT>;
    constexpr bool ENDS = !OUT && !SAVE;
    constexpr int NP = Lds::NP, NJ = Lds::NJ, NS = DKP / 16, KW = Lds::KW;
    const int lane = threadIdx.x % 64, w12 = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), w = w12 % 4;
    const int n = lane & 15, g = lane >> 4;
    // the column groups of a head's segment on one XCD (workgroups go to the 8 XCDs in turn)
    const int nseg = ENDS ? a.nseg - 1 : a.nseg, all_cols = ENDS ? a.dv + a.dk : a.dv;
    const int cols = 16 * waves, cgs = (all_cols + cols - 1) / cols;
    const int vh = (int)(block / (8 * cgs)) * 8 + block % 8;
    if (vh >= a.BH * nseg) return;
    const int bh = vh / nseg, seg = vh % nseg;
    const int c0 = seg * a.seg_chunks, c1 = min(a.nc, c0 + a.seg_chunks);   // its chunks
    const int colg = cols * (int)(block / 8 % cgs), col0 = colg + 16 * w;
    const bool live = w < waves && col0 < (ENDS && seg > 0 ? all_cols : a.dv);
    const size_t so = (size_t)(col0 + n) * a.dk + 4 * g;   // this lane's row of a (dv x dk) state
    if (ENDS && seg == 0 && colg >= a.dv) return;          // the first segment needs no transition
    if (w12 < 4) {
        // ---------------- the state's chain ----------------
        f32x4 S[NS];   // the state times 2^cs
        int cs = 0;
        // all segments start from their copies: the last one's end may go over state0
        const float* from = !ENDS && nseg > 1 ? a.seg_start + (size_t)vh * a.dv * a.dk
                            : seg == 0 && a.state0 ? a.state0 + (size_t)bh * a.dv * a.dk : nullptr;
#pragma unroll
        for (int m = 0; m < NS; ++m) {
            S[m] = from && live && 16 * m < a.dk ? load4(from + so + 16 * m) : f32x4{0.f, 0.f, 0.f, 0.f};
            if (ENDS && col0 >= a.dv)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[m][r] = 16 * m + 4 * g + r == col0 - a.dv + n ? 1.f : 0.f;
        }
        for (int chunk = c0; chunk < c1; ++chunk) {
            const int c = opaque(chunk);
            __syncthreads();
            const float* sc = L.sc[c & 1];
            f16x8 Sh[NJ], Sl[NJ], Bh[2], Bl[2];
            float smax = 0.f;
            int es = 0, er = 0;
            if (live) {
                if constexpr (SAVE) {
                    const float s = pow2(-cs);
                    float* sp = a.S + ((size_t)bh * a.nc + c) * a.dv * a.dk + so;
#pragma unroll
                    for (int m = 0; m < NS; ++m)
                        if (16 * m < a.dk) *reinterpret_cast<f32x4*>(sp + 16 * m) = S[m] * s;
                }
                // ---- X = K S ----
                smax = column_max(S);
                es = h2_exp(smax);
                column_split(S, es, Sh, Sl);
                f32x4 X[4];
                const auto& K = L.K[c & 1];
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
                // ---- R = V - G X ----
                const float is = pow2(-es - cs);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 gk = row4(sc + kGk, i, g);
                    f32x4 v;
                    if constexpr (sizeof(In) == 2) {
                        const f16x4 t = lds_tr_f16x4(&L.V[w][(16 * i + 4 * g + (n >> 2)) * Lds::VW + 2 * (n & 3)]);
                        const uint2 u = __builtin_bit_cast(uint2, t);
                        v = f32x4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                                  __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u)};
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r) v[r] = __uint_as_float(L.V[w][(16 * i + 4 * g + r) * Lds::VW + n]);
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) X[i][r] = v[r] - (gk[r] * is) * X[i][r];
                }
                er = column_exp(X);
                column_split(X, er, Bh, Bl);
            }
            __syncthreads();
            if (!live) continue;
            // ---- E = M R ----
            f32x4 U[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {   // row tiles 2 j and up reach column block j
                f16x8 mh[4], ml[4];
#pragma unroll
                for (int i = 2 * j; i < 4; ++i) {
                    mh[i] = compact_row_operand(L.M, i, j, n, g);
                    ml[i] = compact_row_operand(L.M + kCPlane, i, j, n, g);
                }
#pragma unroll
                for (int i = 2 * j; i < 4; ++i) j ? mfma_acc(U[i], mh[i], Bl[j]) : mfma_first(U[i], mh[i], Bl[j]);
#pragma unroll
                for (int i = 2 * j; i < 4; ++i) mfma_acc(U[i], ml[i], Bh[j]);
#pragma unroll
                for (int i = 2 * j; i < 4; ++i) mfma_acc(U[i], mh[i], Bh[j]);
            }
            if constexpr (OUT) {   // while E is on its way
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    L.ex[w][j][lane] = Sh[j];
                    L.ex[w][NJ + 2 + j][lane] = Sl[j];
                }
                L.is[w][lane] = pow2(-es - cs);
            }
            mfma_done(U);
            const float ir = sc[kMi] * pow2(-er);
#pragma unroll
            for (int i = 0; i < 4; ++i) U[i] *= ir;
            if constexpr (SAVE)
#pragma unroll
                for (int i = 0; i < 4; ++i) L.E[w][tile_slot(i, n, g)] = U[i];
            if constexpr (OUT) {
                const int eu = column_exp(U);
                f16x8 Eh[2], El[2];
                column_split(U, eu, Eh, El);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    L.ex[w][NJ + j][lane] = Eh[j];
                    L.ex[w][2 * NJ + 2 + j][lane] = El[j];
                }
                L.iu[w][lane] = sc[kPi] * pow2(-eu);
            }
            // ---- S' = G_C S + K^T (D_C b E) ----
#pragma unroll
            for (int i = 0; i < 4; ++i) U[i] *= row4(sc + kDb, i, g);
            const int ew = min(column_exp(U), add_exp_cap(smax, es, cs, sc[kGc]));
            column_split(U, ew, Bh, Bl);
            const float gs = __builtin_amdgcn_ldexpf(sc[kGc], ew - cs);
            cs = ew;
#pragma unroll
            for (int m = 0; m < NS; ++m) S[m] *= gs;
            mfma_ready(S);
            const auto& K = L.K[c & 1];
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
        float* to = ENDS ? a.seg_end + (size_t)vh * all_cols * a.dk
                         : a.final_state && seg == nseg - 1 ? a.final_state + (size_t)bh * a.dv * a.dk : nullptr;
        if (to && live) {
            const float s = pow2(-cs);
#pragma unroll
            for (int m = 0; m < NS; ++m)
                if (16 * m < a.dk) *reinterpret_cast<f32x4*>(to + so + 16 * m) = S[m] * s;
        }
        __syncthreads();
    } else if (w12 < 8) {
        // ---------------- outputs of the chunk before, or E out ----------------
        In* Op = OUT ? static_cast<In*>(a.out) + (size_t)bh * a.T * a.dv + col0 : nullptr;
        f32x4 Y[4], zs[4];   // G Q S, and the factors of P diag(b) E's rows
        f16x8 Eh[2], El[2], ph[2][4], pl[2][4];
        auto form_output = [&](int c) {
            if (!live) return;
            const float* sc = L.sc[c & 1];
            f16x8 Sh[NJ], Sl[NJ];
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                Sh[j] = L.ex[w][j][lane];
                Sl[j] = L.ex[w][NJ + 2 + j][lane];
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                Eh[j] = L.ex[w][NJ + j][lane];
                El[j] = L.ex[w][2 * NJ + 2 + j][lane];
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                f16x8 qh[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) qh[i] = row_operand(L.Q[0], KW, i, j, n, g);
#pragma unroll
                for (int i = 0; i < 4; ++i) j ? mfma_acc(Y[i], qh[i], Sl[j]) : mfma_first(Y[i], qh[i], Sl[j]);
                if constexpr (NP == 2)
#pragma unroll
                    for (int i = 0; i < 4; ++i) mfma_acc(Y[i], row_operand(L.Q[NP - 1], KW, i, j, n, g), Sh[j]);
#pragma unroll
                for (int i = 0; i < 4; ++i) mfma_acc(Y[i], qh[i], Sh[j]);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 2 * j; i < 4; ++i) {
                    ph[j][i] = compact_row_operand(L.P, i, j, n, g);
                    pl[j][i] = compact_row_operand(L.P + kCPlane, i, j, n, g);
                }
            mfma_done(Y);
            const float is = L.is[w][lane], iu = L.iu[w][lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                Y[i] *= row4(sc + kGq, i, g) * is;
                zs[i] = row4(sc + kQi, i, g) * iu;
            }
        };
        auto finish_output = [&](int c) {
            if (!live) return;
            f32x4 Z[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int i = 2 * j; i < 4; ++i) j ? mfma_acc(Z[i], ph[j][i], El[j]) : mfma_first(Z[i], ph[j][i], El[j]);
#pragma unroll
                for (int i = 2 * j; i < 4; ++i) mfma_acc(Z[i], pl[j][i], Eh[j]);
#pragma unroll
                for (int i = 2 * j; i < 4; ++i) mfma_acc(Z[i], ph[j][i], Eh[j]);
            }
            mfma_done(Z);
#pragma unroll
            for (int i = 0; i < 4; ++i) Y[i] += zs[i] * Z[i];
            const int valid = min(kDC, a.T - c * kDC);
            In* op = Op + (size_t)c * kDC * a.dv;
            const uint32_t lo = (lane / 4 * a.dv + lane % 4 * 4) * sizeof(In), pitch = fresh(16 * a.dv * sizeof(In), c);
            wave_lds_sync();
            if constexpr (sizeof(In) == 2) {
                uint2* T = L.O[w];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    T[tile_slot(i, n, g)] = make_uint2(bf16_pair(Y[i][0], Y[i][1]), bf16_pair(Y[i][2], Y[i][3]));
                wave_lds_sync();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = lane / 4;
                    const uint16_t* p = reinterpret_cast<const uint16_t*>(T + tile_slot(i, 4 * (lane % 4), row / 4)) + row % 4;
                    const uint2 v = make_uint2(p[0] | (uint32_t)p[4] << 16, p[8] | (uint32_t)p[12] << 16);
                    if (16 * i + row < valid) *reinterpret_cast<uint2*>(lane_at(op, lo + i * pitch)) = v;
                }
            } else {
                f32x4* T = reinterpret_cast<f32x4*>(L.ex[w]);   // which is read
#pragma unroll
                for (int i = 0; i < 4; ++i) T[tile_slot(i, n, g)] = Y[i];
                wave_lds_sync();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 v = tile_row(T, i, lane);
                    if (16 * i + lane / 4 < valid) store4(lane_at(op, lo + i * pitch), v);
                }
            }
        };
        auto e_out = [&](int c) {
            if (!live) return;
            float* ep = a.E + ((size_t)bh * a.nc + c) * kDC * a.dv + col0;
            const uint32_t lo = (lane / 4 * a.dv + lane % 4 * 4) * 4, pitch = fresh(16 * a.dv * 4, c);
#pragma unroll
            for (int i = 0; i < 4; ++i) store4(lane_at(ep, lo + i * pitch), tile_row(L.E[w], i, lane));
        };
        for (int chunk = c0; chunk < c1; ++chunk) {
            const int c = opaque(chunk);
            __syncthreads();
            if (chunk > c0) {
                if constexpr (OUT) form_output(c - 1);
                if constexpr (OUT && !Lds::APART) finish_output(c - 1);
                if constexpr (SAVE) e_out(c - 1);
            }
            __syncthreads();
            if constexpr (Lds::APART)
                if (chunk > c0) finish_output(c - 1);
        }
        __syncthreads();
        if constexpr (OUT) {
            form_output(c1 - 1);
            finish_output(c1 - 1);
        }
        if constexpr (SAVE) e_out(c1 - 1);
    } else {
        // ---------------- staging ----------------
        const int tid = threadIdx.x - 512;
        const int bk = (bh / a.H) * a.Hk + (bh % a.H) / (a.H / a.Hk);
        const In* Kp = static_cast<const In*>(a.k) + (size_t)bk * a.T * a.dk;
        const In* Qp = static_cast<const In*>(a.q) + (size_t)bk * a.T * a.dk;
        const In* Vp = static_cast<const In*>(a.v) + (size_t)bh * a.T * a.dv + colg;
        constexpr bool PBYTES = !SAVE && NP == 1;   // as delta_prep.hip leaves P for the forward
        constexpr size_t image = delta_image_words(PBYTES);
        const uint16_t* img = a.img + (size_t)bh * a.nc * image;
        const float* scal = a.scal + (size_t)bh * a.nc * kScal;
        using Units = RowUnits<DKP, In>;
        using MUnits = PlaneUnits<2>;
        using PUnits = PlaneUnits<1>;
        Units kr, qr;
        MUnits mr;
        PUnits pr[2];
        ValueUnits<In> vr;
        float ksr[Units::n], qsr[Units::n];
        f32x4 scr{0.f, 0.f, 0.f, 0.f};
        // K; V and scalars; M; Q and P of a chunk
        auto fetch_k = [&](int chunk) {
            const int c = opaque(chunk), valid = min(kDC, a.T - c * kDC);
            kr.load(Kp + (size_t)c * kDC * a.dk, a.dk, valid);
            const float* sc = scal + (size_t)c * kScal;
#pragma unroll
            for (int i = 0; i < Units::n; ++i) ksr[i] = *lane_at(sc + kKs, 4 * Units::row(i));
        };
        auto fetch_v = [&](int chunk) {
            const int c = opaque(chunk), valid = min(kDC, a.T - c * kDC);
            vr.load(Vp + (size_t)c * kDC * a.dv, a.dv, cols, a.dv - colg, valid, tid);
            if (tid < kScal / 4) scr = load4(lane_at(scal + (size_t)c * kScal, 16 * tid));
        };
        auto fetch_m = [&](int chunk) { mr.load(img + opaque(chunk) * image); };
        auto fetch_q = [&](int chunk) {
            const int c = opaque(chunk), valid = min(kDC, a.T - c * kDC);
            qr.load(Qp + (size_t)c * kDC * a.dk, a.dk, valid);
            const float* sc = scal + (size_t)c * kScal;
#pragma unroll
            for (int i = 0; i < Units::n; ++i) qsr[i] = *lane_at(sc + kQs, 4 * Units::row(i));
            const uint16_t* p = img + c * image + 2 * kPlaneUnits * 8;
            pr[0].load(p);
            if constexpr (PBYTES) pr[1].load_bytes(p + kPlaneUnits * 8);
            else pr[1].load(p + kPlaneUnits * 8);
        };
        auto put_k = [&](int c) {
#pragma unroll
            for (int i = 0; i < Units::n; ++i) kr.template store<NP>(L.K[c & 1], i, ksr[i]);
        };
        auto put_v = [&](int c) {
            vr.template store<Lds::VW>(L.V, cols, tid);
            if (tid < kScal / 4) *reinterpret_cast<f32x4*>(L.sc[c & 1] + 4 * tid) = scr;
        };
        // every fetch is a whole chunk ahead of its store
        fetch_k(c0);
        fetch_v(c0);
        fetch_m(c0);
        if constexpr (OUT) fetch_q(c0);
        put_k(c0);
        put_v(c0);
        if (c0 + 1 < c1) {
            fetch_k(c0 + 1);
            fetch_v(c0 + 1);
        }
        for (int chunk = c0; chunk < c1; ++chunk) {
            const int c = opaque(chunk);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < MUnits::n; ++i)
                if (MUnits::has(i)) *reinterpret_cast<u32x4*>(compact_unit(L.M, tid + 256 * i)) = mr.raw[i];
            if (chunk + 1 < c1) {
                fetch_m(chunk + 1);
                put_k(c + 1);   // over the chunk before's
                if (chunk + 2 < c1) fetch_k(chunk + 2);
            }
            __syncthreads();
            if constexpr (OUT) {
#pragma unroll
                for (int i = 0; i < Units::n; ++i) qr.template store<NP>(L.Q, i, qsr[i]);
#pragma unroll
                for (int i = 0; i < PUnits::n; ++i)
                    if (PUnits::has(i)) {
                        *reinterpret_cast<u32x4*>(compact_unit(L.P, tid + 256 * i)) = pr[0].raw[i];
                        *reinterpret_cast<u32x4*>(compact_unit(L.P, kPlaneUnits + tid + 256 * i)) = PBYTES ? pr[1].from_bytes(i) : pr[1].raw[i];
                    }
                if (chunk + 1 < c1) fetch_q(chunk + 1);
            }
            if (chunk + 1 < c1) {
                put_v(c + 1);
                if (chunk + 2 < c1) fetch_v(chunk + 2);
            }
        }
        __syncthreads();
    }
}

}  // namespace mesa
