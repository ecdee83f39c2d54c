// ssm_scan.hip -- the state space scan over whole sequences (gfx950): the pass over
// the chunks that writes the outputs, and the passes that only carry the state.
//
// A workgroup takes up to 64 columns of one head's dv and goes over the chunks of its
// part of the sequence; a wave keeps 16 columns of the state in accumulators.  Per
// chunk the four waves of ssm_out_kernel form the 64 x 64 matrix L o (C B^T) diag(D)
// together, through LDS, while the next chunk's rows are on their way; two workgroups
// share a CU.  16 heads of 16384 tokens, dk and dv 128, bfloat16, in 16 segments: 49 us
// for the ends, 8 us to join them, 108 us for the outputs: 3.3 us a chunk and CU, of
// which LDS works 41 %, the VALU 31 %, the matrix units 21 %: the chain from product to
// product is what it waits for.
#include <algorithm>

#include "ssm_core.h"

namespace mesa {

template <int N, typename In>
struct ScanLds {
    Plane<In, N> b, c;
    Plane<In, 64> x;
    Square<In> m;
    Scalars s[2];   // of this chunk and the next
};
template <int N, typename In>
struct CarryLds {
    Plane<In, N> b;
    Plane<In, 64> x;
    Scalars s[2];   // of this chunk and the next
};

// Where a workgroup works.
struct SsmPlace {
    long bh, b;
    int h, v0, cols, seg, valid;   // first column of dv, columns, tokens of the row
};
__device__ __forceinline__ SsmPlace ssm_place(const SsmArgs& a, long i, int nseg) {
    SsmPlace p;
    const int groups = (a.dv + 63) / 64;
    p.v0 = 64 * (int)(i % groups);
    i /= groups;
    p.seg = (int)(i % nseg);
    p.bh = i / nseg;
    p.b = p.bh / a.H;
    p.h = (int)(p.bh % a.H);
    p.cols = min(64, a.dv - p.v0);
    p.valid = a.lens ? min(max(a.lens[p.b], 0), a.T) : a.T;
    return p;
}

// Columns of rows times weights by row, in three parts: rows 32 j .. + 31.
template <typename PV>
__device__ __forceinline__ typename PV::Three weighted(const typename PV::One& x, const float* w, int j, int g) {
    float f[8];
    PV::floats(x, f);
    const f32x4 a = row4(w, 2 * j, g), b = row4(w, 2 * j + 1, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= e < 4 ? a[e] : b[e - 4];
    return PV::three(f);
}

// st = decay st + the rows' columns (transposed) times w, four tiles at a time.
// STATES, for the gradients: the states' columns lie along the lanes' rows, and the
// parts' sums are kept apart; one sum saves 32 additions a chunk.
template <int N, bool STATES, typename PN, typename W>
__device__ __forceinline__ void add_outer(f32x4 (&st)[N / 16], float decay, const PN& rows, const W& w0, const W& w1, int m, int g) {
    constexpr int H = N / 16 < 4 ? N / 16 : 4;
#pragma unroll
    for (int h = 0; h < N / 16; h += H) {
        typename PN::One k0[H], k1[H];
#pragma unroll
        for (int i = 0; i < H; ++i) {
            k0[i] = rows.col(h + i, 0, m, g);
            k1[i] = rows.col(h + i, 1, m, g);
        }
        f32x4 u[H];
        if constexpr (STATES) {
            mma_pair(u, w0, k0, w1, k1);
        } else {
            mma<true>(u, k0, w0);
            mma(u, k1, w1);
            mfma_done(u);
        }
#pragma unroll
        for (int i = 0; i < H; ++i) st[h + i] = st[h + i] * decay + u[i];
    }
}

template <int N, typename In>
__global__ __launch_bounds__(256, sizeof(In) == 2 ? 2 : 1) void ssm_out_kernel(SsmArgs a) {
    const int dk = N > 32 ? N : a.dk;
    typedef Plane<In, N> PN;
    typedef Plane<In, 64> PV;
    __shared__ ScanLds<N, In> S;
    const SsmPlace p = ssm_place(a, xcd_order(), a.nseg);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, m = lane % 16, g = lane / 16, hk = p.h / (a.H / a.Hk);
    const long first = (long)p.seg * a.seg_chunks * kSC;
    const long last = min((long)a.T, first + (long)a.seg_chunks * kSC);   // the segment's tokens
    const int chunks = first < p.valid ? (int)((min((long)p.valid, last) - first + kSC - 1) / kSC) : 0;
    const bool mine = 16 * wave < p.cols;
    const int v = p.v0 + 16 * wave;   // the wave's columns of dv
    const In* xr = static_cast<const In*>(a.x) + p.b * a.xs.batch + p.h * a.xs.head + p.v0;
    const In* br = static_cast<const In*>(a.bm) + p.b * a.bs.batch + hk * a.bs.head;
    const In* cr = static_cast<const In*>(a.cm) + p.b * a.cs.batch + hk * a.cs.head;
    const float A = a.A[p.h], skip = a.D ? a.D[p.h] : 0.0f;
    In* out = static_cast<In*>(a.out) + p.bh * a.T * a.dv + v;

    // the state's columns v + m, rows 16 i + 4 g + r
    f32x4 st[N / 16] = {};
    const float* from = a.nseg > 1 ? a.seg_start + (p.bh * a.nseg + p.seg) * a.dv * dk
                                   : a.state0 ? a.state0 + p.bh * a.dv * dk : nullptr;
    if (from && mine)
#pragma unroll
        for (int i = 0; i < N / 16; ++i)
            if (16 * i < dk) st[i] = load4(from + (long)(v + m) * dk + 16 * i + 4 * g);

    Stage<In, N> sb(a.bs.token, dk), sc(a.cs.token, dk);
    Stage<In, 64> sx(a.xs.token, p.cols);
    uint32_t raw = 0u;   // wave 3: the step sizes to come
    const float bias = step_bias(a, p.h);
    auto tokens = [&](int c) { return (int)min((long)kSC, p.valid - first - (long)c * kSC); };
    auto fetch = [&](int c) {
        const long t0 = first + (long)c * kSC;
        const int n = tokens(c);
        sb.load(br + t0 * a.bs.token, a.bs.token, dk, n);
        sc.load(cr + t0 * a.cs.token, a.cs.token, dk, n);
        sx.load(xr + t0 * a.xs.token, a.xs.token, p.cols, n);
    };
    auto fetch_raw = [&](int c) {
        if (c < chunks && lane < tokens(c)) raw = step_bits(a, p.b, p.h, first + (long)c * kSC + lane);
    };
    auto scalars = [&](int c) {
        if (c < chunks) chunk_scalars(S.s[c % 2], lane < tokens(c) ? step_of(raw_step(a, raw, bias), a.softplus) : 0.0f, A);
        fetch_raw(c + 1);
    };
    if (chunks > 0) {
        fetch(0);
        if (wave == 3) {
            fetch_raw(0);
            scalars(0);
        }
        // above the diagonal blocks, where 32 columns are read
        if (wave < 2) S.m.put4(32 * wave + m, 32 * wave + 16 + 4 * g, f32x4{0.f, 0.f, 0.f, 0.f});
    }
    for (int c = 0; c < chunks; ++c) {
        const long t0 = first + (long)c * kSC;
        sb.store(S.b);
        sc.store(S.c);
        sx.store(S.x);
        __syncthreads();
        if (c + 1 < chunks) fetch(c + 1);
        const Scalars& sl = S.s[c % 2];
        // L o (C B^T) diag(D) + skip I, tiles (i, j): lane's token m of block i, columns
        // 4 g .. of block j.  Waves 0 to 2 take the tiles below the diagonal of one j and
        // one diagonal tile, wave 3 the last one and the next chunk's scalars.
        auto tile = [&](int i, int j, const typename PN::One (&br)[N / 32]) {
            f32x4 acc;
            mma<true>(acc, br[0], S.c.row(i, 0, m, g));
#pragma unroll
            for (int q = 1; q < N / 32; ++q) mma(acc, br[q], S.c.row(i, q, m, g));
            mfma_done(acc);
            const int t = 16 * i + m;
            if (i == j) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int s = 16 * j + 4 * g + r;
                    acc[r] = s <= t ? acc[r] * sl.step[s] * exp2_small(sl.l[t] - sl.l[s]) : 0.0f;
                    if (s == t) acc[r] += skip;
                }
            } else {
                const float e = sl.e1[t] * block_decay(sl, i, j);
                const f32x4 e2 = row4(sl.e2, j, g);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[r] *= e * e2[r];
            }
            S.m.put4(t, 16 * j + 4 * g, acc);
        };
        {
            typename PN::One br[N / 32];
#pragma unroll
            for (int q = 0; q < N / 32; ++q) br[q] = S.b.row(wave, q, m, g);
            for (int i = wave; i < 4; ++i) {
                if (wave == 0 && i == 0) continue;
                tile(i, wave, br);
            }
            if (wave == 2) {
#pragma unroll
                for (int q = 0; q < N / 32; ++q) br[q] = S.b.row(0, q, m, g);
                tile(0, 0, br);
            }
        }
        if (wave == 3) scalars(c + 1);
        // diag(e^l) C S, transposed: rows of dv, columns of tokens
        f32x4 o[4];
        if (mine) {
#pragma unroll
            for (int q = 0; q < N / 32; ++q) {
                float f[8] = {st[2 * q][0], st[2 * q][1], st[2 * q][2], st[2 * q][3],
                              st[2 * q + 1][0], st[2 * q + 1][1], st[2 * q + 1][2], st[2 * q + 1][3]};
                const typename PN::Two s2 = PN::two(f);
                const typename PN::One cr4[4] = {S.c.row(0, q, m, g), S.c.row(1, q, m, g), S.c.row(2, q, m, g), S.c.row(3, q, m, g)};
                if (q == 0) mma<true>(o, s2, cr4);
                else mma(o, s2, cr4);
            }
            mfma_done(o);
        }
        __syncthreads();
        if (mine) {
            const typename PV::One x0 = S.x.col(wave, 0, m, g), x1 = S.x.col(wave, 1, m, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] *= sl.in[16 * i + m];
            mfma_ready(o);
            mma(o, x0, {S.m.row(0, 0, m, g), S.m.row(1, 0, m, g), S.m.row(2, 0, m, g), S.m.row(3, 0, m, g)});
            mma(o[2], x1, S.m.row(2, 1, m, g));
            mma(o[3], x1, S.m.row(3, 1, m, g));
            mfma_done(o);
            In* to = out + t0 * a.dv;
            const int n = tokens(c), rows = (int)min((long)kSC, last - t0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * i + m;
                if (n < kSC) {
                    if (t >= n) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
                    if (t >= rows) continue;
                }
                store4(lane_at(to, (t * a.dv + 4 * g) * sizeof(In)), o[i]);
            }
            // S' = e^{l_63} S + B^T diag(e^{l_63 - l} D) X
            const auto w0 = weighted<PV>(x0, sl.write, 0, g), w1 = weighted<PV>(x1, sl.write, 1, g);
            add_outer<N, false>(st, sl.decay, S.b, w0, w1, m, g);
        }
        __syncthreads();
    }
    if (!mine) return;
    // rows past the length (whole chunks of them)
    for (long t = first + (long)chunks * kSC + lane / 4; t < last; t += 16)
        store4(out + t * a.dv + 4 * (lane % 4), f32x4{0.f, 0.f, 0.f, 0.f});
    if (a.final_state && p.seg == a.nseg - 1)
#pragma unroll
        for (int i = 0; i < N / 16; ++i)
            if (16 * i < dk) store4(a.final_state + (p.bh * a.dv + v + m) * dk + 16 * i + 4 * g, st[i]);
}

// Whole sequences, where one workgroup a CU is what there is: eight waves.  Waves 0 to 3
// keep 16 columns of the state each and take the chunk's products with it; waves 4 to
// 7, on the same SIMDs, prepare the next chunk meanwhile: they bring its rows into LDS
// (and have those after it on their way) and form L o (C B^T) diag(D) + skip I.  The
// two halves of the LDS change places from chunk to chunk.  A chunk takes 3.7 us on a CU
// against 3.3 us with two workgroups of ssm_out_kernel there, but no pass for segments'
// ends comes first: 8 x 32 heads of 4096 tokens, dk 128, dv 64, bfloat16: 237 us, where
// two segments each take 67 + 208 us.  LDS works 40 % of that, the VALU 33 %, the matrix
// units 20 %: what is left are waits of the state waves' chain, product by product.
template <int N, typename In>
struct WalkLds {
    Plane<In, N> b, c;
    Plane<In, 64> x;
    Square<In> m;
};
template <int N, typename In> constexpr bool kWalks = 2 * sizeof(WalkLds<N, In>) + 8192 <= 160 * 1024;

// K tiles (ti, tj) of L o (C B^T) diag(D) + skip I at once, so that their operands'
// reads and their chains of products overlap: a lane's token m of block ti, columns
// 4 g .. of block tj.
template <int K, int N, typename In>
__device__ __forceinline__ void pair_tiles(WalkLds<N, In>& S, const Scalars& sl, const int (&ti)[K], const int (&tj)[K], float skip,
                                           int m, int g) {
    f32x4 acc[K];
#pragma unroll
    for (int q = 0; q < N / 32; ++q)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (q == 0) mma<true>(acc[k], S.b.row(tj[k], q, m, g), S.c.row(ti[k], q, m, g));
            else mma(acc[k], S.b.row(tj[k], q, m, g), S.c.row(ti[k], q, m, g));
        }
    f32x4 f[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int t = 16 * ti[k] + m;
        if (ti[k] == tj[k]) {
            const double lt = sl.l[t];
            const f32x4 d = row4(sl.step, tj[k], g);
#pragma unroll
            for (int r = 0; r < 4; ++r) f[k][r] = 4 * g + r <= m ? d[r] * exp2_small(lt - sl.l[16 * tj[k] + 4 * g + r]) : 0.0f;
        } else {
            f[k] = row4(sl.e2, tj[k], g) * (sl.e1[t] * block_decay(sl, ti[k], tj[k]));
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        mfma_done_with(acc[k], f[k]);
        f32x4 v = acc[k] * f[k];
        if (ti[k] == tj[k])
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = 4 * g + r < m ? v[r] : 4 * g + r == m ? v[r] + skip : 0.0f;
        S.m.put4(16 * ti[k] + m, 16 * tj[k] + 4 * g, v);
    }
}

template <int N, typename In>
__global__ __launch_bounds__(512) void ssm_walk_kernel(SsmArgs a) {
    typedef Plane<In, N> PN;
    typedef Plane<In, 64> PV;
    __shared__ WalkLds<N, In> lds[2];
    __shared__ Scalars scal[4];   // of the chunk passed over, the one prepared, the one after
    const int dk = N > 32 ? N : a.dk;
    const SsmPlace p = ssm_place(a, xcd_order(), 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, m = lane % 16, g = lane / 16;
    const int hk = p.h / (a.H / a.Hk);
    const int chunks = (int)(((long)p.valid + kSC - 1) / kSC);
    const bool carries = wave < 4, mine = carries && 16 * wave < p.cols;
    const int v = p.v0 + 16 * (wave % 4);   // the wave's columns of dv
    const In* xr = static_cast<const In*>(a.x) + p.b * a.xs.batch + p.h * a.xs.head + p.v0;
    const In* br = static_cast<const In*>(a.bm) + p.b * a.bs.batch + hk * a.bs.head;
    const In* cr = static_cast<const In*>(a.cm) + p.b * a.cs.batch + hk * a.cs.head;
    const float A = a.A[p.h], skip = a.D ? a.D[p.h] : 0.0f, bias = step_bias(a, p.h);
    In* out = static_cast<In*>(a.out) + p.bh * a.T * a.dv + v;

    // the state's columns v + m, rows 16 i + 4 g + r
    f32x4 st[N / 16] = {}, o[4];
    const float* from = a.state0 ? a.state0 + p.bh * a.dv * dk : nullptr;
    if (from && mine)
#pragma unroll
        for (int i = 0; i < N / 16; ++i)
            if (16 * i < dk) st[i] = load4(from + (long)(v + m) * dk + 16 * i + 4 * g);

    Stage<In, N> sb(a.bs.token, dk), sc(a.cs.token, dk);
    Stage<In, 64> sx(a.xs.token, p.cols);
    uint32_t raw = 0u;   // wave 7: the step sizes to come
    auto tokens = [&](int c) { return (int)min((long)kSC, p.valid - (long)c * kSC); };
    auto fetch = [&](int c) {
        if (c >= chunks) return;
        const long t0 = (long)c * kSC;
        const int n = tokens(c);
        sb.load(br + t0 * a.bs.token, a.bs.token, dk, n);
        sc.load(cr + t0 * a.cs.token, a.cs.token, dk, n);
        sx.load(xr + t0 * a.xs.token, a.xs.token, p.cols, n);
    };
    // diag(e^l) C S, transposed: rows of dv, columns of tokens
    auto read_state = [&](const WalkLds<N, In>& S, const Scalars& sl) {
#pragma unroll
        for (int q = 0; q < N / 32; ++q) {
            float f[8] = {st[2 * q][0], st[2 * q][1], st[2 * q][2], st[2 * q][3],
                          st[2 * q + 1][0], st[2 * q + 1][1], st[2 * q + 1][2], st[2 * q + 1][3]};
            const typename PN::Two s2 = PN::two(f);
            const typename PN::One c4[4] = {S.c.row(0, q, m, g), S.c.row(1, q, m, g), S.c.row(2, q, m, g), S.c.row(3, q, m, g)};
            if (q == 0) mma<true>(o, s2, c4);
            else mma(o, s2, c4);
        }
        mfma_done(o);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] *= sl.in[16 * i + m];
    };
    auto finish = [&](const WalkLds<N, In>& S, const Scalars& sl, int c) {
        const typename PV::One x0 = S.x.col(wave, 0, m, g), x1 = S.x.col(wave, 1, m, g);
        mfma_ready(o);
        mma(o, x0, {S.m.row(0, 0, m, g), S.m.row(1, 0, m, g), S.m.row(2, 0, m, g), S.m.row(3, 0, m, g)});
        mma(o[2], x1, S.m.row(2, 1, m, g));
        mma(o[3], x1, S.m.row(3, 1, m, g));
        mfma_done(o);
        const long t0 = (long)c * kSC;
        In* to = out + t0 * a.dv;
        const int n = tokens(c), rows = (int)min((long)kSC, a.T - t0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 16 * i + m;
            if (n < kSC) {
                if (t >= n) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (t >= rows) continue;
            }
            store4(lane_at(to, (t * a.dv + 4 * g) * sizeof(In)), o[i]);
        }
        // S' = e^{l_63} S + B^T diag(e^{l_63 - l} D) X
        const auto w0 = weighted<PV>(x0, sl.write, 0, g), w1 = weighted<PV>(x1, sl.write, 1, g);
        add_outer<N, false>(st, sl.decay, S.b, w0, w1, m, g);
    };
    // waves 4 to 6 take the tiles below the diagonal of one column block and one
    // diagonal tile, wave 7 the last one and the scalars of the chunk after
    auto pairs = [&](WalkLds<N, In>& S, int c) {
        const int w = wave - 4;
        if (w < 3) {
            const int ti[3] = {max(w, 1), w == 2 ? 3 : 2, w == 2 ? 0 : 3}, tj[3] = {w, w, w == 2 ? 0 : w};
            pair_tiles<3, N, In>(S, scal[c & 3], ti, tj, skip, m, g);
        } else {
            const int last_tile[1] = {3};
            pair_tiles<1, N, In>(S, scal[c & 3], last_tile, last_tile, skip, m, g);
        }
    };
    auto scalars = [&](int c) {
        if (c < chunks) chunk_scalars(scal[c & 3], lane < tokens(c) ? step_of(raw_step(a, raw, bias), a.softplus) : 0.0f, A);
    };
    auto fetch_raw = [&](int c) {
        if (c < chunks && lane < tokens(c)) raw = step_bits(a, p.b, p.h, (long)c * kSC + lane);
    };
    if (!carries) {
        fetch(0);
        if (wave == 7 && chunks > 0) {
            fetch_raw(0);
            scalars(0);
            fetch_raw(1);
        }
        // above the diagonal blocks, where 32 columns are read
        lds[(wave - 4) / 2].m.put4(32 * (wave % 2) + m, 32 * (wave % 2) + 16 + 4 * g, f32x4{0.f, 0.f, 0.f, 0.f});
    }
    for (int c = chunks > 0 ? -1 : 0; c < chunks; ++c) {
        WalkLds<N, In>& S = lds[(c + 1) & 1];          // being prepared: chunk c + 1
        const WalkLds<N, In>& R = lds[c & 1];          // ready: chunk c
        if (!carries) {
            if (c + 1 < chunks) {
                sb.store(S.b);
                sc.store(S.c);
                sx.store(S.x);
            }
        } else if (mine && c >= 0) {
            read_state(R, scal[c & 3]);
        }
        __syncthreads();
        if (!carries) {
            if (c + 1 < chunks) {
                fetch(c + 2);
                pairs(S, c + 1);
                if (wave == 7) {
                    scalars(c + 2);
                    fetch_raw(c + 3);
                }
            }
        } else if (mine && c >= 0) {
            finish(R, scal[c & 3], c);
        }
        __syncthreads();
    }
    if (!mine) return;
    // rows past the length (whole chunks of them)
    for (long t = (long)chunks * kSC + lane / 4; t < a.T; t += 16)
        store4(out + t * a.dv + 4 * (lane % 4), f32x4{0.f, 0.f, 0.f, 0.f});
    if (a.final_state)
#pragma unroll
        for (int i = 0; i < N / 16; ++i)
            if (16 * i < dk) store4(a.final_state + (p.bh * a.dv + v + m) * dk + 16 * i + 4 * g, st[i]);
}

// Passes that only carry a state: S' = e^{l_63} S + a sum of weighted outer products,
// of b and x from the front, or (BACK) of c and the outputs' gradients from the back:
// R' = e^{l_63} R + C^T diag(e^l) g.  A segment starts from zero (the first from the
// state or gradient that is given) and leaves its end and its decay.  STATES, for the
// gradients: also the states at every chunk's start (BACK: the gradients of its end),
// as far as they come from their segment, and the decay from the segment's start to
// there, with which the gradients add the segments' starts; these states are [dk][dv],
// a lane's rows v + 4 g + r and columns 16 i + m of dk.  Without STATES a lane holds rows
// 16 i + 4 g + r of dk, column v + m.  2 x 32 heads of 4096 tokens, dk 128, dv 64,
// bfloat16, both directions: 90 us for 268 MB of states (3 TB/s); with the segments' ends
// in a pass of their own before, 50 + 98 us.
template <int N, typename In, bool STATES, bool BACK>
__device__ __forceinline__ void ssm_carry(const SsmArgs& a, CarryLds<N, In>& S, const SsmPlace& p) {
    const int dk = N > 32 ? N : a.dk;
    typedef Plane<In, 64> PV;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, m = lane % 16, g = lane / 16;
    const int hk = p.h / (a.H / a.Hk);
    // chunks of the segment, counted from where the pass starts
    const int begin = p.seg * a.seg_chunks, end = min(a.nc, begin + a.seg_chunks), real = (p.valid + kSC - 1) / kSC;
    const bool mine = 16 * wave < p.cols;
    const int v = p.v0 + 16 * wave;
    const RowStrides& ks = BACK ? a.cs : a.bs;
    const In* kr = static_cast<const In*>(BACK ? a.cm : a.bm) + p.b * ks.batch + hk * ks.head;
    const In* xr = BACK ? static_cast<const In*>(a.grad_out) + p.bh * a.T * a.dv + p.v0
                        : static_cast<const In*>(a.x) + p.b * a.xs.batch + p.h * a.xs.head + p.v0;
    const long xt = BACK ? a.dv : a.xs.token;
    const float A = a.A[p.h];
    const long slot = (BACK ? a.BH + p.bh : p.bh) * a.nseg + p.seg;

    f32x4 st[N / 16] = {};
    const float* from = p.seg == 0 ? (BACK ? a.grad_final : a.state0) : nullptr;
    if (from && mine) {
        from += p.bh * a.dv * dk;
#pragma unroll
        for (int i = 0; i < N / 16; ++i) {
            if (16 * i >= dk) continue;
            if constexpr (!STATES) st[i] = load4(from + (long)(v + m) * dk + 16 * i + 4 * g);
            else
#pragma unroll
                for (int r = 0; r < 4; ++r) st[i][r] = from[(long)(v + 4 * g + r) * dk + 16 * i + m];
        }
    }
    // the first segment's start, from where the outputs take it: the final state may
    // take the given one's place while they are formed
    if (!STATES && p.seg == 0 && mine)
#pragma unroll
        for (int i = 0; i < N / 16; ++i)
            if (16 * i < dk) store4(a.seg_start + (slot * a.dv + v + m) * dk + 16 * i + 4 * g, st[i]);
    Stage<In, N> sb(ks.token, dk);
    Stage<In, 64> sx(xt, p.cols);
    uint32_t raw = 0u;   // wave 3: the step sizes to come
    const float bias = step_bias(a, p.h);
    const int k0 = BACK ? max(begin, a.nc - real) : begin, k1 = BACK ? end : min(end, real);
    // chunk of step k; from the back the row's empty chunks come first
    auto chunk_of = [&](int k) { return BACK ? a.nc - 1 - k : k; };
    auto tokens = [&](int k) { return (int)min((long)kSC, p.valid - (long)chunk_of(k) * kSC); };
    auto fetch = [&](int k) {
        const long t0 = (long)chunk_of(k) * kSC;
        sb.load(kr + t0 * ks.token, ks.token, dk, tokens(k));
        sx.load(xr + t0 * xt, xt, p.cols, tokens(k));
    };
    auto fetch_raw = [&](int k) {
        if (k < k1 && lane < tokens(k)) raw = step_bits(a, p.b, p.h, (long)chunk_of(k) * kSC + lane);
    };
    auto scalars = [&](int k) {
        if (k < k1) chunk_scalars(S.s[k % 2], lane < tokens(k) ? step_of(raw_step(a, raw, bias), a.softplus) : 0.0f, A);
        fetch_raw(k + 1);
    };
    if (k0 < k1) {
        fetch(k0);
        if (wave == 3) {
            fetch_raw(k0);
            scalars(k0);
        }
    }
    double total = 0.0;
    for (int k = k0; k < k1; ++k) {
        if (STATES && p.v0 == 0 && threadIdx.x == 0)
            a.chunk_decay[(BACK ? a.BH + p.bh : p.bh) * a.nc + chunk_of(k)] = exp2_small(total);
        if (STATES && mine) {
            float* to = (BACK ? a.R : a.S) + (p.bh * a.nc + chunk_of(k)) * dk * a.dv + v + 4 * g;
#pragma unroll
            for (int i = 0; i < N / 16; ++i)
                if (16 * i < dk) store4(to + (long)(16 * i + m) * a.dv, st[i]);
        }
        sb.store(S.b);
        sx.store(S.x);
        __syncthreads();
        if (k + 1 < k1) fetch(k + 1);
        const Scalars& sl = S.s[k % 2];
        total += sl.l[63];
        if (wave == 3) scalars(k + 1);
        if (mine) {
            const auto w0 = weighted<PV>(S.x.col(wave, 0, m, g), BACK ? sl.in : sl.write, 0, g);
            const auto w1 = weighted<PV>(S.x.col(wave, 1, m, g), BACK ? sl.in : sl.write, 1, g);
            add_outer<N, STATES>(st, sl.decay, S.b, w0, w1, m, g);
        }
        __syncthreads();
    }
    if (!mine) return;
    if (STATES && a.nseg == 1) {
        if (!BACK || !a.grad_state) return;
#pragma unroll
        for (int i = 0; i < N / 16; ++i)
            if (16 * i < dk)
#pragma unroll
                for (int r = 0; r < 4; ++r) a.grad_state[(p.bh * a.dv + v + 4 * g + r) * dk + 16 * i + m] = st[i][r];
        return;
    }
    if (p.v0 == 0 && threadIdx.x == 0) a.seg_decay[slot] = exp2_small(total);
    float* to = a.seg_start + (slot + (STATES ? 0 : 1)) * a.dv * dk;   // the ends' next start
#pragma unroll
    for (int i = 0; i < N / 16; ++i) {
        if (16 * i >= dk) continue;
        if constexpr (STATES) store4(to + (long)(16 * i + m) * a.dv + v + 4 * g, st[i]);
        else store4(to + (long)(v + m) * dk + 16 * i + 4 * g, st[i]);
    }
}

template <int N, typename In>
__global__ __launch_bounds__(256, 2) void ssm_ends_kernel(SsmArgs a) {
    __shared__ CarryLds<N, In> S;
    ssm_carry<N, In, false, false>(a, S, ssm_place(a, xcd_order(), a.nseg - 1));
}
// Both directions of the gradients side by side.
template <int N, typename In>
__global__ __launch_bounds__(256, 2) void ssm_states_kernel(SsmArgs a) {
    __shared__ CarryLds<N, In> S;
    const SsmPlace p = ssm_place(a, xcd_order() / 2, a.nseg);
    if (xcd_order() % 2) ssm_carry<N, In, true, true>(a, S, p);
    else ssm_carry<N, In, true, false>(a, S, p);
}

// Segments' ends, the first's being the real one, into the next segments' starts, in
// place: start_{s+1} = decay_s start_s + end_s.  Of the gradients' second direction
// (rows bh from `back` on) the last segment's end too, as the start state's gradient,
// transposed.
__global__ __launch_bounds__(256) void ssm_join_kernel(float* ends, const float* decay, long n, int dk, int dv, int nseg, long back,
                                                       float* grad_state) {
    const long i = (long)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const int per = dk * dv, at = (int)(i % per);
    const long bh = i / per;
    float* p = ends + bh * nseg * per + at;
    float s = p[0];
    for (int e = 1; e < nseg - 1; ++e) {
        s = decay[bh * nseg + e] * s + p[(long)e * per];
        p[(long)e * per] = s;
    }
    if (grad_state && bh >= back)
        grad_state[(bh - back) * per + (long)(at % dv) * dk + at / dv] = decay[bh * nseg + nseg - 1] * s + p[(nseg - 1L) * per];
}

// Workgroups from which on whole sequences leave too few CUs idle for segments to pay
// (measured per chunk and CU, dk 128, dv 64, bfloat16: 3.7 us in ssm_walk_kernel against
// 3.3 us and 1.05 us for the ends).  256 heads of 4096 tokens, whole and in two segments,
// in us, dk / dv: bfloat16 128/64 217 and 259, 64/64 181 and 198, 16/16 126 and 129; float32
// 64/64 322 and 388, 16/16 189 and 199, and 128/64, where it is ssm_out_kernel with one
// workgroup a CU both times, 688 and 826.  Of 216 heads narrow bfloat16 ones would gain
// from segments (16/16: 126 and 114), the others not (128/64: 217 and 271).
constexpr long kSsmCUs = 256, kSsmWalk = 216;
enum SsmPass { kOut, kEnds, kStates };
template <int N, typename In>
static void scan_go(const SsmArgs& a, SsmPass pass, unsigned blocks, hipStream_t s) {
    const dim3 grid(blocks), block(256);
    switch (pass) {
        case kOut:
            if constexpr (kWalks<N, In>)
                if (a.nseg == 1 && blocks <= kSsmCUs) {
                    hipLaunchKernelGGL((ssm_walk_kernel<N, In>), grid, dim3(512), 0, s, a);
                    break;
                }
            hipLaunchKernelGGL((ssm_out_kernel<N, In>), grid, block, 0, s, a);
            break;
        case kEnds: hipLaunchKernelGGL((ssm_ends_kernel<N, In>), grid, block, 0, s, a); break;
        case kStates: hipLaunchKernelGGL((ssm_states_kernel<N, In>), grid, block, 0, s, a); break;
    }
}
template <int N>
static void scan_type(const SsmArgs& a, SsmPass pass, unsigned blocks, hipStream_t s) {
    if (a.bf16) scan_go<N, bf16_t>(a, pass, blocks, s);
    else scan_go<N, float>(a, pass, blocks, s);
}
static hipError_t scan_pass(const SsmArgs& a, SsmPass pass, hipStream_t s) {
    const unsigned blocks = (unsigned)(a.BH * (pass == kEnds ? a.nseg - 1 : a.nseg) * ((a.dv + 63) / 64) * (pass == kStates ? 2 : 1));
    if (a.dk <= 32) scan_type<32>(a, pass, blocks, s);
    else if (a.dk <= 64) scan_type<64>(a, pass, blocks, s);
    else scan_type<128>(a, pass, blocks, s);
    return hipGetLastError();
}
static hipError_t join(const SsmArgs& a, int sides, float* ends, float* grad_state, hipStream_t s) {
    const long n = sides * a.BH * a.dv * a.dk;
    hipLaunchKernelGGL(ssm_join_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, ends, a.seg_decay, n, a.dk, a.dv, a.nseg,
                       a.BH, grad_state);
    return hipGetLastError();
}
hipError_t launch_ssm_scan(const SsmArgs& a, hipStream_t s) {
    hipError_t e = a.nseg > 1 ? scan_pass(a, kEnds, s) : hipSuccess;
    if (e == hipSuccess && a.nseg > 2) e = join(a, 1, a.seg_start + (long)a.dv * a.dk, nullptr, s);
    return e == hipSuccess ? scan_pass(a, kOut, s) : e;
}
hipError_t launch_ssm_states(const SsmArgs& a, hipStream_t s) {
    const hipError_t e = scan_pass(a, kStates, s);
    return e == hipSuccess && (a.nseg > 2 || (a.nseg > 1 && a.grad_state)) ? join(a, 2, a.seg_start, a.grad_state, s) : e;
}

// Segments of a sequence that are passed over at once: twice as many while the
// workgroups (of `sides` directions) stay below kSsmFill and a segment keeps kSsmLeast
// chunks; for the outputs, which need the ends first, from kSsmShort chunks on.  16
// heads of 16384 tokens, dk and dv 128, bfloat16: 166 us in 16 segments (two workgroups a
// CU), 204 us in 8.  16 heads of 1024 tokens, dk 128, dv 64, bfloat16: 58 us in one segment,
// 37 in four, 28 in eight, their gradients 59, 52 and 50 us; of 256 tokens 19 us in one,
// 23 us in two.  Of float32 rows with dk 128 one workgroup fits a CU: 64 heads of 4096
// tokens 242 us in eight segments, 250 in four; 16 heads 94 in 32, 81 in 16.
constexpr long kSsmFill = 512;
constexpr int kSsmLeast = 2, kSsmShort = 8, kSsmMost = 32;
int ssm_segments(long BH, int nc, int dv, int sides) {
    const long groups = BH * ((dv + 63) / 64) * sides;
    int n = 1;
    if (sides == 1 && ((groups >= kSsmWalk && groups <= kSsmCUs) || nc < kSsmShort)) return n;
    while (n < kSsmMost && groups * n < kSsmFill && nc >= 2 * kSsmLeast * n) n *= 2;
    return n;
}
// n segments or more are taken by up to (kSsmFill - 1) / (n / 2) groups.
long ssm_segment_slots(long BH, int nc, int dv, int sides) {
    long most = 0;
    for (int n = 2; n <= kSsmMost && nc >= kSsmLeast * n; n *= 2)
        most = std::max(most, std::min(BH, (kSsmFill - 1) / (n / 2) / ((dv + 63) / 64 * sides)) * ssm_slots(n, sides));
    return most;
}

}  // namespace mesa
