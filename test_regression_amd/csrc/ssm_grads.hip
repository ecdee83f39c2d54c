// ssm_grads.hip -- gradients of the state space scan, per chunk (gfx950).
//
// With a chunk's start state S (dk x dv), the gradient R of its end state, the
// prefix sums l, L_ij = e^{l_i - l_j} (j <= i), D the step sizes and g the outputs'
// gradients:
//   M = g X^T,  Z = L o M diag(D),  P = L o (C B^T)
//   dC = Z B + diag(e^l) g S^T        dB = Z^T C + diag(D e^{l_63 - l}) X R^T
//   V = P^T g + diag(e^{l_63 - l}) B R,  dX = diag(D) V + skip g
// A token's log decay scales every pair (i >= t > j) of E = Z o (C B^T), what is read
// of the start state after it, what is written before it and stays to the end, and
// the start state's way to the end:
//   da_t = sum_{i >= t > j} E_ij + sum_{i >= t} rd_i + sum_{j < t} wr_j + e^{l_63} <S, R>
//   rd_i = e^{l_i} c_i . S g_i,   wr_j = D_j e^{l_63 - l_j} b_j . R x_j
// the pairs taken as prefix sums of E's column sums less its row sums, in float64.
// Then dD_t = x_t . V_t + A da_t, and the raw step size's gradient through softplus.
//
// A workgroup takes one chunk and some of the heads that share b and c, so that their
// dB and dC are summed in registers; heads of more workgroups are summed in order
// from float32 parts.  dv goes by in pieces of 64 columns, in all of which the
// formulas are sums.
//
// 2 x 32 heads of 4096 tokens that share b and c, dk 128, dv 64, bfloat16: 151 us (354
// MB fetched, of which the states 268 MB), and 90 us for the states.  A head's chunk
// takes 19,000 cycles of a workgroup that fills its CU: pairs 8,000, states 5,000 and
// their wait 2,000, dX 3,000; the VALU issues 47 % of the time (float64 decays, three-part
// splits), the matrix units 11 %.  Strides and addresses do not fit the scalar registers:
// the compiler keeps 178 to 225 of them in lanes of vector registers, and at dk 128 in
// float32 21 vector registers in scratch.  With twice the workgroups in two turns 162 us; so, and
// with wave 7's sums after dX, where the others waited for them, 182 us; with branches
// around the states' loads and the heads' scalars by vector loads, behind which the wave
// waited, 209 us.
#include <algorithm>

#include "ssm_core.h"

namespace mesa {

constexpr int kGradThreads = 512;
// Whether the next head's values, gradients and scalars have their own place to go to
// while those of this one are read: all but the widest float32 rows, which fill the LDS.
template <int N, typename In> constexpr int kGradBuffers = sizeof(In) == 4 && N == 128 ? 1 : 2;

// A state's rows of dk by 64 columns of dv, float32, or for bfloat16 rows the first two
// of its parts: only dX takes it from here, which is stored as bfloat16 (2^-18 of a term
// beside 2^-8 of the sum), and at dk 128 a third plane would not fit the LDS.
template <typename In, int N> struct StatePlane;
template <int N> struct StatePlane<bf16_t, N> {
    static constexpr int pitch = Plane<bf16_t, 64>::pitch;
    uint32_t w[2][N * pitch];
    __device__ __forceinline__ void put(int n, int g, int k, const B3 (&s)[2]) {   // columns 16 k + 4 g ..
        const u32x4 h = __builtin_bit_cast(u32x4, s[k / 2].h), l = __builtin_bit_cast(u32x4, s[k / 2].m);
        const int at = n * pitch + perm32(16 * k + 4 * g) / 2, o = 2 * (k % 2);
        *reinterpret_cast<uint2*>(&w[0][at]) = make_uint2(h[o], h[o + 1]);
        *reinterpret_cast<uint2*>(&w[1][at]) = make_uint2(l[o], l[o + 1]);
    }
    // columns 16 i + m as rows, over rows 32 j ..
    __device__ __forceinline__ B2 col(int i, int j, int m, int g) const {
        return B2{__builtin_bit_cast(bf16x8, col_operand(w[0], pitch, i, j, m, g)),
                  __builtin_bit_cast(bf16x8, col_operand(w[1], pitch, i, j, m, g))};
    }
};
template <int N> struct StatePlane<float, N> {
    static constexpr int pitch = N == 128 ? 64 : 68;   // 68 spreads the reads over the banks, and does not fit
    float w[N * pitch];
    __device__ __forceinline__ void put(int n, int g, int k, const F8 (&s)[2]) {
        const float* v = s[k / 2].v + 4 * (k % 2);
        *reinterpret_cast<f32x4*>(w + n * pitch + 16 * k + 4 * g) = f32x4{v[0], v[1], v[2], v[3]};
    }
    __device__ __forceinline__ F8 col(int i, int j, int m, int g) const {
        F8 r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r.v[e] = w[(32 * j + 4 * g + e % 4 + 16 * (e / 4)) * pitch + 16 * i + m];
        return r;
    }
};

// What the tokens' decays and step sizes take from the pairs and states of a piece.
template <int N>
struct TokenSums {
    double row[10][16], col[10][16];    // by tile: sums of E over j and of L o (C B^T) o M over i, without the diagonal
    float diag[kSC], dx[kSC];           // L o (C B^T) o M on the diagonal, M there
    float rd[N / 16][kSC], wr[N / 16][kSC];   // by 16 rows of dk
    double carry[N / 16];
};
template <int N, typename In>
struct GradLds {
    Plane<In, N> b, c;
    Plane<In, 64> x[kGradBuffers<N, In>], g[kGradBuffers<N, In>];
    Square<In> p;           // rows: the pairs' earlier token
    StatePlane<In, N> r;
    Scalars s[2 * kGradBuffers<N, In> - 1];   // of this head, the one before and the next
    TokenSums<N> sums[kGradBuffers<N, In>];   // of this piece and the one before
};

template <typename In>
__device__ __forceinline__ void zero_rows(In* p, long pitch, int cols, int from, int to) {
    for (int u = threadIdx.x; u < (to - from) * (cols / 4); u += kGradThreads)
        store4_el(p + (from + u / (cols / 4)) * pitch + 4 * (u % (cols / 4)), f32x4{0.f, 0.f, 0.f, 0.f});
}

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xf, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// The sums of four values over 16 neighbouring lanes: lane m gets that of value m % 4,
// by exchanges that halve what is left to sum.
__device__ __forceinline__ double row_sums(const double (&v)[4], int m) {
    const bool odd = m & 1, two = m & 2;
    double a = odd ? v[1] : v[0], b = odd ? v[3] : v[2];
    a += dpp_f64<0xB1>(odd ? v[0] : v[1]);      // quad_perm [1,0,3,2]
    b += dpp_f64<0xB1>(odd ? v[2] : v[3]);
    double c = two ? b : a;
    c += dpp_f64<0x4E>(two ? a : b);            // quad_perm [2,3,0,1]
    c += dpp_f64<0x124>(c);                     // row_ror 4
    return c + dpp_f64<0x128>(c);               // row_ror 8
}
__device__ __forceinline__ double kslot_sum(double v) {
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}
__device__ __forceinline__ float dot4(const f32x4& a, const f32x4& b) {
    return (a[0] * b[0] + a[1] * b[1]) + (a[2] * b[2] + a[3] * b[3]);
}
// Two pieces of a row of the chunk states as eight k-slots.
template <typename PV>
__device__ __forceinline__ typename PV::Three three8(const f32x4& a, const f32x4& b) {
    float f[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    return PV::three(f);
}

// Eight waves.  The pairs' ten tiles go round the first six, while wave 7 sums up the
// tokens' decays of the piece before and wave 6 forms the next head's scalars; a wave
// takes 16 rows of dk and N / 32 tiles of tokens for dB and dC, and leaves the rows of R
// in LDS; then it takes 16 columns of dv and two tiles of tokens for dX.  The next piece's
// rows and states are on their way from the middle of a piece to the middle of the next.
template <int N, typename In>
__global__ __launch_bounds__(kGradThreads) void ssm_grads_kernel(SsmGradArgs ga) {
    typedef Plane<In, N> PN;
    typedef Plane<In, 64> PV;
    constexpr int TT = N / 32, buffers = kGradBuffers<N, In>;
    __shared__ GradLds<N, In> S;
    const SsmArgs& a = ga.f;
    const int dk = N > 32 ? N : a.dk;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, m = lane % 16, g = lane / 16;
    long i0 = xcd_order();
    const int part = (int)(i0 % ga.parts);
    i0 /= ga.parts;
    const int chunk = (int)(i0 % a.nc);
    i0 /= a.nc;
    const int hk = (int)(i0 % a.Hk);
    const long b = i0 / a.Hk;
    const int rep = a.H / a.Hk, h_first = hk * rep + (int)((long)rep * part / ga.parts),
              h_last = hk * rep + (int)((long)rep * (part + 1) / ga.parts);
    const long t0 = (long)chunk * kSC;
    const int rows = (int)min((long)kSC, a.T - t0);
    const int len = a.lens ? min(max(a.lens[b], 0), a.T) : a.T;
    const int n = (int)min((long)rows, max(0L, len - t0));   // the chunk's tokens
    const int nt = wave % (N / 16), first = wave / (N / 16) * TT;   // the wave's rows of dk, its first tile of tokens
    const int vt = wave % 4, half = wave / 4;                       // its columns of dv, its half of the tokens
    const int cols = min(64, a.dv), pieces = (a.dv + 63) / 64;      // a piece: 64 columns of a head's dv, or all
    const int all = (h_last - h_first) * pieces;
    auto head = [&](int k) { return h_first + k / pieces; };
    auto column = [&](int k) { return 64 * (k % pieces); };

    Stage<In, 64, kGradThreads> sx(a.xs.token, cols), sg(a.dv, cols);
    f32x4 s4[4], r4[4];   // the wave's rows of S and R: row m, columns 16 k + 4 g ..
    auto fetch = [&](int k) {
        const int h = head(k), v0 = column(k);
        sx.load(static_cast<const In*>(a.x) + b * a.xs.batch + h * a.xs.head + t0 * a.xs.token + v0, a.xs.token, cols, n);
        sg.load(static_cast<const In*>(a.grad_out) + ((b * a.H + h) * a.T + t0) * a.dv + v0, a.dv, cols, n);
    };
    // 16 rows of a state [dk][dv] from a wave's first on; zeros where there are none and
    // past the columns, by the loads' bounds: a branch around a load waits for it
    auto state_rows = [&](const float* p, bool there, f32x4 (&to)[4]) {
        const int at = 16 * nt * a.dv;
        const auto rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(p + at), (short)0,
                                                          there && 16 * nt < dk ? 16 * a.dv * 4 : 0, 0x00020000);
        const uint32_t lo = (lane_again() % 16 * a.dv + 4 * (lane_again() / 16)) * 4;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            to[q] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, lo + (16 * q < cols ? 64u * q : 1u << 31), 0, 0));
    };
    auto fetch_states = [&](int k) {
        const long at = ((b * a.H + head(k)) * a.nc + chunk) * dk * a.dv + column(k);
        state_rows(a.S + at, true, s4);
        state_rows(a.R + at, true, r4);
    };
    // what the states take from their segments' starts, whose rows are read here (they
    // stay in the caches) while the pairs are formed
    const int seg[2] = {chunk / a.seg_chunks, (a.nc - 1 - chunk) / a.seg_chunks};
    auto fetch_starts = [&](int k, f32x4 (&start)[2][4]) {
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const long bh = (long)side * a.BH + b * a.H + head(k);
            state_rows(a.seg_start + (bh * a.nseg + seg[side] - 1) * dk * a.dv + column(k), seg[side] != 0, start[side]);
        }
    };
    auto add_starts = [&](int k, const f32x4 (&start)[2][4]) {
        const long at = (b * a.H + head(k)) * a.nc + chunk;
        const float ds = seg[0] ? shared_load(a.chunk_decay, at) : 0.0f;
        const float dr = seg[1] ? shared_load(a.chunk_decay, a.BH * a.nc + at) : 0.0f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            s4[q] += ds * start[0][q];
            r4[q] += dr * start[1][q];
        }
    };
    uint32_t next_raw = 0u;   // wave 6: the raw step sizes to come
    auto fetch_raw = [&](int h) {
        if (h < h_last && lane < n) next_raw = step_bits(a, b, h, t0 + lane);
    };
    auto scalars = [&](int h) {
        if (h >= h_last) return;
        chunk_scalars(S.s[h % (2 * buffers - 1)], lane < n ? step_of(raw_step(a, next_raw, step_bias(a, h)), a.softplus) : 0.f, shared_load(a.A, h));
        fetch_raw(h + 1);
    };
    auto tile_of = [&](int q) { return wave < 6 ? wave + 6 * q : 10; };   // of ten
    f32x4 cb[2], zsum[2] = {}, dc[TT] = {}, db[TT] = {};
    if (n > 0) {
        fetch(0);
        fetch_states(0);
        {
            Stage<In, N, kGradThreads> sb(a.bs.token, dk), sc(a.cs.token, dk);
            sb.load(static_cast<const In*>(a.bm) + b * a.bs.batch + hk * a.bs.head + t0 * a.bs.token, a.bs.token, dk, n);
            sc.load(static_cast<const In*>(a.cm) + b * a.cs.batch + hk * a.cs.head + t0 * a.cs.token, a.cs.token, dk, n);
            sb.store(S.b);
            sc.store(S.c);
        }
        if (wave == 6) {
            fetch_raw(h_first);
            scalars(h_first);
        }
        // what is above the pairs, where products read it: six tiles
        if (wave < 6) {
            const int j = wave < 1 ? 1 : wave < 3 ? 2 : 3, i = wave - j * (j - 1) / 2;
            S.p.put4(16 * j + m, 16 * i + 4 * g, f32x4{0.f, 0.f, 0.f, 0.f});
        }
        __syncthreads();
        // C B^T: rows of tokens 16 i + 4 g + r, columns 16 j + m
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int k = min(tile_of(q), 9), i = tile_i(k), j = tile_j(k);
            mma<true>(cb[q], S.c.row(i, 0, m, g), S.b.row(j, 0, m, g));
#pragma unroll
            for (int e = 1; e < N / 32; ++e) mma(cb[q], S.c.row(i, e, m, g), S.b.row(j, e, m, g));
            mfma_done(cb[q]);
        }
    }
    for (int h = h_first; h < h_last; ++h) {
        zero_rows(static_cast<In*>(ga.grad_x) + b * ga.gxs.batch + h * ga.gxs.head + t0 * ga.gxs.token, ga.gxs.token, a.dv, n, rows);
        if (n > 0) continue;
        if (threadIdx.x < rows) {
            const long o = b * ga.gdts.batch + h * ga.gdts.head + (t0 + threadIdx.x) * ga.gdts.token;
            if (a.dt_bf16) store1(static_cast<bf16_t*>(ga.grad_dt) + o, 0.f);
            else static_cast<float*>(ga.grad_dt)[o] = 0.f;
        }
        if (threadIdx.x < 3) ga.sums[((long)h * 3 + threadIdx.x) * a.B * a.nc + b * a.nc + chunk] = 0.0;
    }
    double direct = 0.0, da = 0.0, dskip = 0.0;   // wave 7: of token t's step size and log decay, of skip
    auto token_sums = [&](int k) {
        const int h = head(k), bi = lane / 16, at = lane % 16;
        const TokenSums<N>& U = S.sums[k % buffers];
        const Scalars& sl = S.s[h % (2 * buffers - 1)];
        double row = 0.0, col = 0.0, rdt = 0.0, wrt = 0.0, cr = 0.0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int i = min(q, bi), j = max(q, bi);
            const double r = U.row[bi * (bi + 1) / 2 + i][at], c = U.col[j * (j + 1) / 2 + bi][at];
            row += q <= bi ? r : 0.0;
            col += q >= bi ? c : 0.0;
        }
#pragma unroll
        for (int q = 0; q < N / 16; ++q) {
            if (16 * q >= dk) continue;
            rdt += U.rd[q][lane];
            wrt += U.wr[q][lane];
            cr += U.carry[q];
        }
        const float step = sl.step[lane];
        direct += col + U.diag[lane] + wrt;
        dskip += lane < n ? U.dx[lane] : 0.f;
        // before: of the tokens before t; after: of t and those that follow
        const double own = step * (col + wrt) - row, before = prefix_sum(own) - own;
        const double upto = prefix_sum(rdt), after = __shfl(upto, 63, 64) - upto + rdt;
        da += before + after + (double)sl.decay * cr;
        if ((k + 1) % pieces == 0) {
            double draw = 0.0, dA = 0.0;
            if (lane < n) {
                const double dstep = direct + (double)shared_load(a.A, h) * da;
                // the softplus' slope at a raw value is 1 - e^-step
                draw = a.softplus ? dstep * -expm1f(-step) : dstep;
                dA = step * da;
            }
            if (lane < rows) {
                const long o = b * ga.gdts.batch + h * ga.gdts.head + (t0 + lane) * ga.gdts.token;
                if (a.dt_bf16) store1(static_cast<bf16_t*>(ga.grad_dt) + o, (float)draw);
                else static_cast<float*>(ga.grad_dt)[o] = (float)draw;
            }
            const double sums[3] = {prefix_sum(dA), prefix_sum(dskip), prefix_sum(draw)};
            if (lane == 63)
#pragma unroll
                for (int q = 0; q < 3; ++q) ga.sums[((long)h * 3 + q) * a.B * a.nc + b * a.nc + chunk] = sums[q];
            direct = da = dskip = 0.0;
        }
    };
    for (int k = 0; k < (n > 0 ? all : 0); ++k) {
        const int h = head(k), v0 = column(k);
        Plane<In, 64>& X = S.x[k % buffers];
        Plane<In, 64>& G = S.g[k % buffers];
        const Scalars& sl = S.s[h % (2 * buffers - 1)];
        TokenSums<N>& U = S.sums[k % buffers];
        sx.store(X);
        sg.store(G);
        __syncthreads();
        f32x4 start[2][4];
        fetch_starts(k, start);   // loads come back in order: before the next rows, which come from further away
        if (k + 1 < all) fetch(k + 1);
        if (buffers == 2 && wave == 7 && k > 0) token_sums(k - 1);
        if (buffers == 2 && wave == 6 && (k + 1) % pieces == 0) scalars(h + 1);
        // the pairs
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int lane = lane_again(), m = lane % 16, g = lane / 16, tile = tile_of(q);
            if (tile >= 10) continue;
            const int i = tile_i(tile), j = tile_j(tile), s = 16 * j + m;
            f32x4 M;
            mma<true>(M, G.row(i, 0, m, g), X.row(j, 0, m, g));
            mma(M, G.row(i, 1, m, g), X.row(j, 1, m, g));
            const float D = sl.step[s];
            f32x4 L;   // the pairs' decays, one exponential each
            const double ls = sl.l[s];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = 16 * i + 4 * g + r;
                L[r] = i != j || s <= t ? exp2_small(sl.l[t] - ls) : 0.0f;
            }
            mfma_done(M);
            const f32x4 P = L * cb[q];
            S.p.put4(s, 16 * i + 4 * g, P);
            zsum[q] += L * M * D;
            f32x4 F = P * M;
            if (i == j) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (s == 16 * i + 4 * g + r) {
                        U.diag[s] = F[r];
                        U.dx[s] = M[r];
                        F[r] = 0.f;
                    }
            }
            // not rounded: pairs before a token are in both sums and have to leave nothing
            const double d = D, e[4] = {F[0] * d, F[1] * d, F[2] * d, F[3] * d};
            const double col = kslot_sum(((double)F[0] + F[1]) + ((double)F[2] + F[3])), row = row_sums(e, m);
            if (g == 0) U.col[tile][m] = col;
            if (m < 4) U.row[tile][4 * g + m] = row;
        }
        // dC and dB of the states, transposed: rows of dk, columns of tokens
        if (16 * nt < dk) {
            const int lane = lane_again(), m = lane % 16, g = lane / 16;
            add_starts(k, start);
            __builtin_amdgcn_sched_barrier(0);   // the starts' registers are free from here on
            double carry = 0.0;
#pragma unroll
            for (int q = 0; q < 4; ++q) carry += dot4(s4[q], r4[q]);
            f32x4 o[TT];
            typename PV::One x0[TT], x1[TT];
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                x0[t] = G.row(first + t, 0, m, g);
                x1[t] = G.row(first + t, 1, m, g);
            }
            mma_pair(o, three8<PV>(s4[0], s4[1]), x0, three8<PV>(s4[2], s4[3]), x1);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const int s = 16 * (first + t) + m;
                o[t] *= sl.in[s];
                const float rd = kslot_sum(dot4(o[t], S.c.get4(s, 16 * nt + 4 * g)));
                if (g == 0) U.rd[nt][s] = rd;
                dc[t] += o[t];
                x0[t] = X.row(first + t, 0, m, g);
                x1[t] = X.row(first + t, 1, m, g);
            }
            const typename PV::Three r3[2] = {three8<PV>(r4[0], r4[1]), three8<PV>(r4[2], r4[3])};
            mma_pair(o, r3[0], x0, r3[1], x1);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const int s = 16 * (first + t) + m;
                o[t] *= sl.out[s];
                const float wr = kslot_sum(dot4(o[t], S.b.get4(s, 16 * nt + 4 * g)));
                if (g == 0) U.wr[nt][s] = wr;
                db[t] += o[t] * sl.step[s];
            }
            if (first == 0) {
#pragma unroll
                for (int q = 0; q < 4; ++q) S.r.put(16 * nt + m, g, q, r3);
                carry = prefix_sum(carry);
                if (lane == 63) U.carry[nt] = carry;
            }
        } else if (first == 0) {
            // dk = 16: zeros for the rows that are not there
            const typename PV::Three zero[2] = {};
#pragma unroll
            for (int q = 0; q < 4; ++q) S.r.put(16 * nt + m, g, q, zero);
        }
        if (k + 1 < all) fetch_states(k + 1);
        __syncthreads();
        // dX, transposed: rows of dv, columns of tokens
        if (16 * vt < cols) {
            const int lane = lane_again(), m = lane % 16, g = lane / 16;
            f32x4 o[2];
#pragma unroll
            for (int q = 0; q < N / 32; ++q) {
                const typename PN::One br[2] = {S.b.row(2 * half, q, m, g), S.b.row(2 * half + 1, q, m, g)};
                if (q == 0) mma<true>(o, S.r.col(vt, q, m, g), br);
                else mma(o, S.r.col(vt, q, m, g), br);
            }
            mfma_done(o);
#pragma unroll
            for (int j = 0; j < 2; ++j) o[j] *= sl.out[16 * (2 * half + j) + m];
            mfma_ready(o);
            mma(o, G.col(vt, 1, m, g), {S.p.row(2 * half, 1, m, g), S.p.row(2 * half + 1, 1, m, g)});
            mma(o, G.col(vt, 0, m, g), {S.p.row(2 * half, 0, m, g), S.p.row(2 * half + 1, 0, m, g)});
            mfma_done(o);
            const float skip = a.D ? shared_load(a.D, h) : 0.0f;
            In* gx = static_cast<In*>(ga.grad_x) + b * ga.gxs.batch + h * ga.gxs.head + t0 * ga.gxs.token + v0 + 16 * vt + 4 * g;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int s = 16 * (2 * half + j) + m;
                if (s < n) store4_el(gx + s * ga.gxs.token, o[j] * sl.step[s] + skip * G.get4(s, 16 * vt + 4 * g));
            }
        }
        if (buffers == 1) {
            if (wave == 7) token_sums(k);
            __syncthreads();
            if (wave == 6 && (k + 1) % pieces == 0) scalars(h + 1);
        }
    }
    if (buffers == 2 && wave == 7 && n > 0) token_sums(all - 1);
    // the pairs' dC and dB over the heads' sum of Z
    if (n > 0) {
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (tile_of(q) < 10) S.p.put4(16 * tile_j(tile_of(q)) + m, 16 * tile_i(tile_of(q)) + 4 * g, zsum[q]);
        __syncthreads();
    }
    if (16 * nt >= dk) return;
    if (n > 0) {
        const typename PN::One b0 = S.b.col(nt, 0, m, g), b1 = S.b.col(nt, 1, m, g);
        const typename PN::One c0 = S.c.col(nt, 0, m, g), c1 = S.c.col(nt, 1, m, g);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const int at = first + t;
            mfma_ready(dc[t]);
            mfma_ready(db[t]);
            mma(dc[t], b0, S.p.col(at, 0, m, g));
            mma(db[t], c1, S.p.row(at, 1, m, g));
            mma(dc[t], b1, S.p.col(at, 1, m, g));
            mma(db[t], c0, S.p.row(at, 0, m, g));
            mfma_done(dc[t]);
            mfma_done(db[t]);
        }
    }
    float* pc = ga.part ? ga.part + ((long)part * a.B * a.Hk + b * a.Hk + hk) * 2 * a.T * dk : nullptr;
    In* gc = static_cast<In*>(ga.grad_c) + b * ga.gcs.batch + hk * ga.gcs.head;
    In* gb = static_cast<In*>(ga.grad_b) + b * ga.gbs.batch + hk * ga.gbs.head;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const int s = 16 * (first + t) + m;
        if (s >= rows) continue;
        const f32x4 zero{0.f, 0.f, 0.f, 0.f}, vc = s < n ? dc[t] : zero, vb = s < n ? db[t] : zero;
        if (pc) {
            store4(pc + (t0 + s) * dk + 16 * nt + 4 * g, vc);
            store4(pc + (a.T + t0 + s) * dk + 16 * nt + 4 * g, vb);
        } else {
            store4_el(gc + (t0 + s) * ga.gcs.token + 16 * nt + 4 * g, vc);
            store4_el(gb + (t0 + s) * ga.gbs.token + 16 * nt + 4 * g, vb);
        }
    }
}

// dC and dB over the parts of a group's heads, four features a thread.
template <typename In>
__global__ __launch_bounds__(256) void ssm_head_sums_kernel(SsmGradArgs ga) {
    const SsmArgs& a = ga.f;
    const long per = (long)a.T * a.dk / 4, groups = (long)a.B * a.Hk, i = (long)blockIdx.x * 256 + threadIdx.x;
    if (i >= groups * 2 * per) return;
    f32x4 s{};
    for (int p = 0; p < ga.parts; ++p) s += load4(ga.part + (p * groups * 2 * per + i) * 4);
    const long grp = i / (2 * per), r = i % (2 * per), e = r % per;
    const long b = grp / a.Hk, hk = grp % a.Hk, t = e / (a.dk / 4), d = e % (a.dk / 4) * 4;
    const RowStrides& st = r < per ? ga.gcs : ga.gbs;
    store4_el(static_cast<In*>(r < per ? ga.grad_c : ga.grad_b) + b * st.batch + hk * st.head + t * st.token + d, s);
}

// grad_A, grad_D and grad_dt_bias: a workgroup sums one of them for one head over the
// rows and chunks.
__global__ __launch_bounds__(256) void ssm_sums_kernel(const double* sums, long n, float* gA, float* gD, float* gbias) {
    __shared__ double red[4];
    const double* p = sums + (long)blockIdx.x * n;
    double s = 0.0;
    for (long i = threadIdx.x; i < n; i += 256) s += p[i];
#pragma unroll
    for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o, 64);
    if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = s;
    __syncthreads();
    if (threadIdx.x) return;
    float* to = blockIdx.x % 3 == 0 ? gA : blockIdx.x % 3 == 1 ? gD : gbias;
    if (to) to[blockIdx.x / 3] = (float)((red[0] + red[1]) + (red[2] + red[3]));
}

template <int N>
static void grads_go(const SsmGradArgs& a, unsigned blocks, hipStream_t s) {
    if (a.f.bf16) hipLaunchKernelGGL((ssm_grads_kernel<N, bf16_t>), dim3(blocks), dim3(kGradThreads), 0, s, a);
    else hipLaunchKernelGGL((ssm_grads_kernel<N, float>), dim3(blocks), dim3(kGradThreads), 0, s, a);
}

// Workgroups that share the heads of one b and c.  A CU takes one at a time: the fewest
// turns over the card times a turn's heads, a turn's start and end (b and c staged, their
// products, the parts) counted as one and a half heads (as measured at kSsmGradCUs).
int ssm_grad_parts(long B, int Hk, int H, int nc) {
    const long groups = B * Hk * nc, rep = H / Hk, most = std::min(rep, std::max(1L, kSsmGradMost / groups));
    long best = 1, least = 0;
    for (long n = 1; n <= most; ++n) {
        const long turns = (groups * n + kSsmGradCUs - 1) / kSsmGradCUs, cost = turns * (2 * ((rep + n - 1) / n) + 3);
        if (n == 1 || cost < least) {
            best = n;
            least = cost;
        }
    }
    return (int)best;
}

hipError_t launch_ssm_grads(const SsmGradArgs& a, hipStream_t s) {
    const unsigned blocks = (unsigned)((long)a.f.B * a.f.Hk * a.f.nc * a.parts);
    if (a.f.dk <= 32) grads_go<32>(a, blocks, s);
    else if (a.f.dk <= 64) grads_go<64>(a, blocks, s);
    else grads_go<128>(a, blocks, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.part) {
        const long n = (long)a.f.B * a.f.Hk * 2 * a.f.T * a.f.dk / 4;
        if (a.f.bf16) hipLaunchKernelGGL((ssm_head_sums_kernel<bf16_t>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a);
        else hipLaunchKernelGGL((ssm_head_sums_kernel<float>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    hipLaunchKernelGGL(ssm_sums_kernel, dim3((unsigned)(3 * a.f.H)), dim3(256), 0, s, a.sums, (long)a.f.B * a.f.nc, a.grad_A,
                       a.grad_D, a.grad_dt_bias);
    return hipGetLastError();
}

}  // namespace mesa
