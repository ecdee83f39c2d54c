// ssm_core.h -- what the state space scan's chunk kernels share (gfx950).
//
// Per batch row and head (b and c of head h / (H / Hk)), with the step size D_t,
// the log decay A D_t and the state S_t (stored dk x dv here):
//   S_t = e^{A D_t} S_{t-1} + D_t b_t x_t^T,   o_t = S_t^T c_t + skip x_t.
// Over a chunk of 64 tokens with start state S, l_i the prefix sum of the chunk's
// log decays up to token i and L_ij = e^{l_i - l_j} (j <= i):
//   O = (L o (C B^T) diag(D)) X + diag(e^l) C S + skip X
//   S' = e^{l_63} S + (diag(e^{l_63 - l} D) B)^T X
//
// Rows stored as bfloat16 enter the products as they are.  What is formed in
// float32 is split into bfloat16 parts that need no scale (bfloat16 has float's
// range): two parts (2^-18 of the value) for what only feeds bfloat16 outputs,
// three (2^-27) for what feeds the state.  Rows stored as float32 go through the
// float32 matrix instruction.
//
// MFMA operands: lane 16 g + m holds row (or column) m at eight k-slots, which are
// columns 4 g .. + 3 and 16 + 4 g .. + 3 of a 32-column block.  That is also what
// two 16 x 16 accumulator tiles hold (rows 4 g .. + 3 of column m), so a product's
// result is an operand of the next without leaving its lane.
#pragma once
#include "delta_core.h"

namespace mesa {

constexpr int kSC = kSsmChunk;
static_assert(kSC == 64, "a wave's lanes are a chunk's tokens");

// The workgroup's place in an order in which neighbours share a XCD and its cache:
// workgroups go to the eight XCDs in turn.
__device__ __forceinline__ long xcd_order() {
    const unsigned n = gridDim.x, x = blockIdx.x % 8, q = n / 8, r = n % 8;
    return (long)x * q + min(x, r) + blockIdx.x / 8;
}

// The lane's number again, in a way that the compiler cannot see through: addresses
// formed from it are formed where they are used, not kept in registers over a loop.
__device__ __forceinline__ int lane_again() {
    int l = threadIdx.x % 64;
    asm volatile("" : "+v"(l));
    return l;
}

// Eight k-slots of a lane: exact, in two parts, in three.
struct F8 { float v[8]; };
struct B2 { bf16x8 h, l; };
struct B3 { bf16x8 h, m, l; };

__device__ __forceinline__ bf16x8 bf8(const float (&v)[8]) {
    bf16x8 r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = (__bf16)v[e];
    return r;
}
// v minus its bfloat16 rounding (exact)
__device__ __forceinline__ void bf8_rest(const bf16x8& h, float (&v)[8]) {
    const u32x4 w = __builtin_bit_cast(u32x4, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] -= __uint_as_float(w[i] << 16);
        v[2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ B2 split2(float (&v)[8]) {
    B2 r;
    r.h = bf8(v);
    bf8_rest(r.h, v);
    r.l = bf8(v);
    return r;
}
__device__ __forceinline__ B3 split3(float (&v)[8]) {
    B3 r;
    r.h = bf8(v);
    bf8_rest(r.h, v);
    r.m = bf8(v);
    bf8_rest(r.m, v);
    r.l = bf8(v);
    return r;
}

// Between a VALU instruction's result and a product that takes it, and between the
// products and whatever else takes their result (see delta_core.h).
__device__ __forceinline__ void mfma_ready(f32x4& c) { asm("s_nop 1" : "+v"(c)); }
__device__ __forceinline__ void mfma_done(f32x4& c) { asm("s_nop 11" : "+v"(c)); }
__device__ __forceinline__ void mfma_done(f32x4 (&c)[1]) { mfma_done(c[0]); }
__device__ __forceinline__ void mfma_done(f32x4 (&a)[1], f32x4 (&b)[1]) { asm("s_nop 11" : "+v"(a[0]), "+v"(b[0])); }
__device__ __forceinline__ void mfma_done(f32x4 (&a)[2], f32x4 (&b)[2]) {
    asm("s_nop 11" : "+v"(a[0]), "+v"(a[1]), "+v"(b[0]), "+v"(b[1]));
}
__device__ __forceinline__ void mfma_done(f32x4 (&a)[4], f32x4 (&b)[4]) {
    asm("s_nop 11" : "+v"(a[0]), "+v"(a[1]), "+v"(a[2]), "+v"(a[3]), "+v"(b[0]), "+v"(b[1]), "+v"(b[2]), "+v"(b[3]));
}
// mfma_done once x is there too: what leads to x is issued while the products run.
__device__ __forceinline__ void mfma_done_with(f32x4& c, f32x4& x) { asm("s_nop 11" : "+v"(c), "+v"(x)); }
__device__ __forceinline__ void settle(B2& x) { asm("s_nop 1" : "+v"(x.h), "+v"(x.l)); }
__device__ __forceinline__ void settle(B3& x) { asm("s_nop 1" : "+v"(x.h), "+v"(x.m), "+v"(x.l)); }
__device__ __forceinline__ void settle(F8& x) {
    asm("s_nop 1" : "+v"(x.v[0]), "+v"(x.v[1]), "+v"(x.v[2]), "+v"(x.v[3]), "+v"(x.v[4]), "+v"(x.v[5]), "+v"(x.v[6]), "+v"(x.v[7]));
}

// The products' steps over the 32 k-slots of an operand pair: one bfloat16 MFMA a part,
// or eight float32 ones.  The largest part goes first: the instruction drops the low
// bits of a small accumulator, towards minus infinity, where large products join it.
// Measured over 2^19 sums of 32 products, the mean error is -1.7e-9 of the terms with
// the small parts first, -2e-10 with the large one first and below 3e-11 with the small
// parts in an accumulator of their own; a gradient that sums a sequence's terms of
// mixed sign shows the first two (grad_A of 2x32x4096: 4e-6, 1.7e-6 and 6e-7).  So
// what the gradients sum is taken apart (mma_pair); what the forward's states take keeps
// one accumulator, whose bias is far below a float32 rounding of the state.  Both are
// added to the state outside.  The steps are written with the accumulator
// tied to its destination (delta_core.h says why and what has to stand around them).
template <typename T> inline constexpr int parts_of = 1;
template <> inline constexpr int parts_of<B2> = 2;
template <> inline constexpr int parts_of<B3> = 3;
__device__ __forceinline__ const bf16x8& part_of(const bf16x8& x, int) { return x; }
__device__ __forceinline__ const bf16x8& part_of(const B2& x, int p) { return p == 0 ? x.h : x.l; }
__device__ __forceinline__ const bf16x8& part_of(const B3& x, int p) { return p == 0 ? x.h : p == 1 ? x.m : x.l; }

template <typename A, typename B> inline constexpr int mma_steps = parts_of<A> * parts_of<B>;
template <> inline constexpr int mma_steps<F8, F8> = 8;
template <bool FIRST, typename A, typename B>
__device__ __forceinline__ void mma_step(f32x4& c, const A& a, const B& b, int s) {
    static_assert(parts_of<A> == 1 || parts_of<B> == 1, "one side is exact");
    if constexpr (FIRST) asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, 0" : "=&v"(c) : "v"(part_of(a, s)), "v"(part_of(b, s)));
    else asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+v"(c) : "v"(part_of(a, s)), "v"(part_of(b, s)));
}
template <bool FIRST>
__device__ __forceinline__ void mma_step(f32x4& c, const F8& a, const F8& b, int s) {
    if constexpr (FIRST) asm("v_mfma_f32_16x16x4_f32 %0, %1, %2, 0" : "=&v"(c) : "v"(a.v[s]), "v"(b.v[s]));
    else asm("v_mfma_f32_16x16x4_f32 %0, %1, %2, %0" : "+v"(c) : "v"(a.v[s]), "v"(b.v[s]));
}
// C[i] += a[i] b, or a b[i], the accumulators in turn; FIRST: = instead of +=.
template <bool FIRST = false, int N, typename A, typename B>
__device__ __forceinline__ void mma(f32x4 (&C)[N], const A (&a)[N], const B& b) {
#pragma unroll
    for (int s = 0; s < mma_steps<A, B>; ++s)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (FIRST && s == 0) mma_step<true>(C[i], a[i], b, s);
            else mma_step<false>(C[i], a[i], b, s);
        }
}
template <bool FIRST = false, int N, typename A, typename B>
__device__ __forceinline__ void mma(f32x4 (&C)[N], const A& a, const B (&b)[N]) {
#pragma unroll
    for (int s = 0; s < mma_steps<A, B>; ++s)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (FIRST && s == 0) mma_step<true>(C[i], a, b[i], s);
            else mma_step<false>(C[i], a, b[i], s);
        }
}
// C[i] = a0 b0[i] + a1 b1[i], ready for use, of parts: the largest and the others in
// accumulators of their own.
template <int N, typename A, typename B>
__device__ __forceinline__ void mma_pair(f32x4 (&C)[N], const A& a0, const B (&b0)[N], const A& a1, const B (&b1)[N]) {
    if constexpr (std::is_same_v<A, F8>) {
        mma<true>(C, a0, b0);
        mma(C, a1, b1);
        mfma_done(C);
    } else {
        f32x4 low[N];
#pragma unroll
        for (int s = 0; s < 2 * mma_steps<A, B>; ++s)   // step s / 2 of operand pair s % 2
#pragma unroll
            for (int i = 0; i < N; ++i) {
                f32x4& c = s < 2 ? C[i] : low[i];
                if (s == 0 || s == 2) mma_step<true>(c, a0, b0[i], s / 2);
                else mma_step<false>(c, s % 2 ? a1 : a0, s % 2 ? b1[i] : b0[i], s / 2);
            }
        mfma_done(C, low);
#pragma unroll
        for (int i = 0; i < N; ++i) C[i] += low[i];
    }
}
template <bool FIRST = false, typename A, typename B>
__device__ __forceinline__ void mma(f32x4& c, const A& a, const B& b) {
#pragma unroll
    for (int s = 0; s < mma_steps<A, B>; ++s) {
        if (FIRST && s == 0) mma_step<true>(c, a, b, s);
        else mma_step<false>(c, a, b, s);
    }
}
// Rows of a storage type in LDS and its operands.  W columns (a multiple of 32).
template <typename In, int W> struct Plane;
template <int W> struct Plane<bf16_t, W> {
    typedef bf16x8 One;
    typedef B2 Two;
    typedef B3 Three;
    static constexpr int pitch = W / 2 + 8;   // words; columns in perm32 order
    uint32_t w[kSC * pitch];
    __device__ __forceinline__ bf16x8 row(int i, int j, int m, int g) const {
        return __builtin_bit_cast(bf16x8, row_operand(w, pitch, i, j, m, g));
    }
    __device__ __forceinline__ bf16x8 col(int i, int j, int m, int g) const {
        return __builtin_bit_cast(bf16x8, col_operand(w, pitch, i, j, m, g));
    }
    // columns c .. c + 3 (c a multiple of 4) of row r
    __device__ __forceinline__ f32x4 get4(int r, int c) const {
        return load4(reinterpret_cast<const bf16_t*>(w + r * pitch + perm32(c) / 2));
    }
    __device__ __forceinline__ void put8(int r, int c, const u32x4 (&raw)[1]) {
        *reinterpret_cast<uint2*>(w + r * pitch + perm32(c) / 2) = make_uint2(raw[0][0], raw[0][1]);
        *reinterpret_cast<uint2*>(w + r * pitch + perm32(c + 4) / 2) = make_uint2(raw[0][2], raw[0][3]);
    }
    static __device__ __forceinline__ void floats(const bf16x8& x, float (&v)[8]) {
        const u32x4 u = __builtin_bit_cast(u32x4, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ B2 two(float (&v)[8]) {
        B2 r = split2(v);
        settle(r);
        return r;
    }
    static __device__ __forceinline__ B3 three(float (&v)[8]) {
        B3 r = split3(v);
        settle(r);
        return r;
    }
};
template <int W> struct Plane<float, W> {
    typedef F8 One;
    typedef F8 Two;
    typedef F8 Three;
    static constexpr int pitch = W + 4;   // floats
    float w[kSC * pitch];
    __device__ __forceinline__ F8 row(int i, int j, int m, int g) const {
        const float* p = w + (16 * i + m) * pitch + 32 * j + 4 * g;
        const f32x4 a = load4(p), b = load4(p + 16);
        return F8{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
    }
    __device__ __forceinline__ F8 col(int i, int j, int m, int g) const {
        const float* p = w + (32 * j + 4 * g) * pitch + 16 * i + m;
        F8 r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r.v[e] = p[(e % 4 + 16 * (e / 4)) * pitch];
        return r;
    }
    __device__ __forceinline__ f32x4 get4(int r, int c) const { return load4(w + r * pitch + c); }
    __device__ __forceinline__ void put8(int r, int c, const u32x4 (&raw)[2]) {
        *reinterpret_cast<u32x4*>(w + r * pitch + c) = raw[0];
        *reinterpret_cast<u32x4*>(w + r * pitch + c + 4) = raw[1];
    }
    static __device__ __forceinline__ void floats(const F8& x, float (&v)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = x.v[e];
    }
    static __device__ __forceinline__ F8 two(float (&v)[8]) {
        F8 r{{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]}};
        settle(r);
        return r;
    }
    static __device__ __forceinline__ F8 three(float (&v)[8]) { return two(v); }
};

// A 64 x 64 matrix formed in float32, lower block triangle, row r's columns as k-slots.
// For bfloat16 rows in two parts: what its products give is stored as bfloat16, and 2^-18
// of a term shows there only where terms cancel by more than about 2^9.
template <typename In> struct Square;
template <> struct Square<bf16_t> {
    Plane<bf16_t, 64> p[2];
    __device__ __forceinline__ void put4(int r, int c, const f32x4& v) {
        uint32_t* d = p[0].w + r * Plane<bf16_t, 64>::pitch + perm32(c) / 2;
        const uint32_t a = bf16_pair(v[0], v[1]), b = bf16_pair(v[2], v[3]);
        *reinterpret_cast<uint2*>(d) = make_uint2(a, b);
        d = p[1].w + r * Plane<bf16_t, 64>::pitch + perm32(c) / 2;
        *reinterpret_cast<uint2*>(d) =
            make_uint2(bf16_pair(v[0] - __uint_as_float(a << 16), v[1] - __uint_as_float(a & 0xffff0000u)),
                       bf16_pair(v[2] - __uint_as_float(b << 16), v[3] - __uint_as_float(b & 0xffff0000u)));
    }
    __device__ __forceinline__ B2 row(int i, int j, int m, int g) const { return B2{p[0].row(i, j, m, g), p[1].row(i, j, m, g)}; }
    __device__ __forceinline__ B2 col(int i, int j, int m, int g) const { return B2{p[0].col(i, j, m, g), p[1].col(i, j, m, g)}; }
};
template <> struct Square<float> {
    Plane<float, 64> p;
    __device__ __forceinline__ void put4(int r, int c, const f32x4& v) { *reinterpret_cast<f32x4*>(p.w + r * p.pitch + c) = v; }
    __device__ __forceinline__ F8 row(int i, int j, int m, int g) const { return p.row(i, j, m, g); }
    __device__ __forceinline__ F8 col(int i, int j, int m, int g) const { return p.col(i, j, m, g); }
};

// 64 rows of W columns on their way into a plane, by THREADS threads: units of eight
// columns.  The loads' bounds make zeros of rows `valid` and up and of columns
// `cols` and up, without instructions for it.
template <typename In, int W, int THREADS = 256>
struct Stage {
    static constexpr int per_row = W / 8, n = (kSC * per_row + THREADS - 1) / THREADS, parts = sizeof(In) / 2;
    uint32_t at[n];
    u32x4 raw[n][parts];
    static __device__ __forceinline__ int row(int i) { return ((int)threadIdx.x % THREADS + THREADS * i) / per_row; }
    static __device__ __forceinline__ int col(int i) { return 8 * (((int)threadIdx.x % THREADS + THREADS * i) % per_row); }
    // `pitch` (below kSsmPitch) between the rows
    __device__ __forceinline__ Stage(long pitch, int cols) {
#pragma unroll
        for (int i = 0; i < n; ++i)
            at[i] = row(i) < kSC && col(i) < cols ? ((uint32_t)row(i) * (uint32_t)pitch + col(i)) * (uint32_t)sizeof(In) : 1u << 31;
    }
    __device__ __forceinline__ void load(const In* p, long pitch, int cols, int valid) {
        const int bytes = ((valid - 1) * (int)pitch + cols) * (int)sizeof(In);
        const auto rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<In*>(p), (short)0, bytes, 0x00020000);
#pragma unroll
        for (int i = 0; i < n; ++i)
#pragma unroll
            for (int q = 0; q < parts; ++q) raw[i][q] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, at[i] + 16 * q, 0, 0));
    }
    __device__ __forceinline__ void store(Plane<In, W>& P) const {
#pragma unroll
        for (int i = 0; i < n; ++i)
            if (THREADS * (i + 1) <= kSC * per_row || row(i) < kSC) P.put8(row(i), col(i), raw[i]);
    }
};

// A chunk's scalars, by token.  Pairs (i, j) in different blocks of 16 take their
// decay as e1_i e^{block starts} e2_j, each factor at most 1; pairs in one block from
// the float64 prefix sums.
struct Scalars {
    double l[kSC];        // prefix sums of the log decays, in powers of two
    float e1[kSC];        // 2^(l_t - l before t's block)
    float e2[kSC];        // 2^(l at the block's end - l_t) D_t
    float step[kSC];      // D_t
    float in[kSC];        // 2^(l_t): from the chunk's start
    float out[kSC];       // 2^(l_63 - l_t): to its end
    float write[kSC];     // that times D_t
    float decay;          // 2^(l_63)
};

// 2^x for x <= 0, to the instruction's rounding: what is left after the nearest whole
// power is exact in float32 to 2^-26.
__device__ __forceinline__ float exp2_small(double x) {
    const double n = rint(x);
    return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f((float)(x - n)), (int)n);
}

// The step size of a raw value.
__device__ __forceinline__ float step_of(float raw, int softplus) {
    return softplus ? fmaxf(raw, 0.0f) + log1pf(expf(-fabsf(raw))) : raw;
}
// The raw value of token t, bits as stored: converted where it is used, so that the
// load is not waited for where it is issued.
__device__ __forceinline__ uint32_t step_bits(const SsmArgs& a, long b, int h, long t) {
    const long o = b * a.dts.batch + h * a.dts.head + t * a.dts.token;
    return a.dt_bf16 ? static_cast<const bf16_t*>(a.dt)[o].bits : static_cast<const uint32_t*>(a.dt)[o];
}
__device__ __forceinline__ float raw_step(const SsmArgs& a, uint32_t bits, float bias) {
    return __uint_as_float(a.dt_bf16 ? bits << 16 : bits) + bias;
}
// An element of an array that no kernel writes while this one runs, at an index that
// the wave shares: through the scalar cache, so that it does not wait behind the
// vector loads that are on their way.
__device__ __forceinline__ float shared_load(const float* p, long i) {
    return reinterpret_cast<const __attribute__((address_space(4))) float*>(reinterpret_cast<uintptr_t>(p))[i];
}
__device__ __forceinline__ float step_bias(const SsmArgs& a, int h) { return a.dt_bias ? shared_load(a.dt_bias, h) : 0.0f; }

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, true);
    return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Sum over the lanes up to one's own.
__device__ __forceinline__ double prefix_sum(double x) {
    x = dpp_add<0x111, 0xf>(x);   // row_shr 1, 2, 4, 8
    x = dpp_add<0x112, 0xf>(x);
    x = dpp_add<0x114, 0xf>(x);
    x = dpp_add<0x118, 0xf>(x);
    x = dpp_add<0x142, 0xa>(x);   // row_bcast15: rows 0 and 2 into 1 and 3
    return dpp_add<0x143, 0xc>(x);   // row_bcast31: the lower half into the upper
}

// By a whole wave, lane t for token t of the chunk (step 0 past the row's end).  The
// log decay of one token counts as at least -2^14 powers of two, which float32 has
// as 0; a NaN stays one.
__device__ __forceinline__ void chunk_scalars(Scalars& s, float step, float A) {
    const int t = threadIdx.x % 64;
    double x = (double)step * (double)A * 1.4426950408889634;
    x = prefix_sum(x < -16384.0 ? -16384.0 : x);
    const double before = __shfl(x, t < 16 ? 0 : (t & 48) - 1, 64), after = __shfl(x, t | 15, 64), end = __shfl(x, 63, 64);
    s.l[t] = x;
    s.e1[t] = exp2_small(x - (t < 16 ? 0.0 : before));
    s.e2[t] = exp2_small(after - x) * step;
    s.step[t] = step;
    s.in[t] = exp2_small(x);
    const float out = exp2_small(end - x);
    s.out[t] = out;
    s.write[t] = out * step;
    if (t == 63) s.decay = exp2_small(x);
}

// 2^(l before row block i - l at the end of row block j), j < i
__device__ __forceinline__ float block_decay(const Scalars& s, int i, int j) { return exp2_small(s.l[16 * i - 1] - s.l[16 * j + 15]); }

// The lower block triangle's tiles in order: (0,0), (1,0), (1,1), (2,0), ...
__device__ __forceinline__ constexpr int tile_i(int k) { return k < 1 ? 0 : k < 3 ? 1 : k < 6 ? 2 : 3; }
__device__ __forceinline__ constexpr int tile_j(int k) { return k - tile_i(k) * (tile_i(k) + 1) / 2; }

}  // namespace mesa
