// delta_core.h -- what the gated delta rule's chunk kernels share (gfx950).
//
// Per batch row and head (key/query head h / (H / Hk)), with the state S_t
// (dv x dk), forget gate g_t, write strength b_t, and S_t^T written S (dk x
// dv) below:
//   S_t = g_t (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T,   o_t = S_t^T q_t.
// With e_t = v_t - g_t S_{t-1}^T k_t (what the decayed state still misses of
// v_t) this is S_t = g_t S_{t-1} + b_t k_t e_t^T.  Over a chunk of 64 tokens
// with start state S, G_i the product of the chunk's gates up to token i and
// D_ij = G_i / G_j (j <= i):
//   A_ij = D_ij k_i.k_j (j < i),  P_ij = D_ij q_i.k_j (j <= i)
//   E = M (V - diag(G) K S),   M = (I + A diag(b))^-1  (unit lower triangular)
//   O = diag(G) Q S + (P diag(b)) E
//   S' = G_C S + (diag(D_C.) K)^T diag(b) E
// M and P do not depend on the state: one kernel forms them for all chunks
// at once (delta_prep.hip); the pass over the chunks (delta_scan.hip) is a
// short chain of products per chunk.
//
// Products run on fp16 MFMAs over operands scaled by powers of two and held
// as hi + lo (see cg_h2.h); rows of keys and queries stored as bf16 are exact
// in the hi part alone.
#pragma once
#include "cg_h2.h"
#include "io8.h"
#include "mesa_kernels.h"

#include <type_traits>

namespace mesa {

constexpr int kDC = kDeltaChunk;   // tokens of a chunk
constexpr int kDP = 40;     // words per LDS row of a 64 x 64 plane (fp16, columns perm32)
constexpr int kDF = 68;     // floats per LDS row of a 64 x 64 float matrix

// log2 of a gate for the chunk's double prefix sums.  A gate of 0 (a reset)
// counts as 2^-202, which is 0 in float; a NaN stays one.
__device__ __forceinline__ double log2_gate(float gate) {
    const float x = logf(gate);
    return (double)(x < -140.f ? -140.f : x) * 1.4426950408889634;
}

// Per-chunk scalars in the workspace: powers of two that scale the key and
// query rows into fp16's range, and the factors that undo row scales and apply
// the gates (64 values each, then single ones).
enum DeltaScal {
    kKs = 0,      // 2^EK_t
    kQs = 64,     // 2^EQ_t
    kGk = 128,    // G_t 2^-EK_t
    kGq = 192,    // G_t 2^-EQ_t
    kQi = 256,    // 2^-EQ_t; row t of P diag(b) is scaled by 2^(EQ_t + EP)
    kDb = 320,    // D_Ct b_t 2^-EK_t
    kGc = 384,    // G_C
    kMi = 385,    // 2^-EM, the scale of M undone
    kPi = 386,    // 2^-EP
    kScal = kDeltaScal
};

// A plane of M or P diag(b) in the workspace holds 16-byte units of eight
// columns (perm32): rows below 32 their first 32 columns, the others all 64;
// what is above stays out, being zero in blocks that no product reads.
constexpr int kPlaneUnits = kDeltaPlaneUnits;
__device__ __forceinline__ int unit_row(int u) { return u < 128 ? u / 4 : 16 + u / 8; }
__device__ __forceinline__ int unit_col(int u) { return u < 128 ? u % 4 : u % 8; }

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// p + a lane's byte offset: a scalar base and a 32-bit lane offset.
template <typename T>
__device__ __forceinline__ T* lane_at(T* p, uint32_t bytes) {
    typedef std::conditional_t<std::is_const_v<T>, const char, char> byte;
    return reinterpret_cast<T*>(reinterpret_cast<byte*>(p) + bytes);
}

// A loop counter the compiler cannot see through: addresses formed from it stay
// a scalar base and a lane's 32-bit offset, where it would otherwise keep and
// advance a 64-bit lane pointer for each of a chunk's loads and stores.
__device__ __forceinline__ int opaque(int c) {
    asm("" : "+s"(c));
    return c;
}

// A value that the compiler takes to change with c: what is formed from it is
// not kept in registers from chunk to chunk.
__device__ __forceinline__ uint32_t fresh(uint32_t x, int c) {
    asm("" : "+s"(x) : "s"(c));
    return x;
}
// The 16 values of a wave's 64 x 16 tile of rows of `pitch` bytes that a lane
// holds in accumulator order, at byte lv of the tile: f(byte offset, i) for
// value i of row 16 (i / 4) + i % 4 + 4 g.
template <typename Fn>
__device__ __forceinline__ void each_value(uint32_t lv, uint32_t pitch, Fn f) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        uint32_t o = lv + 16 * t * pitch;
#pragma unroll
        for (int r = 0; r < 4; ++r, o += pitch) f(o, 4 * t + r);
    }
}

// Eight floats, scaled by s (a power of two), rounded to fp16: one instruction each.
__device__ __forceinline__ f16x8 h2_hi_mix(const f32x4& a, const f32x4& b, float s) {
    uint32_t h0, h1, h2, h3;
    asm("v_fma_mixlo_f16 %0, %4, %5, 0\n\t"
        "v_fma_mixhi_f16 %0, %4, %6, 0\n\t"
        "v_fma_mixlo_f16 %1, %4, %7, 0\n\t"
        "v_fma_mixhi_f16 %1, %4, %8, 0\n\t"
        "v_fma_mixlo_f16 %2, %4, %9, 0\n\t"
        "v_fma_mixhi_f16 %2, %4, %10, 0\n\t"
        "v_fma_mixlo_f16 %3, %4, %11, 0\n\t"
        "v_fma_mixhi_f16 %3, %4, %12, 0\n\t"
        "s_nop 1"
        : "=&v"(h0), "=&v"(h1), "=&v"(h2), "=&v"(h3)
        : "v"(s), "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]));
    return __builtin_bit_cast(f16x8, u32x4{h0, h1, h2, h3});
}

// MFMAs with the accumulator tied to its destination, in vector registers.  The
// compiler's own choice gives many of them a separate accumulator input, which
// later instructions then overwrite while it is still read, or keeps the
// accumulators in the other register file, at a copy for every value read and
// written.  Inline asm is opaque to its hazard bookkeeping: mfma_ready() stands
// between VALU writes of the accumulators and the first MFMA on them (two wait
// states), mfma_done() between the last one and the first use of the results
// (12; 8 are asked for, 11 after the float one); codegen_check.py checks the distances in the built
// code.  Operands come from LDS or from the mix splits, which wait by themselves.
__device__ __forceinline__ void mfma_acc(f32x4& c, f16x8 a, f16x8 b) {
    asm("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
}
// four k-slots of float
__device__ __forceinline__ void mfma4_acc(f32x4& c, float a, float b) {
    asm("v_mfma_f32_16x16x4_f32 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
}
// onto zero
__device__ __forceinline__ void mfma_first(f32x4& c, f16x8 a, f16x8 b) {
    asm("v_mfma_f32_16x16x32_f16 %0, %1, %2, 0" : "=&v"(c) : "v"(a), "v"(b));
}
#define MESA_MFMA_FENCE(name, wait)                                                                                   \
    __device__ __forceinline__ void name(f32x4 (&C)[2]) { asm(wait : "+v"(C[0]), "+v"(C[1])); }                       \
    __device__ __forceinline__ void name(f32x4 (&C)[3]) { asm(wait : "+v"(C[0]), "+v"(C[1]), "+v"(C[2])); }           \
    __device__ __forceinline__ void name(f32x4 (&C)[4]) { asm(wait : "+v"(C[0]), "+v"(C[1]), "+v"(C[2]), "+v"(C[3])); } \
    __device__ __forceinline__ void name(f32x4 (&C)[8]) {                                                             \
        asm(wait : "+v"(C[0]), "+v"(C[1]), "+v"(C[2]), "+v"(C[3]), "+v"(C[4]), "+v"(C[5]), "+v"(C[6]), "+v"(C[7]));   \
    }
MESA_MFMA_FENCE(mfma_ready, "s_nop 1")
MESA_MFMA_FENCE(mfma_done, "s_nop 11")
#undef MESA_MFMA_FENCE

// Key planes: 1 where keys and queries are stored as bf16, else 2.
template <typename In> constexpr int delta_planes() { return sizeof(In) == 2 ? 1 : 2; }
constexpr int delta_row_words(int dkp) { return dkp / 2 + 8; }

// 64 rows of DKP features (dk real ones, then zeros) on their way into LDS:
// a thread holds units of eight consecutive features of one row.
template <int DKP, typename In>
struct RowUnits {
    static constexpr int per_row = DKP / 8;
    static constexpr int n = kDC * per_row / 256;
    static constexpr int words = sizeof(In) == 2 ? 4 : 8;
    u32x4 raw[n][words / 4];
    // (a workgroup of 768 threads stages with its last third)
    static __device__ __forceinline__ int row(int i) { return (threadIdx.x % 256 + 256 * i) / per_row; }
    static __device__ __forceinline__ int col(int i) { return 8 * ((threadIdx.x % 256 + 256 * i) % per_row); }
    // Rows `valid` and up repeat the last one: their gates and strengths make
    // them inert (the strength is 0), so only their finiteness matters.
    // Features dk and up are zeros.
    __device__ __forceinline__ void load(const In* p, int dk, int valid) {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const In* s = lane_at(p, ((uint32_t)min(row(i), valid - 1) * (DKP == 32 ? dk : DKP) + col(i)) * sizeof(In));
            u32x4 a{0u, 0u, 0u, 0u}, b = a;
            if (DKP > 32 || col(i) < dk) {
                a = reinterpret_cast<const u32x4*>(s)[0];
                if constexpr (words == 8) b = reinterpret_cast<const u32x4*>(s)[1];
            }
            raw[i][0] = a;
            if constexpr (words == 8) raw[i][1] = b;
        }
    }
    __device__ __forceinline__ float get(int i, int e) const {
        if constexpr (words == 8) return __uint_as_float(raw[i][e / 4][e % 4]);
        else return e % 2 ? __uint_as_float(raw[i][0][e / 2] & 0xffff0000u) : __uint_as_float(raw[i][0][e / 2] << 16);
    }
    __device__ __forceinline__ float absmax(int i) const {
        if constexpr (words == 4) {
            // bf16 magnitudes order as their bit patterns
            uint32_t m = 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
                m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m),
                                                                           __builtin_bit_cast(u16x2, raw[i][0][e] & 0x7fff7fffu)));
            }
            return __uint_as_float(max(m & 0xffff0000u, m << 16));
        } else {
            float m = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(get(i, e)));
            return m;
        }
    }
    // the largest of a row's units, in every lane that holds one of them
    static __device__ __forceinline__ float row_max(float m) {
        m = fmaxf(m, dpp_f32<0xb1>(m));
        m = fmaxf(m, dpp_f32<0x4e>(m));
        if constexpr (per_row > 4) m = fmaxf(m, dpp_f32<0x141>(m));
        if constexpr (per_row > 8) m = fmaxf(m, dpp_f32<0x140>(m));
        return m;
    }
    // into fp16 planes (hi, and lo where there are two), scaled by s
    template <int NP>
    __device__ __forceinline__ void store(uint32_t (&P)[NP][kDC * delta_row_words(DKP)], int i, float s) const {
        uint32_t* d = &P[0][row(i) * delta_row_words(DKP)];
        const int c = col(i);
        const f32x4 x{get(i, 0), get(i, 1), get(i, 2), get(i, 3)}, y{get(i, 4), get(i, 5), get(i, 6), get(i, 7)};
        f16x8 hi, lo;
        if constexpr (NP == 2) h2_split_mix(x, y, s, hi, lo);
        else hi = h2_hi_mix(x, y, s);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int w = perm32(c + 4 * half) / 2;
            *reinterpret_cast<f16x4*>(d + w) = half ? __builtin_shufflevector(hi, hi, 4, 5, 6, 7) : __builtin_shufflevector(hi, hi, 0, 1, 2, 3);
            if constexpr (NP == 2)
                *reinterpret_cast<f16x4*>(&P[1][row(i) * delta_row_words(DKP)] + w) =
                    half ? __builtin_shufflevector(lo, lo, 4, 5, 6, 7) : __builtin_shufflevector(lo, lo, 0, 1, 2, 3);
        }
    }
};

// MFMA operand of rows 16 i .. 16 i + 15 over columns 32 j .. 32 j + 31 of a
// plane of perm32 rows (lane (m, g): row 16 i + m, k-slots 4g.. of the two
// 16-column blocks).
__device__ __forceinline__ f16x8 row_operand(const uint32_t* P, int pitch, int i, int j, int m, int g) {
    return lds_f16x8(P + (16 * i + m) * pitch + 16 * j + 4 * g);
}
// The operand of the transposed plane: columns 16 i .. 16 i + 15 as rows, over
// rows 32 j .. 32 j + 31 in the same k-slot order, through transposed LDS
// reads (lane m addresses row r0 + m / 4, 4-column piece m % 4, and receives
// column m of the four rows).
__device__ __forceinline__ f16x8 col_operand(const uint32_t* P, int pitch, int i, int j, int m, int g) {
    const uint32_t* R = P + perm32(16 * i + 4 * (m & 3)) / 2 + (32 * j + 4 * g + (m >> 2)) * pitch;
    const f16x4 a = lds_tr_f16x4(R), b = lds_tr_f16x4(R + 16 * pitch);
    return f16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// The units of N planes on their way into LDS planes that follow each other.
template <int N>
struct PlaneUnits {
    static constexpr int total = N * kPlaneUnits, n = (total + 255) / 256;
    u32x4 raw[n];
    static __device__ __forceinline__ bool has(int i) { return 256 * (i + 1) <= total || threadIdx.x % 256 + 256 * i < total; }
    __device__ __forceinline__ void load(const uint16_t* img) {
#pragma unroll
        for (int i = 0; i < n; ++i)
            if (has(i)) raw[i] = *lane_at(reinterpret_cast<const u32x4*>(img), 16 * (threadIdx.x % 256 + 256 * i));
    }
    // units that hold a byte an element, the upper byte of its fp16 pattern
    __device__ __forceinline__ void load_bytes(const uint16_t* img) {
#pragma unroll
        for (int i = 0; i < n; ++i)
            if (has(i)) {
                const uint2 b = *lane_at(reinterpret_cast<const uint2*>(img), 8 * (threadIdx.x % 256 + 256 * i));
                raw[i][0] = b.x;
                raw[i][1] = b.y;
            }
    }
    __device__ __forceinline__ u32x4 from_bytes(int i) const {
        const uint32_t x = raw[i][0], y = raw[i][1];
        return u32x4{__builtin_amdgcn_perm(x, x, 0x010c000c), __builtin_amdgcn_perm(x, x, 0x030c020c),
                     __builtin_amdgcn_perm(y, y, 0x010c000c), __builtin_amdgcn_perm(y, y, 0x030c020c)};
    }
    __device__ __forceinline__ void store(uint32_t* P) const {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const int u = threadIdx.x % 256 + 256 * i, pl = u / kPlaneUnits, v = u % kPlaneUnits;
            if (has(i)) *reinterpret_cast<u32x4*>(P + (pl * kDC + unit_row(v)) * kDP + 4 * unit_col(v)) = raw[i];
        }
    }
};

// The column's operands of a block of NT accumulator tiles, scaled by 2^E and
// split in hi and lo (or hi alone).
template <int NT>
__device__ __forceinline__ float column_max(const f32x4 (&X)[NT]) { return kslot_max(absmax(X)); }
template <int NT>
__device__ __forceinline__ int column_exp(const f32x4 (&X)[NT]) { return h2_exp(column_max(X)); }

// The largest scale 2^E for what a chunk adds to a column of the state, whose
// largest magnitude is smax 2^-cs (scaled 2^es into fp16's range) before the
// chunk's gates decay it by gc: the state goes to the same scale and stays
// below 2^41 there.  Where no state is left the additions choose freely: a cap
// from an empty or a forgotten column would push small ones into fp16's
// subnormals.
constexpr int kNoCap = 1 << 16;
__device__ __forceinline__ int add_exp_cap(float smax, int es, int cs, float gc) {
    return smax > 0.f && gc > 0.f ? es + cs + 26 - __builtin_amdgcn_frexp_expf(gc) : kNoCap;
}
// X holds VALU results, or MFMA results from before the last barrier (h2_split_mix).
template <int NT>
__device__ __forceinline__ void column_split(const f32x4 (&X)[NT], int E, f16x8 (&H)[NT / 2], f16x8 (&L)[NT / 2]) {
    const float s = pow2(E);
#pragma unroll
    for (int j = 0; j < NT / 2; ++j) h2_split_mix(X[2 * j], X[2 * j + 1], s, H[j], L[j]);
}
template <int NT>
__device__ __forceinline__ void column_hi(const f32x4 (&X)[NT], int E, f16x8 (&H)[NT / 2]) {
    const float s = pow2(E);
#pragma unroll
    for (int j = 0; j < NT / 2; ++j) H[j] = h2_hi_mix(X[2 * j], X[2 * j + 1], s);
}

__device__ __forceinline__ f32x4 row4(const float* sc, int i, int g) {
    return *reinterpret_cast<const f32x4*>(sc + 16 * i + 4 * g);
}

// The same planes without the block that is never read: rows below 32 hold 32
// columns at a pitch of 24 words, the others 64 at kDP.
constexpr int kCP = 24, kCU = 32 * kCP, kCPlane = kCU + 32 * kDP;
__device__ __forceinline__ uint32_t* compact_unit(uint32_t* P, int u) {
    const int v = u % kPlaneUnits;
    return P + u / kPlaneUnits * kCPlane + (v < 128 ? v / 4 * kCP + 4 * (v % 4) : kCU + (v - 128) / 8 * kDP + 4 * (v % 8));
}
__device__ __forceinline__ f16x8 compact_row_operand(const uint32_t* P, int i, int j, int m, int g) {
    return i < 2 ? lds_f16x8(P + (16 * i + m) * kCP + 4 * g)
                 : lds_f16x8(P + kCU + (16 * (i - 2) + m) * kDP + 16 * j + 4 * g);
}
__device__ __forceinline__ f16x8 compact_col_operand(const uint32_t* P, int i, int j, int m, int g) {
    return j == 0 ? col_operand(P, kCP, i, 0, m, g) : col_operand(P + kCU, kDP, i, 0, m, g);
}

// A wave's 64 x 16 tile in accumulator order, through LDS, as row pieces: lane l
// gets columns 4 (l % 4) .. + 3 of row 16 i + l / 4.  A tile's 16 columns of a
// lane group take 17 slots, so that both sides touch every bank once.
constexpr int kTileSlots = 4 * 17;
__device__ __forceinline__ int tile_slot(int i, int n, int g) { return i * kTileSlots + g * 17 + n; }
__device__ __forceinline__ f32x4 tile_row(const f32x4* T, int i, int lane) {
    const int row = lane / 4;
    const float* p = reinterpret_cast<const float*>(T + tile_slot(i, 4 * (lane % 4), row / 4)) + row % 4;
    return f32x4{p[0], p[4], p[8], p[12]};
}
__device__ __forceinline__ void store4(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
__device__ __forceinline__ void store4(bf16_t* p, f32x4 v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
}

// Waves of a scan's workgroup that take columns: four, unless that leaves
// compute units (256 of them) idle.  A chunk takes 2.5, 2.9 and 3.5 us with one,
// two and four (bf16, dk = 128): 256 column tiles in 256 workgroups of one are
// through in 0.7 of the time of 64 workgroups of four, 1024 in 256 workgroups of
// four in 0.35 of the time of four rounds of one.
inline int scan_waves(long BH, int dv) {
    const long tiles = BH * (dv / 16);
    return tiles <= 256 ? 1 : tiles <= 512 ? 2 : 4;
}
// Its workgroups: heads in eights, one a XCD, and their column groups.
inline unsigned scan_blocks(long heads, int cols, int waves) {
    return (unsigned)((heads + 7) / 8 * 8 * ((cols + 16 * waves - 1) / (16 * waves)));
}

}  // namespace mesa
