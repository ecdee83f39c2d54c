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
//   O = diag(G) Q S + P diag(b) E
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

namespace mesa {

constexpr int kDC = kDeltaChunk;   // tokens of a chunk
constexpr int kDP = 40;     // words per LDS row of a 64 x 64 plane (fp16, columns perm32)
constexpr int kDF = 68;     // floats per LDS row of a 64 x 64 float matrix

// Per-chunk scalars in the workspace, 64 each: powers of two that scale the
// key and query rows into fp16's range; the factors that undo row scales and
// apply the gates.
enum DeltaScal {
    kKs = 0,      // 2^EK_t
    kQs = 64,     // 2^EQ_t
    kGk = 128,    // G_t 2^-EK_t
    kGq = 192,    // G_t 2^-EQ_t
    kMi = 256,    // 2^-EM_t, the scale of row t of M undone
    kPi = 320,    // 2^-EP_t, of row t of P
    kDc = 384,    // D_Ct 2^-EK_t
    kBe = 448,    // b_t
    kGc = 512,    // G_C (one value)
    kScal = kDeltaScal
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Key planes: 1 where keys and queries are stored as bf16, else 2.
template <typename In> constexpr int delta_planes() { return sizeof(In) == 2 ? 1 : 2; }
constexpr int delta_row_words(int dkp) { return dkp / 2 + 8; }

// 64 rows of DKP features (dk real ones, then zeros) on their way into LDS:
// a thread holds units of eight consecutive features of one row.
template <int DKP, typename In, int THREADS = 256>
struct RowUnits {
    static constexpr int per_row = DKP / 8;
    static constexpr int n = kDC * per_row / THREADS;
    static constexpr int words = sizeof(In) == 2 ? 4 : 8;
    u32x4 raw[n][words / 4];
    static __device__ __forceinline__ int row(int i) { return (threadIdx.x + THREADS * i) / per_row; }
    static __device__ __forceinline__ int col(int i) { return 8 * ((threadIdx.x + THREADS * i) % per_row); }
    // rows `valid` and up, and features dk and up, are zeros
    __device__ __forceinline__ void load(const In* p, int dk, int valid) {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const int r = row(i), c = col(i);
            u32x4 a{0u, 0u, 0u, 0u}, b = a;
            if (r < valid && c < dk) {
                const In* s = p + (size_t)r * dk + c;
                a = *reinterpret_cast<const u32x4*>(s);
                if constexpr (words == 8) b = *reinterpret_cast<const u32x4*>(s + 4);
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
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(get(i, e)));
        return m;
    }
    // into fp16 planes (hi, and lo where there are two), scaled by s
    template <int NP>
    __device__ __forceinline__ void store(uint32_t (&P)[NP][kDC * delta_row_words(DKP)], int i, float s) const {
        uint32_t* d = &P[0][row(i) * delta_row_words(DKP)];
        const int c = col(i);
        _Float16 hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float y = get(i, e) * s;
            hi[e] = (_Float16)y;
            lo[e] = (_Float16)(y - (float)hi[e]);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int w = perm32(c + 4 * half) / 2;
            const _Float16* h = hi + 4 * half;
            *reinterpret_cast<f16x4*>(d + w) = f16x4{h[0], h[1], h[2], h[3]};
            if constexpr (NP == 2) {
                const _Float16* l = lo + 4 * half;
                *reinterpret_cast<f16x4*>(&P[1][row(i) * delta_row_words(DKP)] + w) = f16x4{l[0], l[1], l[2], l[3]};
            }
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

// 16-byte pieces of `PLANES` 64 x 64 planes on their way into LDS.
template <int PLANES>
struct PlaneUnits {
    static constexpr int n = PLANES * 2;
    u32x4 raw[n];
    __device__ __forceinline__ void load(const uint16_t* img) {
#pragma unroll
        for (int i = 0; i < n; ++i) raw[i] = reinterpret_cast<const u32x4*>(img)[threadIdx.x + 256 * i];
    }
    __device__ __forceinline__ void store(uint32_t (&P)[PLANES][kDC * kDP]) const {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const int u = threadIdx.x + 256 * i;   // plane u / 512, row (u / 8) % 64, piece u % 8
            *reinterpret_cast<u32x4*>(&P[i / 2][(u / 8 % kDC) * kDP + 4 * (u % 8)]) = raw[i];
        }
    }
};

// The column's operands of a block of NT accumulator tiles: scaled so that
// the largest magnitude lands in [2^14, 2^15), split in hi and lo; returns
// the scale's inverse.
template <int NT>
__device__ __forceinline__ float column_operands(const f32x4 (&X)[NT], f16x8 (&H)[NT / 2], f16x8 (&L)[NT / 2]) {
    const int E = h2_exp(kslot_max(absmax(X)));
    const float s = pow2(E);
#pragma unroll
    for (int j = 0; j < NT / 2; ++j) h2_split(X[2 * j], X[2 * j + 1], s, H[j], L[j]);
    return pow2(-E);
}

__device__ __forceinline__ f32x4 row4(const float* sc, int i, int g) {
    return *reinterpret_cast<const f32x4*>(sc + 16 * i + 4 * g);
}

}  // namespace mesa
