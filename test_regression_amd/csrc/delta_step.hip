// delta_step.hip -- one token of the gated delta rule, state updated in place (gfx950).
//
// Per sequence and head, with the state S (dv x dk), decay g and strength b:
//   e = b (v - g S k),   S' = g S + e k^T,   o = S' q = g S q + e (k . q)
// Row i of S only meets v_i: e_i = b (v_i - g S_i . k) and o_i = g S_i . q +
// e_i (k . q).  So each row is read once, both of its dot products are taken
// from the registers, and it is written back.
//
// HBM-bound: 8 dk dv bytes of state a head against about 7 flops for each
// 8 bytes.  Eight lanes take a row (four at dk = 16), 16-byte pieces
// interleaved over them, so that a wave's accesses are 128-byte runs and the
// row sums take three lane exchanges.  A wave takes one group of 8 or 16 rows:
// 256 sequences x 16 heads of 128 x 128 take 95 us, 5.6 TB/s; with four groups
// a wave 102 us.  One sequence of 4 heads of 64 x 64: 3 us in the kernel.
#include "io8.h"
#include "mesa_kernels.h"

namespace mesa {

template <int dk> struct StepShape {
    static constexpr int lanes = dk >= 32 ? 8 : 4;
    static constexpr int pieces = dk / (4 * lanes);
    static constexpr int rows = 64 / lanes;       // rows of a wave at a time; a head's dv is a multiple of them
};

template <int L>
__device__ __forceinline__ float step_sum(float v) {
    v += dpp<0xB1>(v);                 // lanes 1 apart
    v += dpp<0x4E>(v);                 // lanes 2 apart
    if constexpr (L == 8) v += dpp<0x141>(v);   // row_half_mirror: the other four of the eight
    return v;
}

// A wave takes one group of rows of a head.
template <int dk, typename In>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaStepArgs a) {
    using Sh = StepShape<dk>;
    const long grp = (long)blockIdx.x * 4 + threadIdx.x / 64;
    if (grp >= a.groups) return;
    const int lane = threadIdx.x % 64, li = lane % Sh::lanes, lr = lane / Sh::lanes;
    const long row0 = grp * Sh::rows;
    const long nh = row0 / a.dv;
    const long n = nh / a.H;
    const int h = (int)(nh % a.H);
    const size_t ko = ((size_t)n * a.Hk + h / (a.H / a.Hk)) * dk + 4 * li;
    f32x4 S[Sh::pieces], k[Sh::pieces], q[Sh::pieces];
    float* p = a.state + (size_t)(row0 + lr) * dk + 4 * li;
#pragma unroll
    for (int j = 0; j < Sh::pieces; ++j) S[j] = load4(p + 4 * Sh::lanes * j);
    const float ga = a.gamma[nh], be = a.beta[nh];
    const float v = to_f32(static_cast<const In*>(a.v)[row0 + lr]);
    float kq = 0.f;
#pragma unroll
    for (int j = 0; j < Sh::pieces; ++j) {
        k[j] = load4(static_cast<const In*>(a.k) + ko + 4 * Sh::lanes * j);
        q[j] = load4(static_cast<const In*>(a.q) + ko + 4 * Sh::lanes * j);
#pragma unroll
        for (int e = 0; e < 4; ++e) kq += k[j][e] * q[j][e];
    }
    kq = step_sum<Sh::lanes>(kq);
    float sk = 0.f, sq = 0.f;
#pragma unroll
    for (int j = 0; j < Sh::pieces; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            S[j][e] *= ga;
            sk += S[j][e] * k[j][e];
            sq += S[j][e] * q[j][e];
        }
    sk = step_sum<Sh::lanes>(sk);
    sq = step_sum<Sh::lanes>(sq);
    const float e1 = be * (v - sk);
#pragma unroll
    for (int j = 0; j < Sh::pieces; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) S[j][e] += e1 * k[j][e];
        *reinterpret_cast<f32x4*>(p + 4 * Sh::lanes * j) = S[j];
    }
    if (li == 0) store1(static_cast<In*>(a.out) + row0 + lr, sq + e1 * kq);
}

template <int dk, typename In>
hipError_t step_go(DeltaStepArgs a, hipStream_t s) {
    constexpr int rows = StepShape<dk>::rows;
    a.groups = a.NH * (a.dv / rows);
    hipLaunchKernelGGL((delta_step_kernel<dk, In>), dim3((unsigned)((a.groups + 3) / 4)), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_delta_step(const DeltaStepArgs& a, hipStream_t s) {
    switch (a.dk) {
        case 16: return a.bf16 ? step_go<16, bf16_t>(a, s) : step_go<16, float>(a, s);
        case 32: return a.bf16 ? step_go<32, bf16_t>(a, s) : step_go<32, float>(a, s);
        case 64: return a.bf16 ? step_go<64, bf16_t>(a, s) : step_go<64, float>(a, s);
        case 128: return a.bf16 ? step_go<128, bf16_t>(a, s) : step_go<128, float>(a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace mesa
