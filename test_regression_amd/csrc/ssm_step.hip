// ssm_step.hip -- one token of the state space scan, state updated in place (gfx950).
//
// Per sequence and head, with the state S (dv x dk) and the step size D:
//   S' = e^{A D} S + D x b^T,   o = S' c + skip x
// Row i of S only meets x_i, so each row is read once, its product with c is taken
// from the registers, and it is written back.
//
// HBM-bound: 8 dk dv bytes of state a head against about 5 flops for each 8 bytes.
// Lanes and rows as in the delta rule's step: eight lanes take a row (four at dk =
// 16), 16-byte pieces interleaved over them, a wave one group of 8 or 16 rows.  256
// sequences of 32 heads, dk 128, dv 64: 82 us (6.5 TB/s of states, part of them from the
// last-level cache where calls follow one another).
#include "ssm_core.h"

namespace mesa {

template <int dk, typename In>
__global__ __launch_bounds__(256) void ssm_step_kernel(SsmArgs a, long groups) {
    constexpr int lanes = dk >= 32 ? 8 : 4, pieces = dk / (4 * lanes), rows = 64 / lanes;
    const long grp = (long)blockIdx.x * 4 + threadIdx.x / 64;
    if (grp >= groups) return;
    const int lane = threadIdx.x % 64, li = lane % lanes, lr = lane / lanes;
    const long row = grp * rows + lr, nh = grp * rows / a.dv, n = nh / a.H;
    const int h = (int)(nh % a.H), hk = h / (a.H / a.Hk);
    float* p = a.final_state + row * dk + 4 * li;
    f32x4 S[pieces];
#pragma unroll
    for (int j = 0; j < pieces; ++j) S[j] = load4(p + 4 * lanes * j);
    const float step = step_of(raw_step(a, step_bits(a, n, h, 0), step_bias(a, h)), a.softplus);
    const float decay = expf(step * a.A[h]);
    const float x = to_f32(static_cast<const In*>(a.x)[n * a.xs.batch + h * a.xs.head + row % a.dv]);
    const In* br = static_cast<const In*>(a.bm) + n * a.bs.batch + hk * a.bs.head + 4 * li;
    const In* cr = static_cast<const In*>(a.cm) + n * a.cs.batch + hk * a.cs.head + 4 * li;
    float o = 0.f;
#pragma unroll
    for (int j = 0; j < pieces; ++j) {
        const f32x4 bj = load4_el(br + 4 * lanes * j), cj = load4_el(cr + 4 * lanes * j);
        S[j] = S[j] * decay + (step * x) * bj;
#pragma unroll
        for (int e = 0; e < 4; ++e) o += S[j][e] * cj[e];
        *reinterpret_cast<f32x4*>(p + 4 * lanes * j) = S[j];
    }
    o += dpp<0xB1>(o);                            // lanes 1 apart
    o += dpp<0x4E>(o);                            // lanes 2 apart
    if constexpr (lanes == 8) o += dpp<0x141>(o);   // row_half_mirror: the other four of the eight
    if (li == 0) store1(static_cast<In*>(a.out) + row, o + (a.D ? a.D[h] * x : 0.0f));
}

template <int dk>
static void step_go(const SsmArgs& a, hipStream_t s) {
    const long groups = a.BH * (a.dv / (64 / (dk >= 32 ? 8 : 4)));
    const dim3 grid((unsigned)((groups + 3) / 4));
    if (a.bf16) hipLaunchKernelGGL((ssm_step_kernel<dk, bf16_t>), grid, dim3(256), 0, s, a, groups);
    else hipLaunchKernelGGL((ssm_step_kernel<dk, float>), grid, dim3(256), 0, s, a, groups);
}

hipError_t launch_ssm_step(const SsmArgs& a, hipStream_t s) {
    switch (a.dk) {
        case 16: step_go<16>(a, s); break;
        case 32: step_go<32>(a, s); break;
        case 64: step_go<64>(a, s); break;
        case 128: step_go<128>(a, s); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace mesa
