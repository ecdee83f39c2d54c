// delta_segments.hip -- the start states of a sequence's segments (gfx950).
//
// Over a segment of chunks the gated delta rule is affine in the state it starts
// from: S_end = Phi S_start + B, with Phi (dk x dk) the product of the tokens'
// g_t (I - b_t k_t k_t^T) and B the end state from zero.  With few heads the
// pass over the chunks leaves most of the GPU idle, so the segments are passed
// over at once: a first pass gives B and, from the dk unit states without
// values, Phi (delta_scan_split.hip); this kernel joins them,
//   S_1 = B_0,  S_{s+1} = Phi_s S_s + B_s
// (B_0 from the sequence's own start state), and the real pass then runs all
// segments from their S_s.  States are stored transposed, as rows of dv:
// S_{s+1}^T = S_s^T Phi_s^T + B_s^T, where row j of the stored Phi^T is unit
// state j's end.  A workgroup takes 16 rows of dv through all segments; the
// products are float MFMAs.  Eight segments of 16 heads of 128 x 128: 15-16 us,
// most of it the latency of a segment's rows.
#include "delta_core.h"

namespace mesa {

constexpr int kSegPitch = 132;   // floats of an LDS row of up to 128

// Wave j of the dk / 16 holds column block j of Phi^T; the next segment's is in
// flight meanwhile.
template <int DK>
__global__ __launch_bounds__(DK * 4) void delta_segments_kernel(DeltaArgs a) {
    constexpr int NS = DK / 16;
    __shared__ float L[2][16 * kSegPitch];
    const int lane = threadIdx.x % 64, j = threadIdx.x / 64 * 16, n = lane & 15, g = lane >> 4;
    const int tiles = a.dv / 16, bh = blockIdx.x / tiles, v0 = 16 * (blockIdx.x % tiles);
    const size_t end_rows = a.dv + DK;
    const float* end = a.seg_end + (size_t)bh * (a.nseg - 1) * end_rows * DK;
    float* to = a.seg_start + (size_t)bh * a.nseg * a.dv * DK;
    f32x4 phi[NS], t;
    auto load_b = [&](int s) {
#pragma unroll
        for (int r = 0; r < 4; ++r) t[r] = end[(s * end_rows + v0 + 4 * g + r) * DK + j + n];
    };
    auto load_phi = [&](int s) {
#pragma unroll
        for (int k = 0; k < NS; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) phi[k][e] = end[(s * end_rows + a.dv + 16 * k + 4 * g + e) * DK + j + n];
    };
    load_b(0);
    // the first start is state0 or zeros
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const size_t at = (size_t)(v0 + 4 * g + r) * DK + j + n;
        to[at] = a.state0 ? a.state0[(size_t)bh * a.dv * DK + at] : 0.f;
    }
    for (int s = 0; s + 1 < a.nseg; ++s) {
        f32x4 xy[2] = {t, f32x4{0.f, 0.f, 0.f, 0.f}};
        if (s > 0) {
            mfma_ready(xy);
#pragma unroll
            for (int k = 0; k < NS; ++k) {
                const f32x4 v = load4(&L[s & 1][n * kSegPitch + 16 * k + 4 * g]);
#pragma unroll
                for (int e = 0; e < 4; ++e) mfma4_acc(xy[e & 1], v[e], phi[k][e]);
            }
            mfma_done(xy);
        }
        const f32x4 x = xy[0] + xy[1];   // rows v0 + 4 g + r, column j + n of the start of segment s + 1
        if (s + 2 < a.nseg) {
            load_phi(s + 1);
            load_b(s + 1);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            to[((size_t)(s + 1) * a.dv + v0 + 4 * g + r) * DK + j + n] = x[r];
            L[(s & 1) ^ 1][(4 * g + r) * kSegPitch + j + n] = x[r];
        }
        __syncthreads();
    }
}

// Segments by the passes' modelled time: a chunk takes about 2.5, 2.9 or 3.5 us
// with one, two or four column tiles a workgroup (up to 256, 512, 1024 tiles at
// once; measured with bf16 and dk = 128), the two more launches about 20 us.
// Whole forward calls with 1, 4, 8 and 16 segments, in us, * the model's choice:
//   1x16x16384 128x128 bf16  690 361 305* 339    4x8x4096 64x64 float   183 111 106* 123
//   1x16x4096  128x128 bf16  182 109 104* 131    8x8x8192 16x32 float   343 222 230 242*
//   1x8x2048   128x256 bf16   96  65*  69  95    1x4x16384 16x16 float  516 229 129 82*
//   4x8x4096   64x64   bf16  149  97  84*  97    1x4x16384 32x64 bf16   430 203 118 78*
//   1x1x1024   128x128 bf16   53*  41   -   -    2x16x2048 32x32 bf16    73  50  43* -
// The launches cost less than 20 us for one head, and the chunks of narrow float
// rows less than the model's: at worst a tenth and a quarter are left there.
struct SegmentModel {
    double whole, ends, real;   // us a chunk: the sequence in one piece; the segments' ends, the pass from their starts
};
static SegmentModel segment_model(long BH, int dk, int dv, int n) {
    auto chunk_us = [](long tiles) { return tiles <= 256 ? 2.5 : tiles <= 512 ? 2.9 : 3.5 * ((tiles + 1023) / 1024); };
    const long tiles = BH * (dv / 16);
    return {chunk_us(tiles), chunk_us(tiles + (n - 2) * BH * ((dv + dk) / 16)), chunk_us(tiles * n)};
}
int delta_segments(long BH, int nc, int dk, int dv, int bf16) {
    if (!bf16 && dk == 128) return 1;
    int best = 1;
    double t1 = segment_model(BH, dk, dv, 4).whole * nc;
    for (int n : {4, 8, 16}) {
        const int chunks = (nc + n - 1) / n;
        if (chunks < 4 || (n - 1) * chunks >= nc) continue;   // the last segment is not empty
        const SegmentModel m = segment_model(BH, dk, dv, n);
        const double t = 20.0 + chunks * m.ends + chunks * m.real;
        if (t < 0.9 * t1) { best = n; t1 = t; }
    }
    return best;
}

// The most segments that any sequence of up to nc chunks takes: n is taken for
// nc' chunks only with nc' > 3 n and 20 + (ends + real) nc' / n < 0.9 whole nc',
// and both then hold for nc >= nc' too.
int delta_segments_most(long BH, int nc, int dk, int dv, int bf16) {
    if (!bf16 && dk == 128) return 1;
    for (int n : {16, 8, 4}) {
        const SegmentModel m = segment_model(BH, dk, dv, n);
        if (nc > 3 * n && (0.9 * m.whole - (m.ends + m.real) / n) * nc > 20.0) return n;
    }
    return 1;
}

hipError_t launch_delta_segments(const DeltaArgs& a, hipStream_t s) {
    if (a.nseg <= 1) return hipSuccess;
    const hipError_t e = launch_delta_ends_split(a, s);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)(a.BH * (a.dv / 16)));
    switch (a.dk) {
        case 16: hipLaunchKernelGGL(delta_segments_kernel<16>, grid, dim3(64), 0, s, a); break;
        case 32: hipLaunchKernelGGL(delta_segments_kernel<32>, grid, dim3(128), 0, s, a); break;
        case 64: hipLaunchKernelGGL(delta_segments_kernel<64>, grid, dim3(256), 0, s, a); break;
        default: hipLaunchKernelGGL(delta_segments_kernel<128>, grid, dim3(512), 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace mesa
