// mesa_kernels.h -- host-side launch interface of the gfx950 Mesa-layer kernels.
// Internal to libmesa; the public ABI is include/mesa.h.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mesa {

struct ChunkStatesArgs {
    const void* k; const void* v; const float* gamma;
    long BH; int T; int d; int chunk; int n_chunks; int bf16;
    float* SH; float* SG; float* final_H; float* final_G; int write_chunks;
    int* work_counter;   // zeroed for the CG kernel that follows, or nullptr
    int g_transposed;    // store G^T's blocks in operand order (the adjoint's A operand), not G's
};

struct CgOutputArgs {
    const void* q; const void* k; const void* v; const float* gamma; const float* lambda;
    const float* SH; const float* SG;
    long BH; int H; int T; int d; int chunk; int n_chunks; int bf16;
    int max_iters; float tol;
    float* out; int32_t* iters;
    float* x_out;   // CG solutions [BH, T, d], or nullptr
    int* work_counter;   // chunk claims; zero at launch
};

struct DecodeArgs {
    const void* q; const void* k; const void* v; const float* gamma; const float* lambda;
    float* SH; float* SG;
    long NH; int H; int d; int bf16; int max_iters; float tol;
    float* out; int32_t* iters;
    float* X; int warm_mode;   // warm start: previous solutions [NH, d] (nullptr: cold)
};

hipError_t launch_chunk_states(const ChunkStatesArgs& a, hipStream_t s);
struct QkPreArgs {
    const void* x; const float* w; int W; const void* hist; void* hist_out;
    int H; int T;
    int segs_per_bh; long n_segs;   // token segments of the main kernel (B * H * segs_per_bh)
    long n_hist;                    // elements of hist_out (B * H * (W - 1) * d), when it is set
    int d; int in_bf16; int out_bf16;
    void* y;
};
#ifndef MESA_QK_PRE_SEGMENT
#define MESA_QK_PRE_SEGMENT 32
#endif
constexpr int kQkPreSegment = MESA_QK_PRE_SEGMENT;   // tokens per thread of the pre-processing kernel
constexpr int kQkPreMaxWidth = 4;   // widest convolution window the kernel is built for

// Backward pass (see the bwd_*.hip kernels).
struct BwdAdjointArgs {
    const void* k; const void* v; const float* gamma; const float* lambda;
    const float* x; const float* o; const float* gout; const float* SH; const float* SG;
    long BH; int H; int T; int d; int chunk; int n_chunks; int bf16; int max_iters; float tol;
    float* dq; float* beta; int32_t* z_iters;
    float* lam_part;     // per chunk and wave: sum over the wave's tokens of z (.) x  [BH*n_chunks][C/16][d]
    int* work_counter;   // chunk claims; zero at launch
};
struct BwdStatesArgs {
    const float* g; const float* z; const float* x; const float* gamma;
    long BH; int T; int d; int chunk; int n_chunks;
    float* Pgx; float* Pzx;
    int* Egx; int* Ezx;   // d >= 32: the states' exponents per (head, chunk, row block)
};
struct BwdKvArgs {
    const void* k; const void* v; const float* gamma; const float* x; const float* z; const float* gout;
    const float* Pgx; const float* Pzx;
    const int* Egx; const int* Ezx;
    long BH; int T; int d; int chunk; int n_chunks; int bf16;
    float* dk; float* dv; float* akey;
};
struct BwdGateArgs {
    const float* beta; const float* akey; const float* gamma; const float* lam_part;
    long BH; int B; int H; int T; int d;
    int n_chunks;   // rows of lam_part per (batch, head): chunks times partial sums per chunk
    float* dgamma; float* dlam;
};

hipError_t launch_bwd_adjoint(const BwdAdjointArgs& a, hipStream_t s);
hipError_t launch_bwd_states(const BwdStatesArgs& a, hipStream_t s);
hipError_t launch_bwd_kv(const BwdKvArgs& a, hipStream_t s);
hipError_t launch_bwd_gate(const BwdGateArgs& a, hipStream_t s);
// Hawk layer recurrence (hawk.hip): two-pass chunked scan.
#ifndef MESA_HAWK_CHUNK
#define MESA_HAWK_CHUNK 128
#endif
constexpr int kHawkChunk = MESA_HAWK_CHUNK;   // tokens per chunk of the scan
struct HawkArgs {
    const void* x; const void* ga; const void* gx; const float* lam; float c; const float* h0;
    int B; int T; int D; int nc; int bf16;
    float* Plog; float* S;   // workspace: per (sequence, chunk, channel) log decay product, end state
    float* y; float* h_final;
};
hipError_t launch_hawk(const HawkArgs& a, hipStream_t s);

// Gated delta rule (delta_*.hip).
constexpr int kDeltaChunk = 64;   // tokens per chunk
constexpr int kDeltaScal = 400;   // floats of per-chunk scalars in the workspace
constexpr int kDeltaPlaneUnits = 384;   // 16-byte units of a plane of M or P in the workspace
// A chunk's planes in the workspace, in 2-byte words: two of M, then P's first
// part and its second, which is a plane too or (p_bytes) a byte an element.
constexpr size_t delta_image_words(bool p_bytes) { return (size_t)(p_bytes ? 7 : 8) * kDeltaPlaneUnits * 4; }
struct DeltaArgs {
    const void* q; const void* k; const void* v; const float* gamma; const float* beta; const float* state0;
    long BH; int Hk; int H; int T; int dk; int dv; int nc; int bf16;
    void* out; float* final_state;
    uint16_t* img; float* scal;   // workspace: per head and chunk the planes of M and P, the scalars
    bool p_bytes;                 // how img holds P (delta_image_words): in bytes for the bf16 forward
    float* S; float* E;           // backward workspace: chunk start states [BH][nc][dv][dk], E [BH][nc][64][dv]
    int nseg; int seg_chunks;     // segments of a sequence that are passed over at once, chunks of one
    float* seg_end;               // nseg > 1, workspace: [BH][nseg - 1][dv + dk][dk] (delta_segments.hip)
    float* seg_start;             // and [BH][nseg][dv][dk], the segments' start states
};
struct DeltaBwdArgs {
    DeltaArgs f;                  // q, k, v, gamma, beta, state0, sizes, img, scal, S, E
    const void* grad_out; const float* grad_final;
    void* grad_q; void* grad_k; void* grad_v; float* grad_gamma; float* grad_beta; float* grad_state;
    float* dS; float* dR;         // workspace: gradients of the chunks' end states, of v in float (both as S and E)
    float* part;                  // workspace: dq, then dk of each value head [2][BH][T][dk] (H != Hk), else nullptr
};
hipError_t launch_delta_passes(const DeltaBwdArgs& a, hipStream_t s);        // the forward's pass again, writing S and E, and the backward's
hipError_t launch_delta_passes_split(const DeltaBwdArgs& a, hipStream_t s);
hipError_t launch_delta_grads(const DeltaBwdArgs& a, hipStream_t s);
hipError_t launch_delta_prep(const DeltaArgs& a, hipStream_t s);
hipError_t launch_delta_scan(const DeltaArgs& a, hipStream_t s);
hipError_t launch_delta_scan_split(const DeltaArgs& a, hipStream_t s);   // with its chain on waves of its own (not float, dk 128)
hipError_t launch_delta_ends_split(const DeltaArgs& a, hipStream_t s);    // the segments' end states and transitions
hipError_t launch_delta_segments(const DeltaArgs& a, hipStream_t s);      // and from them the segments' start states
int delta_segments(long BH, int nc, int dk, int dv, int bf16);            // the number of segments
int delta_segments_most(long BH, int nc, int dk, int dv, int bf16);       // the largest of any length up to nc
hipError_t launch_delta_states(const DeltaArgs& a, hipStream_t s);   // the scan without out, writing S and E (float, dk 128)
struct DeltaStepArgs {
    const void* q; const void* k; const void* v; const float* gamma; const float* beta; float* state;
    long NH; int Hk; int H; int dk; int dv; int bf16;
    void* out;
    long groups;   // set by the launch: row groups of a wave
};
hipError_t launch_delta_step(const DeltaStepArgs& a, hipStream_t s);

// Norms around a layer (block_norms.hip).
struct GateNormArgs {
    const void* x; const void* gate; const float* w; float eps;
    int B; int H; int T; int d; int x_bf16; int g_bf16;
    void* y;
};
struct GateNormBwdArgs {
    const void* x; const void* gate; const float* w; float eps;
    int B; int H; int T; int d; int x_bf16; int g_bf16;
    const void* grad_y; void* grad_x; void* grad_gate; float* grad_w;
    float* partial; int parts; long rows_per_part;   // dw per part: [parts][H][d]
};
struct ResidualNormArgs {
    const void* h; const void* y; const float* w; const float* scale; float eps;
    long R; int D; int h_bf16; int y_bf16;
    void* h_out; void* n;
};
struct ResidualNormBwdArgs {
    const void* h; const void* y; const float* w; const float* scale; float eps;
    long R; int D; int h_bf16; int y_bf16;
    const void* grad_n; const void* grad_h_out; void* grad_h; void* grad_y; float* grad_w; float* grad_scale;
    float* partial; int parts;   // dw and ds per part: [parts][2][D]
};
hipError_t launch_gate_norm(const GateNormArgs& a, hipStream_t s);
hipError_t launch_gate_norm_bwd(const GateNormBwdArgs& a, hipStream_t s);
hipError_t launch_residual_norm(const ResidualNormArgs& a, hipStream_t s);
hipError_t launch_residual_norm_bwd(const ResidualNormBwdArgs& a, hipStream_t s);

hipError_t launch_cg_output(const CgOutputArgs& a, hipStream_t s);
hipError_t launch_cg_output_bf16(const CgOutputArgs& a, hipStream_t s);   // bf16 q/k/v, d >= 32
hipError_t launch_qk_preprocess(const QkPreArgs& a, hipStream_t s);
hipError_t launch_decode(const DecodeArgs& a, hipStream_t s);

}  // namespace mesa
