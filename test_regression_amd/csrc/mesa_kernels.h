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

// Element strides of a tensor [B, heads, T, d] whose rows of d are contiguous.
struct RowStrides { long batch, head, token; };

// Short causal convolution over rows [B, T, D] (causal_conv.hip).
constexpr int kConvLeast = 16;      // the fewest tokens a thread takes, if there are as many
constexpr int kConvMaxWidth = 4;    // widest window the kernels are built for
struct ConvArgs {
    const void* x; long xb; long xt;   // batch and token strides
    const float* w; int W; const float* bias; int silu;
    const void* hist; void* hist_out; const int32_t* lens;
    int B; int T; int D; int bf16;
    void* y;
    int run; int segs;                 // set by the launch
};
struct ConvBwdArgs {
    ConvArgs f;
    const void* grad_y; void* grad_x; long gxb; long gxt; void* grad_hist;
    float* grad_w; float* grad_bias;
    float* partial;                    // workspace: [conv_bwd_parts][W + 1][D]
};
long conv_bwd_parts(long B, int T);   // at most
hipError_t launch_causal_conv(ConvArgs a, hipStream_t s);
hipError_t launch_causal_conv_bwd(ConvBwdArgs a, hipStream_t s);

// State space scan (ssm_*.hip).
constexpr int kSsmChunk = 64;       // tokens per chunk
constexpr long kSsmPitch = 1L << 23;   // token strides stay below: a chunk's offsets fit 32 bits
struct SsmArgs {
    const void* x; RowStrides xs; const void* bm; RowStrides bs; const void* cm; RowStrides cs;
    const void* dt; RowStrides dts; int dt_bf16;
    const float* A; const float* D; const float* dt_bias; int softplus;
    const float* state0; const int32_t* lens;
    long BH; int B; int Hk; int H; int T; int dk; int dv; int nc; int bf16;
    void* out; float* final_state;     // the step: its state
    int nseg; int seg_chunks;          // segments of a sequence that are passed over at once, chunks of one
    float* seg_start;                  // nseg > 1, workspace: ssm_slots states of a head, segments' ends that become the next ones' starts
    float* seg_decay;                  // one a state
    const void* grad_out; const float* grad_final; float* grad_state;   // backward
    // backward workspace [BH][nc][dk][dv]: states at the chunks' starts, gradients at their ends, both as they come
    // from their segment; [2][BH][nc]: the decay from the segment's start to there
    float* S; float* R; float* chunk_decay;
};
struct SsmGradArgs {
    SsmArgs f;
    void* grad_x; RowStrides gxs; void* grad_b; RowStrides gbs; void* grad_c; RowStrides gcs; void* grad_dt; RowStrides gdts;
    float* grad_A; float* grad_D; float* grad_dt_bias;
    int parts;       // workgroups that share the heads of one b and c
    float* part;     // parts > 1: [parts][B Hk][2][T][dk], dC and dB
    double* sums;    // [H][3][B nc]
};
// The gradients' workgroups go over the card in turns of kSsmGradCUs; splitting the heads gives at most kSsmGradMost.
// 2 x 32 heads of 4096 tokens, dk 128, dv 64, bfloat16, the gradient kernel: 151 us in one turn of 16 heads, 162 us in
// two of eight.  Whole calls of 3 and 5 such rows: 372 and 615 us in 3 and 5 turns of eight heads, 394 and 718 us
// unsplit in one and two of 32.
constexpr long kSsmGradCUs = 256, kSsmGradMost = 1280;
int ssm_segments(long BH, int nc, int dv, int sides);         // the number of segments; the backward has two sides
// States that a head's segments keep: their starts, for the gradients the ends of both directions.
constexpr int ssm_slots(int nseg, int sides) { return nseg == 1 ? 0 : sides * nseg; }
long ssm_segment_slots(long BH, int nc, int dv, int sides);   // the most BH ssm_slots of any smaller batch and length
int ssm_grad_parts(long B, int Hk, int H, int nc);
hipError_t launch_ssm_scan(const SsmArgs& a, hipStream_t s);
hipError_t launch_ssm_states(const SsmArgs& a, hipStream_t s);   // S and R
hipError_t launch_ssm_grads(const SsmGradArgs& a, hipStream_t s);
hipError_t launch_ssm_step(const SsmArgs& a, hipStream_t s);

// Per-head norm of queries and keys and their rotation (qk_rotate.hip).
constexpr int kRotateParts = 1024;  // workgroups of the backward, each with one partial sum of the weights' gradients
struct RotateArgs {
    const void* q; RowStrides qs; const void* k; RowStrides ks;
    const double* freqs; int rot; int interleaved; float amplitude;
    const int64_t* positions; long pos_stride; long position0;
    const float* wq; const float* wk; int norm; float eps;
    int B; int Hq; int Hk; int T; int d; int bf16;
    void* yq; void* yk;
    int slots;                         // set by the launch: rows of a token side by side
};
struct RotateBwdArgs {
    RotateArgs f;
    const void* grad_yq; const void* grad_yk;
    void* grad_q; RowStrides gqs; void* grad_k; RowStrides gks;
    float* grad_wq; float* grad_wk;
    float* partial;                    // workspace: [kRotateParts][2][d]
};
hipError_t launch_qk_rotate(RotateArgs a, hipStream_t s);
hipError_t launch_qk_rotate_bwd(RotateBwdArgs a, hipStream_t s);

hipError_t launch_cg_output(const CgOutputArgs& a, hipStream_t s);
hipError_t launch_cg_output_bf16(const CgOutputArgs& a, hipStream_t s);   // bf16 q/k/v, d >= 32
hipError_t launch_qk_preprocess(const QkPreArgs& a, hipStream_t s);
hipError_t launch_decode(const DecodeArgs& a, hipStream_t s);

}  // namespace mesa
