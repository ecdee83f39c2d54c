// mesa_host.hip -- the C ABI of libmesa (declared in include/mesa.h).
//
// Host-side only: validates every argument before anything is enqueued,
// carves the caller's workspace, and enqueues the kernels on the caller's
// stream.  Allocates no device memory and never synchronises (except in
// mesa_profile_read, which waits for its own events).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <mutex>
#include <string>
#include <vector>

#include "../../include/mesa.h"
#include "mesa_kernels.h"

namespace {

thread_local std::string g_err;

mesa_status fail(mesa_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_err = buf;
    return s;
}

mesa_status hip_fail(hipError_t e, const char* what) {
    return fail(MESA_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool supported_d(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
bool supported_chunk(int c) { return c == 16 || c == 32 || c == 64; }

constexpr int kMaxIters = 4096;

// ---------------- optional per-kernel timing ----------------
struct ProfRec { hipEvent_t a, b; int kid; };
std::mutex g_prof_mu;
bool g_prof_on = false;
std::vector<ProfRec> g_prof_pending;
double g_prof_ms[MESA_KERNEL_COUNT] = {};
int64_t g_prof_n[MESA_KERNEL_COUNT] = {};

// Launches `fn` on `s`; when profiling is on (and `may_record`), brackets it
// with two events.
template <typename Fn>
hipError_t timed_launch(int kid, hipStream_t s, Fn fn, bool may_record = true) {
    bool on;
    {
        std::lock_guard<std::mutex> g(g_prof_mu);
        on = g_prof_on && may_record;
    }
    if (!on) return fn();
    ProfRec r{nullptr, nullptr, kid};
    hipError_t e = hipEventCreate(&r.a);
    if (e != hipSuccess) return e;
    e = hipEventCreate(&r.b);
    if (e == hipSuccess) e = hipEventRecord(r.a, s);
    if (e == hipSuccess) e = fn();
    if (e == hipSuccess) e = hipEventRecord(r.b, s);
    if (e != hipSuccess) {
        (void)hipEventDestroy(r.a);
        if (r.b) (void)hipEventDestroy(r.b);
        return e;
    }
    std::lock_guard<std::mutex> g(g_prof_mu);
    g_prof_pending.push_back(r);
    return hipSuccess;
}

// Zero-fill with a kernel rather than hipMemsetAsync, so that a caller may
// capture the call in a HIP graph.
__global__ void zero_fill_kernel(uint32_t* p, size_t n_words) {
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n_words;
         i += (size_t)gridDim.x * blockDim.x)
        p[i] = 0u;
}

hipError_t zero_fill(void* p, size_t bytes, hipStream_t s) {
    if (!p || bytes == 0) return hipSuccess;
    const size_t words = bytes / 4;   // every buffer filled here is 4-byte elements
    const unsigned blocks = (unsigned)std::min<size_t>((words + 255) / 256, 4096);
    hipLaunchKernelGGL(zero_fill_kernel, dim3(blocks), dim3(256), 0, s, static_cast<uint32_t*>(p), words);
    return hipGetLastError();
}

__global__ void copy_words_kernel(float* out, const float* in, size_t n) {
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x)
        out[i] = in[i];
}

hipError_t copy_words(float* out, const float* in, size_t n, hipStream_t s) {
    const unsigned blocks = (unsigned)std::min<size_t>((n + 255) / 256, 4096);
    hipLaunchKernelGGL(copy_words_kernel, dim3(blocks), dim3(256), 0, s, out, in, n);
    return hipGetLastError();
}

}  // namespace

extern "C" {

int mesa_abi_version(void) { return MESA_ABI_VERSION; }

const char* mesa_status_string(int s) {
    switch (s) {
        case MESA_OK: return "MESA_OK";
        case MESA_ERR_INVALID_ARGUMENT: return "MESA_ERR_INVALID_ARGUMENT";
        case MESA_ERR_UNSUPPORTED: return "MESA_ERR_UNSUPPORTED";
        case MESA_ERR_WORKSPACE_TOO_SMALL: return "MESA_ERR_WORKSPACE_TOO_SMALL";
        case MESA_ERR_HIP: return "MESA_ERR_HIP";
    }
    return "MESA_ERR_UNKNOWN";
}

const char* mesa_last_error_message(void) { return g_err.c_str(); }

// Bytes of the forward's chunk states: per chunk and head the packed upper
// 16x16-block triangle of H (dk (dk + 16) / 2 floats) and the full G
// (dv x dk), fp32.  A 256-byte tail after them holds the CG/output kernel's
// chunk-claim counter.
static size_t forward_state_bytes(long BH, long nc, int dk, int dv) {
    return (size_t)BH * nc * ((size_t)dk * (dk + 16) / 2 + (size_t)dv * dk) * sizeof(float);
}
constexpr size_t kForwardTailBytes = 256;

size_t mesa_forward_workspace_bytes(int B, int H, int T, int dk, int dv, int chunk) {
    if (B <= 0 || H <= 0 || T < 0 || dk <= 0 || dv <= 0 || chunk <= 0) return 0;
    const long nc = ((long)T + chunk - 1) / chunk;
    if (nc == 0) return 0;
    return forward_state_bytes((long)B * H, nc, dk, dv) + kForwardTailBytes;
}

static mesa_status forward_impl(const void* q, const void* k, const void* v, int qkv_dtype,
                                const float* gamma, const float* lambda, int B, int H, int T, int dk,
                                int dv, int chunk, int max_iters, float tol, float* out, int32_t* iters,
                                float* final_H, float* final_G, float* x_out, void* workspace,
                                size_t workspace_bytes, void* stream, bool may_record = true) {
    if (qkv_dtype != MESA_DTYPE_F32 && qkv_dtype != MESA_DTYPE_BF16)
        return fail(MESA_ERR_INVALID_ARGUMENT, "qkv_dtype %d is not MESA_DTYPE_F32 or MESA_DTYPE_BF16", qkv_dtype);
    if (B <= 0 || H <= 0 || T < 0 || dk <= 0 || dv <= 0 || chunk <= 0)
        return fail(MESA_ERR_INVALID_ARGUMENT, "sizes must be positive (B=%d H=%d T=%d dk=%d dv=%d chunk=%d)",
                    B, H, T, dk, dv, chunk);
    if (max_iters < 0 || max_iters > kMaxIters)
        return fail(MESA_ERR_INVALID_ARGUMENT, "max_iters=%d outside [0, %d]", max_iters, kMaxIters);
    if (!(tol >= 0.0f) || std::isinf(tol))
        return fail(MESA_ERR_INVALID_ARGUMENT, "tol must be finite and >= 0");
    const bool need_ws = max_iters > 0 && T > 0;
    if (T > 0 && (!q || !k || !v || !gamma || !out))
        return fail(MESA_ERR_INVALID_ARGUMENT, "q, k, v, gamma and out must be non-null");
    if (!lambda) return fail(MESA_ERR_INVALID_ARGUMENT, "lambda must be non-null");
    if (need_ws && !workspace) return fail(MESA_ERR_INVALID_ARGUMENT, "workspace must be non-null when max_iters > 0");
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
        !aligned(final_H, 16) || !aligned(final_G, 16) || !aligned(workspace, 16) || !aligned(x_out, 16) ||
        !aligned(gamma, 4) || !aligned(lambda, 4) || !aligned(iters, 4))
        return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer (16 B for tensors/workspace, 4 B for gamma/lambda/iters)");
    if (dk != dv) return fail(MESA_ERR_UNSUPPORTED, "dk (%d) != dv (%d) is not built", dk, dv);
    if (!supported_d(dk)) return fail(MESA_ERR_UNSUPPORTED, "d=%d not built (16, 32, 64, 128)", dk);
    if (!supported_chunk(chunk)) return fail(MESA_ERR_UNSUPPORTED, "chunk=%d not built (16, 32, 64)", chunk);
    const long n_chunks = ((long)T + chunk - 1) / chunk;
    const long BH = (long)B * H;
    if (BH * 4 > 0x7fffffffL || BH * n_chunks > 0x7fffffffL)
        return fail(MESA_ERR_INVALID_ARGUMENT, "grid too large (B*H=%ld, chunks=%ld)", BH, n_chunks);
    if (need_ws) {
        const size_t need = mesa_forward_workspace_bytes(B, H, T, dk, dv, chunk);
        if (workspace_bytes < need)
            return fail(MESA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int bf16 = qkv_dtype == MESA_DTYPE_BF16;
    float* SH = static_cast<float*>(workspace);
    float* SG = need_ws ? SH + (size_t)BH * n_chunks * ((size_t)dk * (dk + 16) / 2) : nullptr;
    int* work_counter =
        need_ws ? reinterpret_cast<int*>(static_cast<char*>(workspace) + forward_state_bytes(BH, n_chunks, dk, dv))
                : nullptr;

    if (T == 0) {
        // Nothing to solve; the final states are the zero initial states.
        hipError_t e = zero_fill(final_H, (size_t)BH * dk * dk * sizeof(float), s);
        if (e == hipSuccess) e = zero_fill(final_G, (size_t)BH * dv * dk * sizeof(float), s);
        if (e != hipSuccess) return hip_fail(e, "zero fill of the final states");
        return MESA_OK;
    }

    if (need_ws || final_H || final_G) {
        mesa::ChunkStatesArgs a{k, v, gamma, BH, T, dk, chunk, (int)n_chunks, bf16,
                                SH, SG, final_H, final_G, need_ws ? 1 : 0, work_counter, 0};
        hipError_t e = timed_launch(
            MESA_KERNEL_CHUNK_STATES, s, [&] { return mesa::launch_chunk_states(a, s); }, may_record);
        if (e != hipSuccess) return hip_fail(e, "chunk-state kernel launch");
    }
    if (!need_ws) {
        // max_iters == 0: x = 0, so out = 0 and no update is made.
        hipError_t e = zero_fill(out, (size_t)BH * T * dv * sizeof(float), s);
        if (e == hipSuccess) e = zero_fill(iters, (size_t)BH * T * sizeof(int32_t), s);
        if (e == hipSuccess) e = zero_fill(x_out, (size_t)BH * T * dk * sizeof(float), s);
        if (e != hipSuccess) return hip_fail(e, "zero fill of out/iters");
        return MESA_OK;
    }
    mesa::CgOutputArgs a{q, k, v, gamma, lambda, SH, SG, BH, H, T, dk, chunk, (int)n_chunks,
                         bf16, max_iters, tol, out, iters, x_out, work_counter};
    hipError_t e =
        timed_launch(MESA_KERNEL_CG_OUTPUT, s, [&] { return mesa::launch_cg_output(a, s); }, may_record);
    if (e != hipSuccess) return hip_fail(e, "CG/output kernel launch");
    return MESA_OK;
}

mesa_status mesa_forward(const void* q, const void* k, const void* v, int qkv_dtype,
                         const float* gamma, const float* lambda, int B, int H, int T, int dk,
                         int dv, int chunk, int max_iters, float tol, float* out, int32_t* iters,
                         float* final_H, float* final_G, void* workspace, size_t workspace_bytes,
                         void* stream) {
    g_err.clear();
    return forward_impl(q, k, v, qkv_dtype, gamma, lambda, B, H, T, dk, dv, chunk, max_iters, tol, out, iters,
                        final_H, final_G, nullptr, workspace, workspace_bytes, stream);
}

mesa_status mesa_forward_train(const void* q, const void* k, const void* v, int qkv_dtype,
                               const float* gamma, const float* lambda, int B, int H, int T, int dk,
                               int dv, int chunk, int max_iters, float tol, float* out, int32_t* iters,
                               float* x_out, void* workspace, size_t workspace_bytes, void* stream) {
    g_err.clear();
    if (T > 0 && !x_out) return fail(MESA_ERR_INVALID_ARGUMENT, "x_out must be non-null");
    return forward_impl(q, k, v, qkv_dtype, gamma, lambda, B, H, T, dk, dv, chunk, max_iters, tol, out, iters,
                        nullptr, nullptr, x_out, workspace, workspace_bytes, stream);
}

}  // extern "C"

// ---- the forward without a caller workspace ----
// The chunk states and the claim counter live in this file-scope device
// array instead.  Each GPU the library runs on holds its own copy until the
// process ends; in host code the name only stands for the array, so the
// library reads each device's address once (with that device current) and
// passes that address to the kernels.
static __device__ __align__(256) unsigned char scratch[MESA_NOALLOC_SCRATCH_BYTES];

namespace {
std::mutex g_scratch_mu;
constexpr int kScratchDevices = 64;
void* g_scratch_ptr[kScratchDevices] = {};

mesa_status scratch_of_current_device(void** out) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
    if (dev < 0 || dev >= kScratchDevices)
        return fail(MESA_ERR_UNSUPPORTED, "device %d beyond the %d this build tracks", dev, kScratchDevices);
    std::lock_guard<std::mutex> g(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        void* p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (e != hipSuccess) return hip_fail(e, "hipGetSymbolAddress of the scratch array");
        if (!p) return fail(MESA_ERR_HIP, "hipGetSymbolAddress gave a null scratch address");
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return MESA_OK;
}
}  // namespace

extern "C" {

mesa_status mesa_forward_noalloc(const void* q, const void* k, const void* v, int qkv_dtype,
                                 const float* gamma, const float* lambda, int B, int H, int T, int dk,
                                 int dv, int chunk, int max_iters, float tol, float* out, int32_t* iters,
                                 float* final_H, float* final_G, void* stream) {
    g_err.clear();
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (max_iters > 0 && T > 0) {
        ws_bytes = mesa_forward_workspace_bytes(B, H, T, dk, dv, chunk);
        if (ws_bytes > MESA_NOALLOC_SCRATCH_BYTES)
            return fail(MESA_ERR_WORKSPACE_TOO_SMALL,
                        "these sizes need %zu bytes of chunk states; the built-in scratch holds %zu "
                        "(use mesa_forward with a caller workspace)",
                        ws_bytes, (size_t)MESA_NOALLOC_SCRATCH_BYTES);
        if (ws_bytes > 0) {
            const mesa_status st = scratch_of_current_device(&ws);
            if (st != MESA_OK) return st;
        }
    }
    return forward_impl(q, k, v, qkv_dtype, gamma, lambda, B, H, T, dk, dv, chunk, max_iters, tol, out, iters,
                        final_H, final_G, nullptr, ws, ws_bytes, stream, /*may_record=*/false);
}

// Backward workspace: forward chunk states, reverse states, per-token totals,
// per-chunk regulariser sums; every segment a multiple of 4 floats.
struct BwdLayout {
    size_t sh, sg, pgx, pzx, egx, ezx, beta, akey, lam, counter, total;   // offsets in floats
};

// lam: one d-vector per chunk and 16-token wave of the adjoint kernel;
// counter: the adjoint kernel's chunk-claim counter (64 floats = 256 bytes).
static BwdLayout bwd_layout(long BH, int T, int d, long nc, int chunk) {
    auto r4 = [](size_t n) { return (n + 3) / 4 * 4; };
    const size_t waves = (size_t)std::max(1, chunk / 16);
    BwdLayout l{};
    size_t o = 0;
    l.sh = o;   o += r4((size_t)BH * nc * ((size_t)d * (d + 16) / 2));
    l.sg = o;   o += r4((size_t)BH * nc * d * d);
    l.pgx = o;  o += r4((size_t)BH * nc * d * d);   // P^gx, accumulator block order
    l.pzx = o;  o += r4((size_t)BH * nc * d * d);   // P^zx + (P^zx)^T, accumulator block order
    l.egx = o;  o += r4((size_t)BH * nc * (d / 16));   // their exponents per 16-row block (d >= 32)
    l.ezx = o;  o += r4((size_t)BH * nc * (d / 16));
    l.beta = o; o += r4((size_t)BH * T);
    l.akey = o; o += r4((size_t)BH * T);
    l.lam = o;  o += r4((size_t)BH * nc * waves * d);
    l.counter = o; o += 64;
    l.total = o;
    return l;
}

size_t mesa_backward_workspace_bytes(int B, int H, int T, int dk, int dv, int chunk) {
    if (B <= 0 || H <= 0 || T < 0 || dk <= 0 || dv <= 0 || chunk <= 0) return 0;
    const long nc = ((long)T + chunk - 1) / chunk;
    return bwd_layout((long)B * H, T, std::max(dk, dv), nc, chunk).total * sizeof(float);
}

mesa_status mesa_backward(const void* k, const void* v, int qkv_dtype, const float* gamma, const float* lambda,
                          const float* x, const float* out, const float* grad_out, int B, int H, int T, int dk,
                          int dv, int chunk, int max_iters, float tol, float* grad_q, float* grad_k, float* grad_v,
                          float* grad_gamma, float* grad_lambda, int32_t* z_iters, void* workspace,
                          size_t workspace_bytes, void* stream) {
    g_err.clear();
    if (qkv_dtype != MESA_DTYPE_F32 && qkv_dtype != MESA_DTYPE_BF16)
        return fail(MESA_ERR_INVALID_ARGUMENT, "qkv_dtype %d is not MESA_DTYPE_F32 or MESA_DTYPE_BF16", qkv_dtype);
    if (B <= 0 || H <= 0 || T < 0 || dk <= 0 || dv <= 0 || chunk <= 0)
        return fail(MESA_ERR_INVALID_ARGUMENT, "sizes must be positive (B=%d H=%d T=%d dk=%d dv=%d chunk=%d)",
                    B, H, T, dk, dv, chunk);
    if (max_iters < 0 || max_iters > kMaxIters)
        return fail(MESA_ERR_INVALID_ARGUMENT, "max_iters=%d outside [0, %d]", max_iters, kMaxIters);
    if (!(tol >= 0.0f) || std::isinf(tol))
        return fail(MESA_ERR_INVALID_ARGUMENT, "tol must be finite and >= 0");
    if (!lambda || !grad_lambda) return fail(MESA_ERR_INVALID_ARGUMENT, "lambda and grad_lambda must be non-null");
    if (T > 0 && (!k || !v || !gamma || !x || !out || !grad_out || !grad_q || !grad_k || !grad_v || !grad_gamma))
        return fail(MESA_ERR_INVALID_ARGUMENT, "k, v, gamma, x, out, grad_out and the gradients must be non-null");
    if (T > 0 && !workspace) return fail(MESA_ERR_INVALID_ARGUMENT, "workspace must be non-null");
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(x, 16) || !aligned(out, 16) || !aligned(grad_out, 16) ||
        !aligned(grad_q, 16) || !aligned(grad_k, 16) || !aligned(grad_v, 16) || !aligned(workspace, 16) ||
        !aligned(gamma, 4) || !aligned(lambda, 4) || !aligned(grad_gamma, 4) || !aligned(grad_lambda, 4) ||
        !aligned(z_iters, 4))
        return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer (16 B for tensors/workspace, 4 B for the rest)");
    if (dk != dv) return fail(MESA_ERR_UNSUPPORTED, "dk (%d) != dv (%d) is not built", dk, dv);
    if (!supported_d(dk)) return fail(MESA_ERR_UNSUPPORTED, "d=%d not built (16, 32, 64, 128)", dk);
    if (!supported_chunk(chunk)) return fail(MESA_ERR_UNSUPPORTED, "chunk=%d not built (16, 32, 64)", chunk);
    const long n_chunks = ((long)T + chunk - 1) / chunk;
    const long BH = (long)B * H;
    if (BH * 4 > 0x7fffffffL || BH * n_chunks > 0x7fffffffL)
        return fail(MESA_ERR_INVALID_ARGUMENT, "grid too large (B*H=%ld, chunks=%ld)", BH, n_chunks);
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (T == 0) {
        hipError_t e = zero_fill(grad_lambda, (size_t)H * dk * sizeof(float), s);
        if (e != hipSuccess) return hip_fail(e, "zero fill of grad_lambda");
        return MESA_OK;
    }
    const BwdLayout lay = bwd_layout(BH, T, dk, n_chunks, chunk);
    const int waves = chunk / 16;   // per-wave partial sums of z (.) x per chunk
    if (workspace_bytes < lay.total * sizeof(float))
        return fail(MESA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", workspace_bytes,
                    lay.total * sizeof(float));
    float* ws = static_cast<float*>(workspace);
    const int bf16 = qkv_dtype == MESA_DTYPE_BF16;
    hipError_t e;
    {
        mesa::ChunkStatesArgs a{k, v, gamma, BH, T, dk, chunk, (int)n_chunks, bf16,
                                ws + lay.sh, ws + lay.sg, nullptr, nullptr, 1,
                                reinterpret_cast<int*>(ws + lay.counter), 1};
        e = timed_launch(MESA_KERNEL_CHUNK_STATES, s, [&] { return mesa::launch_chunk_states(a, s); });
        if (e != hipSuccess) return hip_fail(e, "chunk-state kernel launch");
    }
    {
        mesa::BwdAdjointArgs a{k, v, gamma, lambda, x, out, grad_out, ws + lay.sh, ws + lay.sg, BH, H, T, dk, chunk,
                               (int)n_chunks, bf16, max_iters, tol, grad_q, ws + lay.beta, z_iters, ws + lay.lam,
                               reinterpret_cast<int*>(ws + lay.counter)};
        e = timed_launch(MESA_KERNEL_BWD_ADJOINT, s, [&] { return mesa::launch_bwd_adjoint(a, s); });
        if (e != hipSuccess) return hip_fail(e, "backward adjoint kernel launch");
    }
    {
        mesa::BwdStatesArgs a{grad_out, grad_q, x, gamma, BH, T, dk, chunk, (int)n_chunks, ws + lay.pgx,
                              ws + lay.pzx, reinterpret_cast<int*>(ws + lay.egx),
                              reinterpret_cast<int*>(ws + lay.ezx)};
        e = timed_launch(MESA_KERNEL_BWD_STATES, s, [&] { return mesa::launch_bwd_states(a, s); });
        if (e != hipSuccess) return hip_fail(e, "backward state kernel launch");
    }
    {
        mesa::BwdKvArgs a{k, v, gamma, x, grad_q, grad_out, ws + lay.pgx, ws + lay.pzx,
                          reinterpret_cast<const int*>(ws + lay.egx), reinterpret_cast<const int*>(ws + lay.ezx),
                          BH, T, dk, chunk,
                          (int)n_chunks, bf16, grad_k, grad_v, ws + lay.akey};
        e = timed_launch(MESA_KERNEL_BWD_KV, s, [&] { return mesa::launch_bwd_kv(a, s); });
        if (e != hipSuccess) return hip_fail(e, "backward key/value kernel launch");
    }
    {
        mesa::BwdGateArgs a{ws + lay.beta, ws + lay.akey, gamma, ws + lay.lam, BH, B, H, T, dk,
                            (int)n_chunks * waves, grad_gamma, grad_lambda};
        e = timed_launch(MESA_KERNEL_BWD_GATE, s, [&] { return mesa::launch_bwd_gate(a, s); });
        if (e != hipSuccess) return hip_fail(e, "backward gate kernel launch");
    }
    return MESA_OK;
}

static mesa_status decode_impl(const char* what, const void* q, const void* k, const void* v, int qkv_dtype,
                               const float* gamma, const float* lambda, float* state_H, float* state_G,
                               float* state_x, int warm_mode, int N, int H, int dk, int dv, int max_iters,
                               float tol, float* out, int32_t* iters, void* stream) {
    g_err.clear();
    if (qkv_dtype != MESA_DTYPE_F32 && qkv_dtype != MESA_DTYPE_BF16)
        return fail(MESA_ERR_INVALID_ARGUMENT, "qkv_dtype %d is not MESA_DTYPE_F32 or MESA_DTYPE_BF16", qkv_dtype);
    if (N <= 0 || H <= 0 || dk <= 0 || dv <= 0)
        return fail(MESA_ERR_INVALID_ARGUMENT, "sizes must be positive (N=%d H=%d dk=%d dv=%d)", N, H, dk, dv);
    if (max_iters < 0 || max_iters > kMaxIters)
        return fail(MESA_ERR_INVALID_ARGUMENT, "max_iters=%d outside [0, %d]", max_iters, kMaxIters);
    if (!(tol >= 0.0f) || std::isinf(tol))
        return fail(MESA_ERR_INVALID_ARGUMENT, "tol must be finite and >= 0");
    if (!q || !k || !v || !gamma || !lambda || !state_H || !state_G || !out)
        return fail(MESA_ERR_INVALID_ARGUMENT, "q, k, v, gamma, lambda, state_H, state_G and out must be non-null");
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
        !aligned(state_H, 16) || !aligned(state_G, 16) || !aligned(gamma, 4) ||
        !aligned(lambda, 4) || !aligned(iters, 4) || !aligned(state_x, 16))
        return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer (16 B for tensors, 4 B for gamma/lambda/iters)");
    if (dk != dv) return fail(MESA_ERR_UNSUPPORTED, "dk (%d) != dv (%d) is not built", dk, dv);
    if (!supported_d(dk)) return fail(MESA_ERR_UNSUPPORTED, "d=%d not built (16, 32, 64, 128)", dk);
    const long NH = (long)N * H;
    if (NH > 0x7fffffffL) return fail(MESA_ERR_INVALID_ARGUMENT, "grid too large (N*H=%ld)", NH);
    hipStream_t s = static_cast<hipStream_t>(stream);
    mesa::DecodeArgs a{q, k, v, gamma, lambda, state_H, state_G, NH, H, dk,
                       qkv_dtype == MESA_DTYPE_BF16, max_iters, tol, out, iters, state_x, warm_mode};
    hipError_t e = timed_launch(MESA_KERNEL_DECODE, s, [&] { return mesa::launch_decode(a, s); });
    if (e != hipSuccess) return hip_fail(e, what);
    return MESA_OK;
}

mesa_status mesa_decode_step(const void* q, const void* k, const void* v, int qkv_dtype,
                             const float* gamma, const float* lambda, float* state_H,
                             float* state_G, int N, int H, int dk, int dv, int max_iters,
                             float tol, float* out, int32_t* iters, void* stream) {
    return decode_impl("decode kernel launch", q, k, v, qkv_dtype, gamma, lambda, state_H, state_G, nullptr, 0,
                       N, H, dk, dv, max_iters, tol, out, iters, stream);
}

mesa_status mesa_decode_step_warm(const void* q, const void* k, const void* v, int qkv_dtype,
                                  const float* gamma, const float* lambda, float* state_H,
                                  float* state_G, float* state_x, int N, int H, int dk, int dv,
                                  int max_iters, float tol, int warm_mode, float* out, int32_t* iters,
                                  void* stream) {
    g_err.clear();
    if (!state_x) return fail(MESA_ERR_INVALID_ARGUMENT, "state_x must be non-null");
    if (warm_mode != MESA_WARM_COLD && warm_mode != MESA_WARM_PREVIOUS && warm_mode != MESA_WARM_PROJECTED)
        return fail(MESA_ERR_INVALID_ARGUMENT, "warm_mode %d is not MESA_WARM_COLD, MESA_WARM_PREVIOUS or "
                    "MESA_WARM_PROJECTED", warm_mode);
    return decode_impl("warm decode kernel launch", q, k, v, qkv_dtype, gamma, lambda, state_H, state_G, state_x,
                       warm_mode, N, H, dk, dv, max_iters, tol, out, iters, stream);
}

mesa_status mesa_qk_preprocess(const void* x, int in_dtype, const float* conv_w, int width, const void* hist,
                               void* hist_out, int B, int H, int T, int d, void* y, int out_dtype,
                               void* stream) {
    g_err.clear();
    auto dtype_ok = [](int t) { return t == MESA_DTYPE_F32 || t == MESA_DTYPE_BF16; };
    if (!dtype_ok(in_dtype) || !dtype_ok(out_dtype))
        return fail(MESA_ERR_INVALID_ARGUMENT, "in_dtype %d / out_dtype %d must be MESA_DTYPE_F32 or "
                    "MESA_DTYPE_BF16", in_dtype, out_dtype);
    if (B <= 0 || H <= 0 || T < 0 || d <= 0)
        return fail(MESA_ERR_INVALID_ARGUMENT, "sizes must be positive, T >= 0 (B=%d H=%d T=%d d=%d)", B, H, T, d);
    if (width < 1 || width > 8) return fail(MESA_ERR_INVALID_ARGUMENT, "width=%d outside [1, 8]", width);
    if (!conv_w || (T > 0 && (!x || !y)))
        return fail(MESA_ERR_INVALID_ARGUMENT, "conv_w, and x and y when T > 0, must be non-null");
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(hist, 16) || !aligned(hist_out, 16) ||
        !aligned(conv_w, 16))
        return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer (16 B for every tensor)");
    if (y && y == x) return fail(MESA_ERR_INVALID_ARGUMENT, "y must not alias x");
    if (hist_out && (hist_out == hist || hist_out == x))
        return fail(MESA_ERR_INVALID_ARGUMENT, "hist_out must not alias hist or x");
    if (!supported_d(d)) return fail(MESA_ERR_UNSUPPORTED, "d=%d not built (16, 32, 64, 128)", d);
    if (width > mesa::kQkPreMaxWidth)
        return fail(MESA_ERR_UNSUPPORTED, "width=%d not built (at most %d)", width, mesa::kQkPreMaxWidth);
    const int segs = (T + mesa::kQkPreSegment - 1) / mesa::kQkPreSegment;
    const long n_segs = (long)B * H * segs;
    const long n_hist = (width > 1 && hist_out) ? (long)B * H * (width - 1) * d : 0;
    if (n_segs * d > 0x7fffffffL * 256L || n_hist > 0x7fffffffL * 256L)
        return fail(MESA_ERR_INVALID_ARGUMENT, "grid too large (B*H=%ld)", (long)B * H);
    if (n_segs == 0 && n_hist == 0) return MESA_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    mesa::QkPreArgs a{x, conv_w, width, hist, n_hist ? hist_out : nullptr, H, T, segs, n_segs, n_hist, d,
                      in_dtype == MESA_DTYPE_BF16, out_dtype == MESA_DTYPE_BF16, y};
    hipError_t e = timed_launch(MESA_KERNEL_QK_PREPROCESS, s, [&] { return mesa::launch_qk_preprocess(a, s); });
    if (e != hipSuccess) return hip_fail(e, "q/k pre-processing kernel launch");
    return MESA_OK;
}

size_t mesa_hawk_workspace_bytes(int B, int T, int D) {
    if (B <= 0 || T < 0 || D <= 0) return 0;
    const size_t nc = ((size_t)T + mesa::kHawkChunk - 1) / mesa::kHawkChunk;
    return 2 * (size_t)B * nc * D * sizeof(float);
}

mesa_status mesa_hawk_scan(const void* x, const void* ga, const void* gx, int in_dtype, const float* lam, float c,
                           const float* h0, int B, int T, int D, float* y, float* h_final, void* workspace,
                           size_t workspace_bytes, void* stream) {
    g_err.clear();
    if (in_dtype != MESA_DTYPE_F32 && in_dtype != MESA_DTYPE_BF16)
        return fail(MESA_ERR_INVALID_ARGUMENT, "in_dtype %d is not MESA_DTYPE_F32 or MESA_DTYPE_BF16", in_dtype);
    if (B <= 0 || T < 0 || D <= 0)
        return fail(MESA_ERR_INVALID_ARGUMENT, "sizes must be positive, T >= 0 (B=%d T=%d D=%d)", B, T, D);
    if (!(c >= 0.0f) || std::isinf(c)) return fail(MESA_ERR_INVALID_ARGUMENT, "c must be finite and >= 0");
    if (!lam || (T > 0 && (!x || !ga || !gx || !y || !workspace)))
        return fail(MESA_ERR_INVALID_ARGUMENT, "lam, and x, ga, gx, y and workspace when T > 0, must be non-null");
    const size_t esz = in_dtype == MESA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(x, esz) || !aligned(ga, esz) || !aligned(gx, esz) || !aligned(lam, 4) || !aligned(h0, 4) ||
        !aligned(y, 4) || !aligned(h_final, 4) || !aligned(workspace, 16))
        return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer");
    if (y && (y == x || y == ga || y == gx)) return fail(MESA_ERR_INVALID_ARGUMENT, "y must not alias the inputs");
    const long nc = ((long)T + mesa::kHawkChunk - 1) / mesa::kHawkChunk;
    if ((long)B * nc * D > 0x7fffffffL * 256L) return fail(MESA_ERR_INVALID_ARGUMENT, "grid too large");
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (T == 0) {
        // no token: the final state is the initial one
        hipError_t e = hipSuccess;
        if (h_final) {
            e = h0 ? hipMemcpyAsync(h_final, h0, (size_t)B * D * sizeof(float), hipMemcpyDeviceToDevice, s)
                   : zero_fill(h_final, (size_t)B * D * sizeof(float), s);
        }
        if (e != hipSuccess) return hip_fail(e, "Hawk final state for T = 0");
        return MESA_OK;
    }
    if (workspace_bytes < mesa_hawk_workspace_bytes(B, T, D))
        return fail(MESA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", workspace_bytes,
                    mesa_hawk_workspace_bytes(B, T, D));
    float* ws = static_cast<float*>(workspace);
    const size_t per = (size_t)B * nc * D;
    mesa::HawkArgs a{x, ga, gx, lam, c, h0, B, T, D, (int)nc, in_dtype == MESA_DTYPE_BF16, ws, ws + per, y,
                     h_final};
    hipError_t e = timed_launch(MESA_KERNEL_HAWK, s, [&] { return mesa::launch_hawk(a, s); });
    if (e != hipSuccess) return hip_fail(e, "Hawk scan kernel launch");
    return MESA_OK;
}

// A tensor of a call: its address (NULL when absent), size and name, and for an
// output the input that it may be written over, address for address.
struct Span {
    const void* p;
    size_t bytes;
    const char* name;
    const char* over = nullptr;
};
// Refuses outputs that share memory with an input or with one another: the
// kernels of a call read and write in an order of their own.
static mesa_status no_alias(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    auto shared = [](const Span& a, const Span& b) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
        return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
    };
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        for (const Span& i : ins)
            if (shared(*o, i) && !(o->p == i.p && o->over && !strcmp(o->over, i.name)))
                return fail(MESA_ERR_INVALID_ARGUMENT, "%s must not alias %s", o->name, i.name);
        for (auto q = outs.begin(); q != o; ++q)
            if (shared(*o, *q)) return fail(MESA_ERR_INVALID_ARGUMENT, "%s must not alias %s", o->name, q->name);
    }
    return MESA_OK;
}
static size_t bytes_of(int dtype, double n) { return (size_t)(n * (dtype == MESA_DTYPE_BF16 ? 2 : 4)); }

// ---- gated delta rule ----
static bool dtype_ok(int t) { return t == MESA_DTYPE_F32 || t == MESA_DTYPE_BF16; }

static long delta_chunks(int T) { return ((long)T + mesa::kDeltaChunk - 1) / mesa::kDeltaChunk; }

// Bytes of the segments' end and start states (0 with one segment).
static size_t delta_segment_bytes(long BH, int nseg, int dk, int dv) {
    return nseg > 1 ? (size_t)BH * ((size_t)(nseg - 1) * (dv + dk) + (size_t)nseg * dv) * dk * sizeof(float) : 0;
}
static void delta_use_segments(mesa::DeltaArgs* a, int nseg, float* ws) {
    a->nseg = nseg;
    a->seg_chunks = (a->nc + nseg - 1) / nseg;
    if (nseg == 1) return;
    a->seg_end = ws;
    a->seg_start = ws + (size_t)a->BH * (nseg - 1) * (a->dv + a->dk) * a->dk;
}

// Bytes of a head's chunk: its planes of M and P, its scalars.
static size_t delta_chunk_bytes(int dtype) {
    return mesa::delta_image_words(dtype == MESA_DTYPE_BF16) * 2 + mesa::kDeltaScal * sizeof(float);
}

size_t mesa_delta_workspace_bytes(int B, int H, int T, int dk, int dv, int dtype) {
    if (B <= 0 || H <= 0 || T <= 0 || dk <= 0 || dv <= 0 || !dtype_ok(dtype)) return 0;
    // enough for every smaller batch and shorter sequence too: the states of the
    // segments, which only few heads have, may be more than those of the heads
    // and chunks that come on top.  From 1280 column tiles on there are none
    // (delta_segments_most: ends + real >= 3.5 (2 n - 1) a round of tiles, whole
    // at most 3.5 a started round, and n >= 4).
    const long BH = (long)B * H, nc = delta_chunks(T);
    size_t most = delta_chunk_bytes(dtype) * BH * nc;
    const int bf16 = dtype == MESA_DTYPE_BF16;
    int found = 1;   // segments of the head counts seen so far: fewer heads matter only with more of them
    if (nc > 12)
        for (long b = std::min(BH, 1280L * 16 / std::max(dv, 16)); b > 0 && found < 16; --b) {
            const int n = mesa::delta_segments_most(b, (int)nc, dk, dv, bf16);
            if (n > found) most = std::max(most, delta_chunk_bytes(dtype) * b * nc + delta_segment_bytes(b, found = n, dk, dv));
        }
    return most;
}

// A launch holds fewer than 2^32 threads.
constexpr double kMaxThreads = 4.0e9;

// The checks the delta entry points share; T is 1 for the step.
static mesa_status delta_checks(int dtype, int B, int Hk, int H, int T, int dk, int dv, bool step) {
    if (!dtype_ok(dtype))
        return fail(MESA_ERR_INVALID_ARGUMENT, "dtype %d is not MESA_DTYPE_F32 or MESA_DTYPE_BF16", dtype);
    if (B <= 0 || Hk <= 0 || H <= 0 || T < 0 || dk <= 0 || dv <= 0)
        return fail(MESA_ERR_INVALID_ARGUMENT, "sizes must be positive, T >= 0 (B or N=%d Hk=%d H=%d T=%d dk=%d dv=%d)",
                    B, Hk, H, T, dk, dv);
    if (H % Hk != 0) return fail(MESA_ERR_INVALID_ARGUMENT, "H=%d is not a multiple of Hk=%d", H, Hk);
    if (!supported_d(dk)) return fail(MESA_ERR_UNSUPPORTED, "dk=%d not built (16, 32, 64, 128)", dk);
    if (!supported_d(dv) && dv != 256) return fail(MESA_ERR_UNSUPPORTED, "dv=%d not built (16, 32, 64, 128, 256)", dv);
    // the launches' threads: the step's at most 8 a row of the state; else 256 a
    // head and chunk, two passes of 768 a head (in eights) and 64 columns of dv,
    // and one for four features where the gradients of shared heads are summed
    const double BH = (double)B * H;
    const double threads = step ? BH * dv * 8
                                : std::max({BH * delta_chunks(T) * 256, (BH + 7) * ((dv + 63) / 64) * 2 * 768,
                                            (double)B * Hk * T * dk / 4});
    if (threads > kMaxThreads)
        return fail(MESA_ERR_INVALID_ARGUMENT, "grid too large (B*H=%ld, chunks=%ld)", (long)B * H, delta_chunks(T));
    return MESA_OK;
}

static hipError_t copy_or_zero(float* out, const float* in, size_t n, hipStream_t s) {
    if (!out || out == in) return hipSuccess;
    return in ? copy_words(out, in, n, s) : zero_fill(out, n * sizeof(float), s);
}

mesa_status mesa_delta_forward(const void* q, const void* k, const void* v, int dtype, const float* gamma,
                               const float* beta, const float* state0, int B, int Hk, int H, int T, int dk,
                               int dv, void* out, float* final_state, void* workspace, size_t workspace_bytes,
                               void* stream) {
    g_err.clear();
    const mesa_status st = delta_checks(dtype, B, Hk, H, T, dk, dv, false);
    if (st != MESA_OK) return st;
    if (T > 0 && (!q || !k || !v || !gamma || !beta || !out || !workspace))
        return fail(MESA_ERR_INVALID_ARGUMENT, "q, k, v, gamma, beta, out and workspace must be non-null");
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(state0, 16) ||
        !aligned(final_state, 16) || !aligned(workspace, 16) || !aligned(gamma, 4) || !aligned(beta, 4))
        return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer (16 B for tensors/workspace, 4 B for gamma/beta)");
    const long BH = (long)B * H, nc = delta_chunks(T);
    const int nseg = T > 0 ? mesa::delta_segments(BH, (int)nc, dk, dv, dtype == MESA_DTYPE_BF16) : 1;
    const size_t need = delta_chunk_bytes(dtype) * BH * nc + delta_segment_bytes(BH, nseg, dk, dv);
    if (workspace_bytes < need)
        return fail(MESA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    const size_t kb = bytes_of(dtype, (double)B * Hk * T * dk), vb = bytes_of(dtype, (double)BH * T * dv),
                 gb = (size_t)BH * T * sizeof(float), sb = (size_t)BH * dv * dk * sizeof(float);
    const mesa_status al = no_alias(
        {{out, vb, "out"}, {final_state, sb, "final_state", "state0"}, {workspace, need, "workspace"}},
        {{q, kb, "q"}, {k, kb, "k"}, {v, vb, "v"}, {gamma, gb, "gamma"}, {beta, gb, "beta"}, {state0, sb, "state0"}});
    if (al != MESA_OK) return al;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (T == 0) {
        // no token: the final state is the initial one
        const hipError_t e = copy_or_zero(final_state, state0, (size_t)BH * dv * dk, s);
        if (e != hipSuccess) return hip_fail(e, "final state for T = 0");
        return MESA_OK;
    }
    uint16_t* img = static_cast<uint16_t*>(workspace);
    float* scal = reinterpret_cast<float*>(img + (size_t)BH * nc * mesa::delta_image_words(dtype == MESA_DTYPE_BF16));
    mesa::DeltaArgs a{q, k, v, gamma, beta, state0, BH, Hk, H, T, dk, dv, (int)nc, dtype == MESA_DTYPE_BF16,
                      out, final_state, img, scal, dtype == MESA_DTYPE_BF16};
    delta_use_segments(&a, nseg, scal + (size_t)BH * nc * mesa::kDeltaScal);
    hipError_t e = timed_launch(MESA_KERNEL_DELTA_PREP, s, [&] { return mesa::launch_delta_prep(a, s); });
    if (e != hipSuccess) return hip_fail(e, "delta chunk-matrix kernel launch");
    e = timed_launch(MESA_KERNEL_DELTA_SCAN, s, [&] { return mesa::launch_delta_scan(a, s); });
    if (e != hipSuccess) return hip_fail(e, "delta scan kernel launch");
    return MESA_OK;
}

// Backward workspace, offsets in bytes (every segment a multiple of 16).
struct DeltaBwdLayout {
    size_t scal, S, dS, E, dR, part, total;
};
static DeltaBwdLayout delta_bwd_layout(int B, int Hk, int H, int T, int dk, int dv) {
    const size_t n = (size_t)B * H * delta_chunks(T), C = mesa::kDeltaChunk;
    DeltaBwdLayout l{};
    size_t o = n * mesa::delta_image_words(false) * 2;
    l.scal = o; o += n * mesa::kDeltaScal * sizeof(float);
    l.S = o;    o += n * dv * dk * sizeof(float);
    l.dS = o;   o += n * dv * dk * sizeof(float);
    l.E = o;    o += n * C * dv * sizeof(float);
    l.dR = o;   o += n * C * dv * sizeof(float);
    l.part = o; o += H != Hk ? 2 * (size_t)B * H * T * dk * sizeof(float) : 0;
    l.total = o;
    return l;
}

size_t mesa_delta_backward_workspace_bytes(int B, int Hk, int H, int T, int dk, int dv, int dtype) {
    if (B <= 0 || Hk <= 0 || H <= 0 || T <= 0 || dk <= 0 || dv <= 0 || !dtype_ok(dtype)) return 0;
    return delta_bwd_layout(B, Hk, H, T, dk, dv).total;
}

mesa_status mesa_delta_backward(const void* q, const void* k, const void* v, int dtype, const float* gamma,
                                const float* beta, const float* state0, const void* grad_out,
                                const float* grad_final, int B, int Hk, int H, int T, int dk, int dv, void* grad_q,
                                void* grad_k, void* grad_v, float* grad_gamma, float* grad_beta, float* grad_state,
                                void* workspace, size_t workspace_bytes, void* stream) {
    g_err.clear();
    const mesa_status st = delta_checks(dtype, B, Hk, H, T, dk, dv, false);
    if (st != MESA_OK) return st;
    if (T > 0 && (!q || !k || !v || !gamma || !beta || !grad_out || !grad_q || !grad_k || !grad_v || !grad_gamma ||
                  !grad_beta || !workspace))
        return fail(MESA_ERR_INVALID_ARGUMENT,
                    "q, k, v, gamma, beta, grad_out, their gradients and workspace must be non-null");
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(state0, 16) || !aligned(grad_out, 16) ||
        !aligned(grad_final, 16) || !aligned(grad_q, 16) || !aligned(grad_k, 16) || !aligned(grad_v, 16) ||
        !aligned(grad_state, 16) || !aligned(workspace, 16) || !aligned(gamma, 4) || !aligned(beta, 4) ||
        !aligned(grad_gamma, 4) || !aligned(grad_beta, 4))
        return fail(MESA_ERR_INVALID_ARGUMENT,
                    "misaligned pointer (16 B for tensors/workspace, 4 B for gamma/beta and their gradients)");
    const long BH = (long)B * H, nc = delta_chunks(T);
    const DeltaBwdLayout l = delta_bwd_layout(B, Hk, H, T, dk, dv);
    if (workspace_bytes < l.total)
        return fail(MESA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", workspace_bytes, l.total);
    const size_t kb = bytes_of(dtype, (double)B * Hk * T * dk), vb = bytes_of(dtype, (double)BH * T * dv),
                 gb = (size_t)BH * T * sizeof(float), sb = (size_t)BH * dv * dk * sizeof(float);
    const mesa_status al = no_alias(
        {{grad_q, kb, "grad_q"}, {grad_k, kb, "grad_k"}, {grad_v, vb, "grad_v"}, {grad_gamma, gb, "grad_gamma"},
         {grad_beta, gb, "grad_beta"}, {grad_state, sb, "grad_state", "grad_final"}, {workspace, l.total, "workspace"}},
        {{q, kb, "q"}, {k, kb, "k"}, {v, vb, "v"}, {gamma, gb, "gamma"}, {beta, gb, "beta"}, {state0, sb, "state0"},
         {grad_out, vb, "grad_out"}, {grad_final, sb, "grad_final"}});
    if (al != MESA_OK) return al;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (T == 0) {
        const hipError_t e = copy_or_zero(grad_state, grad_final, (size_t)BH * dv * dk, s);
        if (e != hipSuccess) return hip_fail(e, "state gradient for T = 0");
        return MESA_OK;
    }
    char* ws = static_cast<char*>(workspace);
    auto at = [&](size_t o) { return reinterpret_cast<float*>(ws + o); };
    mesa::DeltaBwdArgs a{};
    a.f = mesa::DeltaArgs{q, k, v, gamma, beta, state0, BH, Hk, H, T, dk, dv, (int)nc, dtype == MESA_DTYPE_BF16,
                          nullptr, nullptr, reinterpret_cast<uint16_t*>(ws), at(l.scal), false, at(l.S), at(l.E)};
    delta_use_segments(&a.f, 1, nullptr);
    a.grad_out = grad_out;
    a.grad_final = grad_final;
    a.grad_q = grad_q;
    a.grad_k = grad_k;
    a.grad_v = grad_v;
    a.grad_gamma = grad_gamma;
    a.grad_beta = grad_beta;
    a.grad_state = grad_state;
    a.dS = at(l.dS);
    a.dR = at(l.dR);
    a.part = H != Hk ? at(l.part) : nullptr;
    hipError_t e = timed_launch(MESA_KERNEL_DELTA_PREP, s, [&] { return mesa::launch_delta_prep(a.f, s); });
    if (e != hipSuccess) return hip_fail(e, "delta chunk-matrix kernel launch");
    e = timed_launch(MESA_KERNEL_DELTA_BWD_SCAN, s, [&] { return mesa::launch_delta_passes(a, s); });
    if (e != hipSuccess) return hip_fail(e, "delta backward pass kernel launch");
    e = timed_launch(MESA_KERNEL_DELTA_GRADS, s, [&] { return mesa::launch_delta_grads(a, s); });
    if (e != hipSuccess) return hip_fail(e, "delta gradient kernel launch");
    return MESA_OK;
}

mesa_status mesa_delta_step(const void* q, const void* k, const void* v, int dtype, const float* gamma,
                            const float* beta, float* state, int N, int Hk, int H, int dk, int dv, void* out,
                            void* stream) {
    g_err.clear();
    const mesa_status st = delta_checks(dtype, N, Hk, H, 1, dk, dv, true);
    if (st != MESA_OK) return st;
    if (!q || !k || !v || !gamma || !beta || !state || !out)
        return fail(MESA_ERR_INVALID_ARGUMENT, "q, k, v, gamma, beta, state and out must be non-null");
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(state, 16) ||
        !aligned(gamma, 4) || !aligned(beta, 4))
        return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer (16 B for tensors, 4 B for gamma/beta)");
    const size_t kb = bytes_of(dtype, (double)N * Hk * dk), vb = bytes_of(dtype, (double)N * H * dv),
                 gb = (size_t)N * H * sizeof(float), sb = (size_t)N * H * dv * dk * sizeof(float);
    const mesa_status al = no_alias({{out, vb, "out"}, {state, sb, "state"}},
                                    {{q, kb, "q"}, {k, kb, "k"}, {v, vb, "v"}, {gamma, gb, "gamma"}, {beta, gb, "beta"}});
    if (al != MESA_OK) return al;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const mesa::DeltaStepArgs a{q, k, v, gamma, beta, state, (long)N * H, Hk, H, dk, dv, dtype == MESA_DTYPE_BF16,
                                out, 0};
    const hipError_t e = timed_launch(MESA_KERNEL_DELTA_STEP, s, [&] { return mesa::launch_delta_step(a, s); });
    if (e != hipSuccess) return hip_fail(e, "delta step kernel launch");
    return MESA_OK;
}

// ---- norms around a layer ----
static mesa_status gate_checks(const void* x, int x_dtype, const void* gate, int dtype, const float* w, float eps,
                               int B, int H, int T, int d) {
    if (!dtype_ok(x_dtype) || !dtype_ok(dtype))
        return fail(MESA_ERR_INVALID_ARGUMENT, "x_dtype %d / dtype %d must be MESA_DTYPE_F32 or MESA_DTYPE_BF16",
                    x_dtype, dtype);
    if (B <= 0 || H <= 0 || T < 0 || d <= 0)
        return fail(MESA_ERR_INVALID_ARGUMENT, "sizes must be positive, T >= 0 (B=%d H=%d T=%d d=%d)", B, H, T, d);
    if (!(eps > 0.0f) || std::isinf(eps)) return fail(MESA_ERR_INVALID_ARGUMENT, "eps must be finite and > 0");
    if (!w || (T > 0 && !x)) return fail(MESA_ERR_INVALID_ARGUMENT, "w, and x when T > 0, must be non-null");
    if (!aligned(x, 16) || !aligned(gate, 16) || !aligned(w, 16))
        return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer (16 B for every tensor)");
    if (!supported_d(d) && d != 256) return fail(MESA_ERR_UNSUPPORTED, "d=%d not built (16, 32, 64, 128, 256)", d);
    if ((double)B * H * ((double)T + 8) * (d / 8) > kMaxThreads)
        return fail(MESA_ERR_INVALID_ARGUMENT, "grid too large (B=%d H=%d T=%d)", B, H, T);
    return MESA_OK;
}

mesa_status mesa_gate_norm(const void* x, int x_dtype, const void* gate, int dtype, const float* w, float eps, int B,
                           int H, int T, int d, void* y, void* stream) {
    g_err.clear();
    const mesa_status st = gate_checks(x, x_dtype, gate, dtype, w, eps, B, H, T, d);
    if (st != MESA_OK) return st;
    if (T > 0 && !y) return fail(MESA_ERR_INVALID_ARGUMENT, "y must be non-null");
    if (!aligned(y, 16)) return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer (16 B for every tensor)");
    const double rows = (double)B * H * T * d;
    const size_t xb = bytes_of(x_dtype, rows), yb = bytes_of(dtype, rows);
    const mesa_status al = no_alias({{y, yb, "y"}}, {{x, xb, "x"}, {gate, yb, "gate"}, {w, (size_t)H * d * sizeof(float), "w"}});
    if (al != MESA_OK) return al;
    if (T == 0) return MESA_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const mesa::GateNormArgs a{x, gate, w, eps, B, H, T, d, x_dtype == MESA_DTYPE_BF16, dtype == MESA_DTYPE_BF16, y};
    const hipError_t e = timed_launch(MESA_KERNEL_GATE_NORM, s, [&] { return mesa::launch_gate_norm(a, s); });
    if (e != hipSuccess) return hip_fail(e, "gate norm kernel launch");
    return MESA_OK;
}

// Workgroups a head of the backward (each keeps one partial sum of grad_w):
// about 1024 in all (134 us at 8x16x4096x128; 139 with 2048, 147 with 4096),
// each with whole passes of its 2048 / d rows.
static void gate_parts(int B, int H, int T, int d, int* parts, long* rows) {
    const long BT = (long)B * T, pass = 2048 / d;
    long p = std::min(std::max(1024L / H, 1L), (BT + pass - 1) / pass);
    const long r = ((BT + p - 1) / p + pass - 1) / pass * pass;
    *rows = r;
    *parts = (int)((BT + r - 1) / r);
}

size_t mesa_gate_norm_backward_workspace_bytes(int B, int H, int T, int d) {
    if (B <= 0 || H <= 0 || T <= 0 || d <= 0 || d > 2048) return 0;
    // before gate_parts rounds them, so that fewer rows or heads never need more
    const long passes = ((long)B * T + 2048 / d - 1) / (2048 / d);
    return (size_t)std::min(passes * H, std::max(1024L, (long)H)) * d * sizeof(float);
}

mesa_status mesa_gate_norm_backward(const void* x, int x_dtype, const void* gate, int dtype, const float* w, float eps,
                                    const void* grad_y, int B, int H, int T, int d, void* grad_x, void* grad_gate,
                                    float* grad_w, void* workspace, size_t workspace_bytes, void* stream) {
    g_err.clear();
    const mesa_status st = gate_checks(x, x_dtype, gate, dtype, w, eps, B, H, T, d);
    if (st != MESA_OK) return st;
    if (!grad_w || (T > 0 && (!grad_y || !grad_x || !workspace)))
        return fail(MESA_ERR_INVALID_ARGUMENT, "grad_w, and grad_y, grad_x and workspace when T > 0, must be non-null");
    if (T > 0 && (gate == nullptr) != (grad_gate == nullptr))
        return fail(MESA_ERR_INVALID_ARGUMENT, "grad_gate must be given exactly when gate is");
    if (!aligned(grad_y, 16) || !aligned(grad_x, 16) || !aligned(grad_gate, 16) || !aligned(workspace, 16) ||
        !aligned(grad_w, 4))
        return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer (16 B for tensors/workspace, 4 B for grad_w)");
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (T == 0) {
        const hipError_t e = zero_fill(grad_w, (size_t)H * d * sizeof(float), s);
        if (e != hipSuccess) return hip_fail(e, "zero fill of grad_w");
        return MESA_OK;
    }
    const size_t need = mesa_gate_norm_backward_workspace_bytes(B, H, T, d);
    if (workspace_bytes < need)
        return fail(MESA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    const double n = (double)B * H * T * d;
    const size_t xb = bytes_of(x_dtype, n), yb = bytes_of(dtype, n), wb = (size_t)H * d * sizeof(float);
    const mesa_status al = no_alias(
        {{grad_x, xb, "grad_x"}, {grad_gate, yb, "grad_gate"}, {grad_w, wb, "grad_w"}, {workspace, need, "workspace"}},
        {{x, xb, "x"}, {gate, yb, "gate"}, {w, wb, "w"}, {grad_y, yb, "grad_y"}});
    if (al != MESA_OK) return al;
    mesa::GateNormBwdArgs a{x, gate, w, eps, B, H, T, d, x_dtype == MESA_DTYPE_BF16, dtype == MESA_DTYPE_BF16,
                            grad_y, grad_x, grad_gate, grad_w, static_cast<float*>(workspace), 0, 0};
    gate_parts(B, H, T, d, &a.parts, &a.rows_per_part);
    const hipError_t e = timed_launch(MESA_KERNEL_GATE_NORM_BWD, s, [&] { return mesa::launch_gate_norm_bwd(a, s); });
    if (e != hipSuccess) return hip_fail(e, "gate norm backward kernel launch");
    return MESA_OK;
}

static mesa_status residual_checks(const void* h, int h_dtype, const void* y, int dtype, const float* scale,
                                   const float* w, float eps, int R, int D) {
    if (!dtype_ok(h_dtype) || !dtype_ok(dtype))
        return fail(MESA_ERR_INVALID_ARGUMENT, "h_dtype %d / dtype %d must be MESA_DTYPE_F32 or MESA_DTYPE_BF16",
                    h_dtype, dtype);
    if (R < 0 || D <= 0) return fail(MESA_ERR_INVALID_ARGUMENT, "sizes must be positive, R >= 0 (R=%d D=%d)", R, D);
    if (!(eps > 0.0f) || std::isinf(eps)) return fail(MESA_ERR_INVALID_ARGUMENT, "eps must be finite and > 0");
    if (!w || (R > 0 && !h)) return fail(MESA_ERR_INVALID_ARGUMENT, "w, and h when R > 0, must be non-null");
    if (scale && !y && R > 0) return fail(MESA_ERR_INVALID_ARGUMENT, "scale needs y");
    if (!aligned(h, 16) || !aligned(y, 16) || !aligned(scale, 16) || !aligned(w, 16))
        return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer (16 B for every tensor)");
    if (D > 16384) return fail(MESA_ERR_UNSUPPORTED, "D=%d not built (at most 16384)", D);
    if ((double)R * (D <= 512 ? 64 : D <= 1024 ? 128 : D <= 2048 ? 256 : D <= 4096 ? 512 : 1024) > kMaxThreads)
        return fail(MESA_ERR_INVALID_ARGUMENT, "grid too large (R=%d)", R);
    return MESA_OK;
}

mesa_status mesa_residual_norm(const void* h, int h_dtype, const void* y, int dtype, const float* scale, const float* w,
                               float eps, int R, int D, void* h_out, void* n, void* stream) {
    g_err.clear();
    const mesa_status st = residual_checks(h, h_dtype, y, dtype, scale, w, eps, R, D);
    if (st != MESA_OK) return st;
    if (R > 0 && !n) return fail(MESA_ERR_INVALID_ARGUMENT, "n must be non-null");
    if (R > 0 && (y == nullptr) != (h_out == nullptr))
        return fail(MESA_ERR_INVALID_ARGUMENT, "h_out must be given exactly when y is");
    if (!aligned(h_out, 16) || !aligned(n, 16))
        return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer (16 B for every tensor)");
    const size_t hb = bytes_of(h_dtype, (double)R * D), yb = bytes_of(dtype, (double)R * D), wb = (size_t)D * sizeof(float);
    const mesa_status al = no_alias({{h_out, hb, "h_out", "h"}, {n, yb, "n"}},
                                    {{h, hb, "h"}, {y, yb, "y"}, {scale, wb, "scale"}, {w, wb, "w"}});
    if (al != MESA_OK) return al;
    if (R == 0) return MESA_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const mesa::ResidualNormArgs a{h, y, w, scale, eps, R, D, h_dtype == MESA_DTYPE_BF16, dtype == MESA_DTYPE_BF16,
                                   h_out, n};
    const hipError_t e = timed_launch(MESA_KERNEL_RESIDUAL_NORM, s, [&] { return mesa::launch_residual_norm(a, s); });
    if (e != hipSuccess) return hip_fail(e, "residual norm kernel launch");
    return MESA_OK;
}

// Workgroups of the backward, each with one partial sum of the parameter
// gradients: at most about 2048 waves.  Twice as many take 201 us and not 177
// at 32768 x 2048 and 69 us and not 50 at 4096 x 4096, half as many 232 us.
static int residual_parts(int R, int D) { return (int)std::min<long>(((long)R + 3) / 4, D <= 2048 ? 512 : 256); }

size_t mesa_residual_norm_backward_workspace_bytes(int R, int D) {
    if (R <= 0 || D <= 0) return 0;
    // up to 2048 columns there may be twice the parts
    return (size_t)std::max((long)residual_parts(R, D) * D, (long)residual_parts(R, 2048) * std::min(D, 2048)) * 2 * sizeof(float);
}

mesa_status mesa_residual_norm_backward(const void* h, int h_dtype, const void* y, int dtype, const float* scale,
                                        const float* w, float eps, const void* grad_n, const void* grad_h_out, int R,
                                        int D, void* grad_h, void* grad_y, float* grad_w, float* grad_scale,
                                        void* workspace, size_t workspace_bytes, void* stream) {
    g_err.clear();
    const mesa_status st = residual_checks(h, h_dtype, y, dtype, scale, w, eps, R, D);
    if (st != MESA_OK) return st;
    if (!grad_w || (R > 0 && (!grad_n || !grad_h || !workspace)))
        return fail(MESA_ERR_INVALID_ARGUMENT, "grad_w, and grad_n, grad_h and workspace when R > 0, must be non-null");
    if ((scale == nullptr) != (grad_scale == nullptr) || (R > 0 && (y == nullptr) != (grad_y == nullptr)))
        return fail(MESA_ERR_INVALID_ARGUMENT, "grad_y and grad_scale must be given exactly when y and scale are");
    if (!aligned(grad_n, 16) || !aligned(grad_h_out, 16) || !aligned(grad_h, 16) || !aligned(grad_y, 16) ||
        !aligned(workspace, 16) || !aligned(grad_w, 4) || !aligned(grad_scale, 4))
        return fail(MESA_ERR_INVALID_ARGUMENT,
                    "misaligned pointer (16 B for tensors/workspace, 4 B for grad_w/grad_scale)");
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (R == 0) {
        hipError_t e = zero_fill(grad_w, (size_t)D * sizeof(float), s);
        if (e == hipSuccess) e = zero_fill(grad_scale, (size_t)D * sizeof(float), s);
        if (e != hipSuccess) return hip_fail(e, "zero fill of the parameter gradients");
        return MESA_OK;
    }
    const size_t need = mesa_residual_norm_backward_workspace_bytes(R, D);
    if (workspace_bytes < need)
        return fail(MESA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    const size_t hb = bytes_of(h_dtype, (double)R * D), yb = bytes_of(dtype, (double)R * D), wb = (size_t)D * sizeof(float);
    const mesa_status al = no_alias(
        {{grad_h, hb, "grad_h"}, {grad_y, yb, "grad_y"}, {grad_w, wb, "grad_w"}, {grad_scale, wb, "grad_scale"},
         {workspace, need, "workspace"}},
        {{h, hb, "h"}, {y, yb, "y"}, {scale, wb, "scale"}, {w, wb, "w"}, {grad_n, yb, "grad_n"}, {grad_h_out, hb, "grad_h_out"}});
    if (al != MESA_OK) return al;
    const mesa::ResidualNormBwdArgs a{h, y, w, scale, eps, R, D, h_dtype == MESA_DTYPE_BF16, dtype == MESA_DTYPE_BF16,
                                      grad_n, grad_h_out, grad_h, grad_y, grad_w, grad_scale,
                                      static_cast<float*>(workspace), residual_parts(R, D)};
    const hipError_t e =
        timed_launch(MESA_KERNEL_RESIDUAL_NORM_BWD, s, [&] { return mesa::launch_residual_norm_bwd(a, s); });
    if (e != hipSuccess) return hip_fail(e, "residual norm backward kernel launch");
    return MESA_OK;
}

mesa_status mesa_profile_enable(int on) {
    std::lock_guard<std::mutex> g(g_prof_mu);
    g_prof_on = on != 0;
    return MESA_OK;
}

mesa_status mesa_profile_reset(void) {
    std::lock_guard<std::mutex> g(g_prof_mu);
    for (auto& r : g_prof_pending) {
        (void)hipEventSynchronize(r.b);
        (void)hipEventDestroy(r.a);
        (void)hipEventDestroy(r.b);
    }
    g_prof_pending.clear();
    for (int i = 0; i < MESA_KERNEL_COUNT; ++i) { g_prof_ms[i] = 0; g_prof_n[i] = 0; }
    return MESA_OK;
}

mesa_status mesa_profile_read(int kernel_id, double* total_ms, int64_t* launches) {
    g_err.clear();
    const bool used = (kernel_id >= 0 && kernel_id <= MESA_KERNEL_HAWK) ||
                      (kernel_id >= MESA_KERNEL_DELTA_PREP && kernel_id < MESA_KERNEL_COUNT);
    if (!used || !total_ms || !launches)
        return fail(MESA_ERR_INVALID_ARGUMENT, "bad kernel id %d or null output", kernel_id);
    std::lock_guard<std::mutex> g(g_prof_mu);
    mesa_status st = MESA_OK;
    for (auto& r : g_prof_pending) {
        float ms = 0.f;
        hipError_t e = hipEventSynchronize(r.b);
        if (e == hipSuccess) e = hipEventElapsedTime(&ms, r.a, r.b);
        if (e != hipSuccess && st == MESA_OK) st = hip_fail(e, "profiling event");
        g_prof_ms[r.kid] += ms;
        g_prof_n[r.kid] += 1;
        (void)hipEventDestroy(r.a);
        (void)hipEventDestroy(r.b);
    }
    g_prof_pending.clear();
    *total_ms = g_prof_ms[kernel_id];
    *launches = g_prof_n[kernel_id];
    return st;
}

const char* mesa_kernel_name(int kernel_id) {
    switch (kernel_id) {
        case MESA_KERNEL_CHUNK_STATES: return "chunk_states_kernel";
        case MESA_KERNEL_CG_OUTPUT: return "cg_output_kernel";
        case MESA_KERNEL_DECODE: return "decode_kernel";
        case MESA_KERNEL_QK_PREPROCESS: return "qk_preprocess_kernel";
        case MESA_KERNEL_BWD_ADJOINT: return "bwd_adjoint_kernel";
        case MESA_KERNEL_BWD_STATES: return "bwd_states_kernel";
        case MESA_KERNEL_BWD_KV: return "bwd_kv_kernel";
        case MESA_KERNEL_BWD_GATE: return "bwd_gate_kernel";
        case MESA_KERNEL_HAWK: return "hawk_kernels";
        case MESA_KERNEL_DELTA_PREP: return "delta_prep_kernel";
        case MESA_KERNEL_DELTA_SCAN: return "delta_scan_kernels";
        case MESA_KERNEL_DELTA_STEP: return "delta_step_kernel";
        case MESA_KERNEL_DELTA_BWD_SCAN: return "delta_bwd_passes";
        case MESA_KERNEL_DELTA_GRADS: return "delta_grads_kernels";
        case MESA_KERNEL_GATE_NORM: return "gate_norm_kernel";
        case MESA_KERNEL_GATE_NORM_BWD: return "gate_norm_bwd_kernels";
        case MESA_KERNEL_RESIDUAL_NORM: return "residual_norm_kernel";
        case MESA_KERNEL_RESIDUAL_NORM_BWD: return "residual_norm_bwd_kernels";
    }
    return "unknown";
}

}  // extern "C"
