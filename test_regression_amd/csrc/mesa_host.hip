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

__global__ void zero_halves_kernel(uint16_t* p, size_t n) {
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x) p[i] = 0u;
}
hipError_t zero_halves(void* p, size_t n, hipStream_t s) {
    if (!p || n == 0) return hipSuccess;
    const unsigned blocks = (unsigned)std::min<size_t>((n + 255) / 256, 4096);
    hipLaunchKernelGGL(zero_halves_kernel, dim3(blocks), dim3(256), 0, s, static_cast<uint16_t*>(p), n);
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

// ---- strided tensors ----
// A tensor [B, heads, T, d] of a call, or with bytes set a plain buffer.
struct View {
    const void* p;
    mesa::RowStrides s;
    long B, H, T, d;
    int size;            // bytes of an element
    const char* name;
    size_t bytes = 0;
    const char* over = nullptr;
};
static View plain(const void* p, size_t bytes, const char* name, const char* over = nullptr) {
    return {p, {0, 0, 0}, 1, 1, 1, 1, 1, name, bytes, over};
}
static View strided(const void* p, const int64_t* st, long B, long H, long T, long d, int dtype, const char* name) {
    View v{p, {}, B, H, T, d, dtype == MESA_DTYPE_BF16 ? 2 : 4, name};
    v.s = st ? mesa::RowStrides{(long)st[0], (long)st[1], (long)st[2]} : mesa::RowStrides{H * T * d, T * d, d};
    return v;
}
static bool empty(const View& v) { return !v.p || (v.bytes == 0 && (v.B <= 0 || v.H <= 0 || v.T <= 0 || v.d <= 0)); }
static double extent(const View& v) {
    if (v.bytes) return (double)v.bytes;
    if (empty(v)) return 0.0;
    return ((double)(v.B - 1) * v.s.batch + (double)(v.H - 1) * v.s.head + (double)(v.T - 1) * v.s.token + v.d) * v.size;
}
// Elements of one row of pitch P, when all strides are multiples of P or stay below it (else 0).
static long width_in(const View& v, long P) {
    long w = v.d;
    const long n[3] = {v.B, v.H, v.T}, s[3] = {v.s.batch, v.s.head, v.s.token};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && s[i] % P != 0) w += (n[i] - 1) * s[i];
    return w <= P ? w : 0;
}
// Whether two views whose memory overlaps lie between one another in rows of a pitch they share.
static bool interleaved(const View& a, const View& b) {
    if (a.bytes || b.bytes || a.size != b.size) return false;
    const intptr_t delta = (intptr_t)((uintptr_t)b.p - (uintptr_t)a.p);
    if (delta % a.size) return false;
    const long of_a[3] = {a.s.batch, a.s.head, a.s.token}, of_b[3] = {b.s.batch, b.s.head, b.s.token};
    for (long P : of_a)
        for (long Q : of_b) {
            if (P != Q || P <= 0) continue;
            const long wa = width_in(a, P), wb = width_in(b, P), x = ((delta / a.size) % P + P) % P;
            if (wa && wb && x >= wa && P - x >= wb) return true;
        }
    return false;
}
static bool share_memory(const View& a, const View& b) {
    if (empty(a) || empty(b)) return false;
    const double d = a.p < b.p ? (double)((uintptr_t)b.p - (uintptr_t)a.p) : -(double)((uintptr_t)a.p - (uintptr_t)b.p);
    return d < extent(a) && -d < extent(b) && !interleaved(a, b);
}
// As no_alias, for views; also refuses strides that are negative, address more than
// 2^62 bytes, or let an output's rows overlap.
static mesa_status check_views(std::initializer_list<View> outs, std::initializer_list<View> ins) {
    for (const auto* list : {&outs, &ins})
        for (const View& v : *list) {
            if (empty(v) || v.bytes) continue;
            if ((v.B > 1 && v.s.batch < 0) || (v.H > 1 && v.s.head < 0) || (v.T > 1 && v.s.token < 0))
                return fail(MESA_ERR_INVALID_ARGUMENT, "strides of %s must not be negative", v.name);
            if (extent(v) > 4.0e18) return fail(MESA_ERR_INVALID_ARGUMENT, "strides of %s are too large", v.name);
            if (!aligned(v.p, v.size)) return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer (%s: an element's size)", v.name);
        }
    for (auto o = outs.begin(); o != outs.end(); ++o) {
        if (!empty(*o) && !o->bytes) {
            long n[3] = {o->B, o->H, o->T}, s[3] = {o->s.batch, o->s.head, o->s.token};
            double reach = (double)o->d;
            for (int k = 0; k < 3; ++k) {   // by growing stride
                int at = -1;
                for (int i = 0; i < 3; ++i)
                    if (n[i] > 1 && (at < 0 || s[i] < s[at])) at = i;
                if (at < 0) break;
                if (s[at] < reach) return fail(MESA_ERR_INVALID_ARGUMENT, "rows of %s must not share memory", o->name);
                reach += (double)(n[at] - 1) * s[at];
                n[at] = 1;
            }
        }
        for (const View& i : ins)
            if (share_memory(*o, i) && !(o->p == i.p && o->over && !strcmp(o->over, i.name)))
                return fail(MESA_ERR_INVALID_ARGUMENT, "%s must not alias %s", o->name, i.name);
        for (auto q = outs.begin(); q != o; ++q)
            if (share_memory(*o, *q)) return fail(MESA_ERR_INVALID_ARGUMENT, "%s must not alias %s", o->name, q->name);
    }
    return MESA_OK;
}

// ---- causal convolution ----
static mesa_status conv_checks(const void* x, int dtype, const float* w, int width, const float* bias, const void* hist,
                               const int32_t* lens, int B, int T, int D) {
    if (!dtype_ok(dtype))
        return fail(MESA_ERR_INVALID_ARGUMENT, "dtype %d is not MESA_DTYPE_F32 or MESA_DTYPE_BF16", dtype);
    if (B <= 0 || T < 0 || D <= 0 || width <= 0)
        return fail(MESA_ERR_INVALID_ARGUMENT, "sizes must be positive, T >= 0 (B=%d T=%d D=%d width=%d)", B, T, D, width);
    if (width > mesa::kConvMaxWidth) return fail(MESA_ERR_UNSUPPORTED, "width %d not built (at most %d)", width, mesa::kConvMaxWidth);
    if (!w || (T > 0 && !x)) return fail(MESA_ERR_INVALID_ARGUMENT, "w, and x when T > 0, must be non-null");
    if (!aligned(w, 16) || !aligned(bias, 16) || !aligned(hist, 16) || !aligned(lens, 4))
        return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer (16 B for w, bias and hist, 4 B for lens)");
    // threads: one for four channels of a run of tokens, in the backward 512 for 256 channels of eight runs
    const double pieces = ((double)D + 255) / 4, runs = (double)T / mesa::kConvLeast + mesa::kConvLeast;
    if (B * pieces * runs > kMaxThreads) return fail(MESA_ERR_INVALID_ARGUMENT, "grid too large (B=%d T=%d D=%d)", B, T, D);
    return MESA_OK;
}
static View rows_view(const void* p, const int64_t* st, int B, int T, int D, int dtype, const char* name) {
    const int64_t s[3] = {st ? st[0] : (int64_t)T * D, 0, st ? st[1] : D};
    return strided(p, s, B, 1, T, D, dtype, name);
}

mesa_status mesa_causal_conv(const void* x, const int64_t* x_strides, int dtype, const float* w, int width, const float* bias,
                             int silu, const void* hist, void* hist_out, const int32_t* lens, int B, int T, int D, void* y,
                             void* stream) {
    g_err.clear();
    mesa_status st = conv_checks(x, dtype, w, width, bias, hist, lens, B, T, D);
    if (st != MESA_OK) return st;
    if (T > 0 && !y) return fail(MESA_ERR_INVALID_ARGUMENT, "y must be non-null");
    if (!aligned(y, 16) || !aligned(hist_out, 16))
        return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer (16 B for y and hist_out)");
    const View vx = rows_view(x, x_strides, B, T, D, dtype, "x");
    const size_t hb = bytes_of(dtype, (double)B * (width - 1) * D), wb = (size_t)width * D * sizeof(float);
    st = check_views({plain(y, bytes_of(dtype, (double)B * T * D), "y"), plain(hist_out, hb, "hist_out", "hist")},
                     {vx, plain(w, wb, "w"), plain(bias, (size_t)D * 4, "bias"), plain(hist, hb, "hist"), plain(lens, (size_t)B * 4, "lens")});
    if (st != MESA_OK) return st;
    if (T == 0 && (!hist_out || hist_out == hist || width == 1)) return MESA_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const mesa::ConvArgs a{x, vx.s.batch, vx.s.token, w, width, bias, silu, hist, hist_out, lens, B, T, D,
                           dtype == MESA_DTYPE_BF16, y, 0, 0};
    const hipError_t e = timed_launch(MESA_KERNEL_CAUSAL_CONV, s, [&] { return mesa::launch_causal_conv(a, s); });
    if (e != hipSuccess) return hip_fail(e, "causal convolution kernel launch");
    return MESA_OK;
}

size_t mesa_causal_conv_backward_workspace_bytes(int B, int T, int D, int width) {
    if (B <= 0 || T <= 0 || D <= 0 || width <= 0) return 0;
    return (size_t)mesa::conv_bwd_parts(B, T) * (width + 1) * D * sizeof(float);
}

mesa_status mesa_causal_conv_backward(const void* x, const int64_t* x_strides, int dtype, const float* w, int width,
                                      const float* bias, int silu, const void* hist, const int32_t* lens,
                                      const void* grad_y, int B, int T, int D, void* grad_x, const int64_t* grad_x_strides,
                                      float* grad_w, float* grad_bias, void* grad_hist, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    g_err.clear();
    mesa_status st = conv_checks(x, dtype, w, width, bias, hist, lens, B, T, D);
    if (st != MESA_OK) return st;
    if (!grad_w || (T > 0 && (!grad_y || !grad_x || !workspace)))
        return fail(MESA_ERR_INVALID_ARGUMENT, "grad_w, and grad_y, grad_x and workspace when T > 0, must be non-null");
    if ((bias == nullptr) != (grad_bias == nullptr))
        return fail(MESA_ERR_INVALID_ARGUMENT, "grad_bias must be given exactly when bias is");
    if (!aligned(grad_y, 16) || !aligned(grad_hist, 16) || !aligned(workspace, 16) || !aligned(grad_w, 4) || !aligned(grad_bias, 4))
        return fail(MESA_ERR_INVALID_ARGUMENT,
                    "misaligned pointer (16 B for grad_y, grad_hist and workspace, 4 B for grad_w and grad_bias)");
    const size_t need = mesa_causal_conv_backward_workspace_bytes(B, T, D, width);
    if (workspace_bytes < need)
        return fail(MESA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    const View vx = rows_view(x, x_strides, B, T, D, dtype, "x"), vg = rows_view(grad_x, grad_x_strides, B, T, D, dtype, "grad_x");
    const size_t hb = bytes_of(dtype, (double)B * (width - 1) * D), wb = (size_t)width * D * 4, db = (size_t)D * 4;
    st = check_views({vg, plain(grad_hist, hb, "grad_hist"), plain(grad_w, wb, "grad_w"), plain(grad_bias, db, "grad_bias"),
                      plain(workspace, need, "workspace")},
                     {vx, plain(w, wb, "w"), plain(bias, db, "bias"), plain(hist, hb, "hist"), plain(lens, (size_t)B * 4, "lens"),
                      plain(grad_y, bytes_of(dtype, (double)B * T * D), "grad_y")});
    if (st != MESA_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (T == 0) {
        hipError_t e = zero_fill(grad_w, wb, s);
        if (e == hipSuccess) e = zero_fill(grad_bias, db, s);
        if (e == hipSuccess) e = zero_halves(grad_hist, hb / 2, s);
        if (e != hipSuccess) return hip_fail(e, "zero fill of the gradients for T = 0");
        return MESA_OK;
    }
    const mesa::ConvBwdArgs a{{x, vx.s.batch, vx.s.token, w, width, bias, silu, hist, nullptr, lens, B, T, D,
                               dtype == MESA_DTYPE_BF16, nullptr, 0, 0},
                              grad_y, grad_x, vg.s.batch, vg.s.token, grad_hist, grad_w, grad_bias,
                              static_cast<float*>(workspace)};
    const hipError_t e = timed_launch(MESA_KERNEL_CAUSAL_CONV_BWD, s, [&] { return mesa::launch_causal_conv_bwd(a, s); });
    if (e != hipSuccess) return hip_fail(e, "causal convolution gradient kernel launch");
    return MESA_OK;
}

// ---- state space scan ----
static long ssm_chunks(int T) { return ((long)T + mesa::kSsmChunk - 1) / mesa::kSsmChunk; }
// Bytes of n segments' states and decays.
static size_t ssm_slot_bytes(size_t n, int dk, int dv) { return (n * ((size_t)dv * dk + 1) * sizeof(float) + 15) / 16 * 16; }

size_t mesa_ssm_workspace_bytes(int B, int H, int T, int dk, int dv, int dtype) {
    if (B <= 0 || H <= 0 || T <= 0 || dk <= 0 || dv <= 0 || !dtype_ok(dtype)) return 0;
    return ssm_slot_bytes(mesa::ssm_segment_slots((long)B * H, (int)ssm_chunks(T), dv, 1), dk, dv);
}

// The checks the scan's entry points share; T is 1 for the step.
static mesa_status ssm_checks(int dtype, int dt_dtype, const float* A, const float* D, const float* dt_bias,
                              const float* state0, const int32_t* lens, int B, int Hk, int H, int T, int dk, int dv, bool step) {
    if (!dtype_ok(dtype) || !dtype_ok(dt_dtype))
        return fail(MESA_ERR_INVALID_ARGUMENT, "dtype %d / dt_dtype %d must be MESA_DTYPE_F32 or MESA_DTYPE_BF16", dtype, dt_dtype);
    if (B <= 0 || Hk <= 0 || H <= 0 || T < 0 || dk <= 0 || dv <= 0)
        return fail(MESA_ERR_INVALID_ARGUMENT, "sizes must be positive, T >= 0 (B or N=%d Hk=%d H=%d T=%d dk=%d dv=%d)", B, Hk, H,
                    T, dk, dv);
    if (H % Hk != 0) return fail(MESA_ERR_INVALID_ARGUMENT, "H=%d is not a multiple of Hk=%d", H, Hk);
    if (!A) return fail(MESA_ERR_INVALID_ARGUMENT, "A must be non-null");
    if (!aligned(A, 4) || !aligned(D, 4) || !aligned(dt_bias, 4) || !aligned(lens, 4) || !aligned(state0, 16))
        return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer (4 B for A, D, dt_bias and lens, 16 B for states)");
    if (!supported_d(dk)) return fail(MESA_ERR_UNSUPPORTED, "dk=%d not built (16, 32, 64, 128)", dk);
    if (!supported_d(dv)) return fail(MESA_ERR_UNSUPPORTED, "dv=%d not built (16, 32, 64, 128)", dv);
    // the launches' threads: the step's at most 8 a row of the state; else 512 for 64
    // columns of dv of a head and segment or chunk, and one for four features of dB and dC
    const double BH = (double)B * H, nc = (double)ssm_chunks(T);
    const double threads = step ? BH * dv * 8 : std::max(BH * std::max(nc, 1.0) * ((dv + 63) / 64) * 512, (double)B * Hk * T * dk / 2);
    if (threads > kMaxThreads) return fail(MESA_ERR_INVALID_ARGUMENT, "grid too large (B*H=%ld, chunks=%ld)", (long)B * H, ssm_chunks(T));
    return MESA_OK;
}

// The kernels address a chunk's rows by 32-bit offsets.
static mesa_status ssm_pitches(std::initializer_list<View> views) {
    for (const View& v : views)
        if (v.T > 1 && v.s.token >= mesa::kSsmPitch)
            return fail(MESA_ERR_UNSUPPORTED, "token stride of %s not built (2^23 elements or more)", v.name);
    return MESA_OK;
}

mesa_status mesa_ssm_forward(const void* x, const int64_t* x_strides, const void* b, const int64_t* b_strides, const void* c,
                             const int64_t* c_strides, int dtype, const void* dt, const int64_t* dt_strides, int dt_dtype,
                             const float* A, const float* D, const float* dt_bias, int softplus, const float* state0,
                             const int32_t* lens, int B, int Hk, int H, int T, int dk, int dv, void* out, float* final_state,
                             void* workspace, size_t workspace_bytes, void* stream) {
    g_err.clear();
    mesa_status st = ssm_checks(dtype, dt_dtype, A, D, dt_bias, state0, lens, B, Hk, H, T, dk, dv, false);
    if (st != MESA_OK) return st;
    if (T > 0 && (!x || !b || !c || !dt || !out))
        return fail(MESA_ERR_INVALID_ARGUMENT, "x, b, c, dt and out must be non-null");
    if (!aligned(out, 16) || !aligned(final_state, 16) || !aligned(workspace, 16))
        return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer (16 B for out, final_state and workspace)");
    const long BH = (long)B * H, nc = ssm_chunks(T);
    const int nseg = T > 0 ? mesa::ssm_segments(BH, (int)nc, dv, 1) : 1;
    const size_t need = ssm_slot_bytes((size_t)BH * mesa::ssm_slots(nseg, 1), dk, dv);
    if (workspace_bytes < need || (need && !workspace))
        return fail(MESA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", workspace ? workspace_bytes : 0, need);
    const size_t sb = (size_t)BH * dv * dk * sizeof(float), hb = (size_t)H * 4;
    const View vx = strided(x, x_strides, B, H, T, dv, dtype, "x"), vb = strided(b, b_strides, B, Hk, T, dk, dtype, "b"),
               vc = strided(c, c_strides, B, Hk, T, dk, dtype, "c"), vd = strided(dt, dt_strides, B, H, T, 1, dt_dtype, "dt");
    st = check_views({plain(out, bytes_of(dtype, (double)BH * T * dv), "out"), plain(final_state, sb, "final_state", "state0"),
                      plain(workspace, need, "workspace")},
                     {vx, vb, vc, vd, plain(A, hb, "A"), plain(D, hb, "D"), plain(dt_bias, hb, "dt_bias"),
                      plain(state0, sb, "state0"), plain(lens, (size_t)B * 4, "lens")});
    if (st != MESA_OK) return st;
    if ((st = ssm_pitches({vx, vb, vc})) != MESA_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (T == 0) {
        const hipError_t e = copy_or_zero(final_state, state0, (size_t)BH * dv * dk, s);
        if (e != hipSuccess) return hip_fail(e, "final state for T = 0");
        return MESA_OK;
    }
    mesa::SsmArgs a{x, vx.s, b, vb.s, c, vc.s, dt, vd.s, dt_dtype == MESA_DTYPE_BF16, A, D, dt_bias, softplus, state0, lens,
                    BH, B, Hk, H, T, dk, dv, (int)nc, dtype == MESA_DTYPE_BF16, out, final_state};
    a.nseg = nseg;
    a.seg_chunks = (int)((nc + nseg - 1) / nseg);
    a.seg_start = static_cast<float*>(workspace);
    a.seg_decay = a.seg_start + (size_t)BH * mesa::ssm_slots(nseg, 1) * dv * dk;
    const hipError_t e = timed_launch(MESA_KERNEL_SSM_SCAN, s, [&] { return mesa::launch_ssm_scan(a, s); });
    if (e != hipSuccess) return hip_fail(e, "state space scan kernel launch");
    return MESA_OK;
}

// Backward workspace, offsets in bytes (every piece a multiple of 16): the chunk
// states S and R, the heads' sums, the segments' `slots`, `parts` of dB and dC for a
// chunk's group of heads.
struct SsmBwdLayout { size_t R, sums, decay, seg, part, total; };
static SsmBwdLayout ssm_bwd_layout(int B, int H, int T, int dk, int dv, size_t slots, size_t parts) {
    const size_t nc = ssm_chunks(T), states = (size_t)B * H * nc * dk * dv * sizeof(float);
    SsmBwdLayout l{};
    l.R = states;
    l.sums = 2 * states;
    l.decay = l.sums + (size_t)H * 3 * B * nc * sizeof(double);
    l.seg = (l.decay + (size_t)H * 2 * B * nc * sizeof(float) + 15) / 16 * 16;
    l.part = l.seg + ssm_slot_bytes(slots, dk, dv);
    l.total = l.part + parts * 2 * mesa::kSsmChunk * dk * sizeof(float);
    return l;
}

size_t mesa_ssm_backward_workspace_bytes(int B, int Hk, int H, int T, int dk, int dv, int dtype) {
    if (B <= 0 || Hk <= 0 || H <= 0 || H % Hk != 0 || T <= 0 || dk <= 0 || dv <= 0 || !dtype_ok(dtype)) return 0;
    // enough for every smaller batch and shorter sequence too: those may split the heads further, but
    // into at most kSsmGradMost workgroups (of a part, row, group and chunk) where there is more than one part
    const size_t parts = H > Hk ? std::min((size_t)mesa::kSsmGradMost, (size_t)B * H * ssm_chunks(T)) : 0;
    return ssm_bwd_layout(B, H, T, dk, dv, mesa::ssm_segment_slots((long)B * H, (int)ssm_chunks(T), dv, 2), parts).total;
}

mesa_status mesa_ssm_backward(const void* x, const int64_t* x_strides, const void* b, const int64_t* b_strides, const void* c,
                              const int64_t* c_strides, int dtype, const void* dt, const int64_t* dt_strides, int dt_dtype,
                              const float* A, const float* D, const float* dt_bias, int softplus, const float* state0,
                              const int32_t* lens, const void* grad_out, const float* grad_final, int B, int Hk, int H, int T,
                              int dk, int dv, void* grad_x, const int64_t* grad_x_strides, void* grad_b,
                              const int64_t* grad_b_strides, void* grad_c, const int64_t* grad_c_strides, void* grad_dt,
                              const int64_t* grad_dt_strides, float* grad_A, float* grad_D, float* grad_dt_bias,
                              float* grad_state, void* workspace, size_t workspace_bytes, void* stream) {
    g_err.clear();
    mesa_status st = ssm_checks(dtype, dt_dtype, A, D, dt_bias, state0, lens, B, Hk, H, T, dk, dv, false);
    if (st != MESA_OK) return st;
    if (!grad_A || (T > 0 && (!x || !b || !c || !dt || !grad_out || !grad_x || !grad_b || !grad_c || !grad_dt || !workspace)))
        return fail(MESA_ERR_INVALID_ARGUMENT, "x, b, c, dt, grad_out, their gradients, grad_A and workspace must be non-null");
    if ((D == nullptr) != (grad_D == nullptr) || (dt_bias == nullptr) != (grad_dt_bias == nullptr))
        return fail(MESA_ERR_INVALID_ARGUMENT, "grad_D and grad_dt_bias must be given exactly when D and dt_bias are");
    if (!aligned(grad_out, 16) || !aligned(grad_final, 16) || !aligned(grad_state, 16) || !aligned(workspace, 16) ||
        !aligned(grad_A, 4) || !aligned(grad_D, 4) || !aligned(grad_dt_bias, 4))
        return fail(MESA_ERR_INVALID_ARGUMENT,
                    "misaligned pointer (16 B for grad_out, states and workspace, 4 B for the heads' gradients)");
    const long BH = (long)B * H, nc = ssm_chunks(T);
    const int parts = T > 0 ? mesa::ssm_grad_parts(B, Hk, H, (int)nc) : 1;
    const int nseg = T > 0 ? mesa::ssm_segments(BH, (int)nc, dv, 2) : 1;
    const SsmBwdLayout l = ssm_bwd_layout(B, H, T, dk, dv, (size_t)BH * mesa::ssm_slots(nseg, 2), parts > 1 ? (size_t)parts * B * Hk * nc : 0);
    if (T > 0 && workspace_bytes < l.total)
        return fail(MESA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", workspace_bytes, l.total);
    const size_t sb = (size_t)BH * dv * dk * sizeof(float), hb = (size_t)H * 4;
    const View vx = strided(x, x_strides, B, H, T, dv, dtype, "x"), vb = strided(b, b_strides, B, Hk, T, dk, dtype, "b"),
               vc = strided(c, c_strides, B, Hk, T, dk, dtype, "c"), vd = strided(dt, dt_strides, B, H, T, 1, dt_dtype, "dt"),
               gx = strided(grad_x, grad_x_strides, B, H, T, dv, dtype, "grad_x"),
               gb = strided(grad_b, grad_b_strides, B, Hk, T, dk, dtype, "grad_b"),
               gc = strided(grad_c, grad_c_strides, B, Hk, T, dk, dtype, "grad_c"),
               gd = strided(grad_dt, grad_dt_strides, B, H, T, 1, dt_dtype, "grad_dt");
    st = check_views({gx, gb, gc, gd, plain(grad_A, hb, "grad_A"), plain(grad_D, hb, "grad_D"),
                      plain(grad_dt_bias, hb, "grad_dt_bias"), plain(grad_state, sb, "grad_state", "grad_final"),
                      plain(workspace, l.total, "workspace")},
                     {vx, vb, vc, vd, plain(A, hb, "A"), plain(D, hb, "D"), plain(dt_bias, hb, "dt_bias"),
                      plain(state0, sb, "state0"), plain(lens, (size_t)B * 4, "lens"),
                      plain(grad_out, bytes_of(dtype, (double)BH * T * dv), "grad_out"), plain(grad_final, sb, "grad_final")});
    if (st != MESA_OK) return st;
    if ((st = ssm_pitches({vx, vb, vc})) != MESA_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (T == 0) {
        hipError_t e = copy_or_zero(grad_state, grad_final, (size_t)BH * dv * dk, s);
        for (float* p : {grad_A, grad_D, grad_dt_bias})
            if (e == hipSuccess) e = zero_fill(p, hb, s);
        if (e != hipSuccess) return hip_fail(e, "gradients for T = 0");
        return MESA_OK;
    }
    char* ws = static_cast<char*>(workspace);
    mesa::SsmGradArgs a{};
    a.f = mesa::SsmArgs{x, vx.s, b, vb.s, c, vc.s, dt, vd.s, dt_dtype == MESA_DTYPE_BF16, A, D, dt_bias, softplus, state0, lens,
                        BH, B, Hk, H, T, dk, dv, (int)nc, dtype == MESA_DTYPE_BF16, nullptr, nullptr, nseg,
                        (int)((nc + nseg - 1) / nseg), reinterpret_cast<float*>(ws + l.seg),
                        reinterpret_cast<float*>(ws + l.seg) + (size_t)BH * mesa::ssm_slots(nseg, 2) * dv * dk, grad_out, grad_final,
                        grad_state, reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + l.R), reinterpret_cast<float*>(ws + l.decay)};
    a.grad_x = grad_x;
    a.gxs = gx.s;
    a.grad_b = grad_b;
    a.gbs = gb.s;
    a.grad_c = grad_c;
    a.gcs = gc.s;
    a.grad_dt = grad_dt;
    a.gdts = gd.s;
    a.grad_A = grad_A;
    a.grad_D = grad_D;
    a.grad_dt_bias = grad_dt_bias;
    a.parts = parts;
    a.part = parts > 1 ? reinterpret_cast<float*>(ws + l.part) : nullptr;
    a.sums = reinterpret_cast<double*>(ws + l.sums);
    hipError_t e = timed_launch(MESA_KERNEL_SSM_STATES, s, [&] { return mesa::launch_ssm_states(a.f, s); });
    if (e != hipSuccess) return hip_fail(e, "state space states kernel launch");
    e = timed_launch(MESA_KERNEL_SSM_GRADS, s, [&] { return mesa::launch_ssm_grads(a, s); });
    if (e != hipSuccess) return hip_fail(e, "state space gradient kernel launch");
    return MESA_OK;
}

mesa_status mesa_ssm_step(const void* x, const int64_t* x_strides, const void* b, const int64_t* b_strides, const void* c,
                          const int64_t* c_strides, int dtype, const void* dt, const int64_t* dt_strides, int dt_dtype,
                          const float* A, const float* D, const float* dt_bias, int softplus, float* state, int N, int Hk,
                          int H, int dk, int dv, void* out, void* stream) {
    g_err.clear();
    mesa_status st = ssm_checks(dtype, dt_dtype, A, D, dt_bias, state, nullptr, N, Hk, H, 1, dk, dv, true);
    if (st != MESA_OK) return st;
    if (!x || !b || !c || !dt || !state || !out) return fail(MESA_ERR_INVALID_ARGUMENT, "x, b, c, dt, state and out must be non-null");
    if (!aligned(out, 16)) return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer (16 B for out)");
    auto token = [&](const void* p, const int64_t* t, int heads, int d, int type, const char* name) {
        const int64_t s[3] = {t ? t[0] : (int64_t)heads * d, t ? t[1] : d, 0};
        return strided(p, s, N, heads, 1, d, type, name);
    };
    const View vx = token(x, x_strides, H, dv, dtype, "x"), vb = token(b, b_strides, Hk, dk, dtype, "b"),
               vc = token(c, c_strides, Hk, dk, dtype, "c"), vd = token(dt, dt_strides, H, 1, dt_dtype, "dt");
    const long BH = (long)N * H;
    const size_t hb = (size_t)H * 4;
    st = check_views({plain(out, bytes_of(dtype, (double)BH * dv), "out"), plain(state, (size_t)BH * dv * dk * sizeof(float), "state")},
                     {vx, vb, vc, vd, plain(A, hb, "A"), plain(D, hb, "D"), plain(dt_bias, hb, "dt_bias")});
    if (st != MESA_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const mesa::SsmArgs a{x, vx.s, b, vb.s, c, vc.s, dt, vd.s, dt_dtype == MESA_DTYPE_BF16, A, D, dt_bias, softplus, nullptr,
                          nullptr, BH, N, Hk, H, 1, dk, dv, 1, dtype == MESA_DTYPE_BF16, out, state};
    const hipError_t e = timed_launch(MESA_KERNEL_SSM_STEP, s, [&] { return mesa::launch_ssm_step(a, s); });
    if (e != hipSuccess) return hip_fail(e, "state space step kernel launch");
    return MESA_OK;
}

// ---- rotation of queries and keys ----
mesa_status mesa_rotary_frequencies(int rot, double base, int scaling, double factor, double context, double fast, double slow,
                                    double* freqs, float* amplitude) {
    g_err.clear();
    if (rot < 2 || rot % 2) return fail(MESA_ERR_INVALID_ARGUMENT, "rot=%d must be even and positive", rot);
    if (!freqs || !amplitude) return fail(MESA_ERR_INVALID_ARGUMENT, "freqs and amplitude must be non-null");
    if (!(base > 1.0) || std::isinf(base)) return fail(MESA_ERR_INVALID_ARGUMENT, "base must be finite and above 1");
    if (!(factor >= 1.0) || std::isinf(factor)) return fail(MESA_ERR_INVALID_ARGUMENT, "factor must be finite and at least 1");
    if (scaling < MESA_ROTARY_PLAIN || scaling > MESA_ROTARY_PARTS) return fail(MESA_ERR_INVALID_ARGUMENT, "scaling %d is not a mesa_rotary_scaling", scaling);
    if (scaling == MESA_ROTARY_PLAIN && factor != 1.0) return fail(MESA_ERR_INVALID_ARGUMENT, "factor must be 1 without scaling");
    if (scaling == MESA_ROTARY_BASE && rot < 4) return fail(MESA_ERR_INVALID_ARGUMENT, "rot=%d has no slowest pair to scale", rot);
    if (scaling == MESA_ROTARY_PARTS && (!(context > 0.0) || std::isinf(context) || !(slow >= 0.0) || !(fast > slow) || std::isinf(fast)))
        return fail(MESA_ERR_INVALID_ARGUMENT, "context must be finite and > 0, fast finite and > slow >= 0");
    if (scaling == MESA_ROTARY_BASE) base *= std::pow(factor, (double)rot / (rot - 2));
    for (int i = 0; i < rot / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rot);
        freqs[i] = f;
        if (scaling == MESA_ROTARY_LINEAR) freqs[i] = f / factor;
        if (scaling == MESA_ROTARY_PARTS) {
            const double turns = context * f / 6.283185307179586477;
            const double keep = std::min(1.0, std::max(0.0, (turns - slow) / (fast - slow)));
            freqs[i] = f * keep + f / factor * (1.0 - keep);
        }
    }
    *amplitude = scaling == MESA_ROTARY_PARTS ? (float)(1.0 + 0.1 * std::log(factor)) : 1.0f;
    return MESA_OK;
}

static View positions_view(const int64_t* p, int64_t stride, int B, int T) {
    return {p, {(long)stride, 0, 1}, B, 1, T, 1, 8, "positions"};
}
static mesa_status rotate_checks(const void* q, const void* k, int dtype, const double* freqs, int rot, float amplitude,
                                 const int64_t* positions, int64_t positions_stride, const float* wq, const float* wk, int norm,
                                 float eps, int B, int Hq, int Hk, int T, int d) {
    if (!dtype_ok(dtype))
        return fail(MESA_ERR_INVALID_ARGUMENT, "dtype %d is not MESA_DTYPE_F32 or MESA_DTYPE_BF16", dtype);
    if (B <= 0 || Hq <= 0 || Hk < 0 || T < 0 || d <= 0)
        return fail(MESA_ERR_INVALID_ARGUMENT, "sizes must be positive, Hk and T >= 0 (B=%d Hq=%d Hk=%d T=%d d=%d)", B, Hq, Hk, T, d);
    if (!freqs || (T > 0 && (!q || (Hk > 0 && !k))))
        return fail(MESA_ERR_INVALID_ARGUMENT, "freqs, and q and k when T > 0, must be non-null");
    if (Hk == 0 && k) return fail(MESA_ERR_INVALID_ARGUMENT, "k is given with Hk = 0");
    if (norm && (!(eps > 0.0f) || std::isinf(eps))) return fail(MESA_ERR_INVALID_ARGUMENT, "eps must be finite and > 0");
    if (!norm && (wq || wk)) return fail(MESA_ERR_INVALID_ARGUMENT, "wq and wk need the norm");
    if (wk && Hk == 0) return fail(MESA_ERR_INVALID_ARGUMENT, "wk is given with Hk = 0");
    if (!(amplitude > 0.0f) || std::isinf(amplitude)) return fail(MESA_ERR_INVALID_ARGUMENT, "amplitude must be finite and > 0");
    if (!aligned(freqs, 8) || !aligned(positions, 8) || !aligned(wq, 16) || !aligned(wk, 16))
        return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer (8 B for freqs and positions, 16 B for weights)");
    if (positions && positions_stride < 0) return fail(MESA_ERR_INVALID_ARGUMENT, "positions_stride must not be negative");
    if (!supported_d(d) && d != 256) return fail(MESA_ERR_UNSUPPORTED, "d=%d not built (16, 32, 64, 128, 256)", d);
    if (rot < 16 || rot > d || rot % 16) return fail(MESA_ERR_UNSUPPORTED, "rot=%d not built (multiples of 16 up to d=%d)", rot, d);
    if ((double)B * T * (d / 8) * (Hq + Hk) + 256.0 * 32 > kMaxThreads)
        return fail(MESA_ERR_INVALID_ARGUMENT, "grid too large (B=%d T=%d heads=%d)", B, T, Hq + Hk);
    return MESA_OK;
}

mesa_status mesa_qk_rotate(const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides, int dtype,
                           const double* freqs, int rot, int interleaved, float amplitude, const int64_t* positions,
                           int64_t positions_stride, int64_t position0, const float* wq, const float* wk, int norm, float eps,
                           int B, int Hq, int Hk, int T, int d, void* yq, void* yk, void* stream) {
    g_err.clear();
    mesa_status st = rotate_checks(q, k, dtype, freqs, rot, amplitude, positions, positions_stride, wq, wk, norm, eps, B, Hq, Hk, T, d);
    if (st != MESA_OK) return st;
    if (T > 0 && (!yq || (Hk > 0 && !yk))) return fail(MESA_ERR_INVALID_ARGUMENT, "yq and yk must be non-null");
    if (!aligned(yq, 16) || !aligned(yk, 16)) return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer (16 B for yq and yk)");
    const View vq = strided(q, q_strides, B, Hq, T, d, dtype, "q"), vk = strided(k, k_strides, B, Hk, T, d, dtype, "k");
    st = check_views({plain(yq, bytes_of(dtype, (double)B * Hq * T * d), "yq"), plain(Hk ? yk : nullptr, bytes_of(dtype, (double)B * Hk * T * d), "yk")},
                     {vq, vk, plain(freqs, (size_t)rot * 4, "freqs"), plain(wq, (size_t)d * 4, "wq"), plain(wk, (size_t)d * 4, "wk"),
                      positions_view(positions, positions_stride, B, T)});
    if (st != MESA_OK) return st;
    if (T == 0) return MESA_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const mesa::RotateArgs a{q, vq.s, k, vk.s, freqs, rot, interleaved, amplitude, positions, (long)positions_stride, (long)position0,
                             wq, wk, norm, eps, B, Hq, Hk, T, d, dtype == MESA_DTYPE_BF16, yq, yk, 1};
    const hipError_t e = timed_launch(MESA_KERNEL_QK_ROTATE, s, [&] { return mesa::launch_qk_rotate(a, s); });
    if (e != hipSuccess) return hip_fail(e, "query and key rotation kernel launch");
    return MESA_OK;
}

size_t mesa_qk_rotate_backward_workspace_bytes(int d) {
    return d > 0 ? (size_t)mesa::kRotateParts * 2 * d * sizeof(float) : 0;
}

mesa_status mesa_qk_rotate_backward(const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides, int dtype,
                                    const double* freqs, int rot, int interleaved, float amplitude, const int64_t* positions,
                                    int64_t positions_stride, int64_t position0, const float* wq, const float* wk, int norm,
                                    float eps, const void* grad_yq, const void* grad_yk, int B, int Hq, int Hk, int T, int d,
                                    void* grad_q, const int64_t* grad_q_strides, void* grad_k, const int64_t* grad_k_strides,
                                    float* grad_wq, float* grad_wk, void* workspace, size_t workspace_bytes, void* stream) {
    g_err.clear();
    mesa_status st = rotate_checks(q, k, dtype, freqs, rot, amplitude, positions, positions_stride, wq, wk, norm, eps, B, Hq, Hk, T, d);
    if (st != MESA_OK) return st;
    if (T > 0 && (!grad_yq || !grad_q || (Hk > 0 && (!grad_yk || !grad_k))))
        return fail(MESA_ERR_INVALID_ARGUMENT, "grad_yq, grad_yk, grad_q and grad_k must be non-null");
    if ((wq == nullptr) != (grad_wq == nullptr) || (wk == nullptr) != (grad_wk == nullptr))
        return fail(MESA_ERR_INVALID_ARGUMENT, "grad_wq and grad_wk must be given exactly when wq and wk are");
    if (!aligned(grad_yq, 16) || !aligned(grad_yk, 16) || !aligned(workspace, 16) || !aligned(grad_wq, 4) || !aligned(grad_wk, 4))
        return fail(MESA_ERR_INVALID_ARGUMENT, "misaligned pointer (16 B for grad_yq, grad_yk and workspace, 4 B for grad_wq and grad_wk)");
    const size_t need = wq || wk ? mesa_qk_rotate_backward_workspace_bytes(d) : 0;
    if (workspace_bytes < need || (need && !workspace))
        return fail(MESA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", workspace ? workspace_bytes : 0, need);
    const View vq = strided(q, q_strides, B, Hq, T, d, dtype, "q"), vk = strided(k, k_strides, B, Hk, T, d, dtype, "k"),
               gq = strided(grad_q, grad_q_strides, B, Hq, T, d, dtype, "grad_q"),
               gk = strided(grad_k, grad_k_strides, B, Hk, T, d, dtype, "grad_k");
    const size_t db = (size_t)d * 4;
    st = check_views({gq, gk, plain(grad_wq, db, "grad_wq"), plain(grad_wk, db, "grad_wk"), plain(workspace, need, "workspace")},
                     {vq, vk, plain(freqs, (size_t)rot * 4, "freqs"), plain(wq, db, "wq"), plain(wk, db, "wk"),
                      positions_view(positions, positions_stride, B, T),
                      plain(grad_yq, bytes_of(dtype, (double)B * Hq * T * d), "grad_yq"),
                      plain(Hk ? grad_yk : nullptr, bytes_of(dtype, (double)B * Hk * T * d), "grad_yk")});
    if (st != MESA_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (T == 0) {
        hipError_t e = zero_fill(grad_wq, db, s);
        if (e == hipSuccess) e = zero_fill(grad_wk, db, s);
        if (e != hipSuccess) return hip_fail(e, "zero fill of the weights' gradients");
        return MESA_OK;
    }
    const mesa::RotateBwdArgs a{{q, vq.s, k, vk.s, freqs, rot, interleaved, amplitude, positions, (long)positions_stride,
                                 (long)position0, wq, wk, norm, eps, B, Hq, Hk, T, d, dtype == MESA_DTYPE_BF16, nullptr, nullptr, 1},
                                grad_yq, grad_yk, grad_q, gq.s, grad_k, gk.s, grad_wq, grad_wk, static_cast<float*>(workspace)};
    const hipError_t e = timed_launch(MESA_KERNEL_QK_ROTATE_BWD, s, [&] { return mesa::launch_qk_rotate_bwd(a, s); });
    if (e != hipSuccess) return hip_fail(e, "query and key rotation gradient kernel launch");
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
                      (kernel_id >= MESA_KERNEL_DELTA_PREP && kernel_id <= MESA_KERNEL_RESIDUAL_NORM_BWD) ||
                      (kernel_id >= MESA_KERNEL_CAUSAL_CONV && kernel_id < MESA_KERNEL_COUNT);
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
        case MESA_KERNEL_CAUSAL_CONV: return "causal_conv_kernel";
        case MESA_KERNEL_CAUSAL_CONV_BWD: return "causal_conv_bwd_kernels";
        case MESA_KERNEL_SSM_SCAN: return "ssm_scan_kernels";
        case MESA_KERNEL_SSM_STATES: return "ssm_state_passes";
        case MESA_KERNEL_SSM_GRADS: return "ssm_grads_kernels";
        case MESA_KERNEL_SSM_STEP: return "ssm_step_kernel";
        case MESA_KERNEL_QK_ROTATE: return "qk_rotate_kernel";
        case MESA_KERNEL_QK_ROTATE_BWD: return "qk_rotate_bwd_kernels";
    }
    return "unknown";
}

}  // extern "C"
