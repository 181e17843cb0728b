// Host side of the C ABI declared in include/lla.h: argument validation,
// path selection (tcgen05 tensor-core path or SIMT path), workspace handling
// and the per-device error word.
#include <initializer_list>
#include <mutex>

#include "../../include/lla.h"
#include "lla_internal.cuh"
#include "lla_linear.cuh"

// One error word per device (each device holds its own copy of this variable).
__device__ int lla_device_error_word;

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_mutex;
int* g_err_ptr[kMaxDevices];
cudaMemPool_t g_pool[kMaxDevices];
bool g_pool_ready[kMaxDevices];

int current_device() {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    return (dev >= 0 && dev < kMaxDevices) ? dev : -1;
}

// Device address of this device's error word (looked up once per device).
int* error_word(int dev) {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!g_err_ptr[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, lla_device_error_word) != cudaSuccess) return nullptr;
        g_err_ptr[dev] = static_cast<int*>(p);
    }
    return g_err_ptr[dev];
}

// Library-private stream-ordered pool: freed workspace stays reserved for the
// next call instead of going back to the CUDA driver.
cudaMemPool_t workspace_pool(int dev) {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!g_pool_ready[dev]) {
        cudaMemPoolProps props = {};
        props.allocType = cudaMemAllocationTypePinned;
        props.location.type = cudaMemLocationTypeDevice;
        props.location.id = dev;
        cudaMemPool_t pool;
        // a process's first call may come while its stream is being captured: creating the pool is no work of
        // that stream, and only the relaxed mode lets it by
        cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
        if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return nullptr;
        cudaError_t e = cudaMemPoolCreate(&pool, &props);
        uint64_t keep = UINT64_MAX;
        if (e == cudaSuccess) cudaMemPoolSetAttribute(pool, cudaMemPoolAttrReleaseThreshold, &keep);
        cudaThreadExchangeStreamCaptureMode(&mode);
        if (e != cudaSuccess) return nullptr;
        g_pool[dev] = pool;
        g_pool_ready[dev] = true;
    }
    return g_pool[dev];
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// lla_forward_host: per device, one copy-in and one copy-out stream and the events that
// order a chunk's copies and kernels; one call at a time per device.
std::mutex g_host_mutex[kMaxDevices];
cudaStream_t g_copy_in[kMaxDevices], g_copy_out[kMaxDevices];
cudaEvent_t g_host_events[kMaxDevices][7];
bool g_host_ready[kMaxDevices];

bool host_streams_ready(int dev) {
    if (g_host_ready[dev]) return true;
    if (cudaStreamCreateWithFlags(&g_copy_in[dev], cudaStreamNonBlocking) != cudaSuccess ||
        cudaStreamCreateWithFlags(&g_copy_out[dev], cudaStreamNonBlocking) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    for (int i = 0; i < 7; i++) {
        if (cudaEventCreateWithFlags(&g_host_events[dev][i], cudaEventDisableTiming) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
    }
    g_host_ready[dev] = true;
    return true;
}

struct ForwardPlan {
    bool tc;
    lla::TcPlan tcp;
    lla::SimtPlan sp;
    size_t bytes;
};

int validate_forward(const void* q, const void* k, const void* v, const float* log_a, const float* lambda,
                     const void* out, int B, int H, int T, int dk, int dv, int chunk, int dtype) {
    if (!q || !k || !v || !log_a || !lambda || !out) return LLA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(log_a) || !aligned16(lambda) || !aligned16(out))
        return LLA_ERR_INVALID_ARG;
    if (dtype != LLA_BF16 && dtype != LLA_F32) return LLA_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || T < 1 || dk < 1 || dv < 1) return LLA_ERR_INVALID_ARG;
    if (chunk != 16 && chunk != 32 && chunk != 64 && chunk != 128) return LLA_ERR_INVALID_ARG;
    if (T % chunk != 0) return LLA_ERR_INVALID_ARG;
    if (dk > 128 || dv > 128) return LLA_ERR_UNSUPPORTED;
    if ((int64_t)B * H > 65535) return LLA_ERR_UNSUPPORTED;
    if ((int64_t)B * H * T * (dk > dv ? dk : dv) > ((int64_t)1 << 40)) return LLA_ERR_UNSUPPORTED;
    return LLA_OK;
}

bool plan_forward(int B, int H, int T, int dk, int dv, int chunk, int dtype, ForwardPlan* fp) {
    fp->tc = lla::tc_supported(dtype, dk, dv, T) && lla::make_tc_plan(B, H, T, dk, dv, &fp->tcp);
    if (fp->tc) {
        fp->bytes = fp->tcp.total_bytes;
    } else {
        if (!lla::make_simt_plan(B, H, T, dk, dv, chunk, &fp->sp)) return false;
        fp->bytes = fp->sp.total_bytes;
    }
    return true;
}

int run_forward(const ForwardPlan& fp, const void* q, const void* k, const void* v, const float* log_a,
                const float* lambda, void* out, int dtype, void* ws, int* err, cudaStream_t stream) {
    cudaError_t e = fp.tc ? lla::tc_forward(fp.tcp, q, k, v, log_a, lambda, out, ws, err, stream)
                          : lla::simt_forward(fp.sp, dtype, q, k, v, log_a, lambda, out, ws, err, stream);
    return e == cudaSuccess ? LLA_OK : LLA_ERR_CUDA;
}

}  // namespace

namespace lla {
LaunchLog*& active_launch_log() {
    static thread_local LaunchLog* log = nullptr;
    return log;
}
}  // namespace lla

extern "C" {

const char* lla_status_string(int status) {
    switch (status) {
        case LLA_OK: return "LLA_OK";
        case LLA_ERR_INVALID_ARG: return "LLA_ERR_INVALID_ARG: null, misaligned or out-of-range argument";
        case LLA_ERR_UNSUPPORTED: return "LLA_ERR_UNSUPPORTED: shape outside the kernels of this build";
        case LLA_ERR_CUDA: return "LLA_ERR_CUDA: a CUDA call or kernel launch failed";
        case LLA_ERR_TIMEOUT: return "LLA_ERR_TIMEOUT: a kernel's bounded wait ran out";
        case LLA_ERR_NOMEM: return "LLA_ERR_NOMEM: workspace missing or too small";
        case LLA_ERR_DEVICE: return "LLA_ERR_DEVICE: a kernel rejected its device-side input";
        default: return "unknown lla status";
    }
}

int lla_num_levels(int64_t T) {
    if (T <= 0) return 0;
    return lla::bitlength(T - 1) + 1;
}

size_t lla_forward_workspace_size(int B, int H, int T, int dk, int dv, int chunk, int dtype) {
    // Pointers are not inspected here; validate sizes with dummy aligned non-null pointers.
    const void* dummy = reinterpret_cast<const void*>(static_cast<uintptr_t>(256));
    if (validate_forward(dummy, dummy, dummy, static_cast<const float*>(dummy), static_cast<const float*>(dummy),
                         dummy, B, H, T, dk, dv, chunk, dtype) != LLA_OK)
        return 0;
    ForwardPlan fp;
    if (!plan_forward(B, H, T, dk, dv, chunk, dtype, &fp)) return 0;
    return fp.bytes;
}

int lla_forward_ws(const void* q, const void* k, const void* v, const float* log_a, const float* lambda, void* out,
                   int B, int H, int T, int dk, int dv, int chunk, void* stream, int dtype, void* workspace,
                   size_t workspace_bytes) {
    int st = validate_forward(q, k, v, log_a, lambda, out, B, H, T, dk, dv, chunk, dtype);
    if (st != LLA_OK) return st;
    ForwardPlan fp;
    if (!plan_forward(B, H, T, dk, dv, chunk, dtype, &fp)) return LLA_ERR_UNSUPPORTED;
    if (fp.bytes > 0 && (!workspace || workspace_bytes < fp.bytes)) return LLA_ERR_NOMEM;
    if (workspace && (reinterpret_cast<uintptr_t>(workspace) & 255u)) return LLA_ERR_INVALID_ARG;
    const int dev = current_device();
    if (dev < 0) return LLA_ERR_CUDA;
    int* err = error_word(dev);
    if (!err) return LLA_ERR_CUDA;
    return run_forward(fp, q, k, v, log_a, lambda, out, dtype, workspace, err, static_cast<cudaStream_t>(stream));
}

int lla_forward(const void* q, const void* k, const void* v, const float* log_a, const float* lambda, void* out,
                int B, int H, int T, int dk, int dv, int chunk, void* stream, int dtype) {
    int st = validate_forward(q, k, v, log_a, lambda, out, B, H, T, dk, dv, chunk, dtype);
    if (st != LLA_OK) return st;
    ForwardPlan fp;
    if (!plan_forward(B, H, T, dk, dv, chunk, dtype, &fp)) return LLA_ERR_UNSUPPORTED;
    const int dev = current_device();
    if (dev < 0) return LLA_ERR_CUDA;
    int* err = error_word(dev);
    if (!err) return LLA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    void* ws = nullptr;
    if (fp.bytes > 0) {
        cudaMemPool_t pool = workspace_pool(dev);
        if (!pool) return LLA_ERR_CUDA;
        if (cudaMallocFromPoolAsync(&ws, fp.bytes, pool, s) != cudaSuccess) {
            cudaGetLastError();
            return LLA_ERR_NOMEM;
        }
    }
    st = run_forward(fp, q, k, v, log_a, lambda, out, dtype, ws, err, s);
    if (ws && cudaFreeAsync(ws, s) != cudaSuccess && st == LLA_OK) st = LLA_ERR_CUDA;
    return st;
}

int lla_forward_host(const void* q, const void* k, const void* v, const float* log_a, const float* lambda,
                     void* out, int B, int H, int T, int dk, int dv, int chunk, void* stream, int dtype) {
    int st = validate_forward(q, k, v, log_a, lambda, out, B, H, T, dk, dv, chunk, dtype);
    if (st != LLA_OK) return st;
    // the buffers must be host memory (pinned or pageable)
    for (const void* p : {q, k, v, static_cast<const void*>(log_a), static_cast<const void*>(lambda),
                          static_cast<const void*>(out)}) {
        cudaPointerAttributes at;
        if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
            cudaGetLastError();
            return LLA_ERR_INVALID_ARG;
        }
        if (at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged) return LLA_ERR_INVALID_ARG;
    }
    const int BH = B * H;
    // head groups of G consecutive (b, h) heads: [BH, T, .] rows, contiguous per group
    const int nchunks = BH < 8 ? BH : 8;
    const int G = (BH + nchunks - 1) / nchunks;
    ForwardPlan fp;
    if (!plan_forward(1, G, T, dk, dv, chunk, dtype, &fp)) return LLA_ERR_UNSUPPORTED;
    const int dev = current_device();
    if (dev < 0) return LLA_ERR_CUDA;
    int* err = error_word(dev);
    if (!err) return LLA_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_host_mutex[dev]);
    if (!host_streams_ready(dev)) return LLA_ERR_CUDA;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    cudaStream_t in_s = g_copy_in[dev], out_s = g_copy_out[dev];
    cudaMemPool_t pool = workspace_pool(dev);
    if (!pool) return LLA_ERR_CUDA;
    const size_t esz = dtype == LLA_BF16 ? 2 : 4;
    const int L = lla_num_levels(T);
    const size_t rq = (size_t)T * dk * esz, rv = (size_t)T * dv * esz, ra = (size_t)T * 4, rl = (size_t)T * L * 4;
    auto up = [](size_t x) { return (x + 1023) / 1024 * 1024; };
    const size_t slot_bytes = 2 * up(G * rq) + 2 * up(G * rv) + up(G * ra) + up(G * rl);
    char* buf = nullptr;
    if (cudaMallocFromPoolAsync(reinterpret_cast<void**>(&buf), 2 * slot_bytes + fp.bytes, pool, cs) != cudaSuccess) {
        cudaGetLastError();
        return LLA_ERR_NOMEM;
    }
    cudaEvent_t* ev = g_host_events[dev];
    cudaError_t e = cudaEventRecord(ev[6], cs);  // the buffers exist from here on
    if (e == cudaSuccess) e = cudaStreamWaitEvent(in_s, ev[6], 0);
    if (e == cudaSuccess) e = cudaStreamWaitEvent(out_s, ev[6], 0);
    char* ws = buf + 2 * slot_bytes;
    const char* hq = static_cast<const char*>(q);
    const char* hk = static_cast<const char*>(k);
    const char* hv = static_cast<const char*>(v);
    const char* ha = reinterpret_cast<const char*>(log_a);
    const char* hl = reinterpret_cast<const char*>(lambda);
    char* ho = static_cast<char*>(out);
    for (int c = 0; c < nchunks && e == cudaSuccess; c++) {
        const int h0 = c * G, g = (BH - h0) < G ? (BH - h0) : G;
        if (g <= 0) break;
        const int slot = c & 1;
        char* sb = buf + slot * slot_bytes;
        char* dq = sb;
        char* dk_ = dq + up(G * rq);
        char* dv_ = dk_ + up(G * rq);
        char* dout = dv_ + up(G * rv);
        char* da = dout + up(G * rv);
        char* dl = da + up(G * ra);
        // the slot's previous chunk has been copied out (and so computed) before it is refilled
        if (c >= 2) e = cudaStreamWaitEvent(in_s, ev[4 + slot], 0);
        auto h2d = [&](char* d, const char* h, size_t row) {
            if (e == cudaSuccess) e = cudaMemcpyAsync(d, h + (size_t)h0 * row, (size_t)g * row, cudaMemcpyHostToDevice, in_s);
        };
        h2d(dq, hq, rq);
        h2d(dk_, hk, rq);
        h2d(dv_, hv, rv);
        h2d(da, ha, ra);
        h2d(dl, hl, rl);
        if (e == cudaSuccess) e = cudaEventRecord(ev[slot], in_s);
        if (e == cudaSuccess) e = cudaStreamWaitEvent(cs, ev[slot], 0);
        if (e != cudaSuccess) break;
        ForwardPlan fg = fp;
        if (g != G && !plan_forward(1, g, T, dk, dv, chunk, dtype, &fg)) {
            e = cudaErrorInvalidValue;
            break;
        }
        if (run_forward(fg, dq, dk_, dv_, reinterpret_cast<float*>(da), reinterpret_cast<float*>(dl), dout, dtype, ws,
                        err, cs) != LLA_OK) {
            e = cudaErrorLaunchFailure;
            break;
        }
        e = cudaEventRecord(ev[2 + slot], cs);
        if (e == cudaSuccess) e = cudaStreamWaitEvent(out_s, ev[2 + slot], 0);
        if (e == cudaSuccess)
            e = cudaMemcpyAsync(ho + (size_t)h0 * rv, dout, (size_t)g * rv, cudaMemcpyDeviceToHost, out_s);
        if (e == cudaSuccess) e = cudaEventRecord(ev[4 + slot], out_s);
    }
    // everything has landed in host memory before the buffers go back to the pool
    const cudaError_t s1 = cudaStreamSynchronize(out_s);
    const cudaError_t s2 = cudaStreamSynchronize(in_s);
    const cudaError_t f = cudaFreeAsync(buf, cs);
    const cudaError_t s3 = cudaStreamSynchronize(cs);
    if (e != cudaSuccess || s1 != cudaSuccess || s2 != cudaSuccess || f != cudaSuccess || s3 != cudaSuccess) {
        cudaGetLastError();
        return LLA_ERR_CUDA;
    }
    return LLA_OK;
}

}  // extern "C"

namespace {

// Runs `call` (which enqueues one library call on `stream`) with the launch log active:
// a CUDA event before the first kernel and after each launch; writes each kernel's device
// time (ms) and name, in launch order, for i < cap. Returns the number of kernels launched
// or a negative lla_status.
template <typename Fn>
int profile_call(cudaStream_t s, float* kernel_ms, const char** kernel_names, int cap, Fn call) {
    if (cap < 0 || (cap > 0 && (!kernel_ms || !kernel_names))) return LLA_ERR_INVALID_ARG;
    lla::LaunchLog log;
    log.count = 0;
    cudaEvent_t start;
    if (cudaEventCreate(&start) != cudaSuccess) return LLA_ERR_CUDA;
    int made = 0;
    for (; made < lla::LaunchLog::kMax; made++)
        if (cudaEventCreate(&log.events[made]) != cudaSuccess) break;
    if (made < lla::LaunchLog::kMax) {
        for (int i = 0; i < made; i++) cudaEventDestroy(log.events[i]);
        cudaEventDestroy(start);
        return LLA_ERR_CUDA;
    }
    cudaEventRecord(start, s);
    lla::active_launch_log() = &log;
    int st = call();
    lla::active_launch_log() = nullptr;
    int n = log.count < lla::LaunchLog::kMax ? log.count : lla::LaunchLog::kMax;
    if (st == LLA_OK && n > 0 && cudaEventSynchronize(log.events[n - 1]) != cudaSuccess) st = LLA_ERR_CUDA;
    if (st == LLA_OK) {
        cudaEvent_t prev = start;
        for (int i = 0; i < n && i < cap; i++) {
            float ms = 0.f;
            cudaEventElapsedTime(&ms, prev, log.events[i]);
            kernel_ms[i] = ms;
            kernel_names[i] = log.names[i];
            prev = log.events[i];
        }
    }
    for (int i = 0; i < lla::LaunchLog::kMax; i++) cudaEventDestroy(log.events[i]);
    cudaEventDestroy(start);
    return st == LLA_OK ? log.count : st;
}

}  // namespace

extern "C" {

int lla_forward_profile(const void* q, const void* k, const void* v, const float* log_a, const float* lambda,
                        void* out, int B, int H, int T, int dk, int dv, int chunk, void* stream, int dtype,
                        float* kernel_ms, const char** kernel_names, int cap) {
    int st = validate_forward(q, k, v, log_a, lambda, out, B, H, T, dk, dv, chunk, dtype);
    if (st != LLA_OK) return st;
    return profile_call(static_cast<cudaStream_t>(stream), kernel_ms, kernel_names, cap, [&] {
        return lla_forward(q, k, v, log_a, lambda, out, B, H, T, dk, dv, chunk, stream, dtype);
    });
}

int lla_gdn_forward_profile(const void* q, const void* k, const void* v, const float* log_a, const float* beta,
                            const float* lambda, void* out, int B, int H, int T, int dk, int dv, int chunk,
                            void* stream, int dtype, float* kernel_ms, const char** kernel_names, int cap) {
    int st = validate_forward(q, k, v, log_a, lambda, out, B, H, T, dk, dv, chunk, dtype);
    if (st != LLA_OK) return st;
    return profile_call(static_cast<cudaStream_t>(stream), kernel_ms, kernel_names, cap, [&] {
        return lla_gdn_forward(q, k, v, log_a, beta, lambda, out, B, H, T, dk, dv, chunk, stream, dtype);
    });
}

int lla_decode_step(const void* q, const void* k, const void* v, const float* log_a, const float* lambda,
                    float* fenwick_states, const int64_t* t, void* out, void* stream, int B, int H, int dk, int dv,
                    int Lmax, int dtype) {
    if (!q || !k || !v || !log_a || !lambda || !fenwick_states || !t || !out) return LLA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(log_a) || !aligned16(lambda) ||
        !aligned16(fenwick_states) || !aligned16(t) || !aligned16(out))
        return LLA_ERR_INVALID_ARG;
    if (dtype != LLA_BF16 && dtype != LLA_F32) return LLA_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || dk < 1 || dv < 1 || Lmax < 1 || Lmax > 40) return LLA_ERR_INVALID_ARG;
    if (dk > 256 || (dv != 16 && dv != 32 && dv != 64 && dv != 128)) return LLA_ERR_UNSUPPORTED;
    if ((int64_t)B * H > 0x7fffffff) return LLA_ERR_UNSUPPORTED;
    const int dev = current_device();
    if (dev < 0) return LLA_ERR_CUDA;
    int* err = error_word(dev);
    if (!err) return LLA_ERR_CUDA;
    cudaError_t e = lla::decode_step(dtype, q, k, v, log_a, lambda, fenwick_states, t, out, B, H, dk, dv, Lmax, err,
                                     static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? LLA_OK : LLA_ERR_CUDA;
}

int lla_prefill_state(const void* k, const void* v, const float* log_a, float* fenwick_states, int B, int H, int T,
                      int dk, int dv, int Lmax, void* stream, int dtype) {
    if (!k || !v || !log_a || !fenwick_states) return LLA_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(log_a) || !aligned16(fenwick_states)) return LLA_ERR_INVALID_ARG;
    if (dtype != LLA_BF16 && dtype != LLA_F32) return LLA_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || T < 1 || dk < 1 || dv < 1 || Lmax < 1 || Lmax > 40) return LLA_ERR_INVALID_ARG;
    if (lla::bitlength((int64_t)T - 1) + 1 > Lmax) return LLA_ERR_INVALID_ARG;
    if (dk > 128 || dv > 128) return LLA_ERR_UNSUPPORTED;
    if ((int64_t)B * H > 65535 || (int64_t)B * H * T * (dk > dv ? dk : dv) > ((int64_t)1 << 40)) return LLA_ERR_UNSUPPORTED;
    const int dev = current_device();
    if (dev < 0) return LLA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool tc = lla::tc_state_supported(dtype, dk, dv, B, H, T);
    const size_t bytes = tc ? lla::tc_state_workspace_bytes(B, H, T, dv) : (size_t)B * H * T * sizeof(float);
    int* err = error_word(dev);
    if (!err) return LLA_ERR_CUDA;
    cudaMemPool_t pool = workspace_pool(dev);
    if (!pool) return LLA_ERR_CUDA;
    void* ws = nullptr;
    if (cudaMallocFromPoolAsync(&ws, bytes, pool, s) != cudaSuccess) {
        cudaGetLastError();
        return LLA_ERR_NOMEM;
    }
    cudaError_t e = tc ? lla::tc_prefill_state(k, v, log_a, fenwick_states, B, H, T, dv, Lmax, ws, err, s)
                       : lla::prefill_state(dtype, k, v, log_a, fenwick_states, B, H, T, dk, dv, Lmax, ws, err, s);
    const cudaError_t f = cudaFreeAsync(ws, s);
    return (e == cudaSuccess && f == cudaSuccess) ? LLA_OK : LLA_ERR_CUDA;
}

int lla_backward(const void* q, const void* k, const void* v, const float* log_a, const float* lambda,
                 const void* dout, void* dq, void* dk, void* dv, float* dlog_a, float* dlambda, int B, int H, int T,
                 int dk_, int dv_, int chunk, void* stream, int dtype) {
    int st = validate_forward(q, k, v, log_a, lambda, dout, B, H, T, dk_, dv_, chunk, dtype);
    if (st != LLA_OK) return st;
    if (!dq || !dk || !dv || !dlog_a || !dlambda) return LLA_ERR_INVALID_ARG;
    if (!aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(dlog_a) || !aligned16(dlambda))
        return LLA_ERR_INVALID_ARG;
    lla::TcPlan tp;
    lla::BwdPlan bp;
    const bool tc = lla::tc_bwd_supported(dtype, dk_, dv_, T) && lla::make_tc_plan(B, H, T, dk_, dv_, &tp);
    if (!tc && !lla::make_bwd_plan(B, H, T, dk_, dv_, chunk, &bp)) return LLA_ERR_UNSUPPORTED;
    const int dev = current_device();
    if (dev < 0) return LLA_ERR_CUDA;
    int* err = error_word(dev);
    if (!err) return LLA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaMemPool_t pool = workspace_pool(dev);
    if (!pool) return LLA_ERR_CUDA;
    void* ws = nullptr;
    const size_t bytes = tc ? lla::tc_bwd_workspace_bytes(tp) : bp.total_bytes;
    if (cudaMallocFromPoolAsync(&ws, bytes, pool, s) != cudaSuccess) {
        cudaGetLastError();
        return LLA_ERR_NOMEM;
    }
    cudaError_t e = tc ? lla::tc_backward(tp, q, k, v, log_a, lambda, dout, dq, dk, dv, dlog_a, dlambda, ws, err, s)
                       : lla::simt_backward(bp, dtype, q, k, v, log_a, lambda, dout, dq, dk, dv, dlog_a, dlambda, ws,
                                            s);
    const cudaError_t f = cudaFreeAsync(ws, s);
    return (e == cudaSuccess && f == cudaSuccess) ? LLA_OK : LLA_ERR_CUDA;
}

int lla_forward_varlen(const void* q, const void* k, const void* v, const float* log_a, const float* lambda,
                       void* out, const int32_t* cu_seqlens, int n_seq, int H, int total_T, int max_T, int dk, int dv,
                       int chunk, void* stream, int dtype) {
    if (!cu_seqlens || !aligned16(cu_seqlens)) return LLA_ERR_INVALID_ARG;
    if (n_seq < 1 || max_T < 1 || total_T < 1) return LLA_ERR_INVALID_ARG;
    if ((int64_t)n_seq * max_T < total_T) return LLA_ERR_INVALID_ARG;
    const int Tpad = (max_T + 127) / 128 * 128;
    int st = validate_forward(q, k, v, log_a, lambda, out, n_seq, H, Tpad, dk, dv, chunk, dtype);
    if (st != LLA_OK) return st;
    if ((int64_t)H * total_T * (dk > dv ? dk : dv) > ((int64_t)1 << 40)) return LLA_ERR_UNSUPPORTED;
    const int dev = current_device();
    if (dev < 0) return LLA_ERR_CUDA;
    int* err = error_word(dev);
    if (!err) return LLA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaMemPool_t pool = workspace_pool(dev);
    if (!pool) return LLA_ERR_CUDA;
    const int L_in = lla_num_levels(max_T), L_pad = lla_num_levels(Tpad);
    lla::TcPlan tp;
    if (lla::tc_varlen_supported(dtype, dk, dv) && (int64_t)H * total_T < ((int64_t)1 << 31) &&
        lla::make_tc_plan(n_seq, H, Tpad, dk, dv, &tp)) {
        // tensor-core kernels over each sequence's own tiles of the packed layout: no padding
        const size_t tbytes = lla::tc_varlen_table_bytes(n_seq);
        char* ws = nullptr;
        if (cudaMallocFromPoolAsync(reinterpret_cast<void**>(&ws), tp.total_bytes + tbytes, pool, s) != cudaSuccess) {
            cudaGetLastError();
            return LLA_ERR_NOMEM;
        }
        const cudaError_t e = lla::tc_forward_varlen(tp, q, k, v, log_a, lambda, out, cu_seqlens, total_T, max_T,
                                                     L_in, ws, ws + tp.total_bytes, err, s);
        const cudaError_t f = cudaFreeAsync(ws, s);
        return (e == cudaSuccess && f == cudaSuccess) ? LLA_OK : LLA_ERR_CUDA;
    }
    ForwardPlan fp;
    if (!plan_forward(n_seq, H, Tpad, dk, dv, chunk, dtype, &fp)) return LLA_ERR_UNSUPPORTED;
    const int esz = dtype == LLA_BF16 ? 2 : 4;
    const size_t rows = (size_t)n_seq * H * Tpad;
    auto up = [](size_t x) { return (x + 1023) / 1024 * 1024; };
    const size_t bq = up(rows * dk * esz), bv = up(rows * dv * esz), ba = up(rows * 4), bl = up(rows * L_pad * 4);
    const size_t bytes = 2 * bq + 2 * bv + ba + bl + fp.bytes;
    char* ws = nullptr;
    if (cudaMallocFromPoolAsync(reinterpret_cast<void**>(&ws), bytes, pool, s) != cudaSuccess) {
        cudaGetLastError();
        return LLA_ERR_NOMEM;
    }
    char* pq = ws;
    char* pk = pq + bq;
    char* pv = pk + bq;
    char* po = pv + bv;
    float* pa = reinterpret_cast<float*>(po + bv);
    float* pl = reinterpret_cast<float*>(po + bv + ba);
    char* fws = po + bv + ba + bl;
    cudaError_t e = cudaSuccess;
    auto chain = [&](cudaError_t x) {
        if (e == cudaSuccess) e = x;
    };
    chain(lla::varlen_pack(esz, q, pq, cu_seqlens, n_seq, H, total_T, Tpad, dk, dk, max_T, err, s));
    chain(lla::varlen_pack(esz, k, pk, cu_seqlens, n_seq, H, total_T, Tpad, dk, dk, max_T, err, s));
    chain(lla::varlen_pack(esz, v, pv, cu_seqlens, n_seq, H, total_T, Tpad, dv, dv, max_T, err, s));
    chain(lla::varlen_pack(4, log_a, pa, cu_seqlens, n_seq, H, total_T, Tpad, 1, 1, max_T, err, s));
    chain(lla::varlen_pack(4, lambda, pl, cu_seqlens, n_seq, H, total_T, Tpad, L_in, L_pad, max_T, err, s));
    if (e == cudaSuccess && run_forward(fp, pq, pk, pv, pa, pl, po, dtype, fws, err, s) != LLA_OK) e = cudaErrorUnknown;
    chain(lla::varlen_unpack(esz, po, out, cu_seqlens, n_seq, H, total_T, Tpad, dv, max_T, err, s));
    const cudaError_t f = cudaFreeAsync(ws, s);
    return (e == cudaSuccess && f == cudaSuccess) ? LLA_OK : LLA_ERR_CUDA;
}

int lla_prefill_state_varlen(const void* k, const void* v, const float* log_a, const int32_t* cu_seqlens,
                             float* fenwick_states, int n_seq, int H, int total_T, int max_T, int dk, int dv, int Lmax,
                             void* stream, int dtype) {
    if (!k || !v || !log_a || !cu_seqlens || !fenwick_states) return LLA_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(log_a) || !aligned16(cu_seqlens) || !aligned16(fenwick_states))
        return LLA_ERR_INVALID_ARG;
    if (dtype != LLA_BF16 && dtype != LLA_F32) return LLA_ERR_INVALID_ARG;
    if (n_seq < 1 || H < 1 || total_T < 1 || max_T < 1 || dk < 1 || dv < 1 || Lmax < 1 || Lmax > 40)
        return LLA_ERR_INVALID_ARG;
    if ((int64_t)n_seq * max_T < total_T) return LLA_ERR_INVALID_ARG;
    if (lla::bitlength((int64_t)max_T - 1) + 1 > Lmax) return LLA_ERR_INVALID_ARG;
    if (dk > 128 || dv > 128) return LLA_ERR_UNSUPPORTED;
    if ((int64_t)n_seq * H > 65535 || (int64_t)H * total_T * (dk > dv ? dk : dv) > ((int64_t)1 << 40))
        return LLA_ERR_UNSUPPORTED;
    const int dev = current_device();
    if (dev < 0) return LLA_ERR_CUDA;
    int* err = error_word(dev);
    if (!err) return LLA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaMemPool_t pool = workspace_pool(dev);
    if (!pool) return LLA_ERR_CUDA;
    const bool tc = lla::tc_state_supported_packed(dtype, dk, dv, n_seq, H, total_T, max_T);
    const size_t bytes = tc ? lla::tc_state_workspace_bytes(n_seq, H, max_T, dv) : (size_t)H * total_T * sizeof(float);
    void* ws = nullptr;
    if (cudaMallocFromPoolAsync(&ws, bytes, pool, s) != cudaSuccess) {
        cudaGetLastError();
        return LLA_ERR_NOMEM;
    }
    cudaError_t e = tc ? lla::tc_prefill_state(k, v, log_a, fenwick_states, n_seq, H, max_T, dv, Lmax, ws, err, s,
                                               cu_seqlens, total_T)
                       : lla::prefill_state(dtype, k, v, log_a, fenwick_states, n_seq, H, max_T, dk, dv, Lmax, ws,
                                            err, s, cu_seqlens, total_T);
    const cudaError_t f = cudaFreeAsync(ws, s);
    return (e == cudaSuccess && f == cudaSuccess) ? LLA_OK : LLA_ERR_CUDA;
}

int lla_gdn_forward(const void* q, const void* k, const void* v, const float* log_a, const float* beta,
                    const float* lambda, void* out, int B, int H, int T, int dk, int dv, int chunk, void* stream,
                    int dtype) {
    int st = validate_forward(q, k, v, log_a, lambda, out, B, H, T, dk, dv, chunk, dtype);
    if (st != LLA_OK) return st;
    if (!beta || !aligned16(beta)) return LLA_ERR_INVALID_ARG;
    lla::GdnPlan pl;
    if (dv % 16 != 0 || !lla::make_gdn_plan(B, H, T, dk, dv, chunk, &pl)) return LLA_ERR_UNSUPPORTED;
    const int dev = current_device();
    if (dev < 0) return LLA_ERR_CUDA;
    int* err = error_word(dev);
    if (!err) return LLA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaMemPool_t pool = workspace_pool(dev);
    if (!pool) return LLA_ERR_CUDA;
    void* ws = nullptr;
    if (cudaMallocFromPoolAsync(&ws, pl.total_bytes, pool, s) != cudaSuccess) {
        cudaGetLastError();
        return LLA_ERR_NOMEM;
    }
    const cudaError_t e = lla::gdn_forward(pl, dtype, q, k, v, log_a, beta, lambda, out, ws, err, s);
    const cudaError_t f = cudaFreeAsync(ws, s);
    return (e == cudaSuccess && f == cudaSuccess) ? LLA_OK : LLA_ERR_CUDA;
}

int lla_gdn_decode_step(const void* q, const void* k, const void* v, const float* log_a, const float* beta,
                        const float* lambda, float* fenwick_states, const int64_t* t, void* out, void* stream, int B,
                        int H, int dk, int dv, int Lmax, int dtype) {
    if (!q || !k || !v || !log_a || !beta || !lambda || !fenwick_states || !t || !out) return LLA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(log_a) || !aligned16(beta) ||
        !aligned16(lambda) || !aligned16(fenwick_states) || !aligned16(t) || !aligned16(out))
        return LLA_ERR_INVALID_ARG;
    if (dtype != LLA_BF16 && dtype != LLA_F32) return LLA_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || dk < 1 || dv < 1 || Lmax < 1 || Lmax > 40) return LLA_ERR_INVALID_ARG;
    if ((dk != 16 && dk != 32 && dk != 64 && dk != 128) || (dv != 16 && dv != 32 && dv != 64 && dv != 128))
        return LLA_ERR_UNSUPPORTED;
    if ((int64_t)B * H > 0x7fffffff) return LLA_ERR_UNSUPPORTED;
    const int dev = current_device();
    if (dev < 0) return LLA_ERR_CUDA;
    int* err = error_word(dev);
    if (!err) return LLA_ERR_CUDA;
    cudaError_t e = lla::gdn_decode_step(dtype, q, k, v, log_a, beta, lambda, fenwick_states, t, out, B, H, dk, dv,
                                         Lmax, err, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? LLA_OK : LLA_ERR_CUDA;
}

int lla_debug_set_waits(int64_t limit_cycles, int hold) {
    if (current_device() < 0) return LLA_ERR_CUDA;
    lla::linear_set_waits({static_cast<long long>(limit_cycles), hold != 0});
    return lla::tc_set_debug_waits(static_cast<long long>(limit_cycles), hold) == cudaSuccess ? LLA_OK : LLA_ERR_CUDA;
}

int lla_device_error(void* stream) {
    const int dev = current_device();
    if (dev < 0) return LLA_ERR_CUDA;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return LLA_ERR_CUDA;
    int word = 0;
    if (cudaMemcpyFromSymbol(&word, lla_device_error_word, sizeof(int)) != cudaSuccess) return LLA_ERR_CUDA;
    const int zero = 0;
    if (cudaMemcpyToSymbol(lla_device_error_word, &zero, sizeof(int)) != cudaSuccess) return LLA_ERR_CUDA;
    if (word == lla::kDevBadInput) return LLA_ERR_DEVICE;
    if (word == lla::kDevTimeout) return LLA_ERR_TIMEOUT;
    return word == 0 ? LLA_OK : LLA_ERR_DEVICE;
}

}  // extern "C"

// ---- linear attention with one decay per head

namespace {

// One argument's bytes (p null: not given).
struct Span {
    const void* p;
    size_t bytes;
};

bool overlap(const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && x < y + b.bytes && y < x + a.bytes;
}

// Whether a written argument overlaps one that is read, or another written one.
bool clash(std::initializer_list<Span> written, std::initializer_list<Span> read) {
    for (const Span* w = written.begin(); w != written.end(); w++) {
        for (const Span& r : read)
            if (overlap(*w, r)) return true;
        for (const Span* o = written.begin(); o != w; o++)
            if (overlap(*w, *o)) return true;
    }
    return false;
}

size_t type_bytes(int dtype) { return dtype == LLA_BF16 ? 2 : 4; }

// Checks shared by the linear prefill, packed prefill and backward: `rows` = rows of one head,
// batch = sequences, b0 = entering states.
int validate_linear(const void* q, const void* k, const void* v, const float* log_a, const float* state0, int batch,
                    int b0, int H, int64_t rows, int T, int dk, int dv, int dtype) {
    if (!q || !k || !v || !log_a) return LLA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(log_a) || !aligned16(state0))
        return LLA_ERR_INVALID_ARG;
    if (dtype != LLA_BF16 && dtype != LLA_F32) return LLA_ERR_INVALID_ARG;
    if (batch < 1 || H < 1 || T < 1 || dk < 1 || dv < 1) return LLA_ERR_INVALID_ARG;
    if ((b0 != 0 && b0 != 1 && b0 != batch) || (b0 == 0) != (state0 == nullptr)) return LLA_ERR_INVALID_ARG;
    if (dk > 128 || dv > 128) return LLA_ERR_UNSUPPORTED;
    if ((int64_t)batch * H > 65535) return LLA_ERR_UNSUPPORTED;
    if (H * rows * (dk > dv ? dk : dv) > ((int64_t)1 << 40)) return LLA_ERR_UNSUPPORTED;
    if (rows / 64 + batch > 0x7fffffff) return LLA_ERR_UNSUPPORTED;  // 64-token chunks of a head are counted in an int
    return LLA_OK;
}

struct PoolBuffer {  // workspace from the library pool on one stream, returned there
    cudaStream_t s;
    char* p = nullptr;
    explicit PoolBuffer(cudaStream_t stream) : s(stream) {}
    int take(int dev, size_t bytes) {
        if (bytes == 0) return LLA_OK;
        cudaMemPool_t pool = workspace_pool(dev);
        if (!pool) return LLA_ERR_CUDA;
        if (cudaMallocFromPoolAsync(reinterpret_cast<void**>(&p), bytes, pool, s) != cudaSuccess) {
            cudaGetLastError();
            return LLA_ERR_NOMEM;
        }
        return LLA_OK;
    }
    int give(cudaError_t e) {
        const cudaError_t f = p ? cudaFreeAsync(p, s) : cudaSuccess;
        if (e != cudaSuccess || f != cudaSuccess) cudaGetLastError();  // reported here, not by the next call
        return (e == cudaSuccess && f == cudaSuccess) ? LLA_OK : LLA_ERR_CUDA;
    }
};

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

lla::LinSeqs dense_seqs(int B, int H, int T) {
    lla::LinSeqs sq = {};
    sq.T = T;
    sq.H = sq.state_heads = H;
    sq.N = (T - 1) / 64 + 1;
    sq.n_chunks = B * sq.N;
    return sq;
}

int pieces64(int d) { return (d + 63) / 64; }

// The CUDA-core path keeps the state of every 64-token chunk of the heads that it runs together: as many heads as stay
// within kMostStates bytes (at least one), so that a long prompt of many heads does not take all its states at once. 1 GiB
// is 16384 states of 128 x 128, 100 times what fills the GPU.
constexpr size_t kMostStates = size_t(1) << 30;
struct HeadGroups {
    int nb, nh;  // sequences and heads of a group: whole sequences, or some heads of one
};
HeadGroups head_groups(int B, int H, size_t head_bytes) {
    const size_t most = kMostStates / head_bytes;
    const size_t b = most / H;
    if (b >= 1) return {b < static_cast<size_t>(B) ? static_cast<int>(b) : B, H};
    return {1, most > 1 ? static_cast<int>(most) : 1};
}

const void* further(const void* p, size_t bytes) { return static_cast<const char*>(p) + bytes; }
void* further(void* p, size_t bytes) { return static_cast<char*>(p) + bytes; }
const float* states_at(const float* p, size_t n) { return p ? p + n : nullptr; }
float* states_at(float* p, size_t n) { return p ? p + n : nullptr; }

}  // namespace

extern "C" {

int lla_linear_forward(const void* q, const void* k, const void* v, const float* log_a, const float* state0, void* out,
                       float* state_out, int B, int B0, int H, int T, int dk, int dv, void* stream, int dtype) {
    int st = validate_linear(q, k, v, log_a, state0, B, B0, H, (int64_t)B * T, T, dk, dv, dtype);
    if (st != LLA_OK) return st;
    if (!out || !aligned16(out) || !aligned16(state_out)) return LLA_ERR_INVALID_ARG;
    const size_t msz = (size_t)dk * dv * sizeof(float);
    const size_t heads = (size_t)B * H, row = heads * T * type_bytes(dtype);
    if (clash({{out, row * dv}, {state_out, heads * msz}},
              {{q, row * dk}, {k, row * dk}, {v, row * dv}, {log_a, H * sizeof(float)}, {state0, B0 * H * msz}}))
        return LLA_ERR_INVALID_ARG;
    const int dev = current_device();
    if (dev < 0) return LLA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int* err = error_word(dev);
    if (!err) return LLA_ERR_CUDA;
    const lla::LinSeqs sq = dense_seqs(B, H, T);
    PoolBuffer ws(s);
    lla::LinTcPlan tp;
    if (lla::linear_tc_supported(dtype, dk, dv) && lla::linear_tc_plan(&tp, B, H, T, (int64_t)B * H * T, pieces64(dv), false)) {
        if ((st = ws.take(dev, tp.seg_bytes)) != LLA_OK) return st;
        const lla::LinTcMap maps[3] = {{q, dk}, {k, dk}, {v, dv}};
        const lla::LinTcScan scan = {0, 1, 2, out, state0, state_out, B0 == 1, 0, dk, dv, pieces64(dv), 0, 0};
        return ws.give(lla::linear_tc_run(tp, maps, 3, &scan, 1, sq, log_a, reinterpret_cast<float*>(ws.p), nullptr,
                                          err, s));
    }
    const HeadGroups gr = head_groups(B, H, sq.N * msz);
    if ((st = ws.take(dev, (size_t)gr.nb * gr.nh * sq.N * msz)) != LLA_OK) return st;
    float* states = reinterpret_cast<float*>(ws.p);
    const size_t ek = (size_t)T * dk * type_bytes(dtype), ev = (size_t)T * dv * type_bytes(dtype), ms = (size_t)dk * dv;
    cudaError_t e = cudaSuccess;
    for (int b = 0; b < B && e == cudaSuccess; b += gr.nb)
        for (int h = 0; h < H && e == cudaSuccess; h += gr.nh) {
            const int nb = B - b < gr.nb ? B - b : gr.nb, nh = H - h < gr.nh ? H - h : gr.nh;
            const size_t at = (size_t)b * H + h;
            const void *kg = further(k, at * ek), *vg = further(v, at * ev);
            lla::LinStateJobs jobs = {{{kg, vg, states, states_at(state0, (B0 == 1 ? h : at) * ms),
                                        states_at(state_out, at * ms), B0 == 1, 0, dk, dv, pieces64(dk) * pieces64(dv)}},
                                      1};
            lla::LinScans scans = {{{further(q, at * ek), kg, vg, further(out, at * ev), states, 0, 0, dk, dv}}, 1};
            e = lla::linear_run(dtype, jobs, scans, dense_seqs(nb, nh, T), log_a + h, s);
        }
    return ws.give(e);
}

int lla_linear_forward_varlen(const void* q, const void* k, const void* v, const float* log_a, const float* state0,
                              void* out, float* state_out, const int32_t* cu_seqlens, int n_seq, int n0, int H,
                              int total_T, int max_T, int dk, int dv, void* stream, int dtype) {
    if (!cu_seqlens || !aligned16(cu_seqlens) || total_T < 1) return LLA_ERR_INVALID_ARG;
    // a bound above the rows that there are (a server's longest context, say) bounds nothing more: it must not count in the
    // plan, nor turn a call away
    const int longest = max_T < total_T ? max_T : total_T;
    int st = validate_linear(q, k, v, log_a, state0, n_seq, n0, H, total_T, longest, dk, dv, dtype);
    if (st != LLA_OK) return st;
    if (!out || !aligned16(out) || !aligned16(state_out)) return LLA_ERR_INVALID_ARG;
    const size_t msz = (size_t)dk * dv * sizeof(float);
    const size_t row = (size_t)H * total_T * type_bytes(dtype);
    if (clash({{out, row * dv}, {state_out, n_seq * H * msz}},
              {{q, row * dk}, {k, row * dk}, {v, row * dv}, {log_a, H * sizeof(float)}, {state0, n0 * H * msz},
               {cu_seqlens, ((size_t)n_seq + 1) * sizeof(int32_t)}}))
        return LLA_ERR_INVALID_ARG;
    const int dev = current_device();
    if (dev < 0) return LLA_ERR_CUDA;
    int* err = error_word(dev);
    if (!err) return LLA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    lla::LinSeqs sq = {};
    sq.n = n_seq;
    sq.T = longest;
    sq.H = sq.state_heads = H;
    sq.total = total_T;
    sq.n_chunks = total_T / 64 + n_seq;
    const size_t tab_b = up256((size_t)n_seq * sizeof(int2)), off_b = up256(((size_t)n_seq + 1) * sizeof(int));
    PoolBuffer ws(s);
    lla::LinTcPlan tp;
    if (lla::linear_tc_supported(dtype, dk, dv) &&
        lla::linear_tc_plan(&tp, n_seq, H, longest, (int64_t)H * total_T, pieces64(dv), false)) {
        if ((st = ws.take(dev, tab_b + 2 * off_b + tp.seg_bytes)) != LLA_OK) return st;
        int2* tab = reinterpret_cast<int2*>(ws.p);
        int* coff = reinterpret_cast<int*>(ws.p + tab_b);
        int* order = reinterpret_cast<int*>(ws.p + tab_b + off_b);
        sq.tab = tab;
        sq.coff = coff;
        sq.order = order;
        cudaError_t e = lla::linear_table(cu_seqlens, n_seq, total_T, longest, tab, coff, order, err, s);
        const lla::LinTcMap maps[3] = {{q, dk}, {k, dk}, {v, dv}};
        const lla::LinTcScan scan = {0, 1, 2, out, state0, state_out, n0 == 1, 0, dk, dv, pieces64(dv), 0, 0};
        if (e == cudaSuccess)
            e = lla::linear_tc_run(tp, maps, 3, &scan, 1, sq, log_a,
                                   reinterpret_cast<float*>(ws.p + tab_b + 2 * off_b), nullptr, err, s);
        return ws.give(e);
    }
    const int group = head_groups(1, H, sq.n_chunks * msz).nh;
    if ((st = ws.take(dev, tab_b + off_b + (size_t)group * sq.n_chunks * msz)) != LLA_OK) return st;
    int2* tab = reinterpret_cast<int2*>(ws.p);
    int* coff = reinterpret_cast<int*>(ws.p + tab_b);
    float* states = reinterpret_cast<float*>(ws.p + tab_b + off_b);
    sq.tab = tab;
    sq.coff = coff;
    cudaError_t e = lla::linear_table(cu_seqlens, n_seq, total_T, longest, tab, coff, nullptr, err, s);
    const size_t ek = (size_t)total_T * dk * type_bytes(dtype), ev = (size_t)total_T * dv * type_bytes(dtype);
    for (int h = 0; h < H && e == cudaSuccess; h += group) {
        const void *kg = further(k, h * ek), *vg = further(v, h * ev);
        const size_t at = (size_t)h * dk * dv;
        sq.H = H - h < group ? H - h : group;
        lla::LinStateJobs jobs = {{{kg, vg, states, states_at(state0, at), states_at(state_out, at), n0 == 1, 0, dk, dv,
                                    pieces64(dk) * pieces64(dv)}},
                                  1};
        lla::LinScans scans = {{{further(q, h * ek), kg, vg, further(out, h * ev), states, 0, 0, dk, dv}}, 1};
        e = lla::linear_run(dtype, jobs, scans, sq, log_a + h, s);
    }
    return ws.give(e);
}

int lla_linear_backward(const void* q, const void* k, const void* v, const float* log_a, const float* state0,
                        const void* dout, const float* dstate_out, void* dq, void* dk, void* dv, float* dstate0, int B,
                        int B0, int H, int T, int dk_, int dv_, void* stream, int dtype) {
    int st = validate_linear(q, k, v, log_a, state0, B, B0, H, (int64_t)B * T, T, dk_, dv_, dtype);
    if (st != LLA_OK) return st;
    if (!dout || !dq || !dk || !dv || !aligned16(dout) || !aligned16(dstate_out) || !aligned16(dq) || !aligned16(dk) ||
        !aligned16(dv) || !aligned16(dstate0))
        return LLA_ERR_INVALID_ARG;
    if (dstate0 && B0 == 0) return LLA_ERR_INVALID_ARG;
    const size_t msz = (size_t)dk_ * dv_ * sizeof(float);
    const size_t heads = (size_t)B * H, row = heads * T * type_bytes(dtype);
    if (clash({{dq, row * dk_}, {dk, row * dk_}, {dv, row * dv_}, {dstate0, B0 * H * msz}},
              {{q, row * dk_}, {k, row * dk_}, {v, row * dv_}, {dout, row * dv_}, {log_a, H * sizeof(float)},
               {state0, B0 * H * msz}, {dstate_out, heads * msz}}))
        return LLA_ERR_INVALID_ARG;
    const int dev = current_device();
    if (dev < 0) return LLA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const lla::LinSeqs sq = dense_seqs(B, H, T);
    int* err = error_word(dev);
    if (!err) return LLA_ERR_CUDA;
    const bool sum = dstate0 && B0 == 1 && B > 1;  // gradients of one shared state: a part per sequence, then their sum
    const size_t sum_b = sum ? up256((size_t)B * H * msz) : 0;
    PoolBuffer ws(s);
    lla::LinTcPlan tp;
    if (lla::linear_tc_supported(dtype, dk_, dv_) &&
        lla::linear_tc_plan(&tp, B, H, T, (int64_t)B * H * T, 2 * pieces64(dv_), true)) {
        const size_t seg_b = up256(tp.seg_bytes);
        if ((st = ws.take(dev, sum_b + seg_b + lla::linear_grad_state_bytes(B * H, T, dv_))) != LLA_OK) return st;
        float* parts = reinterpret_cast<float*>(ws.p);
        void* states = ws.p + sum_b + seg_b;
        const int tiles = pieces64(dv_), chunks = (T - 1) / 128 + 1;
        const lla::LinTcMap maps[4] = {{q, dk_}, {k, dk_}, {v, dv_}, {dout, dv_}};
        const lla::LinTcScan scans[2] = {
            {0, 1, 2, nullptr, state0, nullptr, B0 == 1, 0, dk_, dv_, tiles, 0, 0},
            {0, 0, 3, nullptr, dstate_out, sum ? parts : dstate0, 0, 1, dk_, dv_, tiles, B * H * chunks, 0}};
        cudaError_t e = lla::linear_tc_run(tp, maps, 4, scans, 2, sq, log_a, reinterpret_cast<float*>(ws.p + sum_b),
                                           states, err, s);
        if (e == cudaSuccess)
            e = lla::linear_tc_grads(q, k, v, dout, log_a, states, dq, dk, dv, B * H, H, T, dk_, dv_, err, s);
        if (e == cudaSuccess && sum) e = lla::linear_sum_batch(parts, dstate0, B, (int64_t)H * dk_ * dv_, s);
        return ws.give(e);
    }
    const HeadGroups gr = head_groups(B, H, 2 * sq.N * msz);
    const size_t st_b = up256((size_t)gr.nb * gr.nh * sq.N * msz);
    if ((st = ws.take(dev, 2 * st_b + (sum ? (size_t)B * H * msz : 0))) != LLA_OK) return st;
    float* fw = reinterpret_cast<float*>(ws.p);
    float* bw = reinterpret_cast<float*>(ws.p + st_b);
    float* parts = reinterpret_cast<float*>(ws.p + 2 * st_b);
    const int sp = pieces64(dk_) * pieces64(dv_);
    const size_t ek = (size_t)T * dk_ * type_bytes(dtype), ev = (size_t)T * dv_ * type_bytes(dtype),
                 ms = (size_t)dk_ * dv_;
    cudaError_t e = cudaSuccess;
    for (int b = 0; b < B && e == cudaSuccess; b += gr.nb)
        for (int h = 0; h < H && e == cudaSuccess; h += gr.nh) {
            const int nb = B - b < gr.nb ? B - b : gr.nb, nh = H - h < gr.nh ? H - h : gr.nh;
            const size_t at = (size_t)b * H + h;
            const void *qg = further(q, at * ek), *kg = further(k, at * ek), *vg = further(v, at * ev),
                       *og = further(dout, at * ev);
            lla::LinStateJobs jobs = {{{kg, vg, fw, states_at(state0, (B0 == 1 ? h : at) * ms), nullptr, B0 == 1, 0, dk_,
                                        dv_, sp},
                                       {qg, og, bw, states_at(dstate_out, at * ms),
                                        states_at(sum ? parts : dstate0, at * ms), 0, 1, dk_, dv_, sp}},
                                      2};
            lla::LinScans scans = {{{og, vg, kg, further(dq, at * ek), fw, 1, 0, dv_, dk_},
                                    {vg, og, qg, further(dk, at * ek), bw, 1, 1, dv_, dk_},
                                    {kg, qg, og, further(dv, at * ev), bw, 0, 1, dk_, dv_}},
                                   3};
            e = lla::linear_run(dtype, jobs, scans, dense_seqs(nb, nh, T), log_a + h, s);
        }
    if (e == cudaSuccess && sum) e = lla::linear_sum_batch(parts, dstate0, B, (int64_t)H * dk_ * dv_, s);
    return ws.give(e);
}

int lla_linear_decode_step(const void* q, const void* k, const void* v, const float* log_a, float* state, void* out,
                           void* stream, int B, int H, int dk, int dv, int dtype) {
    if (!q || !k || !v || !log_a || !state || !out) return LLA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(log_a) || !aligned16(state) || !aligned16(out))
        return LLA_ERR_INVALID_ARG;
    if (dtype != LLA_BF16 && dtype != LLA_F32) return LLA_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || dk < 1 || dv < 1) return LLA_ERR_INVALID_ARG;
    if (dk > 128 || dv > 128) return LLA_ERR_UNSUPPORTED;
    if ((int64_t)B * H > 0x7fffffff) return LLA_ERR_UNSUPPORTED;
    const size_t heads = (size_t)B * H, row = heads * type_bytes(dtype);
    if (clash({{out, row * dv}, {state, heads * dk * dv * sizeof(float)}},
              {{q, row * dk}, {k, row * dk}, {v, row * dv}, {log_a, H * sizeof(float)}}))
        return LLA_ERR_INVALID_ARG;
    if (current_device() < 0) return LLA_ERR_CUDA;
    return lla::linear_decode_step(dtype, q, k, v, log_a, state, out, B, H, dk, dv,
                                   static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? LLA_OK
               : LLA_ERR_CUDA;
}

int lla_decode_step_shared(const void* q, const void* k, const void* v, const float* log_a, const float* lambda,
                           const float* prefix_states, int64_t prefix_len, int Lp, float* prefix_decay,
                           float* fenwick_states, const int64_t* t, void* out, void* stream, int B, int H, int dk,
                           int dv, int Lmax, int dtype) {
    if (!q || !k || !v || !log_a || !lambda || !prefix_states || !prefix_decay || !fenwick_states || !t || !out)
        return LLA_ERR_INVALID_ARG;
    for (const void* p : {q, k, v, static_cast<const void*>(log_a), static_cast<const void*>(lambda),
                          static_cast<const void*>(prefix_states), static_cast<const void*>(prefix_decay),
                          static_cast<const void*>(fenwick_states), static_cast<const void*>(t),
                          static_cast<const void*>(out)})
        if (!aligned16(p)) return LLA_ERR_INVALID_ARG;
    if (dtype != LLA_BF16 && dtype != LLA_F32) return LLA_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || dk < 1 || dv < 1 || Lmax < 1 || Lmax > 40 || Lp < 1 || Lp > 40) return LLA_ERR_INVALID_ARG;
    if (prefix_len < 1 || prefix_len >= ((int64_t)1 << (Lmax - 1)) || lla_num_levels(prefix_len) > Lp)
        return LLA_ERR_INVALID_ARG;
    if (dk > 256 || (dv != 16 && dv != 32 && dv != 64 && dv != 128)) return LLA_ERR_UNSUPPORTED;
    if ((int64_t)B * H > 0x7fffffff || H > 65535 || B > 65535) return LLA_ERR_UNSUPPORTED;
    const size_t heads = (size_t)B * H, row = heads * type_bytes(dtype), msz = (size_t)dk * dv * sizeof(float);
    if (clash({{out, row * dv}, {fenwick_states, heads * Lmax * msz}, {prefix_decay, heads * sizeof(float)}},
              {{q, row * dk}, {k, row * dk}, {v, row * dv}, {log_a, heads * sizeof(float)},
               {lambda, heads * Lmax * sizeof(float)}, {prefix_states, (size_t)H * Lp * msz},
               {t, B * sizeof(int64_t)}}))
        return LLA_ERR_INVALID_ARG;
    const int dev = current_device();
    if (dev < 0) return LLA_ERR_CUDA;
    int* err = error_word(dev);
    if (!err) return LLA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    PoolBuffer ws(s);
    const int st = ws.take(dev, lla::shared_workspace_bytes(B, H, dv, prefix_len));
    if (st != LLA_OK) return st;
    return ws.give(lla::decode_step_shared(dtype, q, k, v, log_a, lambda, prefix_states, prefix_len, Lp, prefix_decay,
                                           fenwick_states, t, out, ws.p, B, H, dk, dv, Lmax, err, s));
}

}  // extern "C"
