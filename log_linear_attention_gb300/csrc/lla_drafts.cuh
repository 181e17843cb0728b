// Shared by the host API and the kernels of the gated recurrence (lla_gated.cu) and of trees of
// drafted tokens over recurrent states (lla_tree.cu).
#pragma once

#include <atomic>

#include "lla_internal.cuh"

namespace lla {

// A pass of the gated recurrence over rows [batch][T][D], or [T][D] with cu (packed, batch = 1). Types: dtype and
// gate_dtype are 0 (bf16) or 1 (fp32).
struct GatedPass {
    const void* log_a;
    const void* x;       // forward: the inputs; backward: the forward's outputs
    const void* dout;    // backward
    void* out;           // forward: the outputs; backward: dx
    void* dlog_a;        // backward
    const float* state0;      // [n0][D], or null (n0 = 0)
    const float* dstate_out;  // backward: [n][D], or null for zeros
    float* leave;             // forward: state_out; backward: dstate0 of every sequence; [n][D], or null
    const int32_t* cu;        // packed: [n + 1]
    int n, n0;                // sequences; entering states: 0, 1 or n
    int T, D;                 // rows of a sequence (packed: of all); channels
};
cudaError_t gated_run(const GatedPass& p, bool backward, int dtype, int gate_dtype, int* err, cudaStream_t stream);
// The gradient of one shared state: out [D] from the sequences' parts [n][D] (GatedPass::leave), in order.
cudaError_t gated_sum_shared(const float* parts, float* out, const int32_t* cu, int n, int T, int D, cudaStream_t stream);
cudaError_t gated_decode_step(int dtype, int gate_dtype, const void* x, const void* log_a, float* state, void* out,
                              int64_t size, cudaStream_t stream);
cudaError_t gated_decode_tree(int dtype, int gate_dtype, const void* x, const void* log_a, const float* state,
                              const int32_t* parent, void* out, int B, int BP, int N, int D, int* err,
                              cudaStream_t stream);
cudaError_t gated_decode_commit(int dtype, int gate_dtype, const void* x, const void* log_a, float* state,
                                const int32_t* count, const int32_t* path, int B, int N, int M, int D, int* err,
                                cudaStream_t stream);

// Trees of drafted tokens. t null: linear attention (log_a [H], one state a head, Lmax = 1, lambda unused).
constexpr int kMaxTree = 128;  // nodes of a tree, and accepted tokens of a commit
struct TreeCall {
    const void *q, *k, *v;
    const float *log_a, *lambda, *states;
    const int64_t* t;
    const int32_t* parent;
    void* out;
    int B, BP, H, N, dk, dv, Lmax;
    int* err;
};
cudaError_t decode_tree(int dtype, const TreeCall& c, cudaStream_t stream);
struct CommitCall {
    const void *k, *v;
    const float* log_a;
    float* states;
    const int64_t* t;
    const int32_t *count, *path;  // path null: tokens 0 .. count - 1
    int B, H, N, M, dk, dv, Lmax;
    int* err;
};
cudaError_t decode_commit(int dtype, const CommitCall& c, cudaStream_t stream);

namespace {
// Allows the kernel `bytes` of dynamic shared memory on the current device, once for each (asking costs about a microsecond).
template <typename Kernel>
cudaError_t allow_shared(Kernel* kern, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}
}  // namespace

}  // namespace lla
