// Shared by the host API and the kernels of linear attention with one decay per head
// (lla_linear.cu: CUDA cores, lla_linear_tc.cu: tensor cores) and of the log-linear decode step
// over a shared prefix (lla_shared.cu).
#pragma once

#include "lla_internal.cuh"

namespace lla {

namespace {
// g^n for n >= 0
__device__ __forceinline__ float gpow(float la, int n) { return n == 0 ? 1.f : expf(la * static_cast<float>(n)); }

// Two fp32 values in one register pair: one instruction for both (issue slots bound these kernels).
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 split2(f32x2 x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
}  // namespace

// The sequences of one call. Dense (tab == nullptr): B sequences of T rows, sequence b of head h
// at row (b H + h) T. Packed: n sequences, sequence b of head h has tab[b].y rows from row
// h total + tab[b].x (y = -1: rejected, nothing of it is read or written).
struct LinSeqs {
    const int2* tab;
    const int* coff;   // packed: 64-token chunks before sequence b, [n + 1]
    const int* order;  // packed: sequences by falling length
    int n, T, H, total;
    int N;             // dense: 64-token chunks of a sequence
    int n_chunks;      // 64-token chunks of one head (packed: at most)
    int state_heads;   // heads of the states that enter and leave (packed: H may be a part of them)
};

// A chunk-state job of the CUDA-core path: states [H][n_chunks][d1][d2] of sum w b c^T.
struct LinStateJob {
    const void *b, *c;
    float* states;
    const float* in;  // entering state [batch or 1][H][d1][d2], or null for zeros
    float* out;       // leaving state [batch][H][d1][d2], or null
    int in_shared, reverse, d1, d2, pieces;
};
struct LinStateJobs {
    LinStateJob job[2];
    int count;
};

// A scan of the CUDA-core path (see lla_linear.cu); states as its job leaves them, read as
// [d1][d2], or transposed from [d2][d1].
struct LinScan {
    const void *a, *b, *c;
    void* out;
    const float* states;
    int state_t, reverse, d1, d2;
};
struct LinScans {
    LinScan scan[3];
    int count;
};

cudaError_t linear_run(int dtype, const LinStateJobs& jobs, const LinScans& scans, const LinSeqs& sq,
                       const float* log_a, cudaStream_t stream);
cudaError_t linear_table(const int32_t* cu, int n, int total, int max_T, int2* tab, int* coff, int* order, int* err,
                         cudaStream_t stream);
cudaError_t linear_sum_batch(const float* src, float* dst, int B, int64_t size, cudaStream_t stream);
cudaError_t linear_decode_step(int dtype, const void* q, const void* k, const void* v, const float* log_a,
                               float* state, void* out, int B, int H, int dk, int dv, cudaStream_t stream);

// Tensor-core path (lla_linear_tc.cu): bf16, dk and dv multiples of 8. A scan names its row tensors
// by their index among the call's tensor maps.
struct LinTcMap {
    const void* base;
    int cols;
};
struct LinTcScan {
    int ia, ib, ic;
    void* out;
    const float* in;  // entering state [batch or 1][H][d1][d2], or null for zeros
    float* leave;     // leaving state [batch][H][d1][d2], or null
    int in_shared, reverse, d1, d2;
    int tiles;        // 64-column tiles of c
    int states_base;  // first (b, h, chunk) of this scan in `states`
    int seg_base;     // filled by linear_tc_run
};
struct LinTcPlan {
    int batch;
    int nseg, seg_chunks;      // segments of a sequence, 128-token chunks of a segment
    int npiece, piece_chunks;  // pieces of all segments but the last, whose own states are formed first
    size_t seg_bytes;
};
bool linear_tc_supported(int dtype, int dk, int dv);
// Failure-path test hooks of the tensor-core kernels on the current device, for launches from here on: the bound of their
// pipeline waits in SM cycles (<= 0: the default) and a wait that nothing completes.
struct LinWaits {
    long long cycles;
    int hold;
};
void linear_set_waits(LinWaits waits);
LinWaits linear_waits();
// rows: token rows of the call; tiles: 64-column tiles over all scans of one head; states: only the states are formed
bool linear_tc_plan(LinTcPlan* plan, int batch, int H, int T, int64_t rows, int tiles, bool states);
// One forward scan (states null), or up to two of either direction (dense) that leave the state entering each
// chunk, bf16 [scan][b, h][chunk][tile][128][64], in `states`.
cudaError_t linear_tc_run(const LinTcPlan& plan, const LinTcMap* maps, int n_maps, const LinTcScan* scans, int count,
                          const LinSeqs& sq, const float* log_a, float* seg, void* states, int* err,
                          cudaStream_t stream);
// Gradients from the states entering each chunk (lla_linear_grad.cu): fw of k, v forwards and bw of q, dout backwards,
// both as linear_tc_run leaves them, in one buffer.
size_t linear_grad_state_bytes(int BH, int T, int dv);
cudaError_t linear_tc_grads(const void* q, const void* k, const void* v, const void* dout, const float* log_a,
                            const void* states, void* dq, void* dk, void* dv, int BH, int H, int T, int d_k, int d_v,
                            int* err, cudaStream_t stream);

size_t shared_workspace_bytes(int B, int H, int dv, int64_t prefix_len);
cudaError_t decode_step_shared(int dtype, const void* q, const void* k, const void* v, const float* log_a,
                               const float* lambda, const float* prefix_states, int64_t prefix_len, int Lp,
                               float* prefix_decay, float* states, const int64_t* t, void* out, void* workspace,
                               int B, int H, int dk, int dv, int Lmax, int* err, cudaStream_t stream);

}  // namespace lla
