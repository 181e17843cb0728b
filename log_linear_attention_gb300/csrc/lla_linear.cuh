// Shared by the host API and the kernels of linear attention with one decay per head
// (lla_linear.cu: CUDA cores, lla_linear_tc.cu: tensor cores) and of the log-linear decode step
// over a shared prefix (lla_shared.cu).
#pragma once

#include "lla_internal.cuh"

namespace lla {

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
    int state_t, reverse, d1, d2, pieces;
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

size_t shared_workspace_bytes(int B, int H, int dv, int64_t prefix_len);
cudaError_t decode_step_shared(int dtype, const void* q, const void* k, const void* v, const float* log_a,
                               const float* lambda, const float* prefix_states, int64_t prefix_len, int Lp,
                               float* prefix_decay, float* states, const int64_t* t, void* out, void* workspace,
                               int B, int H, int dk, int dv, int Lmax, int* err, cudaStream_t stream);

}  // namespace lla
