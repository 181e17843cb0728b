// Linear attention with one decay per head, on CUDA cores in fp32: every shape and dtype the
// tensor-core scan (lla_linear_tc.cu) does not take, the decode step, and the packed-sequence
// table both use.
//
//     S_t = g S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t,   g = exp(log_a_h),  S_{-1} = state0
//
// A "scan" is this operator over three row tensors: a (query side), b (key side), c (value side).
// The gradients are scans too. With R_t = q_t dO_t^T + g R_{t+1} (the adjoint of S_t; past the
// last token g R_T stands for dstate_out):
//     dq_t = S_t dO_t    = scan(a = dO, b = v,  c = k)  forwards,   state S^T
//     dk_t = R_t v_t     = scan(a = v,  b = dO, c = q)  backwards,  state R^T
//     dv_t = R_t^T k_t   = scan(a = k,  b = q,  c = dO) backwards,  state R
//     dstate0 = g R_0.
//
// Chunks of 64 tokens, three kernels, each parallel over chunks or state elements:
//   lin_chunk_state : a chunk's own state, sum_i w_i b_i c_i^T (forwards w_i = g^(n-1-i),
//                     backwards w_i = g^(i+1); n = valid rows of the chunk)
//   lin_carry       : entering state of every chunk, in place of its own state:
//                     X <- g^n X + own, and the state that leaves the last chunk
//   lin_out         : out_i = sum_j M_ij (a_i . b_j) c_j + f_i X^T a_i, M_ij = g^|i-j| on the
//                     causal side, f_i = g^(i+1) forwards, g^(n-1-i) backwards.
// All products are 64 x 64 register-tiled fp32 products out of shared memory. No exponent is ever
// negative, so no factor overflows for g <= 1; g^0 is 1 also for g = 0 (log_a = -inf).
#include "lla_internal.cuh"
#include "lla_linear.cuh"

namespace lla {
namespace {

constexpr int kC = 64;         // tokens per chunk
constexpr int kThreads = 256;  // 16 x 16 threads, each a 4 x 4 piece of a 64 x 64 product
constexpr int kLd = kC + 4;    // leading dimension of the transposed tiles (16-byte rows)
constexpr int kMaxD = 128;

// g^n for n >= 0
__device__ __forceinline__ float gpow(float la, int n) { return n == 0 ? 1.f : expf(la * static_cast<float>(n)); }

// One 64-token chunk: its sequence's batch index, its rows and the place of its state.
struct ChunkAt {
    int b, c, n;       // batch index, chunk of the sequence, valid rows
    int64_t row;       // first row
    int64_t state;     // index of its dk x dv state
};

__device__ __forceinline__ bool chunk_at(const LinSeqs& sq, int id, int h, ChunkAt* at) {
    if (!sq.tab) {
        const int b = id / sq.N;
        at->b = b;
        at->c = id - b * sq.N;
        const int left = sq.T - at->c * kC;
        at->n = left < kC ? left : kC;
        at->row = (static_cast<int64_t>(b) * sq.H + h) * sq.T + static_cast<int64_t>(at->c) * kC;
        at->state = static_cast<int64_t>(h) * sq.n_chunks + id;
        return true;
    }
    if (id >= sq.coff[sq.n]) return false;
    int lo = 0, hi = sq.n;  // the last sequence with coff <= id (empty ones share their successor's)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sq.coff[mid] <= id) lo = mid;
        else hi = mid;
    }
    at->b = lo;
    at->c = id - sq.coff[lo];
    const int left = sq.tab[lo].y - at->c * kC;
    at->n = left < kC ? left : kC;
    at->row = static_cast<int64_t>(h) * sq.total + sq.tab[lo].x + static_cast<int64_t>(at->c) * kC;
    at->state = static_cast<int64_t>(h) * sq.n_chunks + id;
    return true;
}

// acc[i][j] += sum_{k < K} X[k][i0 + i] Y[k][j0 + j]; rows of X and Y are ldx and ldy floats.
__device__ __forceinline__ void mul44(float (&acc)[4][4], const float* X, int ldx, const float* Y, int ldy, int K) {
#pragma unroll 4
    for (int k = 0; k < K; k++) {
        const float4 x = *reinterpret_cast<const float4*>(X + k * ldx);
        const float4 y = *reinterpret_cast<const float4*>(Y + k * ldy);
        const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) acc[i][j] += xs[i] * ys[j];
    }
}

// grid (chunks, H, pieces of 64 x 64 over every job), kThreads. states[job] += nothing: written.
template <typename T>
__global__ void __launch_bounds__(kThreads) lin_chunk_state(LinStateJobs jobs, LinSeqs sq, const float* log_a) {
    __shared__ __align__(16) float X[kC][kLd], Y[kC][kLd];
    __shared__ float w[kC];
    const int h = blockIdx.y, tid = threadIdx.x;
    int piece = blockIdx.z, j = 0;
    while (piece >= jobs.job[j].pieces) piece -= jobs.job[j++].pieces;
    const LinStateJob& jb = jobs.job[j];
    const int p2 = (jb.d2 + 63) / 64;
    const int r0 = piece / p2 * 64, c0 = piece % p2 * 64;
    ChunkAt at;
    if (!chunk_at(sq, blockIdx.x, h, &at)) return;
    if (tid < kC) w[tid] = tid < at.n ? gpow(log_a[h], jb.reverse ? tid + 1 : at.n - 1 - tid) : 0.f;
    __syncthreads();
    const T* b = static_cast<const T*>(jb.b);
    const T* c = static_cast<const T*>(jb.c);
    for (int e = tid; e < kC * 64; e += kThreads) {
        const int i = e >> 6, d = e & 63;
        const int64_t row = at.row + i;
        X[i][d] = (i < at.n && r0 + d < jb.d1) ? load_f(b + row * jb.d1 + r0 + d) : 0.f;
        Y[i][d] = (i < at.n && c0 + d < jb.d2) ? w[i] * load_f(c + row * jb.d2 + c0 + d) : 0.f;
    }
    __syncthreads();
    const int i0 = tid / 16 * 4, j0 = tid % 16 * 4;
    float acc[4][4] = {};
    mul44(acc, &X[0][i0], kLd, &Y[0][j0], kLd, kC);
    float* dst = jb.states + at.state * jb.d1 * jb.d2;
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int q = 0; q < 4; q++)
            if (r0 + i0 + i < jb.d1 && c0 + j0 + q < jb.d2)
                dst[static_cast<int64_t>(r0 + i0 + i) * jb.d2 + c0 + j0 + q] = acc[i][q];
}

// Entering state of every chunk in place of its own, and the leaving state of every sequence.
// grid (elements / kThreads, sequences x H, jobs). One thread per state element.
__global__ void __launch_bounds__(kThreads) lin_carry(LinStateJobs jobs, LinSeqs sq, const float* log_a) {
    const LinStateJob& jb = jobs.job[blockIdx.z];
    const int e = blockIdx.x * kThreads + threadIdx.x;
    const int msz = jb.d1 * jb.d2;
    if (e >= msz) return;
    const int b = blockIdx.y / sq.H, h = blockIdx.y % sq.H;
    int len = sq.T, first = b * sq.N;
    if (sq.tab) {
        len = sq.tab[b].y;
        first = sq.coff[b];
        if (len < 0) return;  // rejected by the table kernel: nothing of it is written
    }
    const int N = (len + kC - 1) / kC;
    const float la = log_a[h];
    const float gC = gpow(la, kC), gl = gpow(la, len - (N - 1) * kC);
    float x = jb.in ? jb.in[(static_cast<int64_t>(jb.in_shared ? 0 : b) * sq.H + h) * msz + e] : 0.f;
    float* s = jb.states + (static_cast<int64_t>(h) * sq.n_chunks + first) * msz + e;
    // eight chunks' loads in flight
    for (int c0 = 0; c0 < N; c0 += 8) {
        float own[8];
#pragma unroll
        for (int u = 0; u < 8; u++) {
            const int c = c0 + u;
            if (c < N) own[u] = s[static_cast<int64_t>(jb.reverse ? N - 1 - c : c) * msz];
        }
#pragma unroll
        for (int u = 0; u < 8; u++) {
            const int c = c0 + u;
            if (c < N) {
                const int at = jb.reverse ? N - 1 - c : c;
                s[static_cast<int64_t>(at) * msz] = x;
                x = (at == N - 1 ? gl : gC) * x + own[u];
            }
        }
    }
    if (jb.out) jb.out[(static_cast<int64_t>(b) * sq.H + h) * msz + e] = x;
}

// grid (chunks, H, 64-column pieces over every scan), kThreads.
template <typename T>
__global__ void __launch_bounds__(kThreads) lin_out(LinScans scans, LinSeqs sq, const float* log_a) {
    extern __shared__ __align__(16) float sm[];
    __shared__ float pw[kC + 1];
    const int h = blockIdx.y, tid = threadIdx.x;
    int piece = blockIdx.z, j = 0;
    while (piece >= scans.scan[j].pieces) piece -= scans.scan[j++].pieces;
    const LinScan& sc = scans.scan[j];
    const int c0 = piece * 64, d1 = sc.d1, d2 = sc.d2;
    ChunkAt at;
    if (!chunk_at(sq, blockIdx.x, h, &at)) return;
    const int n = at.n;
    if (tid <= kC) pw[tid] = gpow(log_a[h], tid);
    float* A = sm;             // [d1][kLd], a transposed
    float* Bt = A + d1 * kLd;  // [d1][kLd], b transposed, then X [d1][kLd]
    float* V = Bt + d1 * kLd;  // [kC][kLd]
    float* Pt = V + kC * kLd;  // [kC][kLd], weighted scores transposed
    const T* a = static_cast<const T*>(sc.a);
    const T* b = static_cast<const T*>(sc.b);
    const T* c = static_cast<const T*>(sc.c);
    for (int e = tid; e < kC * d1; e += kThreads) {
        const int i = e / d1, d = e - i * d1;
        A[d * kLd + i] = i < n ? load_f(a + (at.row + i) * d1 + d) : 0.f;
        Bt[d * kLd + i] = i < n ? load_f(b + (at.row + i) * d1 + d) : 0.f;
    }
    for (int e = tid; e < kC * 64; e += kThreads) {
        const int i = e >> 6, d = e & 63;
        V[i * kLd + d] = (i < n && c0 + d < d2) ? load_f(c + (at.row + i) * d2 + c0 + d) : 0.f;
    }
    __syncthreads();
    const int i0 = tid / 16 * 4, j0 = tid % 16 * 4;
    float p[4][4] = {};
    mul44(p, A + i0, kLd, Bt + j0, kLd, d1);
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const int gap = sc.reverse ? j0 + q - (i0 + i) : i0 + i - (j0 + q);
            p[i][q] = gap >= 0 ? p[i][q] * pw[gap] : 0.f;
        }
    __syncthreads();  // Bt is free
#pragma unroll
    for (int q = 0; q < 4; q++)
        *reinterpret_cast<float4*>(Pt + (j0 + q) * kLd + i0) = make_float4(p[0][q], p[1][q], p[2][q], p[3][q]);
    // X[d1][64 columns]: the state is [d1][d2], or [d2][d1] where the scan reads its transpose
    const float* X = sc.states + at.state * d1 * d2;
    for (int e = tid; e < d1 * 64; e += kThreads) {
        int d, col;
        if (sc.state_t) {
            col = e / d1;
            d = e - col * d1;
        } else {
            d = e >> 6;
            col = e & 63;
        }
        float x = 0.f;
        if (c0 + col < d2)
            x = sc.state_t ? X[static_cast<int64_t>(c0 + col) * d1 + d] : X[static_cast<int64_t>(d) * d2 + c0 + col];
        Bt[d * kLd + col] = x;
    }
    __syncthreads();
    float o[4][4] = {}, far[4][4] = {};
    mul44(o, Pt + i0, kLd, V + j0, kLd, kC);
    mul44(far, A + i0, kLd, Bt + j0, kLd, d1);
    T* out = static_cast<T*>(sc.out);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int r = i0 + i;
        if (r >= n) continue;
        const float f = pw[sc.reverse ? n - 1 - r : r + 1];
#pragma unroll
        for (int q = 0; q < 4; q++)
            if (c0 + j0 + q < d2) store_f(out + (at.row + r) * d2 + c0 + j0 + q, o[i][q] + f * far[i][q]);
    }
}

size_t out_smem(int d1) { return static_cast<size_t>(2 * d1 + 2 * kC) * kLd * sizeof(float); }

template <typename T>
cudaError_t run_t(const LinStateJobs& jobs, const LinScans& scans, const LinSeqs& sq, const float* log_a,
                  cudaStream_t stream) {
    const int batch = sq.tab ? sq.n : sq.n_chunks / sq.N;
    int pieces = 0, msz = 0, d1 = 0;
    for (int i = 0; i < jobs.count; i++) {
        pieces += jobs.job[i].pieces;
        msz = jobs.job[i].d1 * jobs.job[i].d2;  // every job has the same d1 x d2
    }
    lin_chunk_state<T><<<dim3(sq.n_chunks, sq.H, pieces), kThreads, 0, stream>>>(jobs, sq, log_a);
    note_launch(stream, "lin_chunk_state");
    lin_carry<<<dim3((msz + kThreads - 1) / kThreads, batch * sq.H, jobs.count), kThreads, 0, stream>>>(jobs, sq,
                                                                                                       log_a);
    note_launch(stream, "lin_carry");
    pieces = 0;
    for (int i = 0; i < scans.count; i++) {
        pieces += scans.scan[i].pieces;
        if (scans.scan[i].d1 > d1) d1 = scans.scan[i].d1;
    }
    const size_t smem = out_smem(d1);
    cudaError_t e = cudaFuncSetAttribute(lin_out<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(out_smem(kMaxD)));
    if (e != cudaSuccess) return e;
    lin_out<T><<<dim3(sq.n_chunks, sq.H, pieces), kThreads, smem, stream>>>(scans, sq, log_a);
    note_launch(stream, "lin_out");
    return cudaGetLastError();
}

// ---- packed sequences

// tab[b] = {first row, length} (length -1: rejected), coff[b] = chunks of kC tokens before
// sequence b, order[i] = the sequence with the i-th largest length. A sequence is accepted when
// its rows lie behind every earlier entry of cu and inside the tensor and it is no longer than
// max_T; accepted ones are disjoint, so their chunks fit the total / kC + n that the host counts
// with. One block of 1024 threads.
__global__ void __launch_bounds__(1024) lin_table(const int32_t* __restrict__ cu, int n, int total, int max_T,
                                                  int2* __restrict__ tab, int* __restrict__ coff,
                                                  int* __restrict__ order, int* err) {
    __shared__ int wsum[32], wmax[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int carry = 0, high = 0;
    for (int b0 = 0; b0 < n; b0 += 1024) {
        const int b = b0 + tid;
        const int c0 = b < n ? cu[b] : 0, c1 = b < n ? cu[b + 1] : 0;
        int m = b < n ? c0 : 0;  // running maximum of cu[0..b]
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, m, off);
            if (lane >= off && y > m) m = y;
        }
        if (lane == 31) wmax[warp] = m;
        __syncthreads();
        int before = high;
        for (int w = 0; w < warp; w++)
            if (wmax[w] > before) before = wmax[w];
        if (before > m) m = before;
        const bool ok = b < n && c0 >= 0 && c0 >= m && c1 >= c0 && c1 <= total && c1 - c0 <= max_T;
        if (b < n && !ok) record_error(err, kDevBadInput);
        const int len = ok ? c1 - c0 : 0;
        const int chunks = (len + kC - 1) / kC;
        int incl = chunks;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        int sum = carry;
        for (int w = 0; w < warp; w++) sum += wsum[w];
        if (b < n) {
            tab[b] = make_int2(ok ? c0 : 0, ok ? len : -1);
            coff[b] = sum + incl - chunks;
        }
        for (int w = warp; w < 32; w++) sum += wsum[w];
        carry = sum;
        for (int w = 0; w < 32; w++)
            if (wmax[w] > high) high = wmax[w];
        __syncthreads();
    }
    if (tid == 0) coff[n] = carry;
    __syncthreads();
    if (!order) return;
    // longest first (ties by index); past 4096 sequences the n^2 comparisons cost more than the
    // order gives, and so many sequences balance by their number
    for (int b = tid; b < n; b += 1024) {
        int rank = b;
        if (n <= 4096) {
            rank = 0;
            const int len = tab[b].y;
            for (int x = 0; x < n; x++) {
                const int y = tab[x].y;
                rank += y > len || (y == len && x < b);
            }
        }
        order[rank] = b;
    }
}

// dst[e] = sum over b of src[b][e], in the order of b
__global__ void __launch_bounds__(kThreads) lin_sum_batch(const float* __restrict__ src, float* __restrict__ dst,
                                                          int B, int64_t size) {
    const int64_t e = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (e >= size) return;
    float s = 0.f;
    for (int b = 0; b < B; b++) s += src[b * size + e];
    dst[e] = s;
}

// ---- decode step

// One CTA per (b, h): S <- g S + k v^T and o = S^T q in one pass. Thread tid owns the column group
// tid % G of VEC columns and rows tid / G + r * (kThreads / G).
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) lin_decode(const T* __restrict__ q, const T* __restrict__ k,
                                                       const T* __restrict__ v, const float* __restrict__ log_a,
                                                       float* __restrict__ state, T* __restrict__ out, int H, int dk,
                                                       int dv) {
    __shared__ float qs[kMaxD], ks[kMaxD], red[kThreads * VEC];
    const int tid = threadIdx.x;
    const int64_t bh = blockIdx.x;
    const int h = static_cast<int>(bh % H);
    for (int x = tid; x < dk; x += kThreads) {
        qs[x] = load_f(q + bh * dk + x);
        ks[x] = load_f(k + bh * dk + x);
    }
    const float g = expf(log_a[h]);
    const int G = (dv + VEC - 1) / VEC, rows = kThreads / G;
    const int col = tid % G * VEC, r0 = tid / G;
    float vv[VEC], o[VEC];
#pragma unroll
    for (int x = 0; x < VEC; x++) {
        vv[x] = r0 < rows ? load_f(v + bh * dv + col + x) : 0.f;
        o[x] = 0.f;
    }
    __syncthreads();
    float* S = state + bh * dk * dv + col;
    if (r0 < rows) {
#pragma unroll 4
        for (int r = r0; r < dk; r += rows) {
            float s[VEC];
            if constexpr (VEC == 4) {
                const float4 x = __ldcs(reinterpret_cast<const float4*>(S + r * dv));
                s[0] = x.x; s[1] = x.y; s[2] = x.z; s[3] = x.w;
            } else {
                s[0] = S[r * dv];
            }
#pragma unroll
            for (int x = 0; x < VEC; x++) {
                s[x] = g * s[x] + ks[r] * vv[x];
                o[x] += qs[r] * s[x];
            }
            if constexpr (VEC == 4) __stcs(reinterpret_cast<float4*>(S + r * dv), make_float4(s[0], s[1], s[2], s[3]));
            else S[r * dv] = s[0];
        }
    }
#pragma unroll
    for (int x = 0; x < VEC; x++) red[tid * VEC + x] = o[x];
    __syncthreads();
    if (tid < dv) {
        float s = 0.f;
        for (int r = 0; r < rows; r++) s += red[(r * G + tid / VEC) * VEC + tid % VEC];
        store_f(out + bh * dv + tid, s);
    }
}

template <typename T>
void decode_t(const void* q, const void* k, const void* v, const float* log_a, float* state, void* out, int B, int H,
              int dk, int dv, cudaStream_t stream) {
    auto go = [&](auto kern) {
        kern<<<static_cast<unsigned>(B) * H, kThreads, 0, stream>>>(static_cast<const T*>(q),
                                                                    static_cast<const T*>(k),
                                                                    static_cast<const T*>(v), log_a, state,
                                                                    static_cast<T*>(out), H, dk, dv);
    };
    if (dv % 4 == 0) go(lin_decode<T, 4>);
    else go(lin_decode<T, 1>);
    note_launch(stream, "lin_decode");
}

}  // namespace

cudaError_t linear_run(int dtype, const LinStateJobs& jobs, const LinScans& scans, const LinSeqs& sq,
                       const float* log_a, cudaStream_t stream) {
    return dtype == 1 ? run_t<float>(jobs, scans, sq, log_a, stream)
                      : run_t<__nv_bfloat16>(jobs, scans, sq, log_a, stream);
}

cudaError_t linear_table(const int32_t* cu, int n, int total, int max_T, int2* tab, int* coff, int* order, int* err,
                         cudaStream_t stream) {
    lin_table<<<1, 1024, 0, stream>>>(cu, n, total, max_T, tab, coff, order, err);
    note_launch(stream, "lin_table");
    return cudaGetLastError();
}

cudaError_t linear_sum_batch(const float* src, float* dst, int B, int64_t size, cudaStream_t stream) {
    lin_sum_batch<<<static_cast<unsigned>((size + kThreads - 1) / kThreads), kThreads, 0, stream>>>(src, dst, B, size);
    note_launch(stream, "lin_sum_batch");
    return cudaGetLastError();
}

cudaError_t linear_decode_step(int dtype, const void* q, const void* k, const void* v, const float* log_a,
                               float* state, void* out, int B, int H, int dk, int dv, cudaStream_t stream) {
    if (dtype == 1) decode_t<float>(q, k, v, log_a, state, out, B, H, dk, dv, stream);
    else decode_t<__nv_bfloat16>(q, k, v, log_a, state, out, B, H, dk, dv, stream);
    return cudaGetLastError();
}

}  // namespace lla
