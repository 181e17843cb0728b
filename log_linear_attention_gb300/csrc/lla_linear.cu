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
// All products are 64 x 64 register-tiled fp32 products out of shared memory. FMAs bound them, over launches of 1.6 waves
// of CTAs: packed FMA instructions, two products each, are 31 to 34% of what the pipe's counter could hold (gradients of
// 3 x 5 heads, T = 1301, 96 x 80: 140 us; prompts of 2 x 16 heads, T = 4096, 128 x 128: 420 us, 31 TFLOP/s counting whole
// squares). No exponent is ever negative, so no factor overflows for g <= 1; g^0 is 1 also for g = 0 (log_a = -inf).
#include <atomic>

#include "lla_internal.cuh"
#include "lla_linear.cuh"
#include "lla_tc_ptx.cuh"

namespace lla {
namespace {

constexpr int kC = 64;         // tokens per chunk
constexpr int kThreads = 256;
constexpr int kMulThreads = 128;  // 8 x 16 threads, each an 8 x 4 piece of a 64 x 64 product
constexpr int kSlab = 32;         // summed indices staged at a time
constexpr int kLd = kC + 4;    // leading dimension of the transposed tiles (16-byte rows)
constexpr int kMaxD = 128;
constexpr int kBlocksPerSm = 4;  // of lin_chunk_state and lin_out

// blocks of lin_out that fill the current device once (asked once of a device)
int64_t full_blocks() {
    constexpr int kMaxDevices = 64;
    static std::atomic<int> sms[kMaxDevices];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return INT64_MAX;
    }
    n = sms[dev].load(std::memory_order_relaxed);
    if (!n) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            return INT64_MAX;
        }
        sms[dev].store(n, std::memory_order_relaxed);
    }
    return static_cast<int64_t>(n) * kBlocksPerSm;
}

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

// A warp's quarter of a 64 x 64 product, 32 x 32, and this thread's 8 x 4 piece of it. Which warp takes which is turned
// from block to block, so that quarters with less to do fall to all sub-partitions of an SM.
struct Piece {
    int wr, wc, i0, j0;
};
__device__ __forceinline__ Piece piece_of(int turn) {
    const int role = ((threadIdx.x >> 5) + turn) & 3, lane = threadIdx.x & 31;
    return {role >> 1, role & 1, (role >> 1) * 32 + (lane >> 3) * 8, (role & 1) * 32 + (lane & 7) * 4};
}

// acc[i][j] += sum_{k < K} X[k][i] Y[k][j], rows of kLd floats: three shared-memory wavefronts for 32 FMAs of a warp
// (4 x 4 pieces took six), two rows to an instruction (prompts and gradients of 128 x 128 heads, T = 4096:
// 460 -> 433 us, 583 -> 564 us).
template <int K>
__device__ __forceinline__ void mul84(float (&acc)[8][4], const float* X, const float* Y) {
    f32x2 s[4][4];
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) s[i][j] = pair2(acc[2 * i][j], acc[2 * i + 1][j]);
#pragma unroll 8
    for (int k = 0; k < K; k++) {
        const ulonglong2 x0 = *reinterpret_cast<const ulonglong2*>(X + k * kLd);
        const ulonglong2 x1 = *reinterpret_cast<const ulonglong2*>(X + k * kLd + 4);
        const float4 y = *reinterpret_cast<const float4*>(Y + k * kLd);
        const f32x2 xs[4] = {x0.x, x0.y, x1.x, x1.y};
        const f32x2 ys[4] = {pair2(y.x, y.x), pair2(y.y, y.y), pair2(y.z, y.z), pair2(y.w, y.w)};
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) s[i][j] = fma2(xs[i], ys[j], s[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float2 f = split2(s[i][j]);
            acc[2 * i][j] = f.x;
            acc[2 * i + 1][j] = f.y;
        }
}

// Four consecutive columns d..d+3 of a row of D columns, zeros past it; one load where rows keep it aligned.
template <typename T>
__device__ __forceinline__ float4 load4(const T* row, int d, int D, bool vec) {
    if (vec && d + 3 < D) {
        if constexpr (sizeof(T) == 4) {
            return *reinterpret_cast<const float4*>(row + d);
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(row + d);
            return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                               __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
        }
    }
    return make_float4(d < D ? load_f(row + d) : 0.f, d + 1 < D ? load_f(row + d + 1) : 0.f,
                       d + 2 < D ? load_f(row + d + 2) : 0.f, d + 3 < D ? load_f(row + d + 3) : 0.f);
}

// A slab of 2048 values passes through four 16-byte registers of each thread, so that the next slab's loads are in
// flight while this one is multiplied.
struct Slab {
    float4 x[4];
};

// kSlab columns d0.. of 64 rows, transposed: S[d - d0][i]. Lanes take rows, so that the stores of a warp fall into 32
// banks. `row` is this thread's row (tid % 64).
template <typename T>
__device__ __forceinline__ void fetch_t(Slab& s, const T* row, int d0, int D, bool vec, bool valid) {
#pragma unroll
    for (int u = 0; u < 4; u++) {
        const int d = d0 + (threadIdx.x >> 6) * (kSlab / 2) + 4 * u;
        s.x[u] = valid && d < D ? load4(row, d, D, vec) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}
__device__ __forceinline__ void put_t(const Slab& s, float (*S)[kLd]) {
    const int i = threadIdx.x & 63, d = (threadIdx.x >> 6) * (kSlab / 2);
#pragma unroll
    for (int u = 0; u < 4; u++) {
        S[d + 4 * u][i] = s.x[u].x;
        S[d + 4 * u + 1][i] = s.x[u].y;
        S[d + 4 * u + 2][i] = s.x[u].z;
        S[d + 4 * u + 3][i] = s.x[u].w;
    }
}

// kSlab rows r0.. of 64 columns c0..: S[r - r0][col]; rows from `rows` on are zeros.
template <typename T>
__device__ __forceinline__ void fetch(Slab& s, const T* base, int r0, int rows, int c0, int D, bool vec) {
#pragma unroll
    for (int u = 0; u < 4; u++) {
        const int e = threadIdx.x + u * kMulThreads, r = r0 + (e >> 4), col = c0 + (e & 15) * 4;
        s.x[u] = r < rows && col < D ? load4(base + static_cast<int64_t>(r) * D, col, D, vec)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}
__device__ __forceinline__ void put(const Slab& s, float (*S)[kLd]) {
#pragma unroll
    for (int u = 0; u < 4; u++) {
        const int e = threadIdx.x + u * kMulThreads;
        *reinterpret_cast<float4*>(&S[e >> 4][(e & 15) * 4]) = s.x[u];
    }
}

// grid (chunks, H, pieces of 64 x 64 over every job), kMulThreads.
template <typename T>
__global__ void __launch_bounds__(kMulThreads, kBlocksPerSm) lin_chunk_state(LinStateJobs jobs, LinSeqs sq, const float* log_a) {
    __shared__ __align__(16) float X[kSlab][kLd], Y[kSlab][kLd];
    __shared__ float w[kC];
    grid_dep_launch();
    const int h = blockIdx.y, tid = threadIdx.x;
    int piece = blockIdx.z, j = 0;
    while (piece >= jobs.job[j].pieces) piece -= jobs.job[j++].pieces;
    const LinStateJob& jb = jobs.job[j];
    const int p2 = (jb.d2 + 63) / 64;
    const int r0 = piece / p2 * 64, c0 = piece % p2 * 64;
    ChunkAt at;
    if (!chunk_at(sq, blockIdx.x, h, &at)) return;
    if (tid < kC) w[tid] = tid < at.n ? gpow(log_a[h], jb.reverse ? tid + 1 : at.n - 1 - tid) : 0.f;
    const T* b = static_cast<const T*>(jb.b) + at.row * jb.d1;
    const T* c = static_cast<const T*>(jb.c) + at.row * jb.d2;
    const bool v1 = jb.d1 % 4 == 0, v2 = jb.d2 % 4 == 0;
    const Piece at_piece = piece_of(0);
    float acc[8][4] = {};
    Slab x, y;
    fetch(x, b, 0, at.n, r0, jb.d1, v1);
    fetch(y, c, 0, at.n, c0, jb.d2, v2);
    for (int t0 = 0; t0 < at.n; t0 += kSlab) {
        __syncthreads();  // the slabs are free, w is written
        put(x, X);
#pragma unroll
        for (int u = 0; u < 4; u++) {
            const int r = t0 + ((tid + u * kMulThreads) >> 4);
            const float f = w[r];
            if (r < at.n) y.x[u] = make_float4(f * y.x[u].x, f * y.x[u].y, f * y.x[u].z, f * y.x[u].w);
        }
        put(y, Y);
        __syncthreads();
        if (t0 + kSlab < at.n) {
            fetch(x, b, t0 + kSlab, at.n, r0, jb.d1, v1);
            fetch(y, c, t0 + kSlab, at.n, c0, jb.d2, v2);
        }
        mul84<kSlab>(acc, &X[0][at_piece.i0], &Y[0][at_piece.j0]);
    }
    const int i0 = at_piece.i0, j0 = c0 + at_piece.j0;
    float* dst = jb.states + at.state * jb.d1 * jb.d2;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        if (r0 + i0 + i >= jb.d1) break;
        float* to = dst + static_cast<int64_t>(r0 + i0 + i) * jb.d2 + j0;
        if (v2 && j0 + 3 < jb.d2) {
            *reinterpret_cast<float4*>(to) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        } else {
#pragma unroll
            for (int q = 0; q < 4; q++)
                if (j0 + q < jb.d2) to[q] = acc[i][q];
        }
    }
}

// Entering state of every chunk in place of its own, and the leaving state of every sequence.
// grid (elements / kThreads, sequences x H, jobs). One thread per state element.
__global__ void __launch_bounds__(kThreads) lin_carry(LinStateJobs jobs, LinSeqs sq, const float* log_a) {
    grid_dep_launch();
    grid_dep_wait();  // the own states
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
    const int N = static_cast<int>((static_cast<unsigned>(len) + kC - 1) / kC);  // len may be 2^31 - 1
    const float la = log_a[h];
    const float gC = gpow(la, kC), gl = gpow(la, len - (N - 1) * kC);
    float x = jb.in ? jb.in[(static_cast<int64_t>(jb.in_shared ? 0 : b) * sq.state_heads + h) * msz + e] : 0.f;
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
    if (jb.out) jb.out[(static_cast<int64_t>(b) * sq.state_heads + h) * msz + e] = x;
}

// grid (chunks, H, scans), kMulThreads. The weighted scores are formed once and serve every 64 columns of c. Operands
// pass through two small slabs (35 KB a block with the scores), so that several blocks share an SM; whole tiles in
// shared memory left two.
template <typename T>
__global__ void __launch_bounds__(kMulThreads, kBlocksPerSm) lin_out(LinScans scans, LinSeqs sq, const float* log_a) {
    __shared__ __align__(16) float X[kSlab][kLd], Y[kSlab][kLd], Pt[kC][kLd];
    __shared__ float pw[kC + 1];
    const int h = blockIdx.y, tid = threadIdx.x;
    const LinScan& sc = scans.scan[blockIdx.z];
    const int d1 = sc.d1, d2 = sc.d2;
    ChunkAt at;
    if (!chunk_at(sq, blockIdx.x, h, &at)) {
        grid_dep_wait();  // with no chunk at all too, this kernel ends after the one that writes the workspace
        return;
    }
    const int n = at.n;
    if (tid <= kC) pw[tid] = gpow(log_a[h], tid);
    const bool v1 = d1 % 4 == 0, v2 = d2 % 4 == 0;
    const int row = tid & 63;
    const T* a = static_cast<const T*>(sc.a) + (at.row + row) * d1;
    const T* b = static_cast<const T*>(sc.b) + (at.row + row) * d1;
    const T* c = static_cast<const T*>(sc.c) + at.row * d2;
    const Piece pc = piece_of(blockIdx.x + blockIdx.y + blockIdx.z);
    const int i0 = pc.i0, j0 = pc.j0;
    const int idle = sc.reverse ? 1 : 0;  // rows of quarter `idle` see no keys of the other half
    T* out = static_cast<T*>(sc.out);
    const float* state = sc.states + at.state * d1 * d2;
    // steps: nd slabs of a and b (scores), then for every 64 columns of c nd slabs of a and the entering state and nt
    // slabs of c
    const int nd = (d1 + kSlab - 1) / kSlab, nt = (n + kSlab - 1) / kSlab, per = nd + nt;
    const int steps = nd + (d2 + 63) / 64 * per;
    Slab x, y;
    auto get = [&](int st) {
        if (st < nd) {
            fetch_t(x, a, st * kSlab, d1, v1, row < n);
            fetch_t(y, b, st * kSlab, d1, v1, row < n);
            return;
        }
        const int c0 = (st - nd) / per * 64, u = (st - nd) % per;
        if (u < nd) {
            fetch_t(x, a, u * kSlab, d1, v1, row < n);
            // the entering state is [d1][d2], or [d2][d1] where the scan reads its transpose
            if (sc.state_t) fetch_t(y, state + static_cast<int64_t>(c0 + row) * d1, u * kSlab, d1, v1, c0 + row < d2);
            else fetch(y, state, u * kSlab, d1, c0, d2, v2);
        } else {
            fetch(y, c, (u - nd) * kSlab, n, c0, d2, v2);
        }
    };
    get(0);
    float o[8][4] = {};
    for (int st = 0; st < steps; st++) {
        const int u = st < nd ? st : (st - nd) % per;  // step of its group
        const bool scores = st < nd, near = !scores && u >= nd;
        __syncthreads();
        if (!near) put_t(x, X);
        if (scores || (!near && sc.state_t)) put_t(y, Y);
        else put(y, Y);
        __syncthreads();
        if (st + 1 == nd) grid_dep_wait();  // the entering states; the scores are formed beside the kernels before
        if (st + 1 < steps) get(st + 1);
        // causality leaves a quarter of the scores out, and a half of the keys for half of the rows
        const bool skip = pc.wr == idle && ((scores && pc.wc != idle) || (near && u - nd != idle));
        if (!skip) mul84<kSlab>(o, near ? &Pt[(u - nd) * kSlab][i0] : &X[0][i0], &Y[0][j0]);
        if (scores && u == nd - 1) {
#pragma unroll
            for (int q = 0; q < 4; q++) {
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const int gap = sc.reverse ? j0 + q - (i0 + i) : i0 + i - (j0 + q);
                    o[i][q] = gap >= 0 ? o[i][q] * pw[gap] : 0.f;
                }
                float4* to = reinterpret_cast<float4*>(&Pt[j0 + q][i0]);
                to[0] = make_float4(o[0][q], o[1][q], o[2][q], o[3][q]);
                to[1] = make_float4(o[4][q], o[5][q], o[6][q], o[7][q]);
#pragma unroll
                for (int i = 0; i < 8; i++) o[i][q] = 0.f;
            }
        } else if (!scores && u == nd - 1) {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const int r = i0 + i;
                const float f = r < n ? pw[sc.reverse ? n - 1 - r : r + 1] : 0.f;
#pragma unroll
                for (int q = 0; q < 4; q++) o[i][q] *= f;
            }
        } else if (near && u == per - 1) {
            const int c0 = (st - nd) / per * 64;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const int r = i0 + i;
                T* to = out + (at.row + r) * d2 + c0 + j0;
                if (r < n && v2 && c0 + j0 + 3 < d2) {
                    if constexpr (sizeof(T) == 4) {
                        *reinterpret_cast<float4*>(to) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
                    } else {
                        const __nv_bfloat162 lo = __floats2bfloat162_rn(o[i][0], o[i][1]),
                                             hi = __floats2bfloat162_rn(o[i][2], o[i][3]);
                        *reinterpret_cast<uint2*>(to) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                                   *reinterpret_cast<const uint32_t*>(&hi));
                    }
                } else if (r < n) {
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        if (c0 + j0 + q < d2) store_f(to + q, o[i][q]);
                }
#pragma unroll
                for (int q = 0; q < 4; q++) o[i][q] = 0.f;
            }
        }
    }
}

template <typename T>
cudaError_t run_t(const LinStateJobs& jobs, const LinScans& scans, const LinSeqs& sq, const float* log_a,
                  cudaStream_t stream) {
    const int batch = sq.tab ? sq.n : sq.n_chunks / sq.N;
    int pieces = 0, msz = 0;
    for (int i = 0; i < jobs.count; i++) {
        pieces += jobs.job[i].pieces;
        msz = jobs.job[i].d1 * jobs.job[i].d2;  // every job has the same d1 x d2
    }
    lin_chunk_state<T><<<dim3(sq.n_chunks, sq.H, pieces), kMulThreads, 0, stream>>>(jobs, sq, log_a);
    note_launch(stream, "lin_chunk_state");
    // Each beside the end of the one before, where lin_out's blocks fill the GPU (four to an SM): fewer would be placed four
    // to an SM on the SMs that the others leave free (240 blocks: 56 us for the three kernels against 39; 2048: 422
    // against 428).
    const dim3 blocks(sq.n_chunks, sq.H, scans.count);
    const bool beside = static_cast<int64_t>(blocks.x) * blocks.y * blocks.z >= full_blocks();
    auto launch = [&](auto kern, dim3 grid, int threads, const auto& what) {
        if (beside) return launch_pdl(kern, grid, dim3(threads), 0, stream, what, sq, log_a);
        kern<<<grid, threads, 0, stream>>>(what, sq, log_a);
        return cudaGetLastError();
    };
    cudaError_t e = launch(lin_carry, dim3((msz + kThreads - 1) / kThreads, batch * sq.H, jobs.count), kThreads, jobs);
    if (e != cudaSuccess) return e;
    note_launch(stream, "lin_carry");
    e = launch(lin_out<T>, blocks, kMulThreads, scans);
    if (e != cudaSuccess) return e;
    note_launch(stream, "lin_out");
    return cudaGetLastError();
}

// ---- packed sequences

// tab[b] = {first row, length} (length -1: rejected), coff[b] = chunks of kC tokens before
// sequence b, order[i] = the sequence with the i-th largest length. A sequence is accepted when
// its rows lie behind every earlier entry of cu and inside the tensor and it is no longer than
// max_T; accepted ones are disjoint, so their chunks fit the total / kC + n that the host counts
// with. One block of 1024 threads.
constexpr int kMostSorted = 1024;
__global__ void __launch_bounds__(1024) lin_table(const int32_t* __restrict__ cu, int n, int total, int max_T,
                                                  int2* __restrict__ tab, int* __restrict__ coff,
                                                  int* __restrict__ order, int* err) {
    __shared__ int wsum[32], wmax[32];
    __shared__ __align__(16) int lens[kMostSorted];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dep_launch();  // the tensor-core scan sets up beside this kernel
    if (tid < kMostSorted) lens[tid] = -2;  // shorter than any sequence
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
        const int chunks = static_cast<int>((static_cast<unsigned>(len) + kC - 1) / kC);
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
            if (b < kMostSorted) lens[b] = ok ? len : -1;
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
    // longest first (ties by index); more sequences than kMostSorted balance by their number
    for (int b = tid; b < n; b += 1024) {
        int rank = b;
        if (n <= kMostSorted) {
            rank = 0;
            const int len = lens[b];
            for (int x = 0; x < n; x += 4) {
                const int4 y = *reinterpret_cast<const int4*>(lens + x);
                rank += (y.x > len || (y.x == len && x < b)) + (y.y > len || (y.y == len && x + 1 < b)) +
                        (y.z > len || (y.z == len && x + 2 < b)) + (y.w > len || (y.w == len && x + 3 < b));
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
// tid % G of VEC columns and rows tid / G + r * (kThreads / G). Bound by the state's bytes: 64 x 16 heads of 128 x 64,
// 67 MB, 8.3 us where half of it stays in L2 from step to step.
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
