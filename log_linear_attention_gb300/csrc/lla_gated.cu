// The gated linear recurrence: every channel by itself, with a gate for each token.
//
//     h_t = a_t h_{t-1} + x_t,   a_t = exp(log_a_t),   h_{-1} = state0
//
// Its gradients are the same recurrence backwards over F_t, the gradient that reaches h_{t-1}:
//     F_t = a_t (dout_t + F_{t+1}),  F_T = dstate_out
//     dx_t = dout_t + F_{t+1},  dlog_a_t = F_t h_{t-1},  dstate0 = F_0.
// h comes from the forward's outputs as they were kept (rounded to their type), so one pass does.
//
// A stretch of rows is the map h -> A h + s with A the product of its gates; maps of neighbours compose. One thread
// block cluster walks 64 channels of one sequence from end to end in steps of (cluster size) x 128 rows: a thread
// keeps 8 rows of 4 channels, forms their map, the block composes its 16 stretches, the blocks hand their maps to
// one another through distributed shared memory, and every thread runs its rows again from the state that enters
// them. Blocks of a cluster are resident together, so nothing waits for a block that may not run yet, and neither
// flags nor workspace are needed. Maps are composed in one fixed order: repeated calls give identical bits.
//
// Packed sequences are one row axis: a map that holds a sequence's first row does not depend on what enters. Its A is
// kept as -1 (a product of exponentials is never negative), so that not even an infinity or NaN crosses over.
#include "lla_drafts.cuh"
#include "lla_tc_ptx.cuh"

namespace lla {
namespace {

constexpr int kThreads = 256;
constexpr int kV = 4;                    // channels of a thread
constexpr int kL = 8;                    // rows of a thread
constexpr int kLanes = 16;               // threads side by side on one row
constexpr int kCols = kLanes * kV;       // channels of a block
constexpr int kSegs = kThreads / kLanes; // stretches of a block
constexpr int kRows = kSegs * kL;        // rows of a block
constexpr int kMaxCluster = 8;

struct Args {
    GatedPass p;
    int cluster, cols, steps;
    int* err;
};

template <typename T> struct Four;  // four neighbouring values as they lie in memory
template <> struct Four<float> { using raw = float4; };
template <> struct Four<__nv_bfloat16> { using raw = uint2; };

__device__ __forceinline__ void widen(const float4& r, float (&f)[4]) { f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w; }
__device__ __forceinline__ void widen(const uint2& r, float (&f)[4]) {
    f[0] = __uint_as_float(r.x << 16); f[1] = __uint_as_float(r.x & 0xffff0000u);
    f[2] = __uint_as_float(r.y << 16); f[3] = __uint_as_float(r.y & 0xffff0000u);
}
__device__ __forceinline__ void put4(float* p, const float (&f)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void put4(__nv_bfloat16* p, const float (&f)[4]) {
    __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    uint2 r;
    r.x = *reinterpret_cast<unsigned*>(&a);
    r.y = *reinterpret_cast<unsigned*>(&b);
    *reinterpret_cast<uint2*>(p) = r;
}

// Four channels of a row: neighbours (kVec; D a multiple of 4), or 16 apart, so that a scalar access of 16 threads is one
// stretch of memory.
template <bool kVec>
struct Chan {
    int c[4];
    bool any;
    int D;
    __device__ __forceinline__ Chan(int col, int lane, int D_) : D(D_) {
#pragma unroll
        for (int v = 0; v < 4; v++) c[v] = col * kCols + (kVec ? lane * 4 + v : lane + 16 * v);
        any = c[0] < D;
    }
    template <typename T> __device__ __forceinline__ void load(const T* row, float (&f)[4]) const {
        if constexpr (kVec) {
            if (any) { widen(__ldg(reinterpret_cast<const typename Four<T>::raw*>(row + c[0])), f); return; }
#pragma unroll
            for (int v = 0; v < 4; v++) f[v] = 0.f;
        } else {
#pragma unroll
            for (int v = 0; v < 4; v++) f[v] = c[v] < D ? load_f(row + c[v]) : 0.f;
        }
    }
    template <typename T> __device__ __forceinline__ void store(T* row, const float (&f)[4]) const {
        if constexpr (kVec) {
            if (any) put4(row + c[0], f);
        } else {
#pragma unroll
            for (int v = 0; v < 4; v++)
                if (c[v] < D) store_f(row + c[v], f[v]);
        }
    }
    // place of the v-th channel among the block's
    __device__ __forceinline__ static int at(int lane, int v) { return kVec ? lane * 4 + v : lane + 16 * v; }
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void store_remote(uint32_t at, uint32_t rank, float x, float y) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(r), "f"(x), "f"(y) : "memory");
}

// (A, s) <- (A2, s2) after (A, s)
template <bool kPacked>
__device__ __forceinline__ void compose(float& A, float& s, float A2, float s2) {
    if (kPacked && A2 < 0.f) {
        A = -1.f;
        s = s2;
        return;
    }
    s = fmaf(A2, s, s2);
    A = kPacked && A < 0.f ? -1.f : A * A2;
}
template <bool kPacked>
__device__ __forceinline__ float apply(float A, float s, float h) {
    return kPacked && A < 0.f ? s : fmaf(A, h, s);
}

// What a row of a packed call is: its sequence, and whether that one's walk begins or ends there. -1: no sequence's.
constexpr int kBegins = 1 << 30, kEnds = 1 << 29, kSeq = kEnds - 1;
template <bool kBack>
__device__ __forceinline__ int row_info(const int32_t* cu, int n, int row) {
    int lo = 0, hi = n;  // the last i with cu[i] <= row
    if (row < cu[0] || row >= cu[n]) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= row) lo = mid;
        else hi = mid;
    }
    const bool first = row == cu[lo], last = row == cu[lo + 1] - 1;
    return lo | ((kBack ? last : first) ? kBegins : 0) | ((kBack ? first : last) ? kEnds : 0);
}

template <typename T, typename G, bool kBack, bool kPacked, bool kVec>
__global__ void __launch_bounds__(kThreads, 2) gated_scan(const Args a) {
    __shared__ __align__(16) float seg_a[2][kSegs][kCols], seg_s[2][kSegs][kCols];
    __shared__ __align__(16) float2 part[2][kMaxCluster][kCols];
    __shared__ __align__(16) float carry[2][kCols];
    __shared__ int info[2][kPacked ? kRows : 1];
    const GatedPass& p = a.p;
    const int tid = threadIdx.x, lane = tid % kLanes, seg = tid / kLanes;
    const int R = p.T, D = p.D, cs = a.cluster;
    const int rank = cs > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int walk = blockIdx.x / cs;  // cluster: a column of one sequence
    const int col = walk % a.cols, b = walk / a.cols;
    const Chan<kVec> ch(col, lane, D);
    if (kPacked) {
        bool bad = false;
        for (int i = tid; i <= p.n; i += kThreads) {
            const int x = p.cu[i];
            bad |= x < 0 || x > R || (i > 0 && x < p.cu[i - 1]);
        }
        if (__syncthreads_or(bad)) {  // every block finds the same
            if (blockIdx.x == 0 && tid == 0) record_error(a.err, kDevBadInput);
            return;
        }
    }
    const float* enter = kBack ? p.dstate_out : p.state0;  // what a walk begins with
    const int64_t row0 = static_cast<int64_t>(b) * R;
    const T* xp = static_cast<const T*>(p.x) + row0 * D;
    const G* gp = static_cast<const G*>(p.log_a) + row0 * D;
    const T* dp = kBack ? static_cast<const T*>(p.dout) + row0 * D : nullptr;
    T* op = static_cast<T*>(p.out) + row0 * D;
    G* ap = kBack ? static_cast<G*>(p.dlog_a) + row0 * D : nullptr;
    auto enters = [&](int i) { return enter + static_cast<int64_t>(kBack || p.n0 > 1 ? i : 0) * D; };
    auto first_state = [&](int i) { return p.state0 + static_cast<int64_t>(p.n0 > 1 ? i : 0) * D; };

    if (kPacked && p.leave) {  // empty sequences: what enters leaves
        for (int i = rank * kSegs + seg; i < p.n; i += cs * kSegs) {
            if (p.cu[i] != p.cu[i + 1]) continue;
            float f[4] = {0.f, 0.f, 0.f, 0.f};
            if (enter) ch.load(enters(i), f);
            ch.store(p.leave + static_cast<int64_t>(i) * D, f);
        }
    }

    const int my_col = col * kCols + tid;  // of the first kCols threads, which carry the walk's state
    float state = 0.f;
    if (!kPacked && enter && tid < kCols && my_col < D) state = enters(b)[my_col];

    for (int st = 0; st < a.steps; st++) {
        const int buf = st & 1;
        const int u0 = (st * cs + rank) * kRows + seg * kL;  // first of this thread's rows, in walking order
        if (kPacked) {
            if (tid < kRows) {
                const int u = (st * cs + rank) * kRows + tid;
                info[buf][tid] = u < R ? row_info<kBack>(p.cu, p.n, kBack ? R - 1 - u : u) : -1;
            }
            __syncthreads();
        }
        float g[kL][4], x[kL][4], hp[kL][4];
#pragma unroll
        for (int j = 0; j < kL; j++) {
            const int u = u0 + j, row = kBack ? R - 1 - u : u;
            const bool in = u < R && (!kPacked || info[buf][seg * kL + j] >= 0);
#pragma unroll
            for (int v = 0; v < 4; v++) g[j][v] = x[j][v] = hp[j][v] = 0.f;
            if (in) {
                ch.load(gp + static_cast<int64_t>(row) * D, g[j]);
                ch.load((kBack ? dp : xp) + static_cast<int64_t>(row) * D, x[j]);
                if (kBack) {
                    const bool first = kPacked ? (info[buf][seg * kL + j] & kEnds) != 0 : row == 0;
                    if (!first) ch.load(xp + static_cast<int64_t>(row - 1) * D, hp[j]);
                    else if (p.state0) ch.load(first_state(kPacked ? info[buf][seg * kL + j] & kSeq : b), hp[j]);
                }
            }
        }
        float A[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kL; j++) {
            const bool begins = kPacked && info[buf][seg * kL + j] >= 0 && (info[buf][seg * kL + j] & kBegins);
            float e[4] = {0.f, 0.f, 0.f, 0.f};
            if (begins && enter) ch.load(enters(info[buf][seg * kL + j] & kSeq), e);
#pragma unroll
            for (int v = 0; v < 4; v++) {
                g[j][v] = expf(g[j][v]);
                if (begins) {
                    s[v] = e[v];
                    A[v] = -1.f;
                }
                if (kBack) s[v] = g[j][v] * (x[j][v] + s[v]);
                else s[v] = fmaf(g[j][v], s[v], x[j][v]);
                if (!kPacked || A[v] >= 0.f) A[v] *= g[j][v];
            }
        }
#pragma unroll
        for (int v = 0; v < 4; v++) {
            seg_a[buf][seg][Chan<kVec>::at(lane, v)] = A[v];
            seg_s[buf][seg][Chan<kVec>::at(lane, v)] = s[v];
        }
        __syncthreads();
        float own_a = 1.f, own_s = 0.f;
        if (tid < kCols) {
#pragma unroll
            for (int i = 0; i < kSegs; i++) {
                const float A2 = seg_a[buf][i][tid], s2 = seg_s[buf][i][tid];
                seg_a[buf][i][tid] = own_a;
                seg_s[buf][i][tid] = own_s;
                compose<kPacked>(own_a, own_s, A2, s2);
            }
            if (cs > 1) {
                const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(&part[buf][rank][tid]));
                for (int r = 0; r < cs; r++) store_remote(at, r, own_a, own_s);
            }
        }
        if (cs > 1) {
            cluster_arrive();
            cluster_wait();
        }
        if (tid < kCols) {
            if (cs > 1) {
                for (int r = 0; r < cs; r++) {
                    if (r == rank) carry[buf][tid] = state;
                    state = apply<kPacked>(part[buf][r][tid].x, part[buf][r][tid].y, state);
                }
            } else {
                carry[buf][tid] = state;
                state = apply<kPacked>(own_a, own_s, state);
            }
        }
        __syncthreads();
        float h[4];
#pragma unroll
        for (int v = 0; v < 4; v++) {
            const int c = Chan<kVec>::at(lane, v);
            h[v] = apply<kPacked>(seg_a[buf][seg][c], seg_s[buf][seg][c], carry[buf][c]);
        }
#pragma unroll
        for (int j = 0; j < kL; j++) {
            const int u = u0 + j, row = kBack ? R - 1 - u : u;
            const int inf = kPacked ? info[buf][seg * kL + j] : 0;
            if (u >= R) continue;
            if (kPacked && inf < 0) {
                if (kBack) {  // rows of no sequence take no part in the sum that is differentiated
                    const float z[4] = {0.f, 0.f, 0.f, 0.f};
                    ch.store(op + static_cast<int64_t>(row) * D, z);
                    ch.store(ap + static_cast<int64_t>(row) * D, z);
                }
                continue;
            }
            if (kPacked && (inf & kBegins)) {
#pragma unroll
                for (int v = 0; v < 4; v++) h[v] = 0.f;
                if (enter) ch.load(enters(inf & kSeq), h);
            }
            if (kBack) {
                float d[4], da[4];
#pragma unroll
                for (int v = 0; v < 4; v++) {
                    d[v] = x[j][v] + h[v];
                    h[v] = g[j][v] * d[v];
                    da[v] = h[v] * hp[j][v];
                }
                ch.store(op + static_cast<int64_t>(row) * D, d);
                ch.store(ap + static_cast<int64_t>(row) * D, da);
            } else {
#pragma unroll
                for (int v = 0; v < 4; v++) h[v] = fmaf(g[j][v], h[v], x[j][v]);
                ch.store(op + static_cast<int64_t>(row) * D, h);
            }
            if (kPacked && (inf & kEnds) && p.leave) ch.store(p.leave + static_cast<int64_t>(inf & kSeq) * D, h);
        }
    }
    if (!kPacked && p.leave && rank == 0 && tid < kCols && my_col < D)
        p.leave[static_cast<int64_t>(b) * D + my_col] = state;
    if (cs > 1) {  // no block leaves while another may still write to it
        cluster_arrive();
        cluster_wait();
    }
}

template <typename T, typename G, bool kBack, bool kPacked, bool kVec>
cudaError_t launch_scan(Args& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.cluster) * a.cols * (kPacked ? 1 : a.p.n));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, gated_scan<T, G, kBack, kPacked, kVec>, static_cast<const Args>(a));
    note_launch(stream, kBack ? "gated_backward" : "gated_forward");
    return e;
}

template <typename T, typename G>
cudaError_t run_t(Args& a, bool back, cudaStream_t stream) {
    const bool vec = a.p.D % 4 == 0;
    auto go = [&](auto kback, auto kpacked) {
        constexpr bool kB = decltype(kback)::value, kP = decltype(kpacked)::value;
        return vec ? launch_scan<T, G, kB, kP, true>(a, stream) : launch_scan<T, G, kB, kP, false>(a, stream);
    };
    using yes = std::true_type;
    using no = std::false_type;
    if (a.p.cu) return back ? go(yes(), yes()) : go(no(), yes());
    return back ? go(yes(), no()) : go(no(), no());
}

// ---- single tokens

template <typename T, typename G>
__global__ void __launch_bounds__(kThreads) gated_step(const T* __restrict__ x, const G* __restrict__ log_a,
                                                       float* __restrict__ state, T* __restrict__ out, int64_t size) {
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * 4;
    if (i >= size) return;
    if (i + 4 <= size) {
        float f[4], g[4], h[4];
        widen(*reinterpret_cast<const typename Four<T>::raw*>(x + i), f);
        widen(*reinterpret_cast<const typename Four<G>::raw*>(log_a + i), g);
        widen(*reinterpret_cast<const float4*>(state + i), h);
#pragma unroll
        for (int v = 0; v < 4; v++) h[v] = fmaf(expf(g[v]), h[v], f[v]);
        put4(state + i, h);
        put4(out + i, h);
        return;
    }
    for (int64_t j = i; j < size; j++) {
        const float h = fmaf(expf(load_f(log_a + j)), state[j], load_f(x + j));
        state[j] = h;
        store_f(out + j, h);
    }
}

// ---- trees: a thread per channel walks the nodes in order; parents come before their children, whose states it keeps in
// shared memory.
constexpr int kTreeThreads = 64;

template <typename T, typename G>
__global__ void __launch_bounds__(kTreeThreads) gated_tree(const T* __restrict__ x, const G* __restrict__ log_a,
                                                           const float* __restrict__ state,
                                                           const int32_t* __restrict__ parent, T* __restrict__ out,
                                                           int BP, int N, int D, int* err) {
    __shared__ int par[kMaxTree];
    extern __shared__ float hs[];  // [N][kTreeThreads]
    const int tid = threadIdx.x, b = blockIdx.y, c = blockIdx.x * kTreeThreads + tid;
    for (int i = tid; i < N; i += kTreeThreads) par[i] = parent[(BP > 1 ? static_cast<int64_t>(b) * N : 0) + i];
    __syncthreads();
    if (tree_is_bad(par, N)) {
        if (tid == 0) record_error(err, kDevBadInput);
        return;
    }
    if (c >= D) return;
    const float h0 = state[static_cast<int64_t>(b) * D + c];
    const int64_t at = static_cast<int64_t>(b) * N * D + c;
    for (int i0 = 0; i0 < N; i0 += 8) {
        float xi[8], gi[8];
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (i0 + j < N) {
                xi[j] = load_f(x + at + static_cast<int64_t>(i0 + j) * D);
                gi[j] = expf(load_f(log_a + at + static_cast<int64_t>(i0 + j) * D));
            }
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (i0 + j < N) {
                const int pi = par[i0 + j];
                if (pi == -2) continue;
                const float h = fmaf(gi[j], pi < 0 ? h0 : hs[pi * kTreeThreads + tid], xi[j]);
                hs[(i0 + j) * kTreeThreads + tid] = h;
                store_f(out + at + static_cast<int64_t>(i0 + j) * D, h);
            }
    }
}

template <typename T, typename G>
__global__ void __launch_bounds__(kTreeThreads) gated_commit(const T* __restrict__ x, const G* __restrict__ log_a,
                                                             float* __restrict__ state,
                                                             const int32_t* __restrict__ count,
                                                             const int32_t* __restrict__ path, int N, int M, int D,
                                                             int* err) {
    __shared__ int node[kMaxTree];
    const int tid = threadIdx.x, b = blockIdx.y, c = blockIdx.x * kTreeThreads + tid;
    const int n = count[b];
    bool bad = n < 0 || n > M;
    if (!bad)
        for (int i = tid; i < n; i += kTreeThreads) {
            const int at = path ? path[static_cast<int64_t>(b) * M + i] : i;
            bad |= at < 0 || at >= N;
            node[i] = at;
        }
    if (__syncthreads_or(bad)) {
        if (tid == 0) record_error(err, kDevBadInput);
        return;
    }
    if (c >= D || n == 0) return;
    float h = state[static_cast<int64_t>(b) * D + c];
    const int64_t at = static_cast<int64_t>(b) * N * D + c;
    for (int i = 0; i < n; i++)
        h = fmaf(expf(load_f(log_a + at + static_cast<int64_t>(node[i]) * D)), h,
                 load_f(x + at + static_cast<int64_t>(node[i]) * D));
    state[static_cast<int64_t>(b) * D + c] = h;
}

// f(T(), G()) for the call's types
template <typename F>
cudaError_t by_types(int dtype, int gate_dtype, F f) {
    if (dtype == 1) return f(float(), float());
    return gate_dtype == 1 ? f(__nv_bfloat16(), float()) : f(__nv_bfloat16(), __nv_bfloat16());
}

}  // namespace

cudaError_t gated_run(const GatedPass& p, bool backward, int dtype, int gate_dtype, int* err, cudaStream_t stream) {
    Args a = {};
    a.p = p;
    a.err = err;
    a.cols = (p.D - 1) / kCols + 1;
    const int64_t walks = static_cast<int64_t>(a.cols) * (p.cu ? 1 : p.n);
    const int pieces = (p.T - 1) / kRows + 1;
    a.cluster = 1;
    while (a.cluster < kMaxCluster && walks * a.cluster < 256 && a.cluster < pieces) a.cluster *= 2;
    a.steps = (pieces - 1) / a.cluster + 1;
    return by_types(dtype, gate_dtype, [&](auto t, auto g) { return run_t<decltype(t), decltype(g)>(a, backward, stream); });
}

cudaError_t gated_decode_step(int dtype, int gate_dtype, const void* x, const void* log_a, float* state, void* out,
                              int64_t size, cudaStream_t stream) {
    return by_types(dtype, gate_dtype, [&](auto t, auto g) {
        using T = decltype(t);
        using G = decltype(g);
        gated_step<T, G><<<static_cast<unsigned>((size + 4 * kThreads - 1) / (4 * kThreads)), kThreads, 0, stream>>>(
            static_cast<const T*>(x), static_cast<const G*>(log_a), state, static_cast<T*>(out), size);
        note_launch(stream, "gated_step");
        return cudaGetLastError();
    });
}

cudaError_t gated_decode_tree(int dtype, int gate_dtype, const void* x, const void* log_a, const float* state,
                              const int32_t* parent, void* out, int B, int BP, int N, int D, int* err,
                              cudaStream_t stream) {
    return by_types(dtype, gate_dtype, [&](auto t, auto g) {
        using T = decltype(t);
        using G = decltype(g);
        gated_tree<T, G><<<dim3((D - 1) / kTreeThreads + 1, B), kTreeThreads, N * kTreeThreads * sizeof(float), stream>>>(
            static_cast<const T*>(x), static_cast<const G*>(log_a), state, parent, static_cast<T*>(out), BP, N, D, err);
        note_launch(stream, "gated_tree");
        return cudaGetLastError();
    });
}

cudaError_t gated_decode_commit(int dtype, int gate_dtype, const void* x, const void* log_a, float* state,
                                const int32_t* count, const int32_t* path, int B, int N, int M, int D, int* err,
                                cudaStream_t stream) {
    return by_types(dtype, gate_dtype, [&](auto t, auto g) {
        using T = decltype(t);
        using G = decltype(g);
        gated_commit<T, G><<<dim3((D - 1) / kTreeThreads + 1, B), kTreeThreads, 0, stream>>>(
            static_cast<const T*>(x), static_cast<const G*>(log_a), state, count, path, N, M, D, err);
        note_launch(stream, "gated_commit");
        return cudaGetLastError();
    });
}

}  // namespace lla
