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
// block cluster walks 64 (32, 16) channels of one sequence from end to end in steps of (cluster size) x 128 (256, 512)
// rows: a thread keeps 8 rows of 4 channels, forms their map, the warps and the block compose them, the blocks send their
// maps to one another through distributed shared memory, and every thread runs its rows again from the state that enters
// them. Blocks of a cluster are resident together, so nothing waits for a block that may not run yet, and neither flags
// nor workspace are needed. Maps are composed in one fixed order: repeated calls give identical bits.
//
// Bound by HBM: 4 x 8192 x 1024, bf16 with fp32 gates, 43 us for 268 MB (91% of the copy rate), gradients 76 us for 470 MB
// (91%); 65536 x 1024 with bf16 gates 67 us for 403 MB (88%; a step's latency, about 2 us with the exchange, shows). What
// got it there: tiles by TMA two steps ahead (69 us with per-thread asynchronous copies, which cost a quarter of all
// instructions and pass through L1), the exchange by stores that signal a barrier (a cluster barrier waits for the step's
// stores to global memory besides: 0.7 us a step), steps without questions asked of a row, two channels to an instruction.
//
// Packed sequences are one row axis: a map that holds a sequence's first row does not depend on what enters. Its A is
// kept as -1 (a product of exponentials is never negative), so that not even an infinity or NaN crosses over.
#include "lla_drafts.cuh"
#include "lla_linear.cuh"
#include "lla_tc_ptx.cuh"

namespace lla {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kFill = 152;    // blocks that a call should have: one for each SM of the GPU
constexpr int kMaxBox = 256;  // rows of a TMA copy

// How rows come to a thread: through shared memory by TMA (rows of a multiple of 16 bytes), or by its own loads a step
// ahead, four channels at a time (D a multiple of 4) or one.
enum Path { kTma, kQuads, kSingles };

// Cut of a block: kLanes threads side by side, four channels each; every thread kL rows. kStages steps' tiles are in flight.
template <typename T, typename G, bool kBack, int kPath>
struct Cut {
    static constexpr int row_bytes = 4 * (sizeof(G) + sizeof(T) * (kBack ? 2 : 1));  // of a thread's row
    static constexpr int kL = kPath == kTma ? 8 : 4;  // kTma with 4 and three stages: 49 us against 43 (4 x 8192 x 1024)
    static constexpr int kStages = 2;
    static constexpr int stage_bytes = row_bytes * kL * kThreads;
    static constexpr int kResident = kPath == kTma && stage_bytes * kStages > 110000 ? 1 : 2;  // blocks of an SM
};

struct Args {
    CUtensorMap map[3];  // kTma: gates; inputs (backward: dout); backward: the forward's outputs
    GatedPass p;
    int cluster, cols;
    int spans;  // packed: parts of the row axis, cut where sequences begin
    LinWaits waits;
    int* err;
};

// Four channels as two register pairs: one instruction for two of them.
struct Quad {
    f32x2 lo, hi;
};
__device__ __forceinline__ Quad quad(const float (&f)[4]) { return {pair2(f[0], f[1]), pair2(f[2], f[3])}; }
__device__ __forceinline__ void split(const Quad& q, float (&f)[4]) {
    const float2 a = split2(q.lo), b = split2(q.hi);
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}
__device__ __forceinline__ Quad mul(const Quad& a, const Quad& b) { return {mul2(a.lo, b.lo), mul2(a.hi, b.hi)}; }
__device__ __forceinline__ Quad fma(const Quad& a, const Quad& b, const Quad& c) {
    return {fma2(a.lo, b.lo, c.lo), fma2(a.hi, b.hi, c.hi)};
}
// exp. kFine: by expf (within 2.5 x 2^-24 of the value wherever measured), as single tokens, trees and commits form their gates.
// Else by the power of two of a rounded product with log2 e: within (|log_a| + 2) x 2^-24 wherever measured, and 0 for gates
// below fp32's normal numbers. That is what a prompt's gates of 16 bits get, whose own step is 2^15 times as wide as what the
// product rounds away: 65536 x 1024 take 67 us so, 78 by expf, whose instructions lie on the step's chain. Other passes feel
// them less: prompts of 4 x 8192 x 1024 with fp32 gates take 43.0 and 43.4 us, their gradients 74.6 and 76, those in fp32 108
// and 114, those with gates of 16 bits 66 and 58.
__device__ __forceinline__ float power2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
template <bool kFine>
__device__ __forceinline__ Quad gate(const Quad& log_a) {
    float f[4];
    if constexpr (kFine) {
        split(log_a, f);
    } else {
        const f32x2 k = pair2(kLog2e, kLog2e);
        split({mul2(log_a.lo, k), mul2(log_a.hi, k)}, f);
    }
#pragma unroll
    for (int v = 0; v < 4; v++) f[v] = kFine ? expf(f[v]) : power2(f[v]);
    return quad(f);
}

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

// Four channels of a row: neighbours (kVec; D a multiple of 4), or kLanes apart, so that a scalar access of kLanes threads
// is one stretch of memory.
template <bool kVec, int kLanes>
struct Chan {
    int c[4];
    bool any;
    int D;
    __device__ __forceinline__ Chan(int col, int lane, int D_) : D(D_) {
#pragma unroll
        for (int v = 0; v < 4; v++) c[v] = col * kLanes * 4 + at(lane, v);
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
    __device__ __forceinline__ static int at(int lane, int v) { return kVec ? lane * 4 + v : lane + kLanes * v; }
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// All blocks of the cluster have got here. No order of memory goes with it (kInit: but the barriers set up before it), so
// nobody waits for stores to global memory to land.
template <bool kInit>
__device__ __forceinline__ void cluster_meet() {
    if (kInit) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    else asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// (x, y) to the place `at` of block `rank`, counted by that block's barrier `bar` when it is there
__device__ __forceinline__ void send(uint32_t at, uint32_t bar, uint32_t rank, float x, float y) {
    uint32_t to, sign;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(at), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(sign) : "r"(bar), "r"(rank));
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(to),
                 "f"(x), "f"(y), "r"(sign)
                 : "memory");
}
__device__ __forceinline__ bool arrived(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "n"(kSuspendNs)
        : "memory");
    return ok != 0;
}

// Bounded wait for a phase of a barrier; what ran out is recorded, for the block in `late`.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, long long limit, int* err, int* late) {
    if (arrived(bar, parity)) return true;
    const long long start = clock64();
    while (!arrived(bar, parity))
        if (clock64() - start > limit) {
            record_error(err, kDevTimeout);
            *late = 1;
            return false;
        }
    return true;
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
// Of a row between an entry of cu, `here`, and the next one
template <bool kBack>
__device__ __forceinline__ int row_flags(int entry, int here, int next, int n, int row) {
    const bool first = row == here, last = row == next - 1;
    return entry < 0 || entry >= n ? -1 : entry | ((kBack ? last : first) ? kBegins : 0) | ((kBack ? first : last) ? kEnds : 0);
}
// The last entry of cu that is not behind the row is at `lo` or above, below `hi`; at(i) is entry i, and one in front of the
// table (i = -1) is in front of every row.
template <bool kBack, typename At>
__device__ __forceinline__ int row_info(At at, int lo, int hi, int n, int row) {
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at(mid) <= row) lo = mid;
        else hi = mid;
    }
    if (lo < 0 || lo >= n) return -1;
    return row_flags<kBack>(lo, at(lo), at(lo + 1), n, row);
}
constexpr int kWindow = 32;  // entries of cu around a block's rows
constexpr int kFew = 8;      // of them that are compared side by side, where the next one lies behind the rows

// Four channels of a row as they lie in memory, loaded before they are needed.
template <typename T, bool kVec>
struct Ahead;
template <typename T>
struct Ahead<T, true> {
    typename Four<T>::raw r;
    __device__ __forceinline__ void load(const T* row, const Chan<true, 16>& ch) {
        if (ch.any) r = __ldg(reinterpret_cast<const typename Four<T>::raw*>(row + ch.c[0]));
    }
    __device__ __forceinline__ void get(float (&f)[4]) const { widen(r, f); }
};
template <typename T>
struct Ahead<T, false> {
    T r[4];
    __device__ __forceinline__ void load(const T* row, const Chan<false, 16>& ch) {
#pragma unroll
        for (int v = 0; v < 4; v++)
            if (ch.c[v] < ch.D) r[v] = row[ch.c[v]];
    }
    __device__ __forceinline__ void get(float (&f)[4]) const {
#pragma unroll
        for (int v = 0; v < 4; v++) f[v] = load_f(&r[v]);
    }
};

// Registers: where shared memory holds one block of an SM, its threads have all of them (fp32 gradients of 16 packed documents of
// 100 to 4000 rows of 512 channels: 55 us, with registers for two blocks 78), but for dense fp32, where the loads that the
// compiler then moves together cost more than they save (gradients of 4 x 8192 x 1024: 114 us for two blocks, 118).
template <typename T, typename G, bool kBack, bool kPacked, int kPath>
constexpr int kBlocks = kPacked || sizeof(T) == 2 ? Cut<T, G, kBack, kPath>::kResident : 2;

template <typename T, typename G, bool kBack, bool kPacked, int kPath, int kLanes>
__global__ void __launch_bounds__(kThreads, (kBlocks<T, G, kBack, kPacked, kPath>)) gated_scan(const __grid_constant__ Args a) {
    using C = Cut<T, G, kBack, kPath>;
    constexpr bool kVec = kPath != kSingles, kFine = kBack || sizeof(G) == 4;
    using Ch = Chan<kVec, kLanes>;
    constexpr int kCols = kLanes * 4;               // channels of a block
    constexpr int kL = C::kL, kStages = C::kStages;
    constexpr int kRows = kThreads / kLanes * kL;   // rows of a block
    constexpr int kStep = 32 / kLanes;              // stretches of a warp
    constexpr int kBoxRows = kRows < kMaxBox ? kRows : kMaxBox;
    __shared__ __align__(16) float warp_a[2][kWarps][kCols], warp_s[2][kWarps][kCols];
    __shared__ __align__(16) float2 part[2][kMaxCluster][kCols];
    __shared__ __align__(16) float carry[2][kCols];
    __shared__ int info[2][kPacked ? kRows : 1];
    __shared__ int late, bounds[4], plain_of[2], near[2], window[2][kPacked ? kWindow : 1];
    __shared__ __align__(8) uint64_t come[2], full[kStages], never;
    extern __shared__ __align__(128) char staged[];
    const GatedPass& p = a.p;
    const int tid = threadIdx.x, lane = tid % kLanes, seg = tid / kLanes, warp = tid / 32;
    const int R = p.T, D = p.D, cs = a.cluster;
    const int rank = cs > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int walk = blockIdx.x / cs;  // cluster: a column of one sequence (packed: of one span)
    const int col = walk % a.cols, b = walk / a.cols;
    const Ch ch(col, lane, D);
    int lo = 0, hi = R;  // the walk's rows
    if (kPacked) {
        // a span's sequences are those that begin in its even share of the rows; the first and the last one also have the
        // rows of no sequence before and behind
        const int64_t cut0 = static_cast<int64_t>(R) * b / a.spans, cut1 = static_cast<int64_t>(R) * (b + 1) / a.spans;
        if (tid < 4) bounds[tid] = tid < 2 ? R : 0;
        __syncthreads();
        bool bad = false;
        int first = R, next = R, before = 0, upto = 0;
        for (int i = tid; i <= p.n; i += kThreads) {
            const int x = p.cu[i];
            bad |= x < 0 || x > R || (i > 0 && x < p.cu[i - 1]);
            if (x < cut0) before++;
            else if (x < first) first = x;
            if (x < cut1) upto++;
            else if (x < next) next = x;
        }
        first = __reduce_min_sync(0xffffffffu, first);
        next = __reduce_min_sync(0xffffffffu, next);
        before = __reduce_add_sync(0xffffffffu, before);
        upto = __reduce_add_sync(0xffffffffu, upto);
        if ((tid & 31) == 0) {
            atomicMin(&bounds[0], first);
            atomicMin(&bounds[1], next);
            atomicAdd(&bounds[2], before);
            atomicAdd(&bounds[3], upto);
        }
        if (__syncthreads_or(bad)) {  // every block finds the same
            if (blockIdx.x == 0 && tid == 0) record_error(a.err, kDevBadInput);
            return;
        }
        lo = b == 0 ? 0 : bounds[0];
        hi = b == a.spans - 1 ? R : bounds[1];
    }
    const int len = hi - lo, steps = (len + cs * kRows - 1) / (cs * kRows);
    if (tid == 0) {
        mbar_init(&come[0], 1);
        mbar_init(&come[1], 1);
        mbar_init(&never, 1);
        late = 0;
        for (int i = 0; i < kStages; i++) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    if (cs > 1) cluster_meet<true>();
    else __syncthreads();
    const float* enter = kBack ? p.dstate_out : p.state0;  // what a walk begins with
    const int64_t row0 = kPacked ? 0 : static_cast<int64_t>(b) * R;
    const T* xp = static_cast<const T*>(p.x) + row0 * D;  // inputs; backward: outputs of the forward
    const G* gp = static_cast<const G*>(p.log_a) + row0 * D;
    const T* dp = kBack ? static_cast<const T*>(p.dout) + row0 * D : nullptr;
    T* op = static_cast<T*>(p.out) + row0 * D;
    G* ap = kBack ? static_cast<G*>(p.dlog_a) + row0 * D : nullptr;
    auto enters = [&](int i) { return enter + static_cast<int64_t>(kBack || p.n0 > 1 ? i : 0) * D; };
    auto first_state = [&](int i) { return p.state0 + static_cast<int64_t>(p.n0 > 1 ? i : 0) * D; };

    // Rows a step ahead. kTma: the block's tiles, rows in the order of memory, in one stage: gates, inputs (backward: dout),
    // and backward the outputs of the row before. Parts of a tile outside the walk belong to others or to nobody and are
    // not used.
    constexpr int kGBytes = kRows * kCols * sizeof(G), kXBytes = kRows * kCols * sizeof(T);
    Ahead<G, kVec> ga[kPath == kTma ? 1 : kL];
    Ahead<T, kVec> xa[kPath == kTma ? 1 : kL], ha[kPath == kTma || !kBack ? 1 : kL];
    int issued = 0;  // kTma, thread 0: steps whose tiles are on their way or there
    auto prefetch = [&](int st) {
        if (st >= steps) return;
        if constexpr (kPath == kTma) {
            if (tid == 0) {
                char* to = staged + (st % kStages) * C::stage_bytes;
                uint64_t* bar = &full[st % kStages];
                const int u = (st * cs + rank) * kRows;
                const int y = static_cast<int>(row0) + (kBack ? hi - u - kRows : lo + u);
                mbar_expect_tx(bar, kGBytes + (kBack ? 2 : 1) * kXBytes);
                for (int r = 0; r < kRows; r += kBoxRows) {
                    tma_load_2d(to + r * kCols * sizeof(G), &a.map[0], bar, col * kCols, y + r);
                    tma_load_2d(to + kGBytes + r * kCols * sizeof(T), &a.map[1], bar, col * kCols, y + r);
                    if (kBack) tma_load_2d(to + kGBytes + kXBytes + r * kCols * sizeof(T), &a.map[2], bar, col * kCols, y + r - 1);
                }
                issued = st + 1;
            }
        } else {
            const int u0 = (st * cs + rank) * kRows + seg * kL;
#pragma unroll
            for (int j = 0; j < kL; j++) {
                const int u = u0 + j;
                const int64_t off = static_cast<int64_t>(kBack ? hi - 1 - u : lo + u) * D;
                if (u < len) {
                    ga[j].load(gp + off, ch);
                    xa[j].load((kBack ? dp : xp) + off, ch);
                    if (kBack && off > 0) ha[kBack ? j : 0].load(xp + off - D, ch);
                }
            }
        }
    };
    for (int st = 0; st < (kPath == kTma ? kStages : 1); st++) prefetch(st);

    if (kPacked && p.leave) {  // empty sequences: what enters leaves
        for (int i = (b * cs + rank) * (kThreads / kLanes) + seg; i < p.n; i += a.spans * cs * (kThreads / kLanes)) {
            if (p.cu[i] != p.cu[i + 1]) continue;
            float f[4] = {0.f, 0.f, 0.f, 0.f};
            if (enter) ch.load(enters(i), f);
            ch.store(p.leave + static_cast<int64_t>(i) * D, f);
        }
    }

    const int my_col = col * kCols + tid;  // of the first kCols threads, which carry the walk's state
    float state = 0.f;
    if (!kPacked && enter && tid < kCols && my_col < D) state = enters(b)[my_col];

    // Packed: the last warp finds ahead of each step whether a sequence begins or ends in the block's rows [y, y + kRows),
    // and lays out the entries of cu around them: `entry` follows the walk, the first one that is not before y.
    int entry = kPacked ? bounds[kBack ? 3 : 2] : 0;
    auto look = [&](int st) {
        const int u = (st * cs + rank) * kRows, l = tid & 31, y = kBack ? hi - u - kRows : lo + u;
        for (int n = 32; n == 32;) {
            const int i = kBack ? entry - 1 - l : entry + l;
            const int x = i < 0 || i > p.n ? 0 : p.cu[i];
            n = __popc(__ballot_sync(0xffffffffu, i >= 0 && i <= p.n && (kBack ? x >= y : x < y)));
            entry += kBack ? -n : n;
        }
        const int e = entry - 1 + l, x = e < 0 ? -1 : e > p.n ? 0x7fffffff : p.cu[e];
        window[st & 1][l] = x;
        if (l == 0) near[st & 1] = entry - 1;
        if (l == 1) plain_of[st & 1] = entry > 0 && entry <= p.n && x > y + kRows;
        // states that walks begin with in these rows
        if (enter && e >= 0 && e < p.n && (kBack ? x < y + kRows : l > 0 && x < y + kRows)) prefetch_l1(enters(e) + col * kCols);
    };
    if (kPacked) {
        if (warp == kWarps - 1) look(0);
        __syncthreads();
    }

    // After a wait that ran out a walk goes on to its end without waiting, sending or copying, its values undefined.
    bool in_time = !a.waits.hold || wait(&never, 0, a.waits.cycles, a.err, &late);
    for (int st = 0; st < steps; st++) {
        const int buf = st & 1;
        const int block0 = (st * cs + rank) * kRows, u0 = block0 + seg * kL;
        // Whether the block's rows and channels are all there and no row is a sequence's first or last: the common step,
        // without a question asked of a row.
        bool plain = kVec && (col + 1) * kCols <= D && block0 + kRows <= len - (kBack && !kPacked ? 1 : 0);
        if (kPacked) {
            plain &= plain_of[buf] != 0;
            if (!plain) {
                const int base = near[buf];  // entry of window[buf][0]
                const int last = kBack ? hi - 1 - block0 : lo + block0 + kRows - 1;
                const bool few = window[buf][kFew] > last, enough = window[buf][kWindow - 1] > last;
                int w[kFew];
#pragma unroll
                for (int e = 0; e < kFew; e++) w[e] = window[buf][e];
                for (int i = tid; i < kRows; i += kThreads) {
                    const int u = block0 + i, row = kBack ? hi - 1 - u : lo + u;
                    int inf = -1;
                    if (u < len && few) {  // side by side
                        int at = 0, here = w[0], next = window[buf][kFew];
#pragma unroll
                        for (int e = 1; e < kFew; e++)
                            if (w[e] <= row) {
                                at = e;
                                here = w[e];
                            }
#pragma unroll
                        for (int e = kFew - 1; e > 0; e--)
                            if (w[e] > row) next = w[e];
                        inf = row_flags<kBack>(base + at, here, next, p.n, row);
                    } else if (u < len && enough) {
                        inf = row_info<kBack>([&](int e) { return window[buf][e - base]; }, base, base + kWindow - 1, p.n, row);
                    } else if (u < len) {
                        inf = row_info<kBack>([&](int e) { return e < 0 ? -1 : p.cu[e]; }, base, p.n + 1, p.n, row);
                    }
                    info[buf][i] = inf;
                }
                __syncthreads();
            }
        }
        // places of this thread's first row in the stage, and from one row to the next
        constexpr int kNextG = (kBack ? -1 : 1) * kCols * static_cast<int>(sizeof(G));
        constexpr int kNextX = (kBack ? -1 : 1) * kCols * static_cast<int>(sizeof(T));
        const int at = (kBack ? kRows - 1 - seg * kL : seg * kL) * kCols + lane * 4;
        const char* sg = staged + (st % kStages) * C::stage_bytes + at * sizeof(G);
        const char* sx = staged + (st % kStages) * C::stage_bytes + kGBytes + at * sizeof(T);
        auto gates_of = [&](int j, float (&f)[4]) {
            if constexpr (kPath == kTma) widen(*reinterpret_cast<const typename Four<G>::raw*>(sg + j * kNextG), f);
            else ga[j].get(f);
        };
        auto inputs_of = [&](int j, float (&f)[4]) {
            if constexpr (kPath == kTma) widen(*reinterpret_cast<const typename Four<T>::raw*>(sx + j * kNextX), f);
            else xa[j].get(f);
        };
        Quad g[kL], x[kL];
        Ahead<T, kVec> hp[kBack ? kL : 1];
        float A[4], s[4];
        if (kPath == kTma && in_time) in_time = wait(&full[st % kStages], (st / kStages) & 1, a.waits.cycles, a.err, &late);
        if (kBack) {
#pragma unroll
            for (int j = 0; j < kL; j++) {
                if constexpr (kPath == kTma) hp[j].r = *reinterpret_cast<const typename Four<T>::raw*>(sx + kXBytes + j * kNextX);
                else hp[j] = ha[j];
            }
        }
        if (plain) {
            Quad pa, ps;
#pragma unroll
            for (int j = 0; j < kL; j++) {
                float f[4];
                gates_of(j, f);
                g[j] = gate<kFine>(quad(f));
                inputs_of(j, f);
                x[j] = quad(f);
                const Quad in = kBack ? mul(g[j], x[j]) : x[j];
                ps = j == 0 ? in : fma(g[j], ps, in);
                pa = j == 0 ? g[j] : mul(g[j], pa);
            }
            split(pa, A);
            split(ps, s);
        } else {
            bool begun = false;
#pragma unroll
            for (int v = 0; v < 4; v++) {
                A[v] = 1.f;
                s[v] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < kL; j++) {
                const int inf = kPacked ? info[buf][seg * kL + j] : 0;
                const bool in = kPacked ? inf >= 0 : u0 + j < len, begins = kPacked && in && (inf & kBegins);
                float gf[4] = {0.f, 0.f, 0.f, 0.f}, xf[4] = {0.f, 0.f, 0.f, 0.f};
                if (kPacked || in) {
                    gates_of(j, gf);
                    inputs_of(j, xf);
                }
                if (kPacked) {  // selects; a branch only where a state enters
#pragma unroll
                    for (int v = 0; v < 4; v++) {
                        gf[v] = in ? gf[v] : 0.f;
                        xf[v] = in ? xf[v] : 0.f;
                        s[v] = begins ? 0.f : s[v];
                    }
                    if (enter && begins) ch.load(enters(inf & kSeq), s);
                    begun |= begins;
                }
                g[j] = gate<kFine>(quad(gf));
                x[j] = quad(xf);
                split(g[j], gf);
#pragma unroll
                for (int v = 0; v < 4; v++) {
                    s[v] = kBack ? fmaf(gf[v], s[v], gf[v] * xf[v]) : fmaf(gf[v], s[v], xf[v]);
                    A[v] *= gf[v];
                }
            }
            if (begun) {
#pragma unroll
                for (int v = 0; v < 4; v++) A[v] = -1.f;
            }
        }
        if (kPath != kTma) prefetch(st + 1);
        // the maps of the warp's stretches up to this thread's, and before it
        float ea[4], es[4];
#pragma unroll
        for (int v = 0; v < 4; v++) {
#pragma unroll
            for (int d = kLanes; d < 32; d *= 2) {
                const float pa = __shfl_up_sync(0xffffffffu, A[v], d), ps = __shfl_up_sync(0xffffffffu, s[v], d);
                if ((tid & 31) >= d) {
                    float na = pa, ns = ps;
                    compose<kPacked>(na, ns, A[v], s[v]);
                    A[v] = na;
                    s[v] = ns;
                }
            }
            ea[v] = __shfl_up_sync(0xffffffffu, A[v], kLanes);
            es[v] = __shfl_up_sync(0xffffffffu, s[v], kLanes);
        }
        if ((tid & 31) / kLanes == kStep - 1) {
#pragma unroll
            for (int v = 0; v < 4; v++) {
                warp_a[buf][warp][Ch::at(lane, v)] = A[v];
                warp_s[buf][warp][Ch::at(lane, v)] = s[v];
            }
        }
        __syncthreads();
        if (kPath == kTma && in_time) prefetch(st + kStages);  // into the stage that all have read
        if (kPacked && warp == kWarps - 1 && st + 1 < steps) look(st + 1);
        if (tid < kCols) {
            float own_a = 1.f, own_s = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; i++) {
                const float A2 = warp_a[buf][i][tid], s2 = warp_s[buf][i][tid];
                warp_a[buf][i][tid] = own_a;
                warp_s[buf][i][tid] = own_s;
                compose<kPacked>(own_a, own_s, A2, s2);
            }
            if (cs > 1) {
                // A place is written again two steps later, by a thread that has by then what this one's block sent a step
                // later, after it had read the place.
                if (in_time) {
                    if (tid == 0) mbar_expect_tx(&come[buf], static_cast<uint32_t>(cs) * kCols * sizeof(float2));
                    const uint32_t to = smem_u32(&part[buf][rank][tid]), sign = smem_u32(&come[buf]);
                    for (int r = 0; r < cs; r++) send(to, sign, r, own_a, own_s);
                    in_time = wait(&come[buf], (st >> 1) & 1, a.waits.cycles, a.err, &late);
                }
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
            const int c = Ch::at(lane, v);
            h[v] = apply<kPacked>(warp_a[buf][warp][c], warp_s[buf][warp][c], carry[buf][c]);
            if ((tid & 31) >= kLanes) h[v] = apply<kPacked>(ea[v], es[v], h[v]);
        }
        if (plain) {
            const int64_t first = static_cast<int64_t>(kBack ? hi - 1 - u0 : lo + u0) * D + ch.c[0];
            const int64_t next = kBack ? -static_cast<int64_t>(D) : static_cast<int64_t>(D);
            T* o = op + first;
            G* da = kBack ? ap + first : nullptr;
            Quad q = quad(h);
#pragma unroll
            for (int j = 0; j < kL; j++) {
                float f[4];
                if constexpr (kBack) {
                    float before[4];
                    hp[j].get(before);
                    q = {add2(x[j].lo, q.lo), add2(x[j].hi, q.hi)};
                    split(q, f);
                    put4(o, f);
                    q = mul(g[j], q);
                    split(mul(q, quad(before)), f);
                    put4(da, f);
                    da += next;
                } else {
                    q = fma(g[j], q, x[j]);
                    split(q, f);
                    put4(o, f);
                }
                o += next;
            }
        } else {
#pragma unroll
            for (int j = 0; j < kL; j++) {
                const int u = u0 + j, row = kBack ? hi - 1 - u : lo + u;
                const int inf = kPacked ? info[buf][seg * kL + j] : 0;
                if (!kPacked && u >= len) continue;
                const bool in = inf >= 0, begins = kPacked && in && (inf & kBegins);
                const bool ends = kPacked ? in && (inf & kEnds) : row == 0;
                const int64_t off = static_cast<int64_t>(row) * D;
                if (kPacked) {
#pragma unroll
                    for (int v = 0; v < 4; v++) h[v] = begins ? 0.f : h[v];
                    if (enter && begins) ch.load(enters(inf & kSeq), h);
                }
                float gf[4], xf[4];
                split(g[j], gf);
                split(x[j], xf);
                if constexpr (kBack) {
                    float before[4] = {0.f, 0.f, 0.f, 0.f}, d[4], da[4];
                    if constexpr (kPacked) {
                        hp[j].get(before);
#pragma unroll
                        for (int v = 0; v < 4; v++) before[v] = ends ? 0.f : before[v];
                        if (ends && p.state0) ch.load(first_state(inf & kSeq), before);
                    } else {
                        if (!ends) hp[j].get(before);
                        else if (p.state0) ch.load(first_state(b), before);
                    }
#pragma unroll
                    for (int v = 0; v < 4; v++) {
                        d[v] = xf[v] + h[v];
                        h[v] = gf[v] * d[v];
                        da[v] = h[v] * before[v];
                        if constexpr (kPacked) {  // rows of no sequence take no part in the sum that is differentiated
                            d[v] = in ? d[v] : 0.f;
                            da[v] = in ? da[v] : 0.f;
                        }
                    }
                    if (!kPacked || u < len) {
                        ch.store(op + off, d);
                        ch.store(ap + off, da);
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < 4; v++) h[v] = fmaf(gf[v], h[v], xf[v]);
                    if (!kPacked || in) ch.store(op + off, h);
                }
                if (kPacked && p.leave && ends) ch.store(p.leave + static_cast<int64_t>(inf & kSeq) * D, h);
            }
        }
    }
    if (!kPacked && p.leave && rank == 0 && tid < kCols && my_col < D)
        p.leave[static_cast<int64_t>(b) * D + my_col] = state;
    // no block leaves while its own copies are under way, or while another may still write to it
    if (kPath == kTma && tid == 0)
        for (int st = issued < kStages ? 0 : issued - kStages; st < issued; st++)
            wait(&full[st % kStages], (st / kStages) & 1, kWaitCycles, a.err, &late);
    if (cs > 1) {
        cluster_meet<false>();
        // The block's own waits took in all that others sent it. One that ran out did not: a block that came late may have sent
        // its maps just before it got here, so stay for half a millisecond, whatever the bound is (those stores take microseconds).
        if (late) wait(&never, 0, 1 << 20, a.err, &late);
    }
}

// The gradient of a state that n sequences share: their parts summed in order. Launched while the scan ends (its results are
// read behind the wait); it writes nothing either where cu is bad.
__global__ void __launch_bounds__(kThreads) gated_sum(const float* parts, float* out, const int32_t* __restrict__ cu, int n,
                                                      int T, int D) {
    bool bad = false;
    if (cu)
        for (int i = threadIdx.x; i <= n; i += kThreads) {
            const int x = cu[i];
            bad |= x < 0 || x > T || (i > 0 && x < cu[i - 1]);
        }
    bad = __syncthreads_or(bad);
    grid_dep_wait();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (bad || c >= D) return;
    float s = 0.f;
#pragma unroll 8
    for (int b = 0; b < n; b++) s += parts[static_cast<int64_t>(b) * D + c];
    out[c] = s;
}

// Tile map of a tensor [rows, D]
bool tile_map(CUtensorMap* m, const void* base, bool f32, int64_t rows, int D, int cols, int box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(D) * (f32 ? 4 : 2)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(cols), static_cast<cuuint32_t>(box_rows)}, one[2] = {1, 1};
    return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
              strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, typename G, bool kBack, bool kPacked, int kPath, int kLanes>
cudaError_t launch_scan(Args& a, cudaStream_t stream) {
    using C = Cut<T, G, kBack, kPath>;
    auto kern = gated_scan<T, G, kBack, kPacked, kPath, kLanes>;
    constexpr int kRows = kThreads / kLanes * C::kL;
    a.cols = (a.p.D - 1) / (kLanes * 4) + 1;
    const int pieces = (a.p.T - 1) / kRows + 1;
    a.spans = kPacked ? 1 : a.p.n;
    // The smallest cluster that gives every SM a block: an exchange costs about as much as a step of 1 us (4 x 8192 x 1024:
    // clusters of 1, 2, 4, 8 take 70, 46, 44, 49 us; one sequence of 65536 x 1024 in 32 columns 258, 164, 86, 67).
    // Packed sequences are cut into spans besides, for what a few waves' blocks leave to chance when lengths differ: 32
    // sequences of 256 to 8192 rows of 1024 channels take 152 us as 2 spans of clusters of 4, 168 as one of 8, 183 as
    // 8 spans of single blocks.
    a.cluster = 1;
    const int most = kPacked && a.p.n > 1 ? 4 : kMaxCluster;
    while (a.cluster < most && static_cast<int64_t>(a.cols) * a.spans * a.cluster < kFill && a.cluster < pieces) a.cluster *= 2;
    if (kPacked) {
        a.spans = 128 * C::kResident / (a.cols * a.cluster);
        if (a.spans > a.p.n) a.spans = a.p.n;
        if (a.spans > pieces) a.spans = pieces;
        if (a.spans < 1) a.spans = 1;
    }
    a.waits = linear_waits();
    if (kPath == kTma) {
        const int64_t rows = static_cast<int64_t>(a.p.T) * (kPacked ? 1 : a.p.n);
        constexpr bool g32 = sizeof(G) == 4, x32 = sizeof(T) == 4;
        constexpr int kBoxRows = kRows < kMaxBox ? kRows : kMaxBox;
        if (!tile_map(&a.map[0], a.p.log_a, g32, rows, a.p.D, kLanes * 4, kBoxRows) ||
            !tile_map(&a.map[1], kBack ? a.p.dout : a.p.x, x32, rows, a.p.D, kLanes * 4, kBoxRows) ||
            (kBack && !tile_map(&a.map[2], a.p.x, x32, rows, a.p.D, kLanes * 4, kBoxRows)))
            return cudaErrorInvalidValue;
    }
    const int64_t walks = static_cast<int64_t>(a.cols) * a.spans;
    const int smem = kPath == kTma ? C::stage_bytes * (pieces <= a.cluster ? 1 : C::kStages) : 0;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = smem > 0 ? allow_shared(kern, C::stage_bytes * C::kStages, allowed) : cudaSuccess;
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.cluster * walks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, static_cast<const Args>(a));
    note_launch(stream, kBack ? "gated_backward" : "gated_forward");
    return e;
}

template <typename T, typename G>
cudaError_t run_t(Args& a, bool back, cudaStream_t stream) {
    const bool tma = static_cast<int64_t>(a.p.D) * sizeof(T) % 16 == 0 && static_cast<int64_t>(a.p.D) * sizeof(G) % 16 == 0 &&
                     static_cast<int64_t>(a.p.T) * (a.p.cu ? 1 : a.p.n) < (int64_t(1) << 31);
    // Columns of 64 channels, whose rows are the longest stretches of memory, where clusters of up to four of them fill the
    // GPU; else of 32, with longer steps of fewer channels (one sequence of 65536 x 1024: 67 us against 110), and of 16
    // where even those leave more than half of it idle (65536 x 64: 30 us against 47; but 73 against 90 the other way for
    // gradients of 65536 x 256). Packed: 32 (the sequences of 256 to 8192 rows: 152 us against 206 with 64).
    const int64_t walks = a.p.cu ? 1 : a.p.n, wide = ((a.p.D - 1) / 64 + 1) * walks, half = ((a.p.D - 1) / 32 + 1) * walks;
    const int lanes = a.p.cu ? 8 : wide * 4 >= kFill ? 16 : half * 8 >= 64 ? 8 : 4;
    auto go = [&](auto kback, auto kpacked) {
        constexpr bool kB = decltype(kback)::value, kP = decltype(kpacked)::value;
        if (tma && lanes == 16) return launch_scan<T, G, kB, kP, kTma, kP ? 8 : 16>(a, stream);
        if (tma && lanes == 8) return launch_scan<T, G, kB, kP, kTma, 8>(a, stream);
        if (tma) return launch_scan<T, G, kB, kP, kTma, kP ? 8 : 4>(a, stream);
        if (a.p.D % 4 == 0) return launch_scan<T, G, kB, kP, kQuads, 16>(a, stream);
        return launch_scan<T, G, kB, kP, kSingles, 16>(a, stream);
    };
    using yes = std::true_type;
    using no = std::false_type;
    if (a.p.cu) return back ? go(yes(), yes()) : go(no(), yes());
    return back ? go(yes(), no()) : go(no(), no());
}

// ---- single tokens: one pass of 16-byte accesses over state, inputs and outputs

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
// shared memory. 64 x 1024 channels, 32 nodes: 6.7 us for 14 MB, bound by latency: the loads of 16 nodes at a time, the next
// ones on their way meanwhile, and the chain of 32 states. (Node by node 34 us; a batch after the other, behind the look at the
// tree, 8.7; each place filled again as it is used 14; 32 nodes' loads at once 12.9; a chain's states passed on in a
// register, behind a branch, 7.5.)
constexpr int kTreeThreads = 64;

// Whether a tree's parents are not as they should be, by every thread of the block together: par[i] (shared memory) < i, not
// below -2, and not a place without a node.
__device__ __forceinline__ bool tree_is_bad(const int* par, int N) {
    bool bad = false;
    for (int i = threadIdx.x; i < N; i += blockDim.x) {
        const int p = par[i];
        if (p >= i || p < -2) bad = true;
        else if (p >= 0 && par[p] == -2) bad = true;
    }
    return __syncthreads_or(bad);
}

template <typename T, typename G>
__global__ void __launch_bounds__(kTreeThreads) gated_tree(const T* __restrict__ x, const G* __restrict__ log_a,
                                                           const float* __restrict__ state,
                                                           const int32_t* __restrict__ parent, T* __restrict__ out,
                                                           int BP, int N, int D, int* err) {
    __shared__ int par[kMaxTree];
    extern __shared__ float hs[];  // [1 + N][kTreeThreads]: the entering state, the nodes'
    const int tid = threadIdx.x, b = blockIdx.y, c = blockIdx.x * kTreeThreads + tid;
    const bool mine = c < D;
    hs[tid] = mine ? state[static_cast<int64_t>(b) * D + c] : 0.f;
    const int64_t at = static_cast<int64_t>(b) * N * D + c;
    constexpr int kAhead = 16;  // nodes whose inputs are loaded together, while those before them are walked
    struct Nodes {
        T x[kAhead];
        G g[kAhead];
    };
    auto load = [&](Nodes& n, int i0) {
        if (i0 >= N || !mine) return;
#pragma unroll
        for (int j = 0; j < kAhead; j++) {
            const int64_t off = at + static_cast<int64_t>(i0 + j < N ? i0 + j : N - 1) * D;
            n.x[j] = x[off];
            n.g[j] = log_a[off];
        }
    };
    auto walk = [&](const Nodes& n, int i0) {
        int at_node[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; j++) at_node[j] = par[i0 + j < kMaxTree ? i0 + j : 0];
#pragma unroll
        for (int j = 0; j < kAhead; j++) {
            if (i0 + j >= N) break;
            const int up = at_node[j] < 0 ? 0 : at_node[j] + 1;  // places without a node go along, but are not stored
            const float h = fmaf(expf(load_f(&n.g[j])), hs[up * kTreeThreads + tid], load_f(&n.x[j]));
            hs[(i0 + j + 1) * kTreeThreads + tid] = h;
            if (at_node[j] != -2) store_f(out + at + static_cast<int64_t>(i0 + j) * D, h);
        }
    };
    Nodes even, odd;
    load(even, 0);
    for (int i = tid; i < N; i += kTreeThreads) par[i] = parent[(BP > 1 ? static_cast<int64_t>(b) * N : 0) + i];
    __syncthreads();
    if (tree_is_bad(par, N)) {
        if (tid == 0) record_error(err, kDevBadInput);
        return;
    }
    if (!mine) return;
    for (int i0 = 0; i0 < N; i0 += 2 * kAhead) {
        load(odd, i0 + kAhead);
        walk(even, i0);
        load(even, i0 + 2 * kAhead);
        walk(odd, i0 + kAhead);
    }
}

// Commits: the same chain over the accepted tokens, 2.8 us for 64 x 1024 channels with 6 tokens at most, about a launch.
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
    return by_types(dtype, gate_dtype, [&](auto t, auto g) { return run_t<decltype(t), decltype(g)>(a, backward, stream); });
}

cudaError_t gated_sum_shared(const float* parts, float* out, const int32_t* cu, int n, int T, int D, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((D - 1) / kThreads + 1);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, gated_sum, parts, out, cu, n, T, D);
    note_launch(stream, "gated_sum");
    return e;
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
        gated_tree<T, G><<<dim3((D - 1) / kTreeThreads + 1, B), kTreeThreads, (N + 1) * kTreeThreads * sizeof(float), stream>>>(
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
