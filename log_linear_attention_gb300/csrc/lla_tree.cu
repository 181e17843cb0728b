// Trees of drafted tokens over recurrent states, and the commit of the accepted tokens.
//
// Node i of a tree hangs on node parent(i) < i, or (-1) on the last token that the states hold, t - 1. At depth d_i its
// position is p_i = t + d_i, and it sees the states and the nodes above it, but no other branch:
//
//     o_i = sum_{j = i or above} lambda_i^(l(p_i, p_j)) e^{D(i,j)} (q_i . k_j) v_j
//         + e^{D_i} sum_m lambda_i^(l(p_i, block m)) (S^(m))^T q_i
//
// D(i,j) sums log_a over the nodes after j on the way to i, D_i over all from the root. The Fenwick walk of t - 1 cuts the
// past into aligned blocks, each inside one bucket of every later position (the highest bit in which they differ lies above
// the block), so the states of t - 1 serve every node as they are: one read of them for the whole tree, no copy of them for
// a branch, nothing to take back for a token that is not accepted. Linear attention is the same with one state, lambda = 1
// and D = d log_a.
//
// The states' part is a product of N queries with (held slots) x dk rows of fp32 states. It runs on mma.sync with both
// operands cut into bf16 parts: bf16 queries are one part, states two (2^-16 of each element, below the output's own
// rounding of 2^-8); fp32 calls take three parts of each and the six products down to 2^-24. The products are summed for
// each slot by itself and weighted in fp32, so queries are never rounded with their weights. The states' rows come to a
// ring in shared memory by TMA, in swizzled boxes of 32 columns, from which a lane reads the four rows' pieces of four
// columns of its MMA operands without bank conflicts and cuts them itself.
//
// Measured (calls in a CUDA graph, inputs larger than L2): 64 sequences x 16 heads of 128 x 64 at t up to 65536, 32 nodes,
// bf16: 63 us for 328 MB (77% of the copy rate); 16 nodes 59 us (80%), 64 nodes 100 us, fp32 with 32 nodes 130 us. One state
// a head (linear) and 64 nodes: 33 us for 84 MB. What a block does before and after its states bounds it: of 26 thousand
// cycles (two blocks on an SM) the first slot is taken at 8.4, a slot of 32 KB every 1.7, the rest is 1.9. fp32 fills no pipe
// either (tensor 38%, issue slots 42%, shared memory 29%): six products and two groups of warps that cut the same states stand
// in a chain that 16 warps of an SM do not hide. Steps: the lanes' own loads of states 85 us, row by row with untiled bulk
// copies 226 (their issue), the ring of boxes 75, walkers beside scorers 62.
#include "lla_drafts.cuh"
#include "lla_linear_tc.cuh"

namespace lla {
namespace {

constexpr int kSlots = 40;
constexpr int kMaxStages = 4;
constexpr int kMostShared = 220 * 1024;  // dynamic; static and reserved shared memory fit beside it in the SM's 228 KB

// bf16 halves of two floats, the first in the low half
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float low(uint32_t r) { return __uint_as_float(r << 16); }
__device__ __forceinline__ float high(uint32_t r) { return __uint_as_float(r & 0xffff0000u); }

// kParts bf16 pairs whose sum is (x, y)
template <int kParts>
__device__ __forceinline__ void cut(float x, float y, uint32_t (&p)[kParts]) {
    f32x2 v = pair2(x, y);
#pragma unroll
    for (int i = 0; i < kParts; i++) {
        const float2 f = split2(v);
        p[i] = pack(f.x, f.y);
        if (i + 1 < kParts) v = fma2(pair2(low(p[i]), high(p[i])), pair2(-1.f, -1.f), v);
    }
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {  // onto zeros
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

// Bytes of a staged q or k row: rows lie 16 bytes further on in the banks each.
__host__ __device__ inline int row_bytes(int dk) { return (dk * 2 + 127) / 128 * 128 + 16; }

__device__ __forceinline__ void load4(const float* p, float (&f)[4]) {
    const float4 y = *reinterpret_cast<const float4*>(p);
    f[0] = y.x; f[1] = y.y; f[2] = y.z; f[3] = y.w;
}
__device__ __forceinline__ void load_nt(const float* p, float (&f)[4]) { load4(p, f); }
__device__ __forceinline__ void load_nt(const float* p, float (&f)[2]) {
    const float2 y = *reinterpret_cast<const float2*>(p);
    f[0] = y.x; f[1] = y.y;
}
__device__ __forceinline__ void load8(const float* p, float (&f)[4], float (&h)[4]) {
    load4(p, f);
    load4(p + 4, h);
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[4], float (&h)[4]) {
    const uint4 y = *reinterpret_cast<const uint4*>(p);
    f[0] = low(y.x); f[1] = high(y.x); f[2] = low(y.y); f[3] = high(y.y);
    h[0] = low(y.z); h[1] = high(y.z); h[2] = low(y.w); h[3] = high(y.w);
}

template <typename T> struct Parts;  // of queries and keys; of states
template <> struct Parts<__nv_bfloat16> { static constexpr int q = 1, s = 2; };
template <> struct Parts<float> { static constexpr int q = 3, s = 3; };

// Blocks of an SM by their registers, and the shared memory of each. (32 nodes in pieces of 16 columns a warp leave room for
// three blocks, but take every query twice as often: 76 us against 69 at that point.)
template <typename T>
__host__ __device__ constexpr int resident(int MT, int NT) { return Parts<T>::q == 1 && MT * NT <= 4 ? 3 : 2; }
template <typename T>
__host__ __device__ constexpr int room(int MT, int NT) { return resident<T>(MT, NT) == 3 ? 69 * 1024 : 107 * 1024; }

// Shared memory of decode_tree_kernel, bytes from a multiple of 1024. The shares' sums take the place
// of q, k and the ring at the end.
struct Layout {
    int q, k;      // kAll: panels of 64 columns, rows of 128 bytes, swizzled; else parts of rows of row_bytes
    int panel_q, panel_k;
    int ring, stage;
    int v, lam, p, far, up, total;
};
__host__ __device__ inline int up1024(int x) { return (x + 1023) / 1024 * 1024; }
// nodes of a block, all nodes, columns of a block, slots; rows of a stage; its stages; shares of the warps
template <typename T>
__host__ __device__ inline Layout layout(int nb, int N, int dk, int cols, int slots, int stage_rows, int stages, int shares,
                                         bool tma) {
    Layout s;
    const int parts = Parts<T>::q, rb = row_bytes(dk), panels = (dk + 63) / 64, sums = shares * nb * (cols + 4) * 4;
    s.panel_q = nb * 128;
    s.panel_k = (N + 7) / 8 * 1024;
    s.q = 0;
    s.k = tma ? panels * s.panel_q : parts * nb * rb;
    const int rows = s.k + (tma ? panels * s.panel_k : parts * N * rb);
    s.ring = up1024(rows);
    s.stage = stage_rows * cols * 4;
    s.v = s.ring + stages * s.stage > sums ? s.ring + stages * s.stage : up1024(sums);
    s.lam = s.v + (N + 7) / 8 * 8 * cols * static_cast<int>(sizeof(T));
    s.p = s.lam + nb * slots * 4;
    s.far = s.p + nb * (N + 1) * 4;
    s.up = s.far + nb * slots * 4;
    s.total = s.up + nb * N + 1024;  // and what aligns the start
    return s;
}

template <int kBytes>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(to)), "l"(from), "n"(kBytes) : "memory");
}
__device__ __forceinline__ void copies_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }

// Loads that may run ahead of stores.
__device__ __forceinline__ float load_nc(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_nc(const __nv_bfloat16* p) {
    return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p))) << 16);
}

// Rows of q or k into shared memory as bf16 parts, zeros behind dk and behind the valid rows.
template <typename T, int kThreads>
__device__ __forceinline__ void stage_rows(char* to, const T* from, int rows, int valid, int dk, int dkp) {
    constexpr int kParts = Parts<T>::q;
    const int rb = row_bytes(dk);
    if (dk % 8 == 0) {  // rows of whole 16-byte pieces: eight values at a time
        const int per = dkp / 8, step = kThreads / per, first = threadIdx.x / per, c = (threadIdx.x - first * per) * 8;
#pragma unroll 4
        for (int i = first < step ? first : rows; i < rows; i += step) {
            char* at = to + i * rb + c * 2;
            const T* src = from + static_cast<int64_t>(i) * dk + c;
            const bool in = i < valid && c < dk;
            if constexpr (kParts == 1) {
                if (in) copy_async<16>(at, src);
                else *reinterpret_cast<uint4*>(at) = make_uint4(0u, 0u, 0u, 0u);
            } else {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
                if (in) {
                    x = __ldg(reinterpret_cast<const float4*>(src));
                    y = __ldg(reinterpret_cast<const float4*>(src) + 1);
                }
                uint32_t p0[kParts], p1[kParts], p2[kParts], p3[kParts];
                cut<kParts>(x.x, x.y, p0);
                cut<kParts>(x.z, x.w, p1);
                cut<kParts>(y.x, y.y, p2);
                cut<kParts>(y.z, y.w, p3);
#pragma unroll
                for (int w = 0; w < kParts; w++)
                    *reinterpret_cast<uint4*>(at + w * rows * rb) = make_uint4(p0[w], p1[w], p2[w], p3[w]);
            }
        }
        return;
    }
    const int pairs = dkp / 2;
#pragma unroll 4
    for (int e = threadIdx.x; e < rows * pairs; e += kThreads) {
        const int i = e / pairs, c = (e - i * pairs) * 2;
        const T* src = from + static_cast<int64_t>(i) * dk + c;
        const float x = i < valid && c < dk ? load_nc(src) : 0.f, y = i < valid && c + 1 < dk ? load_nc(src + 1) : 0.f;
        uint32_t p[kParts];
        cut<kParts>(x, y, p);
#pragma unroll
        for (int w = 0; w < kParts; w++) *reinterpret_cast<uint32_t*>(to + (w * rows + i) * rb + c * 2) = p[w];
    }
}

// d (+)= a b over the parts, the small products first
template <bool kFirst, int kQ, int kS>
__device__ __forceinline__ void mma_parts(float (&d)[4], const uint32_t (&a)[kQ][4], const uint32_t (&b0)[kS],
                                          const uint32_t (&b1)[kS]) {
    constexpr int kTop = kQ == 1 ? kS - 1 : 2;
#pragma unroll
    for (int sum = kTop; sum >= 0; sum--)
#pragma unroll
        for (int i = 0; i < kQ; i++) {
            const int j = sum - i;
            if (j < 0 || j >= kS) continue;
            if (kFirst && sum == kTop && (i == 0 || (kTop - i + 1 >= kS))) mma_first(d, a[i], b0[j], b1[j]);
            else mma(d, a[i], b0[j], b1[j]);
        }
}

// What lies between a node and the one that its jump leads to (-1: past the root). At the end jumps lead past the root
// everywhere, and what lies between a node and one above it is the difference of the two, so the sum of log decays carries what
// its additions round away in a second float: behind gates of -100 each, a difference of plain fp32 sums has lost 2^-10 of the
// weight. A gate that is 0 in fp32 forgets whatever it is (-inf, -1e9), and one that is infinite or NaN spoils the weight; both
// are counted instead of summed.
struct __align__(16) Link {
    int jump;
    unsigned counts;  // steps, gates of zero << 8, gates that are not finite << 16: 128 of each at most
    float decay, rest;
    __device__ __forceinline__ int steps() const { return static_cast<int>(counts & 255u); }
};
constexpr unsigned kZero = 1u << 8, kOdd = 1u << 16;
__device__ __forceinline__ void add_decays(Link& a, const Link& b) {  // the first sum's rounding error is exact
    const float s = a.decay + b.decay, part = s - a.decay;
    a.rest += b.rest + ((a.decay - (s - part)) + (b.decay - part));
    a.decay = s;
}
// e^(sum of log decays) between a node and one above it, or past the root: `counts` and sums are differences
__device__ __forceinline__ float weight(unsigned counts, float decay, float rest) {
    return counts < kZero ? expf(decay + rest) : counts < kOdd ? 0.f : __int_as_float(0x7fffffff);
}
__device__ __forceinline__ void scorers_meet() { asm volatile("bar.sync 2, 128;" ::: "memory"); }
// Walkers' barrier; any(x): whether one of them has x.
__device__ __forceinline__ void walkers_meet() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool walkers_any(bool x) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.s32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, 128, p;\n\t"
        "selp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<int>(x))
        : "memory");
    return r != 0;
}
enum Mode { kNone, kStates, kAll };

// Maps of the tensors that come by TMA, each [heads (states: slots)][rows][columns].
struct Maps {
    CUtensorMap states, q, k, v;
};

// Grid: (heads of all sequences times blocks of 16 MT NG nodes, column blocks of 8 CW NT). The warps are CW column pieces of
// 8 NT times NG groups of 16 MT nodes times KS shares of the 16-row units. kStageRows: state rows of a stage of the ring.
// kMode: what comes by TMA, as rows of multiples of 16 bytes can; the states' ring is else filled by copies of every thread,
// of 4 bytes (8 where dv is even), in two stages.
//
// Four warps walk the tree and form the weights while the other four multiply queries and keys, as most of what comes before
// the first slot is latency: 75 us as one after the other, 62 side by side (32 nodes, the batch above).
template <typename T, int MT, int NG, int CW, int NT, int kStageRows, int kMode>
__global__ void __launch_bounds__(256, resident<T>(MT, NT))
    decode_tree_kernel(const TreeCall c, const __grid_constant__ Maps maps, const int stages, const LinWaits waits) {
    constexpr int kWarps = 8, kThreads = kWarps * 32, kNb = 16 * MT * NG, kCols = 8 * CW * NT, KS = kWarps / (CW * NG);
    constexpr int kQ = Parts<T>::q, kS = Parts<T>::s, CU = kCols / 32;
    constexpr bool kTma = kMode >= kStates, kTmaIn = kMode == kAll;
    constexpr int kUnits = kStageRows / 16;  // of a stage
    constexpr int kWalkers = 128;            // threads that form the weights
    extern __shared__ __align__(16) char smem_any[];
    __shared__ int par[kMaxTree], slot_of[kSlots];
    __shared__ float la[kMaxTree];
    __shared__ Link link[kMaxTree];
    __shared__ uint4 above[kMaxTree];
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], inputs, never;
    char* smem = smem_any + (-smem_u32(smem_any) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, cc = lane & 3;
    const int blocks = (c.N - 1) / kNb + 1;  // of nodes: those of one head run side by side, so that its states come once
    const unsigned head = blockIdx.x / blocks;
    const int b = static_cast<int>(head / c.H), h = static_cast<int>(head - b * static_cast<unsigned>(c.H));
    const int64_t bh = head;
    const int N = c.N, dk = c.dk, dv = c.dv, dkp = (dk + 15) / 16 * 16, rb = row_bytes(dk), ksteps = dkp / 16;
    const int i0 = static_cast<int>(blockIdx.x % blocks) * kNb, col0 = blockIdx.y * kCols, live = N - i0 < kNb ? N - i0 : kNb;
    const bool linear = c.t == nullptr;
    const Layout s = layout<T>(kNb, N, dk, kCols, c.Lmax, kStageRows, stages, KS, kTmaIn);
    char *qs = smem + s.q, *ks = smem + s.k, *ring = smem + s.ring;
    T* vs = reinterpret_cast<T*>(smem + s.v);               // [N][kCols]
    float* lam = reinterpret_cast<float*>(smem + s.lam);    // [kNb][Lmax]
    float* P = reinterpret_cast<float*>(smem + s.p);        // [kNb][N + 1]: weights, then scores times weights
    float* far = reinterpret_cast<float*>(smem + s.far);    // [slots][kNb]
    uint8_t* up = reinterpret_cast<uint8_t*>(smem + s.up);  // [kNb][N]: a node and those above it, upwards
    float* acc = reinterpret_cast<float*>(smem);            // [KS][kNb][kCols + 4], once q, k and the ring are done with
    const int wide = dv - col0 < kCols ? dv - col0 : kCols; // columns of the block

    // The held slots of t - 1, in pieces of kStageRows rows (dk <= 128).
    const int pieces = kStageRows >= 128 ? 1 : (dk - 1) / kStageRows + 1;
    constexpr int kBox = kStageRows * 128;          // bytes of a stage's 32 columns
    auto copy = [&](int at, int slot, int piece) {  // into stage `at`, by one thread
        uint64_t* bar = &full[at];
        mbar_expect_tx(bar, CU * kBox);
        for (int u = 0; u < CU; u++)
            tma_load_3d(ring + at * s.stage + u * kBox, &maps.states, bar, col0 + u * 32, piece * kStageRows,
                        static_cast<int>(bh * c.Lmax + slot));
    };
    auto held = [&](int64_t t) {  // none where there are none, or the call is bad
        const bool there = t > 0 && (linear || t < (int64_t(1) << (c.Lmax - 1)));
        return !there ? 0 : linear ? 1 : 1 + __popcll(static_cast<unsigned long long>(t - 1));
    };

    // Everything that the block reads is on its way before the first wait.
    if (warp == kWarps - 1) {
        if (lane == 0) {
            for (int i = 0; i < kMaxStages; i++) {
                mbar_init(&full[i], 1);
                mbar_init(&empty[i], kWarps);
            }
            mbar_init(&inputs, 1);
            mbar_init(&never, 1);
            fence_mbar_init();
            if constexpr (kTmaIn) {
                const int panels = (dk + 63) / 64;
                mbar_expect_tx(&inputs, panels * (s.panel_q + s.panel_k) + (N + 7) / 8 * 8 * kCols * 2);
                for (int y = 0; y < panels; y++) {
                    tma_load_3d(qs + y * s.panel_q, &maps.q, &inputs, y * 64, i0, static_cast<int>(bh));
                    tma_load_3d(ks + y * s.panel_k, &maps.k, &inputs, y * 64, 0, static_cast<int>(bh));
                }
                tma_load_3d(vs, &maps.v, &inputs, col0, 0, static_cast<int>(bh));
            }
        }
        __syncwarp();
        if (kTmaIn) scorers_meet();
        const int64_t t = linear ? 1 : c.t[b];
        const int rounds = held(t) * pieces;
        for (int l = lane; l < kSlots && rounds > 0; l += 32)
            if (l == 0 || (!linear && ((t - 1) >> (l - 1) & 1))) {
                const int64_t below = l == 0 ? 0 : (int64_t(1) << (l - 1)) - 1;
                const int at = l == 0 ? 0 : 1 + __popcll(static_cast<unsigned long long>((t - 1) & below));
                slot_of[at] = l;
            }
        __syncwarp();
        if (kTma)
            for (int r = 0; r < stages && r < rounds && lane == 0; r++) copy(r, slot_of[r / pieces], r % pieces);
    }
    if (tid < kWalkers) {
        for (int i = tid; i < N; i += kWalkers) {
            copy_async<4>(&par[i], c.parent + (c.BP > 1 ? static_cast<int64_t>(b) * N : 0) + i);
            if (!linear) copy_async<4>(&la[i], c.log_a + bh * N + i);
        }
        if (!linear)
            for (int e = tid; e < live * c.Lmax; e += kWalkers) copy_async<4>(&lam[e], c.lambda + (bh * N + i0) * c.Lmax + e);
        copies_group();
    }
    const float lg = linear && tid < kWalkers ? c.log_a[h] : 0.f;
    const int64_t t = linear ? 1 : c.t[b];
    const int slots = held(t), rounds = slots * pieces;
    // A round's rows into stage `at` as TMA lays them, by all threads, zeros behind them; columns behind the last stay zero.
    // A warp to every eighth row, whose places differ by a constant (64 x 16 heads of 128 x 50, 12 nodes: 92 us, with every
    // element's place worked out 178; four stages instead of two: no change).
    auto fill_by = [&](int at, int slot, int piece, auto width) {
        constexpr int kW = decltype(width)::value;  // columns of a copy
        const int r0 = piece * kStageRows, rows = dk - r0 < kStageRows ? dk - r0 : kStageRows;
        const float* from = c.states + ((bh * c.Lmax + slot) * dk + r0) * dv + col0;
        static_assert(kWarps == 8);  // a warp's rows lie alike in their swizzled lines
        for (int x = lane * kW; x < wide; x += 32 * kW) {
            char* place = ring + at * s.stage + x / 32 * kBox + warp * 128 + ((x % 32 / 4 ^ warp) << 4) + x % 4 * 4;
            const float* src = from + static_cast<int64_t>(warp) * dv + x;
#pragma unroll 4
            for (int r = warp; r < (rows + 15) / 16 * 16; r += 8, place += 1024, src += 8 * dv) {
                if (r < rows) {
                    copy_async<4 * kW>(place, src);
                } else {
#pragma unroll
                    for (int v = 0; v < kW; v++) reinterpret_cast<float*>(place)[v] = 0.f;
                }
            }
        }
        copies_group();
    };
    auto fill = [&](int at, int slot, int piece) {
        if (dv % 2 == 0) fill_by(at, slot, piece, std::integral_constant<int, 2>());
        else fill_by(at, slot, piece, std::integral_constant<int, 1>());
    };
    if constexpr (!kTma) {
        for (int e = tid; e < stages * s.stage / 16; e += kThreads) reinterpret_cast<uint4*>(ring)[e] = make_uint4(0u, 0u, 0u, 0u);
    }
    if constexpr (!kTmaIn) {
        stage_rows<T, kThreads>(qs, static_cast<const T*>(c.q) + (bh * N + i0) * dk, kNb, live, dk, dkp);
        stage_rows<T, kThreads>(ks, static_cast<const T*>(c.k) + bh * N * dk, N, N, dk, dkp);
        const T* vg = static_cast<const T*>(c.v) + bh * N * dv + col0;
#pragma unroll 4
        for (int e = tid; e < N * kCols; e += kThreads) {
            const int j = e / kCols, x = e - j * kCols;
            if (x < wide) store_f(vs + e, load_nc(vg + static_cast<int64_t>(j) * dv + x));
        }
        copies_group();
        copies_done<0>();
        __syncthreads();
    } else if (warp >= kWalkers / 32 && warp < kWarps - 1) {
        scorers_meet();  // the barriers are set up
    }

    // Operands of 16 queries (from row r0, summed indexes 16 kk ..), and of 8 keys (from row j0, 16 kk .. + 31).
    auto load_q = [&](uint32_t (&a)[kQ][4], int r0, int kk) {
        if constexpr (kTmaIn) {
            ldmatrix4(a[0], smem_u32(qs) + (kk >> 2) * s.panel_q + (r0 + (lane & 15)) * 128 +
                                ((((kk & 3) * 2 + (lane >> 4)) ^ (lane & 7)) << 4));
        } else {
#pragma unroll
            for (int w = 0; w < kQ; w++)
                ldmatrix4(a[w], smem_u32(qs) + (w * kNb + r0 + (lane & 15)) * rb + kk * 32 + (lane >> 4) * 16);
        }
    };
    auto load_k = [&](uint32_t (&z)[kQ][4], int j0, int kk) {
        if constexpr (kTmaIn) {
            ldmatrix4(z[0], smem_u32(ks) + (kk >> 2) * s.panel_k + (j0 + (lane & 7)) * 128 +
                                ((((kk & 3) * 2 + (lane >> 3)) ^ (lane & 7)) << 4));
        } else {
            const int j = j0 + (lane & 7) < N ? j0 + (lane & 7) : N - 1;  // behind the last key: that one, not kept
#pragma unroll
            for (int w = 0; w < kQ; w++)
                ldmatrix4(z[w], smem_u32(ks) + (w * N + j) * rb + kk * 32 + (lane >> 3) * 16);
        }
    };
    // scores: units of kMany 16 x 8 pieces side by side (those behind the last key are not kept)
    constexpr int kMany = kNb / 16;
    const int mts = (live + 15) / 16, nts = (N + 7) / 8, groups = (nts + kMany - 1) / kMany;
    auto score = [&](float (&d)[kMany][4], int u) {
        const int mt = u % mts, nt0 = u / mts * kMany;
#pragma unroll
        for (int y = 0; y < kMany; y++)
#pragma unroll
            for (int r = 0; r < 4; r++) d[y][r] = 0.f;
        for (int kk = 0; kk < ksteps; kk += 2) {
            uint32_t a[2][kQ][4], z[kMany][kQ][4];
            const bool two = kk + 1 < ksteps;
            load_q(a[0], mt * 16, kk);
            if (two) load_q(a[1], mt * 16, kk + 1);
#pragma unroll
            for (int y = 0; y < kMany; y++) load_k(z[y], (nt0 + y) * 8, kk);
#pragma unroll
            for (int half = 0; half < 2; half++) {
                if (half == 1 && !two) break;
#pragma unroll
                for (int y = 0; y < kMany; y++) {
                    uint32_t b0[kQ], b1[kQ];
#pragma unroll
                    for (int w = 0; w < kQ; w++) {
                        b0[w] = z[y][w][half * 2];
                        b1[w] = z[y][w][half * 2 + 1];
                    }
                    mma_parts<false>(d[y], a[half], b0, b1);
                }
            }
        }
    };
    auto onto_weights = [&](const float (&d)[kMany][4], int u) {
        const int mt = u % mts, nt0 = u / mts * kMany;
#pragma unroll
        for (int y = 0; y < kMany; y++)
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const int i = mt * 16 + g + (r >> 1) * 8, x = (nt0 + y) * 8 + cc * 2 + (r & 1);
                if (x < N) P[i * (N + 1) + x] *= d[y][r];
            }
    };

    const int64_t limit = linear ? 2 : int64_t(1) << (c.Lmax - 1);  // of positions
    bool bad = t < 0 || t >= limit, in_time = true;
    float held_scores[2][kMany][4];
    const int scorer = warp - kWalkers / 32;
    if (tid < kWalkers) {
        // Depths, sums of log decays and the nodes above each node, by jumps that double in length: log2 of the depth
        // rounds. A thread to a node (N <= 128).
        static_assert(kMaxTree == kWalkers);
        copies_done<0>();
        walkers_meet();
        const int p = tid < N ? par[tid] : -2;
        Link me = {p, p >= 0 ? 1u : 0u, 0.f, 0.f};
        uint4 mask = make_uint4(0u, 0u, 0u, 0u);
        if (tid < N) {
            if (p >= tid || p < -2 || (p >= 0 && par[p] == -2)) {
                bad = true;
                me.jump = -1;
            }
            const float x = linear ? 0.f : la[tid], gate = expf(x);
            if (gate == 0.f) me.counts += kZero;
            else if (!(gate < INFINITY)) me.counts += kOdd;
            else me.decay = x;
            const uint32_t bit = 1u << (tid & 31);
            (tid < 32 ? mask.x : tid < 64 ? mask.y : tid < 96 ? mask.z : mask.w) = bit;
        }
        for (;;) {
            link[tid] = me;
            above[tid] = mask;
            walkers_meet();
            if (me.jump >= 0) {
                const Link to = link[me.jump];
                const uint4 m = above[me.jump];
                me.jump = to.jump;
                me.counts += to.counts;
                add_decays(me, to);
                mask = make_uint4(mask.x | m.x, mask.y | m.y, mask.z | m.z, mask.w | m.w);
            }
            if (!walkers_any(me.jump >= 0)) break;
        }
        if (!linear && tid < N && t < limit && t + me.steps() >= limit) bad = true;
        link[tid] = me;
        above[tid] = mask;
        walkers_meet();
        // weights: kEach threads to a node, each with every so many of the nodes above it and of the held slots
        constexpr int kEach = kWalkers / kNb;
        const int i = tid % kNb, first = tid / kNb, node = i0 + i;
        if (i < live && par[node] != -2 && t >= 0 && t < limit) {
            const Link at = link[node];
            const uint4 line = above[node];
            const int64_t pos = t + at.steps();
            const float* lam_i = lam + i * c.Lmax;
            // nodes j of j % kEach == first, four at a time, so that their links are read side by side
            constexpr unsigned long long kMine = ~0ull / ((1ull << kEach) - 1);
            unsigned long long lo = (line.x | static_cast<unsigned long long>(line.y) << 32) & kMine << first;
            unsigned long long hi = (line.z | static_cast<unsigned long long>(line.w) << 32) & kMine << first;
            int base = 0, j[4];
            do {
                Link other[4];
#pragma unroll
                for (int y = 0; y < 4; y++) {
                    if (lo == 0) {
                        lo = hi;
                        hi = 0;
                        base = 64;
                    }
                    j[y] = lo == 0 ? -1 : base + __ffsll(static_cast<long long>(lo)) - 1;
                    lo &= lo - 1;
                    other[y] = link[j[y] < 0 ? node : j[y]];
                }
                float w[4];
#pragma unroll
                for (int y = 0; y < 4; y++) {
                    const int n = at.steps() - other[y].steps();
                    if (linear) w[y] = n == 0 ? 1.f : expf(lg * static_cast<float>(n));
                    else
                        w[y] = lam_i[64 - __clzll(static_cast<long long>(pos ^ (pos - n)))] *
                               weight(at.counts - other[y].counts, at.decay - other[y].decay, at.rest - other[y].rest);
                }
#pragma unroll
                for (int y = 0; y < 4; y++)
                    if (j[y] >= 0) {
                        up[i * N + at.steps() - other[y].steps()] = static_cast<uint8_t>(j[y]);
                        P[i * (N + 1) + j[y]] = w[y];
                    }
            } while (j[3] >= 0);
            const float whole = linear ? expf(lg * static_cast<float>(at.steps() + 1)) : weight(at.counts, at.decay, at.rest);
            // the blocks of the walk of t - 1 begin at t - 1 and where its set bits are cleared one by one
            if (linear) {
                if (first == 0) far[i] = whole;
            } else {
                int64_t begin = t - 1;
                for (int m = 0; m < slots; m++, begin &= begin - 1) {
                    if (m % kEach != first) continue;
                    far[m * kNb + i] = whole * lam_i[64 - __clzll(static_cast<long long>(pos ^ begin))];
                }
            }
        }
    } else {
        if (kTmaIn) in_time = mbar_try_wait(&inputs, 0) || mbar_wait(&inputs, 0, waits.cycles);
#pragma unroll
        for (int y = 0; y < 2; y++)
            if (scorer + 4 * y < mts * groups) score(held_scores[y], scorer + 4 * y);
    }
    bad = __syncthreads_or(bad);
    if (bad && tid == 0) record_error(c.err, kDevBadInput);
    if (tid >= kWalkers) {
#pragma unroll
        for (int y = 0; y < 2; y++)
            if (scorer + 4 * y < mts * groups) onto_weights(held_scores[y], scorer + 4 * y);
    } else if (kTmaIn) {
        in_time = mbar_try_wait(&inputs, 0) || mbar_wait(&inputs, 0, waits.cycles);
    }
    for (int u = 8 + warp; u < mts * groups; u += kWarps) {
        score(held_scores[0], u);
        onto_weights(held_scores[0], u);
    }

    // the states' part: a slot's units of 16 rows summed, then weighted
    const int cw = warp % CW, ng = warp / CW % NG, share = warp / (CW * NG);
    const int colw = cw * 8 * NT + g * NT;  // of the lane's pieces
    float out[MT][NT][4], d[MT][NT][4];
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int r = 0; r < 4; r++) out[mt][n][r] = 0.f;
    // one unit's products; f: rows 2 cc, 2 cc + 1, 2 cc + 8, 2 cc + 9 and the lane's NT columns
    auto multiply = [&](const float (&f)[4][NT], int kk, auto first) {  // first: onto zeros
        uint32_t b0[NT][kS], b1[NT][kS];
#pragma unroll
        for (int n = 0; n < NT; n++) {
            cut<kS>(f[0][n], f[1][n], b0[n]);
            cut<kS>(f[2][n], f[3][n], b1[n]);
        }
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
            uint32_t a[kQ][4];
            load_q(a, (ng * MT + mt) * 16, kk);
#pragma unroll
            for (int n = 0; n < NT; n++) mma_parts<decltype(first)::value>(d[mt][n], a, b0[n], b1[n]);
        }
    };
    auto weigh = [&](int m) {
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
            const int row = (ng * MT + mt) * 16 + g;
            const float w0 = far[m * kNb + row], w1 = far[m * kNb + row + 8];
#pragma unroll
            for (int n = 0; n < NT; n++) {
#pragma unroll
                for (int r = 0; r < 4; r += 2) {
                    const float w = r == 0 ? w0 : w1;
                    const float2 y = split2(fma2(pair2(w, w), pair2(d[mt][n][r], d[mt][n][r + 1]),
                                                 pair2(out[mt][n][r], out[mt][n][r + 1])));
                    out[mt][n][r] = y.x;
                    out[mt][n][r + 1] = y.y;
                }
            }
        }
    };
    using yes = std::true_type;
    using no = std::false_type;
    // places of the lane's pieces in a unit's swizzled rows 2 cc and 2 cc + 1; those 8 rows on lie alike
    const int chunk = colw % 32 / 4, rest = colw % 4 * 4;
    const int even = cc * 256 + ((chunk ^ (cc * 2)) << 4) + rest, odd = cc * 256 + 128 + ((chunk ^ (cc * 2 + 1)) << 4) + rest;
    const bool mine = share < ksteps;  // whether any unit of a slot is this warp's
    // a stage's units; read(): once the last of them is in registers
    auto consume = [&](int at, int piece, auto read) {
        const char* st = ring + at * s.stage + colw / 32 * kBox;
        const int left = dk - piece * kStageRows;  // rows of the stage that are the slot's; zeros lie behind them
        constexpr int kTimes = (kUnits + KS - 1) / KS;
        float f[kTimes][4][NT];
#pragma unroll
        for (int k = 0; k < kTimes; k++) {
            const int u = share + k * KS;
            if (u * 16 >= left || u >= kUnits) break;
#pragma unroll
            for (int r = 0; r < 4; r++)
                load_nt(reinterpret_cast<const float*>(st + u * 2048 + (r & 1 ? odd : even) + (r >> 1) * 1024), f[k][r]);
            if (k + 1 == kTimes || (u + KS) * 16 >= left || u + KS >= kUnits) read();
            if (k == 0 && piece == 0) multiply(f[k], piece * kUnits + u, yes());
            else multiply(f[k], piece * kUnits + u, no());
        }
        if (share * 16 >= left || share >= kUnits) read();  // nothing here for this warp
    };
    int m = 0, piece = 0;
    if constexpr (kTma) {
        if (waits.hold && in_time) in_time = mbar_wait(&never, 0, waits.cycles);
        int slot_ahead = stages / pieces, piece_ahead = stages % pieces, at = 0, issued = -1;
        uint32_t parity = 0;
        for (int round = 0; round < rounds; round++) {
            if (in_time && !mbar_try_wait(&full[at], parity)) in_time = mbar_wait(&full[at], parity, waits.cycles);
            consume(at, piece, [&] {
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[at]);
            });
            if (warp == (round & (kWarps - 1)) && round + stages < rounds) {  // the stage's next rows, by one warp in turn
                if (in_time && !mbar_try_wait(&empty[at], parity)) in_time = mbar_wait(&empty[at], parity, waits.cycles);
                in_time = __all_sync(0xffffffffu, in_time);
                if (in_time) {
                    if (lane == 0) copy(at, slot_of[slot_ahead], piece_ahead);
                    issued = round + stages;
                }
            }
            if (++piece_ahead == pieces) {
                piece_ahead = 0;
                slot_ahead++;
            }
            if (++piece == pieces) {
                if (mine) weigh(m);
                piece = 0;
                m++;
            }
            if (++at == stages) {
                at = 0;
                parity ^= 1u;
            }
        }
        if (!in_time && lane == 0) {  // no block leaves while its own copies are under way
            record_error(c.err, kDevTimeout);
            if (issued >= 0) mbar_wait(&full[issued % stages], (issued / stages) & 1);
            if (warp == kWarps - 1)
                for (int r = 0; r < stages && r < rounds; r++) mbar_wait(&full[r], 0);
            if (kTmaIn && warp == kWarps - 1) mbar_wait(&inputs, 0);
        }
    } else {
        if (rounds > 0) fill(0, slot_of[0], 0);
        for (int round = 0; round < rounds; round++) {
            copies_done<0>();
            __syncthreads();  // this round's rows are there, and the other stage's have been read
            if (round + 1 < rounds) fill((round + 1) & 1, slot_of[(round + 1) / pieces], (round + 1) % pieces);
            consume(round & 1, piece, [] {});
            if (++piece == pieces) {
                if (mine) weigh(m);
                piece = 0;
                m++;
            }
        }
    }
    if (bad) return;
    __syncthreads();  // q is not read any more
    // the shares' sums; a lane holds 2 NT neighbouring columns of its rows
    constexpr int kSums = kNb * (kCols + 4);
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
        for (int r = 0; r < 4; r += 2) {
            float* at = acc + share * kSums + ((ng * MT + mt) * 16 + g + r * 4) * (kCols + 4) + cw * 8 * NT + cc * 2 * NT;
#pragma unroll
            for (int x = 0; x < 2 * NT; x += 4)
                *reinterpret_cast<float4*>(at + x) =
                    make_float4(out[mt][x % NT][r + x / NT], out[mt][(x + 1) % NT][r + (x + 1) / NT],
                                out[mt][(x + 2) % NT][r + (x + 2) / NT], out[mt][(x + 3) % NT][r + (x + 3) / NT]);
        }
    __syncthreads();
    // the nodes above, in fp32, and the result; eight columns of a node to a thread
    T* og = static_cast<T*>(c.out) + (bh * N + i0) * dv + col0;
    for (int e = tid; e < live * (kCols / 8); e += kThreads) {
        const int i = e / (kCols / 8), x = (e - i * (kCols / 8)) * 8;
        if (par[i0 + i] == -2 || x >= wide) continue;
        f32x2 o[4];
#pragma unroll
        for (int sh = 0; sh < KS; sh++) {  // in order
            const float4* sum = reinterpret_cast<const float4*>(acc + sh * kSums + i * (kCols + 4) + x);
            const float4 y = sum[0], z = sum[1];
            const f32x2 add[4] = {pair2(y.x, y.y), pair2(y.z, y.w), pair2(z.x, z.y), pair2(z.z, z.w)};
#pragma unroll
            for (int v = 0; v < 4; v++) o[v] = sh == 0 ? add[v] : add2(o[v], add[v]);
        }
        const int d = link[i0 + i].steps();
#pragma unroll 4
        for (int n = 0; n <= d; n++) {
            const int j = up[i * N + n];
            const float p = P[i * (N + 1) + j];
            const f32x2 pp = pair2(p, p);
            float f[4], h[4];
            load8(vs + j * kCols + x, f, h);
            o[0] = fma2(pp, pair2(f[0], f[1]), o[0]);
            o[1] = fma2(pp, pair2(f[2], f[3]), o[1]);
            o[2] = fma2(pp, pair2(h[0], h[1]), o[2]);
            o[3] = fma2(pp, pair2(h[2], h[3]), o[3]);
        }
        T* to = og + static_cast<int64_t>(i) * dv + x;
        float y[8];
#pragma unroll
        for (int v = 0; v < 4; v++) {
            const float2 z = split2(o[v]);
            y[2 * v] = z.x;
            y[2 * v + 1] = z.y;
        }
        if (kTma && x + 8 <= wide) {  // rows of multiples of four values at least
            if constexpr (sizeof(T) == 4) {
                *reinterpret_cast<float4*>(to) = make_float4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<float4*>(to + 4) = make_float4(y[4], y[5], y[6], y[7]);
            } else {
                *reinterpret_cast<uint2*>(to) = make_uint2(pack(y[0], y[1]), pack(y[2], y[3]));
                *reinterpret_cast<uint2*>(to + 4) = make_uint2(pack(y[4], y[5]), pack(y[6], y[7]));
            }
        } else {
#pragma unroll
            for (int v = 0; v < 8; v++)
                if (x + v < wide) store_f(to + v, y[v]);
        }
    }
}

// Map of a tensor [z][rows][cols]; parts of a box outside a matrix read as zeros.
bool map_3d(CUtensorMap* m, const void* base, bool f32, int64_t z, int rows, int cols, int box_cols, int box_rows, bool swizzle) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t e = f32 ? 4 : 2, row = static_cast<cuuint64_t>(cols) * e;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(z)};
    const cuuint64_t strides[2] = {row, row * rows};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1}, one[3] = {1, 1, 1};
    return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
              strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int MT, int NG, int CW, int NT, int kStageRows, int kMode>
cudaError_t launch_tree(const TreeCall& c, int stages, cudaStream_t stream) {
    constexpr int kNb = 16 * MT * NG, kCols = 8 * CW * NT;
    const int64_t heads = static_cast<int64_t>(c.B) * c.H;
    Maps maps = {};
    if (kMode >= kStates) {
        if (!map_3d(&maps.states, c.states, true, heads * c.Lmax, c.dk, c.dv, 32, kStageRows, true)) return cudaErrorInvalidValue;
        const int keys = (c.N + 7) / 8 * 8;
        if (kMode == kAll &&
            (!map_3d(&maps.q, c.q, false, heads, c.N, c.dk, 64, kNb, true) ||
             !map_3d(&maps.k, c.k, false, heads, c.N, c.dk, 64, keys, true) ||
             !map_3d(&maps.v, c.v, false, heads, c.N, c.dv, kCols, keys, false)))
            return cudaErrorInvalidValue;
    }
    const Layout s = layout<T>(kNb, c.N, c.dk, kCols, c.Lmax, kStageRows, stages, 8 / (CW * NG), kMode == kAll);
    auto kern = decode_tree_kernel<T, MT, NG, CW, NT, kStageRows, kMode>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_shared(kern, kMostShared, allowed);
    if (e != cudaSuccess) return e;
    if (s.total > kMostShared) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(heads * ((c.N - 1) / kNb + 1)), (c.dv - 1) / kCols + 1);
    kern<<<grid, 256, s.total, stream>>>(c, maps, stages, linear_waits());
    note_launch(stream, "decode_tree");
    return cudaGetLastError();
}

// The ring: stages of a whole slot's columns, or of part of its rows, the largest of which two fit beside the other blocks of
// an SM (one, where there is one slot); by TMA up to four of them. (Two stages of 128 rows against four of 64: 62 us and
// 66 for 32 nodes, alike for 16.)
template <typename T, int MT, int NG, int CW, int NT, int kMode>
cudaError_t pick_stage(const TreeCall& c, cudaStream_t stream) {
    constexpr int KS = 8 / (CW * NG), least = KS * 16 > 32 ? KS * 16 : 32;  // every warp has a unit of a stage
    constexpr int middle = least > 64 ? least : 64;
    auto fit = [&](int rows) {
        const Layout s = layout<T>(16 * MT * NG, c.N, c.dk, 8 * CW * NT, c.Lmax, rows, 0, KS, kMode == kAll);
        const int all = c.Lmax * ((c.dk - 1) / rows + 1), most = all < kMaxStages ? all : kMaxStages;
        const int n = (room<T>(MT, NT) - (s.total - s.v) - s.ring) / s.stage;
        return kMode == kNone ? n < 2 ? n : 2 : n < most ? n : most;
    };
    const int want = c.Lmax > 1 || kMode == kNone ? 2 : 1;
    if ((c.dk > 64 || middle == 128) && fit(128) >= want) return launch_tree<T, MT, NG, CW, NT, 128, kMode>(c, fit(128), stream);
    if ((c.dk > 32 || least == middle) && fit(middle) >= want)
        return launch_tree<T, MT, NG, CW, NT, middle, kMode>(c, fit(middle), stream);
    const int n = fit(least);
    return launch_tree<T, MT, NG, CW, NT, least, kMode>(c, n < want ? want : n, stream);
}

template <typename T, int MT, int NG, int CW, int NT>
cudaError_t pick_copies(const TreeCall& c, cudaStream_t stream) {
    if (c.dv % 4 != 0 || static_cast<int64_t>(c.B) * c.H * c.Lmax >= (int64_t(1) << 31))
        return pick_stage<T, MT, NG, CW, NT, kNone>(c, stream);
    if constexpr (Parts<T>::q == 1)  // fp32 queries and keys are cut on their way
        if (c.dk % 8 == 0 && c.dv % 8 == 0) return pick_stage<T, MT, NG, CW, NT, kAll>(c, stream);
    return pick_stage<T, MT, NG, CW, NT, kStates>(c, stream);
}

// ---- commit

constexpr int kThreads = 256;

// Slot of position s <= e in the Fenwick walk of e
__device__ __forceinline__ int slot_in_walk(int64_t e, int64_t s) { return 64 - __clzll(static_cast<long long>(e ^ s)); }

// Every held slot of the last accepted position e = t + n - 1 from the old slots and the new tokens inside it. Each old
// slot lies inside one new slot of its own number or above, so a thread, which takes its elements through all slots, goes
// from the highest slot down and never reads what it has written. Elements are independent: grid (heads of all sequences,
// shares of a state's elements). Bound by HBM: 64 x 16 heads of 128 x 64 with 6 tokens at most, 96 us for 531 MB read and
// written (82% of the copy rate), four elements of a thread at a time (two 107 us, eight 151).
template <typename T, int kW, int kU>  // kW columns of a thread, kU of its elements at a time
__global__ void __launch_bounds__(kThreads) decode_commit_kernel(const CommitCall c, int share) {
    extern __shared__ float tok[];  // [n][dk] weighted keys, [n][dv] values
    __shared__ int node[kMaxTree], first[kSlots + 1];
    __shared__ float w[kMaxTree], la[kMaxTree];
    __shared__ unsigned long long from[kSlots];
    __shared__ float whole_s;
    const int tid = threadIdx.x, dk = c.dk, dv = c.dv;
    const int64_t bh = blockIdx.x;
    const int b = static_cast<int>(bh / c.H), h = static_cast<int>(bh - static_cast<int64_t>(b) * c.H);
    const bool linear = c.t == nullptr;
    const int64_t t = linear ? 0 : c.t[b];
    const int n = c.count[b];
    const int64_t e = t + n - 1;
    bool bad = n < 0 || n > c.M || t < 0 || (!linear && t > (int64_t(1) << (c.Lmax - 1)) - n);
    if (!bad)
        for (int i = tid; i < n; i += kThreads) {
            const int at = c.path ? c.path[static_cast<int64_t>(b) * c.M + i] : i;
            bad |= at < 0 || at >= c.N;
            node[i] = at;
        }
    if (__syncthreads_or(bad)) {
        if (tid == 0) record_error(c.err, kDevBadInput);
        return;
    }
    if (n == 0) return;
    // weights: what the tokens after one make of it; of the old slots (thread n): what all make of them
    if (linear) {
        const float g = c.log_a[h];
        if (tid < n) w[tid] = tid == n - 1 ? 1.f : expf(g * static_cast<float>(n - 1 - tid));
        if (tid == n) whole_s = expf(g * static_cast<float>(n));
    } else {
        if (tid < n) la[tid] = c.log_a[bh * c.N + node[tid]];
        __syncthreads();
        if (tid <= n) {
            const int stop = tid < n ? tid : -1;
            float D = 0.f;
            for (int i = n - 1; i > stop; i--) D += la[i];
            (tid < n ? w[tid] : whole_s) = expf(D);
        }
    }
    // old slots that go into slot l, and its first token (tokens of slot l: first[l] .. the first of the next lower held one)
    if (tid < c.Lmax) {
        unsigned long long m = 0;
        if (linear) m = 1;
        else if (t > 0)
            for (int o = 0; o < c.Lmax; o++)
                if ((o == 0 || ((t - 1) >> (o - 1) & 1)) && slot_in_walk(e, ((t - 1) >> o) << o) == tid) m |= 1ull << o;
        from[tid] = m;
        int f = 0;
        while (!linear && f < n && slot_in_walk(e, t + f) > tid) f++;
        first[tid] = f;
    }
    __syncthreads();
    float* kw = tok;
    float* vv = tok + n * dk;
    for (int x = tid; x < n * dk; x += kThreads) {
        const int i = x / dk;
        kw[x] = w[i] * load_f(static_cast<const T*>(c.k) + (bh * c.N + node[i]) * dk + (x - i * dk));
    }
    for (int x = tid; x < n * dv; x += kThreads) {
        const int i = x / dv;
        vv[x] = load_f(static_cast<const T*>(c.v) + (bh * c.N + node[i]) * dv + (x - i * dv));
    }
    __syncthreads();
    const float whole = whole_s;
    const int64_t msz = static_cast<int64_t>(dk) * dv;
    float* S = c.states + bh * c.Lmax * msz;
    const int groups = dv / kW, items = dk * groups;
    const int end = (static_cast<int>(blockIdx.y) + 1) * share < items ? (static_cast<int>(blockIdx.y) + 1) * share : items;
    for (int it0 = blockIdx.y * share + tid; it0 < end; it0 += kThreads * kU) {
        int row[kU], col[kU];
        float* at[kU];
#pragma unroll
        for (int r = 0; r < kU; r++) {
            const int it = it0 + r * kThreads < end ? it0 + r * kThreads : it0;  // past the end: the first again, not stored
            row[r] = it / groups;
            col[r] = (it - row[r] * groups) * kW;
            at[r] = S + static_cast<int64_t>(row[r]) * dv + col[r];
        }
        for (int l = c.Lmax - 1; l >= 0; l--) {
            if (!linear && l > 0 && !((e >> (l - 1)) & 1)) continue;
            float a[kU][kW];
#pragma unroll
            for (int r = 0; r < kU; r++)
#pragma unroll
                for (int v = 0; v < kW; v++) a[r][v] = 0.f;
            for (unsigned long long m = from[l]; m; m &= m - 1) {
                const int64_t off = (__ffsll(static_cast<long long>(m)) - 1) * msz;
                if constexpr (kW == 4) {
                    float4 y[kU];
#pragma unroll
                    for (int r = 0; r < kU; r++) y[r] = __ldcs(reinterpret_cast<const float4*>(at[r] + off));
#pragma unroll
                    for (int r = 0; r < kU; r++) {
                        a[r][0] += y[r].x; a[r][1] += y[r].y; a[r][2] += y[r].z; a[r][3] += y[r].w;
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < kU; r++) a[r][0] += at[r][off];
                }
            }
            if (from[l] != 0) {  // a slot of new tokens alone stays clear of gates that are not finite before them
#pragma unroll
                for (int r = 0; r < kU; r++)
#pragma unroll
                    for (int v = 0; v < kW; v++) a[r][v] *= whole;
            }
            // this slot's tokens end where the next lower held slot's begin
            const int stop = l == 0 ? n : first[l - 1];
            for (int s = first[l]; s < stop; s++) {
#pragma unroll
                for (int r = 0; r < kU; r++) {
                    const float ki = kw[s * dk + row[r]];
#pragma unroll
                    for (int v = 0; v < kW; v++) a[r][v] = fmaf(ki, vv[s * dv + col[r] + v], a[r][v]);
                }
            }
#pragma unroll
            for (int r = 0; r < kU; r++) {
                if (r > 0 && it0 + r * kThreads >= end) continue;
                float* to = at[r] + l * msz;
                if constexpr (kW == 4) __stcs(reinterpret_cast<float4*>(to), make_float4(a[r][0], a[r][1], a[r][2], a[r][3]));
                else *to = a[r][0];
            }
        }
    }
}

template <typename T>
cudaError_t launch_commit(const CommitCall& c, cudaStream_t stream) {
    const size_t smem = static_cast<size_t>(c.M) * (c.dk + c.dv) * sizeof(float);
    const int64_t heads = static_cast<int64_t>(c.B) * c.H;
    const int width = c.dv % 4 == 0 ? 4 : 1, items = c.dk * (c.dv / width), most = (items - 1) / kThreads + 1;
    // Blocks for a few waves (64 x 16 heads of 128 x 64: 97 us as one block a head, 94 as two, 108 as four, which leave a
    // thread fewer rows in flight).
    int parts = 1;
    while (parts < most && heads * parts < 2000) parts *= 2;
    const int share = (items - 1) / parts + 1;
    auto go = [&](auto kern, std::atomic<uint64_t>& allowed) {
        // always: the kernel's static memory counts to what a launch has without asking
        cudaError_t e = allow_shared(kern, kMaxTree * 256 * 4, allowed);
        if (e != cudaSuccess) return e;
        kern<<<dim3(static_cast<unsigned>(heads), parts), kThreads, smem, stream>>>(c, share);
        note_launch(stream, "decode_commit");
        return cudaGetLastError();
    };
    static std::atomic<uint64_t> allowed[3];
    if (width == 1) return go(decode_commit_kernel<T, 1, 4>, allowed[0]);
    return share > kThreads ? go(decode_commit_kernel<T, 4, 4>, allowed[1]) : go(decode_commit_kernel<T, 4, 1>, allowed[2]);
}

}  // namespace

cudaError_t decode_tree(int dtype, const TreeCall& c, cudaStream_t stream) {
    // 64 columns to a block, or 32 where that leaves half of the SMs without one (4 x 16 heads of 128 x 64, 8 nodes: 9.8 us
    // against 16). More than 32 nodes: blocks of 64 nodes with 16 columns a warp (64 nodes at that point: 113 us; two groups
    // of warps of 32 nodes 119, two blocks of 32 nodes 147). fp32: two groups, whose three parts of a query fit registers.
    const bool wide = c.dv > 32 && static_cast<int64_t>(c.B) * c.H * ((c.dv - 1) / 64 + 1) > 76;
    if (dtype == 1) {
        if (c.N <= 16) return wide ? pick_copies<float, 1, 1, 2, 4>(c, stream) : pick_copies<float, 1, 1, 1, 4>(c, stream);
        return wide ? pick_copies<float, 1, 2, 2, 4>(c, stream) : pick_copies<float, 1, 2, 1, 4>(c, stream);
    }
    using T = __nv_bfloat16;
    if (c.N <= 16) return wide ? pick_copies<T, 1, 1, 2, 4>(c, stream) : pick_copies<T, 1, 1, 1, 4>(c, stream);
    if (c.N <= 32) return wide ? pick_copies<T, 2, 1, 2, 4>(c, stream) : pick_copies<T, 2, 1, 1, 4>(c, stream);
    return wide ? pick_copies<T, 4, 1, 4, 2>(c, stream) : pick_copies<T, 4, 1, 2, 2>(c, stream);
}

cudaError_t decode_commit(int dtype, const CommitCall& c, cudaStream_t stream) {
    return dtype == 1 ? launch_commit<float>(c, stream) : launch_commit<__nv_bfloat16>(c, stream);
}

}  // namespace lla
