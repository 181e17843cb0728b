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
#include "lla_drafts.cuh"
#include "lla_tc_ptx.cuh"

namespace lla {
namespace {

constexpr int kSlots = 40;
constexpr int kMaxStages = 4;
constexpr int kHalfSm = 111 * 1024;  // shared memory of a block of which an SM holds two

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
#pragma unroll
    for (int i = 0; i < kParts; i++) {
        p[i] = pack(x, y);
        x -= low(p[i]);
        y -= high(p[i]);
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
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&f)[4]) {
    const uint2 y = *reinterpret_cast<const uint2*>(p);
    f[0] = low(y.x); f[1] = high(y.x); f[2] = low(y.y); f[3] = high(y.y);
}

template <typename T> struct Parts;  // of queries and keys; of states
template <> struct Parts<__nv_bfloat16> { static constexpr int q = 1, s = 2; };
template <> struct Parts<float> { static constexpr int q = 3, s = 3; };

struct Layout {  // shared memory of decode_tree_kernel, bytes from its start; the sums take the place of q and k
    int q, k, v, lam, p, far, ring, stage;
};
// nodes of a block, all nodes, columns of a block
template <typename T>
__host__ __device__ inline Layout layout(int nb, int N, int dk, int cols, int slots, int stage_rows) {
    Layout s;
    const int parts = Parts<T>::q, rb = row_bytes(dk), rows = parts * (nb + N) * rb, sums = nb * (cols + 4) * 4;
    s.q = 0;
    s.k = s.q + parts * nb * rb;
    s.v = rows > sums ? rows : sums;
    s.lam = s.v + N * cols * static_cast<int>(sizeof(T));
    s.p = s.lam + nb * slots * 4;
    s.far = s.p + nb * (N + 1) * 4;
    s.ring = s.far + nb * slots * 4;
    s.stage = stage_rows * cols * 4;
    return s;
}

template <int kBytes>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(to)), "l"(from), "n"(kBytes) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Rows of q or k into shared memory as bf16 parts, zeros behind dk and behind the valid rows.
template <typename T, int kThreads>
__device__ __forceinline__ void stage(char* to, const T* from, int rows, int valid, int dk, int dkp) {
    constexpr int kParts = Parts<T>::q;
    const int rb = row_bytes(dk);
    if (dk % 8 == 0) {  // rows of whole 16-byte pieces: eight values at a time
        const int per = dkp / 8;
        const float inv = 1.f / static_cast<float>(per);
        for (int e = threadIdx.x; e < rows * per; e += kThreads) {
            const int i = static_cast<int>((static_cast<float>(e) + 0.5f) * inv), c = (e - i * per) * 8;  // e < 2^12
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
    for (int e = threadIdx.x; e < rows * pairs; e += kThreads) {
        const int i = e / pairs, c = (e - i * pairs) * 2;
        const T* src = from + static_cast<int64_t>(i) * dk + c;
        const float x = i < valid && c < dk ? load_f(src) : 0.f, y = i < valid && c + 1 < dk ? load_f(src + 1) : 0.f;
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

// Four 8 x 8 pieces of a staged matrix of bf16 rows: rows r0 .. r0 + 15 (lanes 0-15 name them) and summed indexes 16 ks ..
// + 15, as the A operand takes them.
__device__ __forceinline__ uint32_t piece_at(const char* m, int rb, int r0, int ks, int lane) {
    return smem_u32(m + (r0 + (lane & 15)) * rb + ks * 32 + (lane >> 4) * 16);
}

// Grid: (heads of all sequences, blocks of 16 MT NG nodes, column blocks of 32 CU). The warps are CU column pieces of 32
// times NG groups of 16 MT nodes times KS shares of the 16-row units. kStageRows: state rows of a
// stage of the ring, or 0 where it is not used (rows that are no multiples of 16 bytes, or less than 128).
template <typename T, int MT, int NG, int CU, int kStageRows>
__global__ void __launch_bounds__(256, 2) decode_tree_kernel(const TreeCall c, const __grid_constant__ CUtensorMap map, const int stages) {
    constexpr int kWarps = 8, kThreads = kWarps * 32, kNb = 16 * MT * NG, kCols = 32 * CU, KS = kWarps / (CU * NG);
    constexpr int kQ = Parts<T>::q, kS = Parts<T>::s;
    constexpr int kUnits = kStageRows / 16;  // of a stage
    constexpr bool kRing = kStageRows > 0;
    extern __shared__ __align__(16) char smem[];
    __shared__ int par[kMaxTree], dep[kMaxTree], slot_of[kSlots];
    __shared__ float la[kMaxTree];
    __shared__ int64_t slot_at[kSlots];
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, cc = lane & 3;
    const int64_t bh = blockIdx.x;
    const int b = static_cast<int>(bh / c.H), h = static_cast<int>(bh - static_cast<int64_t>(b) * c.H);
    const int N = c.N, dk = c.dk, dv = c.dv, dkp = (dk + 15) / 16 * 16, rb = row_bytes(dk), ksteps = dkp / 16;
    const int i0 = blockIdx.y * kNb, col0 = blockIdx.z * kCols, live = N - i0 < kNb ? N - i0 : kNb;
    const bool linear = c.t == nullptr;
    const int64_t t = linear ? 1 : c.t[b];
    const Layout s = layout<T>(kNb, N, dk, kCols, c.Lmax, kStageRows);
    char *qs = smem + s.q, *ks = smem + s.k;
    T* vs = reinterpret_cast<T*>(smem + s.v);             // [N][kCols]
    float* lam = reinterpret_cast<float*>(smem + s.lam);  // [kNb][Lmax]
    float* P = reinterpret_cast<float*>(smem + s.p);      // [kNb][N + 1]
    float* far = reinterpret_cast<float*>(smem + s.far);  // [slots][kNb]
    float* acc = reinterpret_cast<float*>(smem);          // [kNb][kCols + 4], once q and k are done with

    // the held slots of t - 1, in pieces of kStageRows rows
    const bool there = t > 0 && (linear || t < (int64_t(1) << (c.Lmax - 1)));  // else there are none, or the call is bad
    const int slots = !there ? 0 : linear ? 1 : 1 + __popcll(static_cast<unsigned long long>(t - 1));
    const int pieces = kRing ? (dk - 1) / (kRing ? kStageRows : 1) + 1 : 1, rounds = slots * pieces;
    const int64_t msz = static_cast<int64_t>(dk) * dv;
    const float* S = c.states + bh * c.Lmax * msz + col0;
    const int wide = dv - col0 < kCols ? dv - col0 : kCols;  // columns of the block
    char* ring = smem + s.ring + (-smem_u32(smem + s.ring) & 1023u);  // boxes begin at multiples of 1024 bytes
    constexpr int kBox = kStageRows * 128;                            // bytes of a stage's 32 columns
    auto copy = [&](int at, int slot, int piece) {                    // into stage `at`, by one thread
        uint64_t* bar = &full[at];
        mbar_expect_tx(bar, CU * kBox);
        const int y = static_cast<int>((bh * c.Lmax + slot) * dk) + piece * kStageRows;
        for (int u = 0; u < CU; u++) tma_load_2d(ring + at * s.stage + u * kBox, &map, bar, col0 + u * 32, y);
    };
    if (warp == kWarps - 1) {
        for (int l = lane; l < kSlots && there; l += 32)
            if (l == 0 || (!linear && ((t - 1) >> (l - 1) & 1))) {
                const int64_t below = l == 0 ? 0 : (int64_t(1) << (l - 1)) - 1;
                const int at = l == 0 ? 0 : 1 + __popcll(static_cast<unsigned long long>((t - 1) & below));
                slot_of[at] = l;
                slot_at[at] = ((t - 1) >> l) << l;
            }
        if (kRing) {
            if (lane < stages) {
                mbar_init(&full[lane], 1);
                mbar_init(&empty[lane], kWarps);
                fence_mbar_init();
            }
            __syncwarp();
            for (int r = 0; r < stages && r < rounds && lane == 0; r++) copy(r, slot_of[r / pieces], r % pieces);
        }
    }

    // everything else that the block reads is on its way before the first wait
    for (int i = tid; i < N; i += kThreads) {
        copy_async<4>(&par[i], c.parent + (c.BP > 1 ? static_cast<int64_t>(b) * N : 0) + i);
        if (!linear) copy_async<4>(&la[i], c.log_a + bh * N + i);
    }
    stage<T, kThreads>(qs, static_cast<const T*>(c.q) + (bh * N + i0) * dk, kNb, live, dk, dkp);
    stage<T, kThreads>(ks, static_cast<const T*>(c.k) + bh * N * dk, N, N, dk, dkp);
    const T* vg = static_cast<const T*>(c.v) + bh * N * dv + col0;
    constexpr int kE = 16 / sizeof(T);
    if (dv % kE == 0) {
        for (int e = tid; e < N * (kCols / kE); e += kThreads) {
            const int j = e / (kCols / kE), x = (e - j * (kCols / kE)) * kE;
            if (col0 + x < dv) copy_async<16>(vs + j * kCols + x, vg + static_cast<int64_t>(j) * dv + x);
        }
    } else {
        for (int e = tid; e < N * kCols; e += kThreads) {
            const int j = e / kCols, x = e - j * kCols;
            if (col0 + x < dv) vs[e] = vg[static_cast<int64_t>(j) * dv + x];
        }
    }
    if (!linear)
        for (int e = tid; e < live * c.Lmax; e += kThreads) copy_async<4>(&lam[e], c.lambda + (bh * N + i0) * c.Lmax + e);
    copies_done();
    __syncthreads();

    // scores: 16 x 8 pieces dealt to the warps
    {
        const int mts = (live + 15) / 16, nts = (N + 7) / 8;
        for (int u = warp; u < mts * nts; u += kWarps) {
            const int mt = u % mts, nt = u / mts;
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            const int j = nt * 8 + g < N ? nt * 8 + g : N - 1;  // columns behind the last are not kept
            for (int kk = 0; kk < ksteps; kk++) {
                uint32_t a[kQ][4], b0[kQ], b1[kQ];
#pragma unroll
                for (int w = 0; w < kQ; w++) {
                    ldmatrix4(a[w], piece_at(qs + w * kNb * rb, rb, mt * 16, kk, lane));
                    const char* at = ks + (w * N + j) * rb + (kk * 16 + cc * 2) * 2;
                    b0[w] = *reinterpret_cast<const uint32_t*>(at);
                    b1[w] = *reinterpret_cast<const uint32_t*>(at + 16);
                }
                mma_parts<false>(d, a, b0, b1);
            }
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const int i = mt * 16 + g + (r >> 1) * 8, x = nt * 8 + cc * 2 + (r & 1);
                if (x < N) P[i * (N + 1) + x] = d[r];
            }
        }
    }
    // depths; a walk up only goes to smaller indexes, so it ends in a bad tree too
    bool bad = t < 0;
    for (int i = tid; i < N; i += kThreads) {
        int d = -1;
        for (int j = i; j >= 0; d++) {
            const int up = par[j];
            if (up >= j || up < -2 || (up == -2 && j != i)) {
                bad = true;
                break;
            }
            j = up;
        }
        dep[i] = d;
        if (!linear && t + d >= (int64_t(1) << (c.Lmax - 1))) bad = true;
    }
    bad = __syncthreads_or(bad);
    if (bad && tid == 0) record_error(c.err, kDevBadInput);

    // weights of the nodes above, onto their scores, and of the held slots: kThreads / kNb threads walk up from each node,
    // each with every so many of the steps
    if (!bad) {
        constexpr int kEach = kThreads / kNb;
        const int i = tid % kNb, first = tid / kNb;
        if (i < live && par[i0 + i] != -2) {
            const int d = dep[i0 + i];
            const float lg = linear ? c.log_a[h] : 0.f;
            float D = 0.f;
            int turn = first, n = 0;
            for (int j = i0 + i; j >= 0; j = par[j], n++) {
                if (turn-- == 0) {
                    turn = kEach - 1;
                    P[i * (N + 1) + j] *=
                        linear ? (n == 0 ? 1.f : expf(lg * static_cast<float>(n)))
                               : lam[i * c.Lmax + 64 - __clzll(static_cast<long long>((t + d) ^ (t + d - n)))] * expf(D);
                }
                if (!linear) D += la[j];
            }
            const float whole = linear ? expf(lg * static_cast<float>(d + 1)) : expf(D);
            for (int m = first; m < slots; m += kEach)
                far[m * kNb + i] =
                    linear ? whole
                           : whole * lam[i * c.Lmax + 64 - __clzll(static_cast<long long>((t + d) ^ slot_at[m]))];
        }
    }
    __syncthreads();

    // the states' part: a slot's units of 16 rows summed, then weighted
    const int cu = warp % CU, ng = warp / CU % NG, share = warp / (CU * NG);
    const int colw = cu * 32 + g * 4;  // of the lane's pieces
    float out[MT][4][4], d[MT][4][4];
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
        for (int n = 0; n < 4; n++)
#pragma unroll
            for (int r = 0; r < 4; r++) out[mt][n][r] = d[mt][n][r] = 0.f;
    // one unit's products; f: rows 2 cc, 2 cc + 1, 2 cc + 8, 2 cc + 9 and the lane's four columns
    auto multiply = [&](const float (&f)[4][4], int kk) {
        uint32_t b0[4][kS], b1[4][kS];
#pragma unroll
        for (int n = 0; n < 4; n++) {
            cut<kS>(f[0][n], f[1][n], b0[n]);
            cut<kS>(f[2][n], f[3][n], b1[n]);
        }
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
            uint32_t a[kQ][4];
#pragma unroll
            for (int w = 0; w < kQ; w++)
                ldmatrix4(a[w], piece_at(qs + w * kNb * rb, rb, (ng * MT + mt) * 16, kk, lane));
#pragma unroll
            for (int n = 0; n < 4; n++) mma_parts<false>(d[mt][n], a, b0[n], b1[n]);
        }
    };
    auto weigh = [&](int m) {
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
            const int row = (ng * MT + mt) * 16 + g;
            const float w0 = far[m * kNb + row], w1 = far[m * kNb + row + 8];
#pragma unroll
            for (int n = 0; n < 4; n++) {
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    out[mt][n][r] = fmaf(r < 2 ? w0 : w1, d[mt][n][r], out[mt][n][r]);
                    d[mt][n][r] = 0.f;
                }
            }
        }
    };
    constexpr int kRow[4] = {0, 1, 8, 9};
    if constexpr (kRing) {
        bool in_time = true;
        int m = 0, piece = 0, slot_ahead = stages / pieces, piece_ahead = stages % pieces, at = 0, issued = -1;
        uint32_t parity = 0;
        for (int round = 0; round < rounds; round++) {
            if (in_time && !mbar_try_wait(&full[at], parity)) in_time = mbar_wait(&full[at], parity);
            const char* st = ring + at * s.stage + cu * kBox;
            const int left = dk - piece * kStageRows;  // rows of the stage that are the slot's
            constexpr int kTimes = (kUnits + KS - 1) / KS;
            float f[kTimes][4][4];
#pragma unroll
            for (int k = 0; k < kTimes; k++) {
                const int u = share + k * KS;
                if (u * 16 >= left || u >= kUnits) break;
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const int row = u * 16 + cc * 2 + kRow[r];
                    load4(reinterpret_cast<const float*>(st + row * 128 + ((g ^ (row & 7)) << 4)), f[k][r]);
                    if (u * 16 + 16 > left && row >= left) {  // the next slot's
#pragma unroll
                        for (int v = 0; v < 4; v++) f[k][r][v] = 0.f;
                    }
                }
                if (k + 1 == kTimes || (u + KS) * 16 >= left || u + KS >= kUnits) {  // read to the end
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[at]);
                }
                multiply(f[k], piece * kUnits + u);
            }
            if (share * 16 >= left || share >= kUnits) {  // nothing here for this warp
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[at]);
            }
            if (warp == (round & (kWarps - 1)) && round + stages < rounds) {  // the stage's next rows, by one warp in turn
                if (in_time && !mbar_try_wait(&empty[at], parity)) in_time = mbar_wait(&empty[at], parity);
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
                weigh(m);
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
        }
    } else {
        // the lane's own loads, a unit ahead
        auto fetch = [&](float (&f)[4][4], int m, int kk) {
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const int row = kk * 16 + cc * 2 + kRow[r];
                const float* from = S + slot_of[m] * msz + static_cast<int64_t>(row) * dv + colw;
#pragma unroll
                for (int v = 0; v < 4; v++) f[r][v] = row < dk && colw + v < wide ? __ldcs(from + v) : 0.f;
            }
        };
        float f[4][4], next[4][4];
        if (slots > 0 && share < ksteps) fetch(f, 0, share);
        for (int m = 0; m < slots; m++) {
            for (int kk = share; kk < ksteps; kk += KS) {
                const bool more = kk + KS < ksteps;
                if (more || m + 1 < slots) fetch(next, more ? m : m + 1, more ? kk + KS : share);
                multiply(f, kk);
#pragma unroll
                for (int r = 0; r < 4; r++)
#pragma unroll
                    for (int v = 0; v < 4; v++) f[r][v] = next[r][v];
            }
            weigh(m);
        }
    }
    if (bad) return;
    __syncthreads();  // q is not read any more
    // the shares are added in order; a lane holds columns 8 cc + {0..3, 4..7} of its rows
    for (int sh = 0; sh < KS; sh++) {
        if (share == sh) {
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    float4* at = reinterpret_cast<float4*>(acc + ((ng * MT + mt) * 16 + g + (r >> 1) * 8) * (kCols + 4) +
                                                           cu * 32 + cc * 8 + (r & 1) * 4);
                    float4 x = make_float4(out[mt][0][r], out[mt][1][r], out[mt][2][r], out[mt][3][r]);
                    if (sh > 0) {
                        const float4 y = *at;
                        x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
                    }
                    *at = x;
                }
        }
        __syncthreads();
    }
    // the nodes above, in fp32, and the result; four columns of a node to a thread
    T* og = static_cast<T*>(c.out) + (bh * N + i0) * dv + col0;
    for (int e = tid; e < live * (kCols / 4); e += kThreads) {
        const int i = e / (kCols / 4), x = (e - i * (kCols / 4)) * 4;
        if (par[i0 + i] == -2 || x >= wide) continue;
        float o[4] = {0.f, 0.f, 0.f, 0.f};
        for (int j = i0 + i; j >= 0; j = par[j]) {
            const float p = P[i * (N + 1) + j];
            float f[4];
            load4(vs + j * kCols + x, f);
#pragma unroll
            for (int v = 0; v < 4; v++) o[v] = fmaf(p, f[v], o[v]);
        }
        T* to = og + static_cast<int64_t>(i) * dv + x;
        float sum[4];
        load4(acc + i * (kCols + 4) + x, sum);
#pragma unroll
        for (int v = 0; v < 4; v++) {
            o[v] += sum[v];
            if (!kRing && x + v < wide) store_f(to + v, o[v]);
        }
        if constexpr (kRing) {
            if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(to) = make_float4(o[0], o[1], o[2], o[3]);
            else *reinterpret_cast<uint2*>(to) = make_uint2(pack(o[0], o[1]), pack(o[2], o[3]));
        }
    }
}

template <typename T, int MT, int NG, int CU, int kStageRows>
cudaError_t launch_tree(const TreeCall& c, cudaStream_t stream) {
    constexpr int kNb = 16 * MT * NG;
    constexpr bool ring = kStageRows > 0;
    const Layout s = layout<T>(kNb, c.N, c.dk, 32 * CU, c.Lmax, kStageRows);
    const dim3 grid(static_cast<unsigned>(c.B) * c.H, (c.N - 1) / kNb + 1, (c.dv - 1) / (32 * CU) + 1);
    // stages of the ring: four, or as many as leave room for two blocks on an SM, two at least
    const int64_t rows = static_cast<int64_t>(c.B) * c.H * c.Lmax * c.dk;
    int stages = 0;
    CUtensorMap map = {};
    if (ring) {
        if (!make_map_box(&map, c.states, true, static_cast<uint64_t>(rows), static_cast<uint64_t>(c.dv), 32, kStageRows))
            return cudaErrorInvalidValue;
        const int most = c.Lmax * ((c.dk - 1) / (ring ? kStageRows : 1) + 1);
        stages = (kHalfSm - s.ring - 1024) / s.stage;
        stages = stages > kMaxStages ? kMaxStages : stages < 2 ? 2 : stages;
        if (stages > most) stages = most;
    }
    const int smem = s.ring + stages * s.stage + (ring ? 1024 : 0);
    auto go = [&](auto kern) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        kern<<<grid, 256, smem, stream>>>(c, map, stages);
        note_launch(stream, "decode_tree");
        return cudaGetLastError();
    };
    return go(decode_tree_kernel<T, MT, NG, CU, kStageRows>);
}

// The stage's size: a whole slot's columns where two of them and another block fit on an SM, else half of its rows.
template <typename T, int MT, int NG, int CU>
cudaError_t pick_stage(const TreeCall& c, cudaStream_t stream) {
    constexpr int most = 8 / (CU * NG) * 16 > 64 ? 8 / (CU * NG) * 16 : 64;  // every warp has a unit of a stage
    if (c.dv % 4 != 0 || c.dv < 32 || static_cast<int64_t>(c.B) * c.H * c.Lmax * c.dk >= (int64_t(1) << 31))
        return launch_tree<T, MT, NG, CU, 0>(c, stream);
    const Layout s = layout<T>(16 * MT * NG, c.N, c.dk, 32 * CU, c.Lmax, 128);
    const int want = c.Lmax > 1 ? 2 : 1;
    if (c.dk > 64 && s.ring + want * s.stage + 1024 <= kHalfSm) return launch_tree<T, MT, NG, CU, 128>(c, stream);
    return launch_tree<T, MT, NG, CU, most>(c, stream);
}

// ---- commit

constexpr int kThreads = 256;

// Slot of position s <= e in the Fenwick walk of e
__device__ __forceinline__ int slot_in_walk(int64_t e, int64_t s) { return 64 - __clzll(static_cast<long long>(e ^ s)); }

// Every held slot of the last accepted position e = t + n - 1 from the old slots and the new tokens inside it. Each old
// slot lies inside one new slot of its own number or above, so a thread, which takes its elements through all slots, goes
// from the highest slot down and never reads what it has written. Elements are independent: grid (heads of all sequences,
// shares of a state's elements).
template <typename T, int kW, int kU>  // kW columns of a thread, kU of its elements at a time
__global__ void __launch_bounds__(kThreads) decode_commit_kernel(const CommitCall c, int share) {
    extern __shared__ float tok[];  // [n][dk] weighted keys, [n][dv] values
    __shared__ int node[kMaxTree], first[kSlots + 1];
    __shared__ float w[kMaxTree];
    __shared__ unsigned long long from[kSlots];
    __shared__ float whole_s;
    const int tid = threadIdx.x, dk = c.dk, dv = c.dv;
    const int64_t bh = blockIdx.x;
    const int b = static_cast<int>(bh / c.H), h = static_cast<int>(bh - static_cast<int64_t>(b) * c.H);
    const bool linear = c.t == nullptr;
    const int64_t t = linear ? 0 : c.t[b];
    const int n = c.count[b];
    const int64_t e = t + n - 1;
    bool bad = n < 0 || n > c.M || t < 0 || (!linear && e >= (int64_t(1) << (c.Lmax - 1)));
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
    if (tid == 0) {
        if (linear) {
            const float g = c.log_a[h];
            for (int i = 0; i < n; i++) w[i] = i == n - 1 ? 1.f : expf(g * static_cast<float>(n - 1 - i));
            whole_s = expf(g * static_cast<float>(n));
        } else {
            float D = 0.f;
            for (int i = n - 1; i >= 0; i--) {
                w[i] = expf(D);
                D += c.log_a[bh * c.N + node[i]];
            }
            whole_s = expf(D);
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
#pragma unroll
            for (int r = 0; r < kU; r++)
#pragma unroll
                for (int v = 0; v < kW; v++) a[r][v] *= whole;
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
    int parts = 1;
    while (parts < most && heads * parts < 600) parts *= 2;
    const int share = (items - 1) / parts + 1;
    auto go = [&](auto kern) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        kern<<<dim3(static_cast<unsigned>(heads), parts), kThreads, smem, stream>>>(c, share);
        note_launch(stream, "decode_commit");
        return cudaGetLastError();
    };
    if (width == 1) return go(decode_commit_kernel<T, 1, 4>);
    return share > kThreads ? go(decode_commit_kernel<T, 4, 4>) : go(decode_commit_kernel<T, 4, 1>);
}

}  // namespace

cudaError_t decode_tree(int dtype, const TreeCall& c, cudaStream_t stream) {
    const bool wide = c.dv > 32;
    if (dtype == 1) {
        if (c.N <= 16) return wide ? pick_stage<float, 1, 1, 2>(c, stream) : pick_stage<float, 1, 1, 1>(c, stream);
        return wide ? pick_stage<float, 1, 2, 2>(c, stream) : pick_stage<float, 1, 2, 1>(c, stream);
    }
    using T = __nv_bfloat16;
    if (c.N <= 16) return wide ? pick_stage<T, 1, 1, 2>(c, stream) : pick_stage<T, 1, 1, 1>(c, stream);
    if (c.N <= 32) return wide ? pick_stage<T, 2, 1, 2>(c, stream) : pick_stage<T, 2, 1, 1>(c, stream);
    return wide ? pick_stage<T, 2, 2, 2>(c, stream) : pick_stage<T, 2, 2, 1>(c, stream);
}

cudaError_t decode_commit(int dtype, const CommitCall& c, cudaStream_t stream) {
    return dtype == 1 ? launch_commit<float>(c, stream) : launch_commit<__nv_bfloat16>(c, stream);
}

}  // namespace lla
