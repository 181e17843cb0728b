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
// each slot by itself and weighted in fp32, so queries are never rounded with their weights. Each lane loads the states in
// the order in which it feeds the MMA: rows 4c..4c+3 and columns 4n..4n+3 of a 16 x 32 piece, four 16-byte loads that cover
// 128 bytes of a row each; the order of the summed index does not matter as long as the queries are read in the same one.
// So the states go from memory to registers once, past shared memory.
#include "lla_drafts.cuh"
#include "lla_tc_ptx.cuh"

namespace lla {
namespace {

constexpr int kSlots = 40;

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

__host__ __device__ inline int row_bytes(int dk) { return (dk * 2 + 127) / 128 * 128 + 32; }  // of a staged q or k row

template <typename T> struct Parts;  // of queries and keys; of states
template <> struct Parts<__nv_bfloat16> { static constexpr int q = 1, s = 2; };
template <> struct Parts<float> { static constexpr int q = 3, s = 3; };

struct Layout {  // shared memory of decode_tree_kernel, bytes from its start
    int q, k, v, lam, p, acc, far, total;
};
// nodes of a block, all nodes, columns of a block
template <typename T>
__host__ __device__ inline Layout layout(int nb, int N, int dk, int cols, int slots) {
    Layout s;
    const int parts = Parts<T>::q, rb = row_bytes(dk);
    s.q = 0;
    s.k = s.q + parts * nb * rb;
    s.v = s.k + parts * N * rb;
    s.lam = s.v + N * cols * static_cast<int>(sizeof(T));
    s.p = s.lam + nb * slots * 4;
    s.acc = (s.p + nb * (N + 1) * 4 + 15) / 16 * 16;
    s.far = s.acc + nb * cols * 4;
    s.total = s.far + nb * slots * 4;
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

// d += a b over the parts, the small products first
template <int kQ, int kS>
__device__ __forceinline__ void mma_parts(float (&d)[4], const uint32_t (&a)[kQ][4], const uint32_t (&b0)[kS],
                                          const uint32_t (&b1)[kS]) {
#pragma unroll
    for (int sum = (kQ == 1 ? kS - 1 : 2); sum >= 0; sum--)
#pragma unroll
        for (int i = 0; i < kQ; i++) {
            const int j = sum - i;
            if (j >= 0 && j < kS) mma(d, a[i], b0[j], b1[j]);
        }
}

// The A operand of rows 16 mt + {g, g + 8}, summed indexes 16 ks + {4c .. 4c + 3}
template <int kQ>
__device__ __forceinline__ void load_a(uint32_t (&a)[kQ][4], const char* q, int rows, int rb, int mt, int ks, int lane) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int w = 0; w < kQ; w++) {
        const char* at = q + (w * rows + mt * 16 + g) * rb + (ks * 16 + c * 4) * 2;
        const uint2 x = *reinterpret_cast<const uint2*>(at), y = *reinterpret_cast<const uint2*>(at + 8 * rb);
        a[w][0] = x.x;
        a[w][1] = y.x;
        a[w][2] = x.y;
        a[w][3] = y.y;
    }
}

// A lane's piece of the states: rows 4c..4c+3 of a unit's 16, columns 4g..4g+3 of a warp's 32.
struct Piece {
    float f[4][4];
};
template <bool kVec>
__device__ __forceinline__ void load_piece(Piece& p, const float* row, int rows, int cols, int dv) {
#pragma unroll
    for (int r = 0; r < 4; r++) {
        if constexpr (kVec) {
            const float4 y = r < rows && cols > 0 ? __ldcs(reinterpret_cast<const float4*>(row + static_cast<int64_t>(r) * dv))
                                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            p.f[r][0] = y.x; p.f[r][1] = y.y; p.f[r][2] = y.z; p.f[r][3] = y.w;
        } else {
#pragma unroll
            for (int v = 0; v < 4; v++) p.f[r][v] = r < rows && v < cols ? row[static_cast<int64_t>(r) * dv + v] : 0.f;
        }
    }
}

// Grid: (heads of all sequences, blocks of 16 MT NG nodes, column blocks of 32 CU). The warps are CU column pieces of 32
// times NG groups of 16 MT nodes times KS shares of the (slot, 16 rows) units.
template <typename T, int kWarps, int MT, int NG, int CU, bool kVec>
__global__ void __launch_bounds__(kWarps * 32, kWarps == 8 ? 2 : 1) decode_tree_kernel(const TreeCall c) {
    constexpr int kThreads = kWarps * 32, kNb = 16 * MT * NG, kCols = 32 * CU, KS = kWarps / (CU * NG);
    constexpr int kQ = Parts<T>::q, kS = Parts<T>::s;
    extern __shared__ __align__(16) char smem[];
    __shared__ int par[kMaxTree], dep[kMaxTree], slot_of[kSlots];
    __shared__ float la[kMaxTree];
    __shared__ int64_t slot_at[kSlots];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, cc = lane & 3;
    const int64_t bh = blockIdx.x;
    const int b = static_cast<int>(bh / c.H), h = static_cast<int>(bh - static_cast<int64_t>(b) * c.H);
    const int N = c.N, dk = c.dk, dv = c.dv, dkp = (dk + 15) / 16 * 16, rb = row_bytes(dk), ksteps = dkp / 16;
    const int i0 = blockIdx.y * kNb, col0 = blockIdx.z * kCols, live = N - i0 < kNb ? N - i0 : kNb;
    const bool linear = c.t == nullptr;
    const int64_t t = linear ? 1 : c.t[b];
    const Layout s = layout<T>(kNb, N, dk, kCols, c.Lmax);
    char *qs = smem + s.q, *ks = smem + s.k;
    T* vs = reinterpret_cast<T*>(smem + s.v);             // [N][kCols]
    float* lam = reinterpret_cast<float*>(smem + s.lam);  // [kNb][Lmax]
    float* P = reinterpret_cast<float*>(smem + s.p);      // [kNb][N + 1]
    float* acc = reinterpret_cast<float*>(smem + s.acc);  // [kNb][kCols]
    float* far = reinterpret_cast<float*>(smem + s.far);  // [slots][kNb]

    // everything that the block reads but the states is on its way before the first wait
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

    // units of (slot, 16 rows) of this warp's share; the first one is of slot 0, which is always held
    const int slots = linear ? 1 : t <= 0 ? 0 : 1 + __popcll(static_cast<unsigned long long>(t - 1));
    const int cu = warp % CU, ng = warp / CU % NG, share = warp / (CU * NG);
    const int colw = col0 + cu * 32 + g * 4;  // of the lane's pieces
    const int units = slots * ksteps;
    const float* S = c.states + bh * c.Lmax * dk * dv + colw;
    auto fetch = [&](Piece& p, int slot, int kk) {
        const int r = kk * 16 + cc * 4;
        load_piece<kVec>(p, S + (static_cast<int64_t>(slot) * dk + r) * dv, dk - r, dv - colw, dv);
    };
    Piece piece;
    const bool early = share < ksteps && share < units;
    if (early) fetch(piece, 0, share);

    if (tid < kSlots && !linear && t > 0 && (tid == 0 || ((t - 1) >> (tid - 1) & 1))) {
        const int64_t below = tid == 0 ? 0 : (int64_t(1) << (tid - 1)) - 1;
        const int at = tid == 0 ? 0 : 1 + __popcll(static_cast<unsigned long long>((t - 1) & below));
        slot_of[at] = tid;
        slot_at[at] = ((t - 1) >> tid) << tid;
    }
    if (linear && tid == 0) slot_of[0] = 0;
    copies_done();
    __syncthreads();
    if (tree_is_bad(par, N)) {
        if (tid == 0) record_error(c.err, kDevBadInput);
        return;
    }
    bool far_off = t < 0;
    for (int i = tid; i < N; i += kThreads) {
        int d = -1;
        for (int j = i; j >= 0; j = par[j]) d++;
        dep[i] = d;
        if (!linear && t + d >= (int64_t(1) << (c.Lmax - 1))) far_off = true;
    }
    if (__syncthreads_or(far_off)) {
        if (tid == 0) record_error(c.err, kDevBadInput);
        return;
    }

    // weights of the nodes above (P, for now without the scores) and of the held slots: kThreads / kNb threads walk up from
    // each node, each with every so many of the steps
    {
        constexpr int kEach = kThreads / kNb;
        const int i = tid % kNb, first = tid / kNb;
        if (i < live && par[i0 + i] != -2) {
            const int d = dep[i0 + i];
            const float lg = linear ? c.log_a[h] : 0.f;
            float D = 0.f;
            int turn = first;
            for (int j = i0 + i; j >= 0; j = par[j]) {
                if (turn-- == 0) {
                    turn = kEach - 1;
                    float w;
                    if (linear) {
                        const int n = d - dep[j];
                        w = n == 0 ? 1.f : expf(lg * static_cast<float>(n));
                    } else {
                        const int64_t x = (t + d) ^ (t + dep[j]);
                        w = lam[i * c.Lmax + 64 - __clzll(static_cast<long long>(x))] * expf(D);
                    }
                    P[i * (N + 1) + j] = w;
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

    // scores: 16 x 8 pieces dealt to the warps; a lane's four scores take their weights in place
    {
        const int mts = (live + 15) / 16, nts = (N + 7) / 8;
        for (int u = warp; u < mts * nts; u += kWarps) {
            const int mt = u % mts, nt = u / mts;
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            const int j = nt * 8 + g;
            for (int kk = 0; kk < ksteps; kk++) {
                uint32_t a[kQ][4], b0[kQ], b1[kQ];
                load_a<kQ>(a, qs, kNb, rb, mt, kk, lane);
#pragma unroll
                for (int w = 0; w < kQ; w++) {
                    uint2 x = make_uint2(0u, 0u);
                    if (j < N) x = *reinterpret_cast<const uint2*>(ks + (w * N + j) * rb + (kk * 16 + cc * 4) * 2);
                    b0[w] = x.x;
                    b1[w] = x.y;
                }
                mma_parts<kQ, kQ>(d, a, b0, b1);
            }
#pragma unroll
            for (int r = 0; r < 4; r++) {
                const int i = mt * 16 + g + (r >> 1) * 8, x = nt * 8 + cc * 2 + (r & 1);
                if (x < N) P[i * (N + 1) + x] *= d[r];
            }
        }
    }

    // the states' part, weighted unit by unit; the next unit's piece is on its way during this one's products
    float out[MT][4][4];
#pragma unroll
    for (int m = 0; m < MT; m++)
#pragma unroll
        for (int n = 0; n < 4; n++)
#pragma unroll
            for (int r = 0; r < 4; r++) out[m][n][r] = 0.f;
    int m = share / ksteps, kk = share - m * ksteps;
    if (!early && share < units) fetch(piece, slot_of[m], kk);
    for (int u = share; u < units; u += KS) {
        uint32_t b0[4][kS], b1[4][kS];
#pragma unroll
        for (int n = 0; n < 4; n++) {
            cut<kS>(piece.f[0][n], piece.f[1][n], b0[n]);
            cut<kS>(piece.f[2][n], piece.f[3][n], b1[n]);
        }
        const int um = m, uk = kk;
        kk += KS;
        while (kk >= ksteps) {
            kk -= ksteps;
            m++;
        }
        if (u + KS < units) fetch(piece, slot_of[m], kk);
#pragma unroll
        for (int mt = 0; mt < MT; mt++) {
            const int row = (ng * MT + mt) * 16 + g;
            uint32_t a[kQ][4];
            load_a<kQ>(a, qs, kNb, rb, ng * MT + mt, uk, lane);
            const float w0 = far[um * kNb + row], w1 = far[um * kNb + row + 8];
#pragma unroll
            for (int n = 0; n < 4; n++) {
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                mma_parts<kQ, kS>(d, a, b0[n], b1[n]);
                out[mt][n][0] = fmaf(w0, d[0], out[mt][n][0]);
                out[mt][n][1] = fmaf(w0, d[1], out[mt][n][1]);
                out[mt][n][2] = fmaf(w1, d[2], out[mt][n][2]);
                out[mt][n][3] = fmaf(w1, d[3], out[mt][n][3]);
            }
        }
    }
    // the shares are added in order; a lane holds columns 8 cc + {0..3, 4..7} of its rows
    for (int sh = 0; sh < KS; sh++) {
        if (share == sh) {
#pragma unroll
            for (int mt = 0; mt < MT; mt++)
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    float4* at = reinterpret_cast<float4*>(acc + ((ng * MT + mt) * 16 + g + (r >> 1) * 8) * kCols + cu * 32 +
                                                           cc * 8 + (r & 1) * 4);
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
        if (par[i0 + i] == -2 || col0 + x >= dv) continue;
        float o[4] = {0.f, 0.f, 0.f, 0.f};
        for (int j = i0 + i; j >= 0; j = par[j]) {
            const float p = P[i * (N + 1) + j];
#pragma unroll
            for (int v = 0; v < 4; v++) o[v] = fmaf(p, load_f(vs + j * kCols + x + v), o[v]);
        }
        T* to = og + static_cast<int64_t>(i) * dv + x;
#pragma unroll
        for (int v = 0; v < 4; v++) {
            o[v] += acc[i * kCols + x + v];
            if (!kVec && col0 + x + v < dv) store_f(to + v, o[v]);
        }
        if constexpr (kVec) {
            if constexpr (sizeof(T) == 4) {
                *reinterpret_cast<float4*>(to) = make_float4(o[0], o[1], o[2], o[3]);
            } else {
                *reinterpret_cast<uint2*>(to) = make_uint2(pack(o[0], o[1]), pack(o[2], o[3]));
            }
        }
    }
}

template <typename T, int kWarps, int MT, int NG, int CU>
cudaError_t launch_tree(const TreeCall& c, cudaStream_t stream) {
    constexpr int kNb = 16 * MT * NG;
    const Layout s = layout<T>(kNb, c.N, c.dk, 32 * CU, c.Lmax);
    const dim3 grid(static_cast<unsigned>(c.B) * c.H, (c.N - 1) / kNb + 1, (c.dv - 1) / (32 * CU) + 1);
    auto go = [&](auto kern) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, s.total);
        if (e != cudaSuccess) return e;
        kern<<<grid, kWarps * 32, s.total, stream>>>(c);
        note_launch(stream, "decode_tree");
        return cudaGetLastError();
    };
    return c.dv % 4 == 0 ? go(decode_tree_kernel<T, kWarps, MT, NG, CU, true>)
                         : go(decode_tree_kernel<T, kWarps, MT, NG, CU, false>);
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
        if (c.N <= 16) return wide ? launch_tree<float, 8, 1, 1, 2>(c, stream) : launch_tree<float, 8, 1, 1, 1>(c, stream);
        return wide ? launch_tree<float, 8, 1, 2, 2>(c, stream) : launch_tree<float, 8, 1, 2, 1>(c, stream);
    }
    using T = __nv_bfloat16;
    if (c.N <= 16) return wide ? launch_tree<T, 8, 1, 1, 2>(c, stream) : launch_tree<T, 8, 1, 1, 1>(c, stream);
    if (c.N <= 32) return wide ? launch_tree<T, 8, 2, 1, 2>(c, stream) : launch_tree<T, 8, 2, 1, 1>(c, stream);
    return wide ? launch_tree<T, 16, 2, 2, 2>(c, stream) : launch_tree<T, 16, 2, 2, 1>(c, stream);
}

cudaError_t decode_commit(int dtype, const CommitCall& c, cudaStream_t stream) {
    return dtype == 1 ? launch_commit<float>(c, stream) : launch_commit<__nv_bfloat16>(c, stream);
}

}  // namespace lla
