// Gradients of linear attention with one decay per head on tensor cores, from the states that enter each
// chunk (bf16, formed by lla_linear_tc.cu: S forwards, R backwards; see lla_linear.cu for the formulas):
//
//     dq_i = sum_{j <= i} g^(i-j) (dO_i . v_j) k_j + g^(i+1)   S dO_i
//     dk_i = sum_{j >= i} g^(j-i) (v_i . dO_j) q_j + g^(n-1-i) R v_i
//     dv_i = sum_{j >= i} g^(j-i) (k_i . q_j) dO_j + g^(n-1-i) R^T k_i
//
// An item is 64 columns of one of them for one 128-token chunk, with rows a (d1 wide), b (d1 wide) and
// c (64 columns) and the chunk's state X:
//     scores  A B^T  [128 x 128] -> P = scores o g^|i-j| (two bf16 parts, in TMEM in place of the scores)
//     far     A X    [128 x 64]     X as it lies (dv), or the same rows read as its transpose (dq, dk)
//     near    P C    [128 x 64]     out_i = near_i + f_i far_i
// With the states given, chunks do not wait for one another: items are dealt out evenly to one CTA per SM whatever the
// number of heads, where one scan per gradient took whole waves of CTAs (320 equal scans on 152 SMs at 4 x 16 heads,
// T = 8192, 128 x 64: three waves for 2.1 waves of work). A CTA holds a chunk's rows of all four tensors, copied once
// for its items (two chunks where they fit), and S and R; the items of one gradient share scores and P. Two items are in
// flight: both kinds of accumulator are double.
//
// Measured there: the whole backward 231 us; under ncu, cold, this kernel 143 and the state scans before it 96. With every
// item's operands copied for itself, its own scores and the places of its operands looked up by the issuing thread this
// kernel took 42 us more (gradients as scans: the whole 278); the rows shared, but looked up: 36. The instructions of the
// thread that issues the MMAs are the chain that is left, and the bytes that it moves (844 MB) take 125 us at the copy rate.
#include <atomic>
#include <type_traits>

#include "lla_linear_tc.cuh"

namespace lla {
namespace {

constexpr int kGradThreads = 640;
constexpr int kXPanel = 64 * 128;  // 64 rows of 64 bf16
constexpr int kSmemMost = 232448 - 2048;  // 227 KB less the static part
// TMEM columns: two buffers of scores, two of [near | far]
constexpr uint32_t kColS = 0, kColO = 256;

struct GradKind {
    int d1, tiles, reverse;
    int cols;  // of the output
};

struct GradParams {
    CUtensorMap map[4];
    GradKind kind[3];
    __nv_bfloat16* out[3];
    const float* log_a;
    const __nv_bfloat16* states;  // tiles of 128 rows of 64, each row's 16-byte pieces swizzled as shared memory wants them
    int rows_at[4], panels[4];    // a stage's rows of each tensor: first byte, panels of 64 columns
    int stage_bytes, nst;
    int BH, H, T, nch, v_tiles, k_panels, per_chunk;  // per_chunk: items of one chunk
    bool wide;  // 32-byte stores
    LinWaits waits;
};

// An item and its successors; every role walks its CTA's items with one of these. The items of one gradient and chunk
// (its columns' tiles) are a group: they share scores and P.
struct Item {
    int bh, h, ch, k, tile;
    __device__ __forceinline__ void next_group(const GradParams& pr) {
        tile = 0;
        if (++k < 3) return;
        k = 0;
        if (++ch < pr.nch) return;
        ch = 0;
        bh++;
        if (++h == pr.H) h = 0;
    }
    __device__ __forceinline__ void next(const GradParams& pr) {
        if (++tile == pr.kind[k].tiles) next_group(pr);
    }
};

__device__ __forceinline__ Item item_at(const GradParams& pr, int64_t i) {
    Item it;
    const int64_t c = i / pr.per_chunk;
    int r = static_cast<int>(i - c * pr.per_chunk);
    it.bh = static_cast<int>(c / pr.nch);
    it.h = it.bh % pr.H;
    it.ch = static_cast<int>(c - static_cast<int64_t>(it.bh) * pr.nch);
    it.k = 0;
    while (r >= pr.kind[it.k].tiles) r -= pr.kind[it.k++].tiles;
    it.tile = r;
    return it;
}

// Warps: 0 copies a chunk's rows, 2 S and 3 R; 1 issues the MMAs; 4..11 P (every other block of 32 keys), 12..19 write out
// (32 columns each). Warp w reaches TMEM lanes 32 (w % 4)..+31.
__global__ void __launch_bounds__(kGradThreads, 1) linear_grad_kernel(const __grid_constant__ GradParams pr, int* err) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t rows_full[2], rows_free[2];  // of a stage
    __shared__ uint64_t x_full[2], x_free[2];        // of S, of R
    __shared__ uint64_t s_full[2], p_ready[2], o_full[2], o_read[2], drain;
    __shared__ uint64_t never;  // nothing arrives here: for the test hook
    __shared__ uint32_t tmem_base_sh;
    __shared__ Bound bound;
    // forwards and backwards: weight of key c for row r of a diagonal 32-key block at 31 + r - c, and of key c of another
    // block. Each P warp writes what it reads, all the same, and none is a head's two groups of one direction ahead.
    __shared__ __align__(16) float weights[2][96];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t total = static_cast<int64_t>(pr.BH) * pr.nch * pr.per_chunk;
    const int64_t first = total * blockIdx.x / gridDim.x;
    const int m = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x - first);  // items of this CTA
    const int nst = pr.nst, x_bytes = pr.v_tiles * pr.k_panels * kXPanel;
    uint8_t* xs = smem + nst * pr.stage_bytes;  // the entering states S and R of a chunk, all their tiles
    volatile Bound* const fail = &bound;

    if (tid == 0) {
        for (int i = 0; i < 2; i++) {
            mbar_init(&rows_full[i], 1);
            mbar_init(&rows_free[i], 1);
            mbar_init(&x_full[i], 1);
            mbar_init(&x_free[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], 8);
            mbar_init(&o_full[i], 1);
            mbar_init(&o_read[i], 8);
        }
        mbar_init(&drain, 1);
        mbar_init(&never, 1);
        fence_mbar_init();
        bound = {pr.waits.cycles, 0};
    }
    if (warp == 1) tmem_alloc(&tmem_base_sh, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_dep_wait();  // the states
    const uint32_t tmem = tmem_base_sh;
    auto fail_now = [&]() {
        if (atomicExch(&bound.fail, 1) == 0) record_error(err, kDevTimeout);
    };

    if (warp == 0 || warp == 2 || warp == 3) {
        if (m > 0 && elect_one()) {
            const int64_t c0 = first / pr.per_chunk, c1 = (first + m - 1) / pr.per_chunk;
            if (warp == 0) {
                int s = 0, sent = 0;
                uint32_t ph = 1;
                for (int64_t c = c0; c <= c1; c++) {
                    if (sent >= nst && !wait_one(&rows_free[s], ph, fail)) {
                        fail_now();
                        break;
                    }
                    const int bh = static_cast<int>(c / pr.nch);
                    const int t0 = static_cast<int>(c - static_cast<int64_t>(bh) * pr.nch) * kTile;
                    mbar_expect_tx(&rows_full[s], pr.stage_bytes);
                    // in the order of their use
                    for (int u = 0; u < 4; u++) {
                        const int i = u == 0 ? 3 : u == 1 ? 2 : u == 2 ? 1 : 0;
                        for (int p = 0; p < pr.panels[i]; p++)
                            tma_load_3d(smem + s * pr.stage_bytes + pr.rows_at[i] + p * kPanelBytes, &pr.map[i],
                                        &rows_full[s], 64 * p, t0, bh);
                    }
                    sent++;
                    if (++s == nst) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                // every copy has landed before the shared memory goes away
                for (int i = sent > nst ? sent - nst : 0; i < sent; i++) mbar_wait(&rows_full[i % nst], (i / nst) & 1);
            } else {
                // S for the first gradient's items, R for the others'
                const int r = warp - 2, firsts = pr.kind[0].tiles;
                const int64_t from = r == 0 && first - c0 * pr.per_chunk >= firsts ? c0 + 1 : c0;
                const int64_t to = r == 1 && first + m - 1 - c1 * pr.per_chunk < firsts ? c1 - 1 : c1;
                int sent = 0;
                for (int64_t c = from; c <= to; c++, sent++) {
                    if (sent > 0 && !wait_one(&x_free[r], (sent - 1) & 1, fail)) {
                        fail_now();
                        break;
                    }
                    mbar_expect_tx(&x_full[r], x_bytes);
                    const __nv_bfloat16* x =
                        pr.states + (static_cast<int64_t>(r) * pr.BH * pr.nch + c) * pr.v_tiles * (kTile * kDepth);
                    for (int t = 0; t < pr.v_tiles; t++)
                        bulk_load(xs + r * x_bytes + t * pr.k_panels * kXPanel, x + t * (kTile * kDepth),
                                  pr.k_panels * kXPanel, &x_full[r]);
                }
                if (sent > 0) mbar_wait(&x_full[r], (sent - 1) & 1);
            }
        }
    } else if (warp == 1) {
        if (m > 0 && elect_one()) {
            constexpr uint32_t kIdS = idesc_bf16(kTile, kTile, 0, 0);
            constexpr uint32_t kIdMn = idesc_bf16(kTile, kDepth, 0, 1), kIdK = idesc_bf16(kTile, kDepth, 0, 0);
            // descriptors of the first stage's rows and of the states; a stage, a 64-column tile of X, a panel further
            const uint64_t base = sdesc(smem_u32(smem), 16, 1024), mn = sdesc(0, kPanelBytes, 1024) - sdesc(0, 16, 1024);
            const uint64_t at[4] = {further(base, pr.rows_at[0] >> 4), further(base, pr.rows_at[1] >> 4),
                                    further(base, pr.rows_at[2] >> 4), further(base, pr.rows_at[3] >> 4)};
            const uint64_t x_at[2] = {sdesc(smem_u32(xs), 16, 1024), sdesc(smem_u32(xs) + x_bytes, 16, 1024)};
            const uint64_t st_step = static_cast<uint64_t>(pr.stage_bytes >> 4);
            const uint64_t t_step = static_cast<uint64_t>((pr.k_panels * kXPanel) >> 4);
            const int k_tiles = pr.kind[0].tiles, v_tiles = pr.kind[2].tiles;
            const int v_steps = (pr.kind[0].d1 + 15) / 16, k_steps = (pr.kind[2].d1 + 15) / 16;
            auto kstep = [](int kk) { return static_cast<uint64_t>(((kk >> 2) * kPanelBytes + (kk & 3) * 32) >> 4); };
            // a gradient's row tensors a, b, c
            constexpr int kA[3] = {3, 2, 1}, kB[3] = {2, 3, 0}, kC[3] = {1, 0, 3};
            auto scores = [&](auto kind, uint64_t stage, uint32_t buf) {
                constexpr int K = decltype(kind)::value;
                const uint64_t a = further(at[kA[K]], stage), b = further(at[kB[K]], stage);
                const int steps = K == 2 ? k_steps : v_steps;
#pragma unroll
                for (int kk = 0; kk < 8; kk++)
                    if (kk < steps) mma_bf16(tmem + kColS + buf * kTile, further(a, kstep(kk)), further(b, kstep(kk)), kIdS, kk > 0);
                mma_commit(&s_full[buf]);
            };
            using K0 = std::integral_constant<int, 0>;
            using K1 = std::integral_constant<int, 1>;
            using K2 = std::integral_constant<int, 2>;
            Item it = item_at(pr, first);
            int k = it.k, tile = it.tile, j = 0, s = 0;  // s: stage of the chunk
            uint64_t stage = 0;                          // and what it adds to a descriptor
            uint32_t ph = 0, grp = 0;                    // its phase; groups so far
            uint32_t xph[2] = {0, 0};                    // phases of S and R
            bool ok = wait_one(&rows_full[0], 0, fail);
            if (ok) {
                tc_fence_after();
                if (k == 0) scores(K0(), 0, 0);
                else if (k == 1) scores(K1(), 0, 0);
                else scores(K2(), 0, 0);
            }
            // one item of gradient K; each gradient's code has its operands' places as constants, as this thread's
            // instructions are what the kernel waits for
            auto item = [&](auto kind) {
                constexpr int K = decltype(kind)::value, R = K == 0 ? 0 : 1;
                const int tiles = K == 2 ? v_tiles : k_tiles, steps = K == 2 ? k_steps : v_steps;
                const uint32_t buf = j & 1, use = (j >> 1) & 1, sbuf = grp & 1;
                const uint32_t d = tmem + kColO + buf * kTile;
                const bool opens = j == 0 || tile == 0, closes = tile + 1 == tiles;
                if (j >= 2 && !wait_one(&o_read[buf], use ^ 1u, fail)) return false;
                if (opens && (K < 2 || j == 0)) {  // the first item here that reads this state
                    if (!wait_one(&x_full[R], xph[R], fail)) return false;
                    xph[R] ^= 1u;
                }
                tc_fence_after();
                const uint64_t a = further(at[kA[K]], stage);
                if constexpr (K < 2) {
                    const uint64_t xt = further(x_at[R], (tile * kXPanel) >> 4);
#pragma unroll
                    for (int kk = 0; kk < 8; kk++)
                        if (kk < steps)
                            mma_bf16(d + kDepth, further(a, kstep(kk)), further(xt, (kk >> 2) * t_step + (kk & 3) * 2), kIdK,
                                     kk > 0);
                } else {
                    const uint64_t xt = further(x_at[R], mn + tile * t_step);
#pragma unroll
                    for (int kk = 0; kk < 8; kk++)
                        if (kk < steps) mma_bf16(d + kDepth, further(a, kstep(kk)), further(xt, 128u * kk), kIdMn, kk > 0);
                }
                if (closes && K != 1) mma_commit(&x_free[R]);
                // the next group's scores, so that its P is built while this one's is multiplied. With one stage the next
                // chunk's rows come only when this chunk is done
                const bool wrap = s + 1 == nst;
                if (opens && j + tiles - tile < m && (K < 2 || nst > 1)) {
                    // they take the place of the P that the item before this one read: MMAs of different accumulators are
                    // ordered by their completion only. This item's far product runs meanwhile
                    if (j > 0 && !wait_one(&o_full[buf ^ 1u], ((j - 1) >> 1) & 1, fail)) return false;
                    tc_fence_after();
                    if constexpr (K < 2) {
                        scores(std::integral_constant<int, K < 2 ? K + 1 : 0>(), stage, sbuf ^ 1u);
                    } else {
                        if (!wait_one(&rows_full[wrap ? 0 : s + 1], wrap ? ph ^ 1u : ph, fail)) return false;
                        tc_fence_after();
                        scores(K0(), wrap ? 0 : stage + st_step, sbuf ^ 1u);
                    }
                }
                if (opens) {
                    if (!wait_one(&p_ready[sbuf], (grp >> 1) & 1, fail)) return false;
                    tc_fence_after();
                }
                const uint64_t c = further(at[kC[K]], stage + ((tile * kPanelBytes) >> 4) + mn);
                const uint32_t p = tmem + kColS + sbuf * kTile;
#pragma unroll
                for (int kk = 0; kk < kTile / 16; kk++) {
                    mma_bf16_ta(d, p + 16 * kk, further(c, 128u * kk), kIdMn, kk > 0);
                    mma_bf16_ta(d, p + 16 * kk + 8, further(c, 128u * kk), kIdMn, 1);
                }
                mma_commit(&o_full[buf]);
                if (K == 2 && closes) {
                    mma_commit(&rows_free[s]);
                    ph = wrap ? ph ^ 1u : ph;
                    stage = wrap ? 0 : stage + st_step;
                    s = wrap ? 0 : s + 1;
                    if (nst == 1 && j + 1 < m) {
                        if (!wait_one(&rows_full[0], ph, fail)) return false;
                        tc_fence_after();
                        scores(K0(), 0, sbuf ^ 1u);
                    }
                }
                grp += closes;
                tile = closes ? 0 : tile + 1;
                j++;
                return true;
            };
            while (ok && j < m) {
                for (; k == 0 && ok && j < m; k += ok && tile == 0) ok = item(K0());
                for (; k == 1 && ok && j < m; k += ok && tile == 0) ok = item(K1());
                for (; k == 2 && ok && j < m; k = ok && tile == 0 ? 0 : k) ok = item(K2());
            }
            if (!ok) fail_now();
            // every MMA issued above has completed before TMEM and shared memory go away
            mma_commit(&drain);
            if (!mbar_wait(&drain, 0)) fail_now();
        }
    } else if (warp >= 4 && warp < 12) {
        const int w = warp & 3;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(w * 32) << 16);
        Item it = item_at(pr, first);
        int made[2] = {-1, -1};  // head of the tables
        float far[2][3] = {};    // the row's part of the weight of a block one, two, three blocks off
        for (int j = 0, grp = 0; j < m; grp++) {
            const int rev = pr.kind[it.k].reverse, buf = grp & 1;
            float* wt = weights[rev];
            if (!wait_warp(&s_full[buf], (grp >> 1) & 1, fail)) {
                if (lane == 0) fail_now();
                break;
            }
            // these scores came after the P of every warp for the group before the last
            if (it.h != (rev ? made[1] : made[0])) {
                const float la = pr.log_a[it.h];
#pragma unroll
                for (int u = 0; u < 2; u++) {
                    const int x = lane + 32 * u, gap = rev ? 31 - x : x - 31;
                    wt[x] = gap >= 0 ? gpow(la, gap) : 0.f;
                }
                wt[64 + lane] = gpow(la, rev ? lane : 31 - lane);
                made[0] = rev ? made[0] : it.h;
                made[1] = rev ? it.h : made[1];
#pragma unroll
                for (int u = 0; u < 3; u++) {
                    const float f = gpow(la, rev ? 32 * (u + 1) - lane : 32 * u + lane + 1);
                    far[0][u] = rev ? far[0][u] : f;
                    far[1][u] = rev ? f : far[1][u];
                }
                __syncwarp();
            }
            tc_fence_after();
            const uint32_t cols = lanes + kColS + buf * kTile;
#pragma unroll 1
            for (int cb = (warp - 4) >> 2; cb < 4; cb += 2) {
                const int side = cb == w ? 0 : (rev ? cb > w : cb < w) ? 1 : -1;
                const int off = rev ? cb - w : w - cb;
                const float rw = rev ? (off == 1 ? far[1][0] : off == 2 ? far[1][1] : far[1][2])
                                     : (off == 1 ? far[0][0] : off == 2 ? far[0][1] : far[0][2]);
                weigh_block<2>(cols + 32 * cb, side, wt + 31 + lane, wt + 64, rw);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready[buf]);
            j += pr.kind[it.k].tiles - it.tile;
            it.next_group(pr);
        }
    } else {
        const int row = (warp & 3) * 32 + lane, cw = (warp - 12) / 4 * 32;
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        Item it = item_at(pr, first);
        int made = -1;
        float la = 0.f;
        const bool held = pr.waits.hold && !wait_warp(&never, 0, fail);
        if (held && lane == 0) fail_now();
        for (int j = 0; j < m && !held; j++) {
            const GradKind& kd = pr.kind[it.k];
            const int rev = kd.reverse;
            if (it.h != made) {
                made = it.h;
                la = pr.log_a[it.h];
            }
            const int nr = pr.T - it.ch * kTile < kTile ? pr.T - it.ch * kTile : kTile;
            const float f = row < nr ? gpow(la, rev ? nr - 1 - row : row + 1) : 0.f;
            const f32x2 f2 = pair2(f, f);
            const int col = it.tile * kDepth + cw;
            __nv_bfloat16* to = pr.out[it.k] + (static_cast<int64_t>(it.bh) * pr.T + it.ch * kTile + row) * kd.cols + col;
            if (!wait_warp(&o_full[j & 1], (j >> 1) & 1, fail)) {
                if (lane == 0) fail_now();
                break;
            }
            tc_fence_after();
            const uint32_t from = lanes + kColO + (j & 1) * kTile + cw;
            uint32_t o[2][8];
#pragma unroll
            for (int c = 0; c < 2; c++) {
                f32x2 a[8], y[8];
                tmem_ld16x2(from + 16 * c, from + kDepth + 16 * c, a, y);
#pragma unroll
                for (int i = 0; i < 8; i++) o[c][i] = pack_bf16(fma2(f2, y[i], a[i]));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_read[j & 1]);
            // rows past T and columns past the tensor's are not written
#pragma unroll
            for (int c = 0; c < 2; c++)
                if (row < nr && col + 16 * c < kd.cols)
                    store32(to + 16 * c, o[c], pr.wide && kd.cols % 16 == 0, col + 16 * c + 8 < kd.cols);
            it.next(pr);
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

constexpr int kMaxDevices = 64;
std::atomic<int> g_sms[kMaxDevices];  // asked once of a device, with the kernel's shared memory set

int grad_sms() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return 0;
    }
    int sms = g_sms[dev].load(std::memory_order_acquire);
    if (sms) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaFuncSetAttribute(linear_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost) !=
            cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    g_sms[dev].store(sms, std::memory_order_release);
    return sms;
}

}  // namespace

size_t linear_grad_state_bytes(int BH, int T, int dv) {
    return static_cast<size_t>(2) * BH * ((T - 1) / kTile + 1) * ((dv + kDepth - 1) / kDepth) * kTile * kDepth *
           sizeof(__nv_bfloat16);
}

cudaError_t linear_tc_grads(const void* q, const void* k, const void* v, const void* dout, const float* log_a,
                            const void* states, void* dq, void* dk, void* dv, int BH, int H, int T, int d_k, int d_v,
                            int* err, cudaStream_t stream) {
    const int sms = grad_sms();
    if (sms <= 0) return cudaErrorUnknown;
    GradParams pr = {};
    const int nch = (T - 1) / kTile + 1;
    const int kt = (d_k + kDepth - 1) / kDepth, vt = (d_v + kDepth - 1) / kDepth;
    const void* rows[4] = {q, k, v, dout};
    for (int i = 0; i < 4; i++) {
        if (!make_map_3d(&pr.map[i], rows[i], BH, T, i < 2 ? d_k : d_v, kTile)) return cudaErrorInvalidValue;
        pr.panels[i] = i < 2 ? kt : vt;
        pr.rows_at[i] = pr.stage_bytes;
        pr.stage_bytes += pr.panels[i] * kPanelBytes;
    }
    void* outs[3] = {dq, dk, dv};
    pr.wide = true;
    for (int i = 0; i < 3; i++) {
        pr.out[i] = static_cast<__nv_bfloat16*>(outs[i]);
        if (reinterpret_cast<uintptr_t>(outs[i]) % 32) pr.wide = false;
    }
    pr.kind[0] = {d_v, kt, 0, d_k};
    pr.kind[1] = {d_v, kt, 1, d_k};
    pr.kind[2] = {d_k, vt, 1, d_v};
    pr.states = static_cast<const __nv_bfloat16*>(states);
    pr.log_a = log_a;
    pr.BH = BH;
    pr.H = H;
    pr.T = T;
    pr.nch = nch;
    pr.waits = linear_waits();
    pr.v_tiles = vt;
    pr.k_panels = kt;
    pr.per_chunk = 2 * kt + vt;
    // two stages but where both dk and dv are above 64
    const int x_bytes = 2 * vt * kt * kXPanel + 1024;
    pr.nst = 2 * pr.stage_bytes + x_bytes <= kSmemMost ? 2 : 1;
    const int smem = pr.nst * pr.stage_bytes + x_bytes;
    const int64_t items = static_cast<int64_t>(BH) * nch * pr.per_chunk;
    const unsigned grid = static_cast<unsigned>(items < sms ? items : sms);
    const cudaError_t e = launch_pdl(linear_grad_kernel, dim3(grid), dim3(kGradThreads), smem, stream, pr, err);
    if (e != cudaSuccess) return e;
    note_launch(stream, "linear_grad");
    return cudaGetLastError();
}

}  // namespace lla
