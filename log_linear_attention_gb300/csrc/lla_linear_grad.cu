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
// With the states given, chunks do not wait for one another: items are dealt out evenly to one CTA per SM
// whatever the number of heads, where one scan per gradient took whole waves of CTAs (320 equal scans on 152
// SMs at 4 x 16 heads, T = 8192, 128 x 64: three waves for 2.1 waves of work, 367 us for the backward against 270).
// Consecutive items share their chunk's rows in L2. Two items are in flight: both kinds of accumulator are double.
//
// Measured there: 184 us for 20480 items, 848 MB at 4.6 TB/s (68% of the copy rate), tensor pipe 38% and issue slots 54%
// busy; an item is 1.3 us. What bounds it is the chain scores -> P -> near -> out of two items in flight, with the
// issue slots that P and out take; the two state scans before it take 89 us (514 MB at 5.8 TB/s).
#include <atomic>

#include "lla_linear_tc.cuh"

namespace lla {
namespace {

constexpr int kGradThreads = 640;
constexpr int kMaxStages = 3;
constexpr int kXPanel = 64 * 128;  // 64 rows of 64 bf16
constexpr int kSmemMost = 232448 - 6144;
// TMEM columns: two buffers of scores, two of [near | far]
constexpr uint32_t kColS = 0, kColO = 256;

struct GradKind {
    int ia, ib, ic;  // tensor maps: 0 q, 1 k, 2 v, 3 dout
    int d1, tiles, reverse;
    int state_t;      // X is read as the transpose of the stored rows
    int states_base;  // first (b, h, chunk) of its state in the buffer
};

struct GradParams {
    CUtensorMap map[4], omap[3];
    GradKind kind[3];
    const float* log_a;
    const __nv_bfloat16* states;  // tiles of 128 rows of 64, each row's 16-byte pieces swizzled as shared memory wants them
    int BH, H, T, nch, v_tiles, per_chunk;  // per_chunk: items of one chunk
};

// An item and its successor; every role walks its CTA's items with one of these.
struct Item {
    int bh, h, ch, k, tile;
    __device__ __forceinline__ void next(const GradParams& pr) {
        if (++tile < pr.kind[k].tiles) return;
        tile = 0;
        if (++k < 3) return;
        k = 0;
        if (++ch < pr.nch) return;
        ch = 0;
        bh++;
        if (++h == pr.H) h = 0;
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

// Warps: 0 copies a and X, 2 b, 3 c; 1 issues the MMAs; 4..11 P (every other block of 32 keys), 12..19 write out
// (32 columns each). Warp w reaches TMEM lanes 32 (w % 4)..+31.
__global__ void __launch_bounds__(kGradThreads, 1) linear_grad_kernel(const __grid_constant__ GradParams pr, int nst,
                                                                      int np_most, int* err) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t ax_full[kMaxStages], b_full[kMaxStages], c_full[kMaxStages];
    __shared__ uint64_t ax_free[kMaxStages], b_free[kMaxStages], c_free[kMaxStages];
    __shared__ uint64_t s_full[2], p_ready[2], o_full[2], o_read[2], out_put, out_free, drain;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int fail_sh;
    // per P warp: weight of key c for row r of a diagonal 32-key block at 31 + r - c, and of key c of another block
    __shared__ __align__(16) float weights[8][96];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t total = static_cast<int64_t>(pr.BH) * pr.nch * pr.per_chunk;
    const int64_t first = total * blockIdx.x / gridDim.x;
    const int m = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x - first);  // items of this CTA
    // a stage: a | b | c | X
    const int b_off = np_most * kPanelBytes, c_off = 2 * b_off, x_off = c_off + kPanelBytes;
    const int stage_bytes = x_off + np_most * kXPanel;
    uint8_t* stage_out = smem + nst * stage_bytes;  // an item's output rows on their way to memory
    volatile int* fail = &fail_sh;

    if (tid == 0) {
        for (int s = 0; s < nst; s++) {
            mbar_init(&ax_full[s], 1);
            mbar_init(&b_full[s], 1);
            mbar_init(&c_full[s], 1);
            mbar_init(&ax_free[s], 1);
            mbar_init(&b_free[s], 1);
            mbar_init(&c_free[s], 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], 8);
            mbar_init(&o_full[i], 1);
            mbar_init(&o_read[i], 8);
        }
        mbar_init(&out_put, 8);
        mbar_init(&out_free, 1);
        mbar_init(&drain, 1);
        fence_mbar_init();
        fail_sh = 0;
    }
    if (warp == 1) tmem_alloc(&tmem_base_sh, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_dep_wait();  // the states
    const uint32_t tmem = tmem_base_sh;
    auto fail_now = [&]() {
        if (atomicExch(&fail_sh, 1) == 0) record_error(err, kDevTimeout);
    };

    if (warp == 0 || warp == 2 || warp == 3) {
        // each operand is free at another time, so each is waited for by a warp of its own
        if (m > 0 && elect_one()) {
            uint64_t* full = warp == 0 ? ax_full : warp == 2 ? b_full : c_full;
            uint64_t* free_ = warp == 0 ? ax_free : warp == 2 ? b_free : c_free;
            Item it = item_at(pr, first);
            int s = 0, sent = 0;
            uint32_t ph = 1;
            for (int j = 0; j < m; j++) {
                if (j >= nst && !wait_one(&free_[s], ph, fail)) {
                    fail_now();
                    break;
                }
                const GradKind& kd = pr.kind[it.k];
                const int np = kd.d1 > 64 ? 2 : 1, t0 = it.ch * kTile;
                uint8_t* st = smem + s * stage_bytes;
                if (warp == 0) {
                    mbar_expect_tx(&full[s], np * (kPanelBytes + kXPanel));
                    const int64_t x0 = static_cast<int64_t>(kd.states_base + it.bh * pr.nch + it.ch) * pr.v_tiles;
                    for (int p = 0; p < np; p++) {
                        tma_load_3d(st + p * kPanelBytes, &pr.map[kd.ia], &full[s], 64 * p, t0, it.bh);
                        // 64 state rows of one 64-column tile: rows of X, or of 64 columns of d1 of its transpose
                        bulk_load(st + x_off + p * kXPanel,
                                  pr.states + ((x0 + (kd.state_t ? p : it.tile)) * 2 + (kd.state_t ? it.tile : p)) *
                                                  (kXPanel / 2),
                                  kXPanel, &full[s]);
                    }
                } else if (warp == 2) {
                    mbar_expect_tx(&full[s], np * kPanelBytes);
                    for (int p = 0; p < np; p++)
                        tma_load_3d(st + b_off + p * kPanelBytes, &pr.map[kd.ib], &full[s], 64 * p, t0, it.bh);
                } else {
                    mbar_expect_tx(&full[s], kPanelBytes);
                    tma_load_3d(st + c_off, &pr.map[kd.ic], &full[s], it.tile * kDepth, t0, it.bh);
                }
                sent++;
                it.next(pr);
                if (++s == nst) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            // every copy has landed before the shared memory goes away
            for (int i = sent > nst ? sent - nst : 0; i < sent; i++) mbar_wait(&full[i % nst], (i / nst) & 1);
        }
    } else if (warp == 1) {
        if (m > 0 && elect_one()) {
            constexpr uint32_t kIdS = idesc_bf16(kTile, kTile, 0, 0);
            constexpr uint32_t kIdMn = idesc_bf16(kTile, kDepth, 0, 1), kIdK = idesc_bf16(kTile, kDepth, 0, 0);
            const uint64_t step = static_cast<uint64_t>(stage_bytes >> 4);
            const uint64_t a_first = sdesc(smem_u32(smem), 16, 1024), mn = sdesc(0, kPanelBytes, 1024) - sdesc(0, 16, 1024);
            const uint64_t to_b = static_cast<uint64_t>(b_off >> 4), to_c = static_cast<uint64_t>(c_off >> 4) + mn;
            const uint64_t to_x = static_cast<uint64_t>(x_off >> 4);
            auto kstep = [](int kk) { return static_cast<uint64_t>(((kk >> 2) * kPanelBytes + (kk & 3) * 32) >> 4); };
            auto scores = [&](uint64_t a, int s, uint32_t ph, uint32_t buf, int ksteps) {
                if (!wait_one(&ax_full[s], ph, fail) || !wait_one(&b_full[s], ph, fail)) return false;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 8; kk++)
                    if (kk < ksteps)
                        mma_bf16(tmem + kColS + buf * kTile, a + kstep(kk), a + to_b + kstep(kk), kIdS, kk > 0);
                mma_commit(&s_full[buf]);
                mma_commit(&b_free[s]);
                return true;
            };
            Item it = item_at(pr, first);
            int s = 0;
            uint32_t ph = 0;
            uint64_t a = a_first;
            int ksteps = (pr.kind[it.k].d1 + 15) / 16;
            bool ok = scores(a, 0, 0, 0, ksteps);
            for (int j = 0; j < m && ok; j++) {
                const uint32_t buf = j & 1, use = (j >> 1) & 1;
                const uint32_t d = tmem + kColO + buf * kTile;
                if (j >= 2) ok = wait_one(&o_read[buf], use ^ 1u, fail);
                if (!ok) break;
                tc_fence_after();
                if (pr.kind[it.k].state_t) {
#pragma unroll
                    for (int kk = 0; kk < 8; kk++)
                        if (kk < ksteps)
                            mma_bf16(d + kDepth, a + kstep(kk),
                                     a + to_x + static_cast<uint64_t>(((kk >> 2) * kXPanel + (kk & 3) * 32) >> 4), kIdK,
                                     kk > 0);
                } else {
#pragma unroll
                    for (int kk = 0; kk < 8; kk++)
                        if (kk < ksteps) mma_bf16(d + kDepth, a + kstep(kk), a + to_x + mn + 128u * kk, kIdMn, kk > 0);
                }
                mma_commit(&ax_free[s]);
                // the next item's scores, so that its P is built while this one's is multiplied
                const uint64_t ct = a + to_c;
                const int cs = s;
                const uint32_t cph = ph;
                a += step;
                if (++s == nst) {
                    s = 0;
                    ph ^= 1u;
                    a = a_first;
                }
                it.next(pr);
                if (j + 1 < m) {
                    ksteps = (pr.kind[it.k].d1 + 15) / 16;
                    ok = scores(a, s, ph, buf ^ 1u, ksteps);
                }
                ok = ok && wait_one(&p_ready[buf], use, fail) && wait_one(&c_full[cs], cph, fail);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < kTile / 16; kk++) {
                    const uint32_t p = tmem + kColS + buf * kTile + 16 * kk;
                    mma_bf16_ta(d, p, ct + 128u * kk, kIdMn, kk > 0);
                    mma_bf16_ta(d, p + 8, ct + 128u * kk, kIdMn, 1);
                }
                mma_commit(&o_full[buf]);
                mma_commit(&c_free[cs]);
            }
            if (!ok) fail_now();
            // every MMA issued above has completed before TMEM and shared memory go away
            mma_commit(&drain);
            if (!mbar_wait(&drain, 0)) fail_now();
        }
    } else if (warp >= 4 && warp < 12) {
        const int w = warp & 3;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(w * 32) << 16);
        float* wt = weights[warp - 4];
        Item it = item_at(pr, first);
        int made = -1;  // head and direction of the table
        float far[3] = {};  // the row's part of the weight of a block one, two, three blocks off
        for (int j = 0; j < m; j++) {
            const int rev = pr.kind[it.k].reverse, key = 2 * it.h + rev;
            if (key != made) {
                made = key;
                const float la = pr.log_a[it.h];
                __syncwarp();
#pragma unroll
                for (int u = 0; u < 2; u++) {
                    const int x = lane + 32 * u, gap = rev ? 31 - x : x - 31;
                    wt[x] = gap >= 0 ? gpow(la, gap) : 0.f;
                }
                wt[64 + lane] = gpow(la, rev ? lane : 31 - lane);
#pragma unroll
                for (int u = 0; u < 3; u++) far[u] = gpow(la, rev ? 32 * (u + 1) - lane : 32 * u + lane + 1);
                __syncwarp();
            }
            if (!wait_warp(&s_full[j & 1], (j >> 1) & 1, fail)) {
                if (lane == 0) fail_now();
                break;
            }
            tc_fence_after();
            const uint32_t cols = lanes + kColS + (j & 1) * kTile;
#pragma unroll 1
            for (int cb = (warp - 4) >> 2; cb < 4; cb += 2) {
                const int side = cb == w ? 0 : (rev ? cb > w : cb < w) ? 1 : -1;
                const int off = rev ? cb - w : w - cb;
                const float rw = off == 1 ? far[0] : off == 2 ? far[1] : far[2];
                weigh_block<2>(cols + 32 * cb, side, wt + 31 + lane, wt + 64, rw);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready[j & 1]);
            it.next(pr);
        }
    } else {
        const int row = (warp & 3) * 32 + lane, cw = (warp - 12) / 4 * 32;
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        Item it = item_at(pr, first);
        int made = -1;
        float la = 0.f;
        for (int j = 0; j < m; j++) {
            const int rev = pr.kind[it.k].reverse;
            if (it.h != made) {
                made = it.h;
                la = pr.log_a[it.h];
            }
            const int nr = pr.T - it.ch * kTile < kTile ? pr.T - it.ch * kTile : kTile;
            const float f = row < nr ? gpow(la, rev ? nr - 1 - row : row + 1) : 0.f;
            const f32x2 f2 = pair2(f, f);
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
            if (j > 0 && !wait_warp(&out_free, (j - 1) & 1, fail)) {
                if (lane == 0) fail_now();
                break;
            }
#pragma unroll
            for (int c = 0; c < 4; c++)
                *reinterpret_cast<uint4*>(stage_out + sw128_off(row, cw / 8 + c)) =
                    make_uint4(o[c / 2][c % 2 * 4], o[c / 2][c % 2 * 4 + 1], o[c / 2][c % 2 * 4 + 2],
                               o[c / 2][c % 2 * 4 + 3]);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&out_put);
            if (warp == 12) {
                if (elect_one()) {
                    // rows past T and columns past the tensor's are not written
                    if (wait_one(&out_put, j & 1, fail)) {
                        tma_store_3d(&pr.omap[it.k], stage_out, it.tile * kDepth, it.ch * kTile, it.bh);
                        bulk_commit();
                        bulk_wait_read0();
                        mbar_arrive(&out_free);
                    } else {
                        fail_now();
                    }
                }
                __syncwarp();
            }
            it.next(pr);
        }
        if (warp == 12) bulk_wait0();
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
    for (int i = 0; i < 4; i++)
        if (!make_map_3d(&pr.map[i], rows[i], BH, T, i < 2 ? d_k : d_v, kTile)) return cudaErrorInvalidValue;
    void* outs[3] = {dq, dk, dv};
    for (int i = 0; i < 3; i++)
        if (!make_map_3d(&pr.omap[i], outs[i], BH, T, i < 2 ? d_k : d_v, kTile)) return cudaErrorInvalidValue;
    pr.kind[0] = {3, 2, 1, d_v, kt, 0, 1, 0};
    pr.kind[1] = {2, 3, 0, d_v, kt, 1, 1, BH * nch};
    pr.kind[2] = {1, 0, 3, d_k, vt, 1, 0, BH * nch};
    pr.states = static_cast<const __nv_bfloat16*>(states);
    pr.log_a = log_a;
    pr.BH = BH;
    pr.H = H;
    pr.T = T;
    pr.nch = nch;
    pr.v_tiles = vt;
    pr.per_chunk = 2 * kt + vt;
    const int np = (d_k > d_v ? d_k : d_v) > 64 ? 2 : 1, nst = np == 2 ? 2 : 3;
    const int smem = nst * ((2 * np + 1) * kPanelBytes + np * kXPanel) + kPanelBytes + 1024;
    const int64_t items = static_cast<int64_t>(BH) * nch * pr.per_chunk;
    const unsigned grid = static_cast<unsigned>(items < sms ? items : sms);
    const cudaError_t e = launch_pdl(linear_grad_kernel, dim3(grid), dim3(kGradThreads), smem, stream, pr, nst, np, err);
    if (e != cudaSuccess) return e;
    note_launch(stream, "linear_grad");
    return cudaGetLastError();
}

}  // namespace lla
