// Linear attention with one decay per head on tensor cores: bf16 rows, dk and dv multiples of 8.
//
// One kernel walks a scan (see lla_linear.cu: out_t = S_t^T a_t, S_t = g S_{t-1} + b_t c_t^T) over one
// (sequence, head, 64 columns of c) in chunks of 128 tokens. The state (d1 x 64, fp32) never leaves the
// registers of eight warps. Per chunk, n valid rows:
//     scores  A B^T                      [128 x 128]  -> TMEM
//     own     B^T [hi | mid + lo]        [d1 x 128]   -> TMEM, w o C cut into three bf16 parts, so that the
//                                                     state keeps the 24 bits of fp32 (only states: [hi | mid | lo])
//     far     A X                        [128 x 64]   X = entering state, rounded to bf16
//     near    P C                        [128 x 64]   P = scores o g^|i-j|, two bf16 parts in TMEM
//     out_i = near_i + f_i far_i,   X <- g^n X + own
// with w_i = g^(n-1-i), f_i = g^(i+1) (states formed backwards: w_i = g^(i+1)). X is rounded to bf16 as an operand of a
// bf16 product must be (2^-8 of each term, as the output itself). P is given in two bf16 parts, 16 bits: with one the
// outputs' error was 1.4 times that of fp32 arithmetic rounded once, with two it is 1.2 times, for 2% of the time.
// Scores, sums, weights and the state are fp32.
//
// Heads alone do not fill the GPU when they are few, so a scan may be cut into segments, one CTA each: a first
// launch (kPieces) forms the own states of pieces of every segment but the last (smaller than segments, as
// it is launched without the last segment's share), and each segment's CTA sums those before it, decayed, in
// order. kFull does all of the above, forwards; kStates only forms the states, forwards or backwards, and
// writes the one that enters each chunk in bf16 for the kernel of the gradients (lla_linear_grad.cu).
//
// Measured (GB300): a chunk takes about 2.1 us (1.2 where only the state is formed). What bounds it is shared memory: at
// d = 128 its products read 288 KB of operands, the copies write 80 KB, the cut reads and writes 64 KB and X takes 16: 448 KB,
// 3500 of the 4000 cycles at 128 bytes each. (Two warps issuing the MMAs, each half of them, took 101 us where one took
// 97.) Two stages, as shared memory is full: 224 KB.
// 4 x 16 heads, T = 8192, 128 x 64: 99 us for 403 MB, 492 with the pieces'. 16 heads, T = 65536, 128 x 128: 366 us. 32
// packed sequences of 256..8192: 252 us for 1.53 GB, 90% of the copy rate.
//
// Rows of a chunk behind its sequence's end (another sequence's, when packed) are set to zero in shared
// memory before any product sums over them. Every wait is bounded; on overrun the kernel records
// LLA_ERR_TIMEOUT in the device error word, lets its own copies and MMAs land and returns.
#include <atomic>
#include <cmath>

#include "lla_linear_tc.cuh"

namespace lla {
namespace {

constexpr int kScanThreads = 1024;
constexpr int kWcBytes = 3 * kPanelBytes;
constexpr int kSmemMost = 232448 - 2048;  // 227 KB less the static part

// TMEM columns
// two buffers of scores (P takes the place of its scores: per 16 keys eight columns of high parts, eight of low); own: the
// high part's product, then that of the middle and low parts. Only states: two buffers of own, each part's product apart
constexpr uint32_t kColS = 0, kColNear = 256, kColFar = 320, kColOwn = 384, kOwnStates = 3 * kDepth;

enum { kFull, kPieces, kStates };  // what a launch forms: see above

struct ScanParams {
    CUtensorMap map[4];
    LinTcScan scan[2];
    const float* log_a;
    float* seg;             // pieces' own states
    __nv_bfloat16* states;  // kStates: the entering states
    LinSeqs sq;
    int count, nseg, seg_chunks, npiece, piece_chunks, seg_pieces, packed;
    LinWaits waits;
};

// Warps: 0 and 2 TMA producers, 1 TMEM owner and MMA issuer, 4..11 P (every other block of 32 keys), 12..19 state
// (32 columns each), 20..23 write out, 24..31 cut w o C. Warp w reaches TMEM lanes 32 (w % 4)..+31: rows of scores and
// out, rows of the state.
template <int kMode>
__global__ void __launch_bounds__(kScanThreads, 1) linear_scan_kernel(const __grid_constant__ ScanParams pr, int* err) {
    constexpr bool kStateOnly = kMode != kFull;
    constexpr int kCutWarps = kStateOnly ? 16 : 8;  // where there is no P, its warps cut w o C too
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // one barrier per lane of the warp that sets them up, and one more
    __shared__ uint64_t bars[33];
    uint64_t *const qk_full = bars, *const v_full = bars + 4, *const qk_free = bars + 8, *const v_free = bars + 12;
    uint64_t *const scaled = bars + 16, *const own_full = bars + 18, *const own_read = bars + 20, *const s_full = bars + 22;
    uint64_t &x_ready = bars[24], &x_free = bars[25], &x_put = bars[26], &x_sent = bars[27];
    // p_ready of even and odd chunks: the next chunk's scores may be there before a P warp is done with this one's
    uint64_t *const p_ready = bars + 28, &o_full = bars[30], &o_read = bars[31], &drain = bars[32];
    __shared__ uint32_t tmem_base_sh;
    __shared__ Bound bound;
    __shared__ float pw[132];    // g^n
    __shared__ __align__(16) float colw[32];  // weight of key c of an off-diagonal 32-key block
    __shared__ float diag[64];   // weight of key c for row r of a diagonal block, at 31 + r - c

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (pr.packed) grid_dep_wait();  // the sequence table; pieces' states are waited for below
    grid_dep_launch();
    // ---- which scan, segment and 64 columns (one or two of them), sequence and head. Divisions are kept out: a CTA's
    // start is a quarter of a short prompt
    const int ncta = kMode == kPieces ? pr.npiece : pr.nseg;  // of one sequence, head and 64 columns
    int x = blockIdx.x, si = 0;
    if (pr.count > 1 && x >= ncta * pr.scan[0].tiles) x -= ncta * pr.scan[si++].tiles;
    const LinTcScan& sc = pr.scan[si];
    const int tile = x & (sc.tiles - 1), g = x >> (sc.tiles - 1);
    int b = blockIdx.y / pr.sq.H, len = pr.sq.T, row0 = 0;
    const int h = blockIdx.y - b * pr.sq.H;
    if (pr.packed) {
        b = pr.sq.order[b];
        row0 = pr.sq.tab[b].x;
        len = pr.sq.tab[b].y;
        if (len < 0) return;
    }
    const int bh = b * pr.sq.H + h;
    const int z = pr.packed ? h : bh;  // outermost coordinate of the tensor maps
    const int nch = static_cast<int>((static_cast<unsigned>(len) + kTile - 1) / kTile);  // len may be 2^31 - 1
    const int have = nch <= pr.seg_chunks ? 1 : pr.packed ? (nch + pr.seg_chunks - 1) / pr.seg_chunks : pr.nseg;
    const int span = kMode == kPieces ? pr.piece_chunks : pr.seg_chunks;
    const int p0 = g * span;
    if (kMode == kPieces ? p0 >= (have - 1) * pr.seg_chunks : g >= have) return;
    const int n = nch - p0 < span ? nch - p0 : span;  // chunks of this CTA
    const bool rev = kStateOnly && sc.reverse != 0;
    auto chunk_of = [&](int j) { return rev ? nch - 1 - (p0 + j) : p0 + j; };
    auto rows_of = [&](int c) { return len - c * kTile < kTile ? len - c * kTile : kTile; };
    // tokens ahead of the p-th chunk in scan order
    auto before = [&](int p) { return !rev ? p * kTile : (p == 0 ? 0 : len - (nch - p) * kTile); };
    const int d1 = sc.d1, d2 = sc.d2, c0 = tile * kDepth;
    const int np = d1 > 64 ? 2 : 1, ksteps = (d1 + 15) / 16;
    // Shared memory. kFull: stages of a | b | c, two (three of narrow rows), then the parts of w o C and X. Only states:
    // as many of b, four of c (free once cut; kStates: three, and one of the states on its way to memory) and two of the
    // parts, so that copies, cutting and product all overlap.
    const int k_bytes = np * kPanelBytes;
    const int nk = np == 1 ? 3 : 2, nv = kMode == kFull ? nk : kMode == kPieces ? 4 : 3;
    const int k_step = kStateOnly ? k_bytes : 2 * k_bytes + kPanelBytes;  // from one stage of b to the next
    const int v_step = kStateOnly ? kPanelBytes : k_step;
    const int k_off = kStateOnly ? 0 : k_bytes, v_off = kStateOnly ? nk * k_bytes : 2 * k_bytes;
    uint8_t* wc = smem + (kStateOnly ? v_off + nv * kPanelBytes : nk * k_step);
    uint8_t* xs = wc + (kStateOnly ? 2 : 1) * kWcBytes;  // kFull, kStates
    volatile Bound* const fail = &bound;
    uint64_t* const never = kStateOnly ? s_full : &x_put;  // a barrier that no role of this mode uses, for the test hook

    if (warp == 0) {
        // arrivals of a phase: one but where several warps take part
        const int parties = lane >= 12 && lane < 16 ? (kStateOnly ? kCutWarps : 1) : lane == 16 || lane == 17 ? kCutWarps :
                            lane == 20 || lane == 21 || lane == 24 || lane == 26 || lane == 28 || lane == 29 ? 8 :
                            lane == 31 ? 4 : 1;
        mbar_init(&bars[lane], parties);
        if (lane == 0) mbar_init(&drain, 1);
        fence_mbar_init();
        if (lane == 0) bound = {pr.waits.cycles, 0};
    }
    if (warp == 1) tmem_alloc(&tmem_base_sh, 512);
    const float la = pr.log_a[h];
    if (tid >= 64 && tid < 64 + 129) pw[tid - 64] = gpow(la, tid - 64);
    if (tid >= 256 && tid < 288) colw[tid - 256] = gpow(la, 31 - (tid - 256));
    if (tid >= 320 && tid < 383) {
        const int u = tid - 320 - 31;  // r - c
        diag[tid - 320] = u >= 0 ? gpow(la, u) : 0.f;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    // own states of the sequence's pieces, [64 columns][prow rows] each, at every 64 x 128
    const int prow = 64 * np;
    float* seg0 = pr.seg + (static_cast<int64_t>(sc.seg_base) +
                            static_cast<int64_t>(bh) * pr.npiece * sc.tiles + tile) * (kDepth * kTile);
    const int64_t seg_step = static_cast<int64_t>(sc.tiles) * (kDepth * kTile);
    if (kMode != kPieces && g > 0 && warp >= 4 && warp < 20) {
        // the pieces before this segment, decayed to its start and summed in order, while the first copies and scores run
        grid_dep_wait();
        constexpr int kSumThreads = 512;
        const float gp = gpow(la, pr.piece_chunks * kTile);
        const int count = g * pr.seg_pieces;
        // round trips are what this takes, so four pieces' loads are in flight (2 x 4 heads, T = 2048: 18.4 -> 15.9 us;
        // eight take 0.3 off that and cost the roles registers: 97 -> 99.7 us at 4 x 16 heads, T = 8192)
        constexpr int kAhead = 4;
#pragma unroll 1
        for (int at = tid - 128; at < 16 * prow; at += kSumThreads) {
            const float4* src = reinterpret_cast<const float4*>(seg0) + at;
            float4 sum = {};
#pragma unroll 1
            for (int left = count; left > 0; left -= kAhead, src += kAhead * (seg_step / 4)) {
                float4 y[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; u++)
                    if (u < left) y[u] = src[u * (seg_step / 4)];
#pragma unroll
                for (int u = 0; u < kAhead; u++)
                    if (u < left) {
                        sum.x = gp * sum.x + y[u].x;
                        sum.y = gp * sum.y + y[u].y;
                        sum.z = gp * sum.z + y[u].z;
                        sum.w = gp * sum.w + y[u].w;
                    }
            }
            reinterpret_cast<float4*>(wc)[at] = sum;
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kSumThreads) : "memory");
    }
    // A CTA's last chunk adds to no state that is read, unless the state leaves here; a ragged one has its rows set to
    // zero on the way. Where it is left out no warp cuts that chunk's c, so nobody tells the thread that issues the MMAs
    // that c has landed: it waits for the copy itself before the product that reads it.
    const int n_own =
        n > 0 && !kStateOnly && !(sc.leave && g == have - 1) && rows_of(chunk_of(n - 1)) == kTile ? n - 1 : n;
    auto fail_now = [&]() {
        if (atomicExch(&bound.fail, 1) == 0) record_error(err, kDevTimeout);
    };

    if (warp == 0 || warp == 2) {
        // a and b, and in a warp of its own c: its place is free earlier, and waited for longer
        if (elect_one()) {
            const bool is_c = warp == 2;
            uint64_t* full = is_c ? v_full : qk_full;
            uint64_t* free_ = is_c ? v_free : qk_free;
            const int nst = is_c ? nv : nk;
            int s = 0, sent = 0, t0 = row0 + chunk_of(0) * kTile;
            const int dt = rev ? -kTile : kTile;
            uint32_t ph = 1;
            for (int j = 0; j < n; j++, t0 += dt) {
                uint8_t* st = smem + s * (is_c ? v_step : k_step);
                if (j >= nst && !wait_one(&free_[s], ph, fail)) {
                    fail_now();
                    break;
                }
                if (is_c) {
                    // kFull with two stages: a chunk's c is waited for longest (its place is free last and the cutting takes the
                    // time before its product), so that of two chunks on comes from L2 (4% of the headline prompt; three
                    // stages do without, and prefetching a and b too costs more than it gives)
                    if (kMode == kFull && np == 2 && j + 2 < n) tma_prefetch_l2_3d(&pr.map[sc.ic], c0, t0 + 2 * dt, z);
                    mbar_expect_tx(&v_full[s], kPanelBytes);
                    tma_load_3d(st + v_off, &pr.map[sc.ic], &v_full[s], c0, t0, z);
                } else {
                    mbar_expect_tx(&qk_full[s], kStateOnly ? k_bytes : 2 * k_bytes);
                    for (int p = 0; p < np; p++) {
                        if (!kStateOnly) tma_load_3d(st + p * kPanelBytes, &pr.map[sc.ia], &qk_full[s], 64 * p, t0, z);
                        tma_load_3d(st + k_off + p * kPanelBytes, &pr.map[sc.ib], &qk_full[s], 64 * p, t0, z);
                    }
                }
                sent++;
                if (++s == nst) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            // every copy has landed before the shared memory goes away
            for (int i = sent > nst ? sent - nst : 0; i < sent; i++) mbar_wait(&full[i % nst], (i / nst) & 1);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            constexpr uint32_t kIdS = idesc_bf16(kTile, kTile, 0, 0);    // A B^T, both K-major
            constexpr uint32_t kIdX = idesc_bf16(kTile, kDepth, 0, 1);   // A X and P C: B MN-major
            constexpr uint32_t kIdOwn = idesc_bf16(kTile, kDepth, 1, 1), kIdOwn3 = idesc_bf16(kTile, 3 * kDepth, 1, 1);
            // operands of the current stage and what a stage, a 16-column step of a K-major operand and a 16-row
            // step of an MN-major one (128) add to a descriptor's address field
            const uint64_t step = static_cast<uint64_t>(k_step >> 4);
            const uint64_t a_first = sdesc(smem_u32(smem), 16, 1024), kmaj = sdesc(0, kPanelBytes, 1024) - sdesc(0, 16, 1024);
            const uint64_t w0 = sdesc(smem_u32(wc), kPanelBytes, 1024), x0 = sdesc(smem_u32(xs), kPanelBytes, 1024);
            const uint64_t to_b = static_cast<uint64_t>(k_off >> 4), to_c = static_cast<uint64_t>(v_off >> 4);
            auto kstep = [](int kk) { return static_cast<uint64_t>(((kk >> 2) * kPanelBytes + (kk & 3) * 32) >> 4); };
            auto scores = [&](uint64_t a, uint64_t* full, uint32_t ph, uint32_t buf) {
                if (!wait_one(full, ph, fail)) return false;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; kk++)
                    if (kk < ksteps) mma_bf16(tmem + kColS + buf * kTile, further(a, kstep(kk)), further(a, to_b + kstep(kk)), kIdS, kk > 0);
                if (ksteps > 4) {
#pragma unroll
                    for (int kk = 4; kk < 8; kk++)
                        if (kk < ksteps) mma_bf16(tmem + kColS + buf * kTile, further(a, kstep(kk)), further(a, to_b + kstep(kk)), kIdS, 1);
                }
                mma_commit(&s_full[buf]);
                return true;
            };
            bool ok = true;
            int s = 0;
            uint32_t ph = 0;       // phase of stage s
            uint32_t par = 0;      // j & 1
            uint64_t a = a_first;  // stage s
            if (!kStateOnly && n > 0) ok = scores(a, &qk_full[0], 0, 0);
            for (int j = 0; j < n && ok; j++) {
                if (j < n_own) {
                    // the parts and their product: two places of each where only the states are formed
                    const uint32_t pl = kStateOnly ? par : 0u, use = kStateOnly ? (j >> 1) & 1 : par;
                    ok = wait_one(&scaled[pl], use, fail) && (!kStateOnly || wait_one(&qk_full[s], ph, fail)) &&
                         (j < (kStateOnly ? 2 : 1) || wait_one(&own_read[pl], use ^ 1u, fail));
                    if (!ok) break;
                    tc_fence_after();
                    // Only MMAs of one accumulator and one shape are ordered among themselves, so columns that two parts are
                    // added to see one shape. (High and middle part as one product of 128 columns, the low part onto the
                    // last 64 of them, took 2% off the headline prompt and rested on an order that nothing promises.)
                    const uint64_t bt = further(a, to_b + kmaj), wp = further(w0, static_cast<uint64_t>(kWcBytes >> 4) * pl);
                    const uint64_t part = kPanelBytes >> 4;
                    const uint32_t own = tmem + (kStateOnly ? kOwnStates * pl : kColOwn);
                    if (kStateOnly) {
#pragma unroll
                        for (int kk = 0; kk < kTile / 16; kk++)
                            mma_bf16(own, further(bt, 128u * kk), further(wp, 128u * kk), kIdOwn3, kk > 0);
                    } else {
#pragma unroll
                        for (int kk = 0; kk < kTile / 16; kk++)
                            mma_bf16(own, further(bt, 128u * kk), further(wp, 128u * kk), kIdOwn, kk > 0);
#pragma unroll
                        for (int kk = 0; kk < kTile / 16; kk++) {
                            mma_bf16(own + kDepth, further(bt, 128u * kk), further(wp, part + 128u * kk), kIdOwn, kk > 0);
                            mma_bf16(own + kDepth, further(bt, 128u * kk), further(wp, 2 * part + 128u * kk), kIdOwn, 1);
                        }
                    }
                    mma_commit(&own_full[pl]);
                }
                if (kStateOnly) {
                    mma_commit(&qk_free[s]);
                } else {
                    ok = wait_one(&x_ready, par, fail) && (j == 0 || wait_one(&o_read, par ^ 1u, fail));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 8; kk++)
                        if (kk < ksteps) mma_bf16(tmem + kColFar, further(a, kstep(kk)), further(x0, 128u * kk), kIdX, kk > 0);
                    mma_commit(&x_free);
                    mma_commit(&qk_free[s]);
                    // the next chunk's scores, so that its P is built while this one's is multiplied
                    const uint64_t ct = further(a, to_c + kmaj);
                    const bool wrap = s + 1 == nk;
                    if (j + 1 < n)
                        ok = scores(wrap ? a_first : further(a, step), &qk_full[wrap ? 0 : s + 1], wrap ? ph ^ 1u : ph, par ^ 1u);
                    ok = ok && wait_one(&p_ready[par], (j >> 1) & 1, fail) && (j < n_own || wait_one(&v_full[s], ph, fail));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; kk++) {
                        const uint32_t p = tmem + kColS + par * kTile + 16 * kk;
                        mma_bf16_ta(tmem + kColNear, p, further(ct, 128u * kk), kIdX, kk > 0);
                        mma_bf16_ta(tmem + kColNear, p + 8, further(ct, 128u * kk), kIdX, 1);
                    }
                    mma_commit(&v_free[s]);
                    mma_commit(&o_full);
                }
                a = further(a, step);
                if (++s == nk) {
                    s = 0;
                    ph ^= 1u;
                    a = a_first;
                }
                par ^= 1u;
            }
            if (!ok) fail_now();
            // every MMA issued above has completed before TMEM and shared memory go away
            mma_commit(&drain);
            if (!mbar_wait(&drain, 0)) fail_now();
        }
    } else if (warp == 3 && kMode == kStates) {
        // the states to memory, as they lie in shared memory (rows of 128 bytes, swizzled)
        if (elect_one()) {
            for (int j = 0; j < n; j++) {
                if (!wait_one(&x_put, j & 1, fail)) {
                    fail_now();
                    break;
                }
                const int64_t at = (static_cast<int64_t>(sc.states_base) + static_cast<int64_t>(bh) * nch + chunk_of(j)) *
                                       sc.tiles + tile;
                bulk_store(pr.states + at * (kTile * kDepth), xs, np * (kPanelBytes / 2));
                bulk_commit();
                bulk_wait_read0();
                mbar_arrive(&x_sent);
            }
            bulk_wait0();
        }
    } else if (warp >= 4 && warp < 12 && !kStateOnly) {
        const int w = warp & 3;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(w * 32) << 16);
        for (int j = 0; j < n; j++) {
            if (!wait_warp(&s_full[j & 1], (j >> 1) & 1, fail)) {
                if (lane == 0) fail_now();
                break;
            }
            tc_fence_after();
            const uint32_t cols = lanes + kColS + (j & 1) * kTile;
#pragma unroll 1
            for (int cb = (warp - 4) >> 2; cb < 4; cb += 2) {
                const float rw = cb < w ? pw[32 * w + lane - 32 * cb - 31] : 0.f;
                weigh_block<1>(cols + 32 * cb, cb == w ? 0 : cb < w ? 1 : -1, diag + 31 + lane, colw, rw);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready[j & 1]);
        }
    } else if (warp >= 12 && warp < 20) {
        const int d = (warp & 3) * 32 + lane;  // row of the state
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const int cw = (warp - 12) / 4 * 32, cg = c0 + cw;  // first of this warp's columns, in the tile and in c
        f32x2 x2[16];  // column pairs
        if (kMode != kPieces) {
            float x[32];
#pragma unroll
            for (int c = 0; c < 32; c++) x[c] = 0.f;
            if (sc.in && d < d1) {
                const float* in = sc.in + static_cast<int64_t>(sc.in_shared ? h : bh) * d1 * d2;
                const float f = gpow(la, before(p0));
#pragma unroll
                for (int c = 0; c < 32; c += 4)
                    if (cg + c < d2) {
                        const float4 y = *reinterpret_cast<const float4*>(in + static_cast<int64_t>(d) * d2 + cg + c);
                        x[c] = f * y.x;
                        x[c + 1] = f * y.y;
                        x[c + 2] = f * y.z;
                        x[c + 3] = f * y.w;
                    }
            }
            if (g > 0) {
                const float* sum = reinterpret_cast<const float*>(wc) + (d < prow ? d : 0);  // rows past d1 are not used
#pragma unroll
                for (int c = 0; c < 32; c++) x[c] += sum[(cw + c) * prow];
            }
#pragma unroll
            for (int c = 0; c < 16; c++) x2[c] = pair2(x[2 * c], x[2 * c + 1]);
        } else {
#pragma unroll
            for (int c = 0; c < 16; c++) x2[c] = 0ull;
        }
        auto stage_x = [&](uint8_t* to) {
            if (d < 64 * np) {
#pragma unroll
                for (int c = 0; c < 4; c++)
                    *reinterpret_cast<uint4*>(to + sw128_off(d, cw / 8 + c)) =
                        make_uint4(pack_bf16(x2[4 * c]), pack_bf16(x2[4 * c + 1]), pack_bf16(x2[4 * c + 2]),
                                   pack_bf16(x2[4 * c + 3]));
            }
            fence_async_smem();
            __syncwarp();
        };
        auto put_x = [&]() {
            stage_x(xs);
            if (lane == 0) mbar_arrive(&x_ready);
        };
        if (kMode == kFull && n > 0) put_x();
        if (kMode == kStates) {  // the sum of the pieces is read
            __syncwarp();
            if (lane == 0) mbar_arrive(&x_ready);
        }
        bool ok = true;
        if (kStateOnly && pr.waits.hold && !wait_warp(never, 0, fail)) {
            if (lane == 0) fail_now();
            ok = false;
        }
        for (int j = 0; j < n_own && ok; j++) {
            if (kMode == kStates) {
                // the entering state of this chunk, on its way to memory by warp 3
                if (j > 0 && !wait_warp(&x_sent, (j - 1) & 1, fail)) {
                    if (lane == 0) fail_now();
                    ok = false;
                    break;
                }
                stage_x(xs);
                if (lane == 0) mbar_arrive(&x_put);
            }
            const int pl = kStateOnly ? j & 1 : 0;
            if (!wait_warp(&own_full[pl], kStateOnly ? (j >> 1) & 1 : j & 1, fail)) {
                if (lane == 0) fail_now();
                ok = false;
                break;
            }
            tc_fence_after();
            const float gn = pw[rows_of(chunk_of(j))];
            f32x2 decay = pair2(gn, gn);
#pragma unroll 1
            for (int part = kStateOnly ? 2 : 1; part >= 0; part--) {  // the smaller first
                f32x2 y[8], u[8];
                const uint32_t from = lanes + (kStateOnly ? kOwnStates * pl : kColOwn) + part * kDepth + cw;
                tmem_ld16x2(from, from + 16, y, u);
#pragma unroll
                for (int c = 0; c < 8; c++) {
                    x2[c] = fma2(decay, x2[c], y[c]);
                    x2[c + 8] = fma2(decay, x2[c + 8], u[c]);
                }
                decay = pair2(1.f, 1.f);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&own_read[pl]);
            if (kMode == kFull && j + 1 < n) {
                if (!wait_warp(&x_free, j & 1, fail)) {
                    if (lane == 0) fail_now();
                    ok = false;
                    break;
                }
                put_x();
            }
        }
        if (ok) {
            if (kMode == kPieces) {
                float* sg = seg0 + static_cast<int64_t>(g) * seg_step + d;
                if (d < prow) {
#pragma unroll
                    for (int c = 0; c < 16; c++) {
                        const float2 y = split2(x2[c]);
                        sg[(cw + 2 * c) * prow] = y.x;
                        sg[(cw + 2 * c + 1) * prow] = y.y;
                    }
                }
            } else if (sc.leave && g == have - 1 && d < d1) {
                float* o = sc.leave + (static_cast<int64_t>(bh) * d1 + d) * d2 + cg;
#pragma unroll
                for (int c = 0; c < 32; c += 4)
                    if (cg + c < d2) *reinterpret_cast<ulonglong2*>(o + c) = make_ulonglong2(x2[c / 2], x2[c / 2 + 1]);
            }
        }
    } else if (warp >= 20 && warp < 24 && !kStateOnly) {
        const int quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(sc.out) +
                             (pr.packed ? static_cast<int64_t>(h) * pr.sq.total + row0
                                        : static_cast<int64_t>(bh) * pr.sq.T) * d2 + c0;
        const bool wide = d2 % 16 == 0 && (reinterpret_cast<uintptr_t>(sc.out) & 31) == 0;
        const bool held = pr.waits.hold && !wait_warp(never, 0, fail);
        if (held && lane == 0) fail_now();
        for (int j = 0; j < n && !held; j++) {
            if (!wait_warp(&o_full, j & 1, fail)) {
                if (lane == 0) fail_now();
                break;
            }
            tc_fence_after();
            const int ch = chunk_of(j), nr = rows_of(ch);
            const float f = row < nr ? pw[row + 1] : 0.f;
            const f32x2 f2 = pair2(f, f);
            __nv_bfloat16* orow = out + (static_cast<int64_t>(ch) * kTile + row) * d2;
#pragma unroll 1
            for (int c = 0; c < kDepth; c += 16) {
                f32x2 a[8], y[8];
                tmem_ld16x2(lanes + kColNear + c, lanes + kColFar + c, a, y);
                if (c == kDepth - 16) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&o_read);
                }
                uint32_t o[8];
#pragma unroll
                for (int i = 0; i < 8; i++) o[i] = pack_bf16(fma2(f2, y[i], a[i]));
                if (row < nr && c0 + c < d2) store32(orow + c, o, wide, c0 + c + 8 < d2);
            }
        }
    } else if (warp >= 24 || (kStateOnly && warp >= 4 && warp < 12)) {
        // thread: a half or a quarter of a row of c, 16-byte pieces c_first..
        constexpr int kCut = 32 / kCutWarps;
        const int row = (warp & 3) * 32 + lane, c_first = (warp >= 24 ? (warp - 24) >> 2 : (warp - 4) / 4 + 2) * kCut;
        bool ok = true;
        int s = 0, ks = 0;            // stages of c and of b
        uint32_t ph = 0, kph = 0;
        for (int j = 0; j < n_own; j++) {
            const int nr = rows_of(chunk_of(j));
            uint8_t* st = smem + v_off + s * v_step;
            ok = wait_warp(&v_full[s], ph, fail);
            // the products of the chunk (only states: two chunks) before are done with the parts' place
            const int pl = kStateOnly ? j & 1 : 0;
            if (ok && j >= (kStateOnly ? 2 : 1))
                ok = wait_warp(&own_full[pl], kStateOnly ? ((j >> 1) & 1) ^ 1 : (j - 1) & 1, fail);
            if (ok && nr < kTile) {
                // Rows behind the sequence's end count nothing, whatever they hold. Behind the wait above, as only then
                // the stage's rows before these have landed for sure and the barrier's phase tells these from them.
                ok = wait_warp(&qk_full[ks], kph, fail);
                if (ok && row >= nr) {
                    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
                    for (int c = c_first; c < c_first + kCut; c++) {
                        const uint32_t off = sw128_off(row, c);
                        *reinterpret_cast<uint4*>(st + off) = zero;
                        for (int p = 0; p < np; p++)
                            *reinterpret_cast<uint4*>(smem + k_off + ks * k_step + p * kPanelBytes + off) = zero;
                    }
                }
            }
            // and at first the state warps with the sum that lies there
            if (ok && j == 0 && kMode != kPieces) ok = wait_warp(&x_ready, 0, fail);
            if (!ok) break;
            const float wt = row < nr ? pw[rev ? row + 1 : nr - 1 - row] : 0.f;
            const f32x2 wt2 = pair2(wt, wt), minus = pair2(-1.f, -1.f);
            auto cut = [](f32x2 f) {
                const float2 y = split2(f);
                return __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x7632);
            };
            auto less = [&](f32x2 f, uint32_t p) {
                return fma2(pair2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u)), minus, f);
            };
            uint8_t* to = wc + pl * kWcBytes;
            // rolled: the unrolled loop's 300 instructions were fetched anew for every chunk and took three times as long
#pragma unroll 1
            for (int c = c_first; c < c_first + kCut; c++) {
                const uint32_t off = sw128_off(row, c);
                const uint4 xv = *reinterpret_cast<const uint4*>(st + off);
                const uint32_t in[4] = {xv.x, xv.y, xv.z, xv.w};
                uint32_t p1[4], p2[4], p3[4];
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    // three cuts of 8 bits: exact, 24 bits in all
                    f32x2 f = mul2(pair2(__uint_as_float(in[q] << 16), __uint_as_float(in[q] & 0xffff0000u)), wt2);
                    p1[q] = cut(f);
                    f = less(f, p1[q]);
                    p2[q] = cut(f);
                    f = less(f, p2[q]);
                    p3[q] = cut(f);
                }
                *reinterpret_cast<uint4*>(to + off) = make_uint4(p1[0], p1[1], p1[2], p1[3]);
                *reinterpret_cast<uint4*>(to + kPanelBytes + off) = make_uint4(p2[0], p2[1], p2[2], p2[3]);
                *reinterpret_cast<uint4*>(to + 2 * kPanelBytes + off) = make_uint4(p3[0], p3[1], p3[2], p3[3]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&scaled[pl]);
                if (kStateOnly) mbar_arrive(&v_free[s]);
            }
            if (++s == nv) {
                s = 0;
                ph ^= 1u;
            }
            if (++ks == nk) {
                ks = 0;
                kph ^= 1u;
            }
        }
        if (!ok && lane == 0) fail_now();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// What is asked of a device once: its SMs, and the kernels' shared memory (0: not asked yet).
constexpr int kMaxDevices = 64;
std::atomic<int> g_sms[kMaxDevices];

int sm_count() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return 0;
    }
    int sms = g_sms[dev].load(std::memory_order_acquire);
    if (sms) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaFuncSetAttribute(linear_scan_kernel<kFull>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost) !=
            cudaSuccess ||
        cudaFuncSetAttribute(linear_scan_kernel<kPieces>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost) !=
            cudaSuccess ||
        cudaFuncSetAttribute(linear_scan_kernel<kStates>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost) !=
            cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    g_sms[dev].store(sms, std::memory_order_release);
    return sms;
}

std::atomic<long long> g_wait_cycles[kMaxDevices];  // 0: the default
std::atomic<int> g_hold[kMaxDevices];

constexpr int64_t kMostPieces = 16384;  // 512 MB of workspace

int smem_bytes(int mode, int d1) {
    const int np = d1 > 64 ? 2 : 1;
    int panels;
    if (mode == kFull) panels = (np == 1 ? 3 : 2) * (2 * np + 1) + 3 + 1;
    else panels = (np == 1 ? 3 : 2) * np + 4 + 6;
    return panels * kPanelBytes + 1024;
}

}  // namespace

void linear_set_waits(LinWaits waits) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return;
    g_wait_cycles[dev].store(waits.cycles > 0 ? waits.cycles : 0);
    g_hold[dev].store(waits.hold);
}

LinWaits linear_waits() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return {kWaitCycles, 0};
    const long long cycles = g_wait_cycles[dev].load(std::memory_order_relaxed);
    return {cycles ? cycles : kWaitCycles, g_hold[dev].load(std::memory_order_relaxed)};
}

bool linear_tc_supported(int dtype, int dk, int dv) { return dtype == 0 && dk % 8 == 0 && dv % 8 == 0; }

bool linear_tc_plan(LinTcPlan* pl, int batch, int H, int T, int64_t rows, int tiles, bool states) {
    if (T > (1 << 30) || rows / H > (1 << 30)) return false;  // token offsets are ints
    pl->batch = batch;
    const int64_t items = static_cast<int64_t>(batch) * H * tiles;
    const int nch = (T - 1) / kTile + 1;
    if (states && static_cast<int64_t>(batch) * H * nch * 4 > 0x7fffffff) return false;  // state tiles are counted in ints
    const double sms = sm_count();
    if (sms <= 0) return false;
    const bool ragged = rows < static_cast<int64_t>(batch) * H * T;
    const double total = static_cast<double>(rows) / kTile * tiles;  // chunks of all items
    // Microseconds of `it` CTAs of L chunks at c a chunk and `fixed` a CTA, one CTA per SM at a time; ragged sequences
    // (longest first) end about one CTA after the even share.
    auto cost = [&](double it, int L, double share, double c, double fixed) {
        const double waves = std::ceil(it / sms) * (L * c + fixed);
        if (!ragged) return waves;
        const double even = total * share / sms * (c + fixed / L) + L * c + fixed;
        return even < waves ? even : waves;
    };
    // As measured at d = 128 and 64, for a choice between cuts: a chunk 2.1 us (1.4 where only the state is formed), a
    // CTA's start and end 5 (4), the second launch 3, a piece in a segment's sum 0.2. Against every cut of eleven shapes its
    // choice was within 5% of the fastest.
    const double chunk = states ? 1.4 : 2.1, fixed = states ? 4.0 : 5.0;
    double best = cost(static_cast<double>(items), nch, 1.0, chunk, fixed);
    pl->nseg = 1;
    pl->seg_chunks = pl->piece_chunks = nch;
    pl->npiece = 0;
    for (int s = 2, last = 0; s <= 64 && s <= nch; s++) {
        const int base = (nch + s - 1) / s;  // chunks of a segment; the same ones for several s
        if (base == last) continue;
        last = base;
        for (int r = 1; r <= 8 && r <= base; r++) {  // pieces of a segment
            const int P = (base + r - 1) / r, L = P * r;
            const int n = (nch + L - 1) / L, np = (n - 1) * r;
            if (n < 2 || items * np > kMostPieces) continue;
            const double share = static_cast<double>(np) * P / nch;
            const double c = cost(static_cast<double>(items) * n, L, 1.0, chunk, fixed) +
                             cost(static_cast<double>(items) * np, P, share, 1.4, 4.0) + 3.0 + 0.2 * np;
            if (c < best) {
                best = c;
                pl->nseg = n;
                pl->seg_chunks = L;
                pl->npiece = np;
                pl->piece_chunks = P;
            }
        }
    }
    pl->seg_bytes = static_cast<size_t>(items) * pl->npiece * kDepth * kTile * sizeof(float);
    return items * (pl->nseg > pl->npiece ? pl->nseg : pl->npiece) <= 0x7fffffff;
}

cudaError_t linear_tc_run(const LinTcPlan& pl, const LinTcMap* maps, int n_maps, const LinTcScan* scans, int count,
                          const LinSeqs& sq, const float* log_a, float* seg, void* states, int* err,
                          cudaStream_t stream) {
    ScanParams pr = {};
    const bool packed = sq.tab != nullptr;
    for (int i = 0; i < n_maps; i++)
        if (!make_map_3d(&pr.map[i], maps[i].base, packed ? sq.H : static_cast<uint64_t>(pl.batch) * sq.H,
                         packed ? sq.total : sq.T, maps[i].cols, kTile))
            return cudaErrorInvalidValue;
    pr.log_a = log_a;
    pr.seg = seg;
    pr.states = static_cast<__nv_bfloat16*>(states);
    pr.sq = sq;
    pr.count = count;
    pr.nseg = pl.nseg;
    pr.seg_chunks = pl.seg_chunks;
    pr.npiece = pl.npiece;
    pr.piece_chunks = pl.piece_chunks;
    pr.seg_pieces = pl.seg_chunks / pl.piece_chunks;
    pr.packed = packed;
    pr.waits = linear_waits();
    int base = 0, tiles = 0, d1 = 0;
    for (int i = 0; i < count; i++) {
        pr.scan[i] = scans[i];
        pr.scan[i].seg_base = base;
        base += pl.batch * sq.H * pl.npiece * scans[i].tiles;
        tiles += scans[i].tiles;
        if (scans[i].d1 > d1) d1 = scans[i].d1;
    }
    // beside the end of the kernel before it, where that is the table's or the pieces'
    auto launch = [&](auto kern, int ncta, int smem, bool beside) {
        const dim3 grid(tiles * ncta, pl.batch * sq.H);
        if (beside) return launch_pdl(kern, grid, dim3(kScanThreads), smem, stream, pr, err);
        kern<<<grid, kScanThreads, smem, stream>>>(pr, err);
        return cudaSuccess;
    };
    if (pl.nseg > 1) {
        const cudaError_t e = launch(linear_scan_kernel<kPieces>, pl.npiece, smem_bytes(kPieces, d1), packed);
        if (e != cudaSuccess) return e;
        note_launch(stream, "linear_scan_pieces");
    }
    const auto kern = states ? linear_scan_kernel<kStates> : linear_scan_kernel<kFull>;
    const int smem = smem_bytes(states ? kStates : kFull, d1);
    const cudaError_t e = launch(kern, pl.nseg, smem, packed || pl.nseg > 1);
    if (e != cudaSuccess) return e;
    note_launch(stream, states ? "linear_scan_states" : "linear_scan");
    return cudaGetLastError();
}

}  // namespace lla
