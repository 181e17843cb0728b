// Linear attention with one decay per head on tensor cores: bf16 rows, dk and dv multiples of 8.
//
// One kernel walks a scan (see lla_linear.cu: out_t = S_t^T a_t, S_t = g S_{t-1} + b_t c_t^T) over one (sequence, head, 64 columns of c) in chunks of 128 tokens. The state
// (d1 x 64, fp32) never leaves the registers of four warps. Per chunk, n valid rows:
//     scores  A B^T                      [128 x 128]  -> TMEM
//     own     B^T [hi | mid + lo]        [d1 x 128]   -> TMEM, w o C cut into three bf16 parts, so that the
//                                                     state keeps the 24 bits of fp32
//     far     A X                        [128 x 64]   X = entering state, rounded to bf16
//     near    P C                        [128 x 64]   P = scores o g^|i-j|, bf16, in TMEM
//     out_i = near_i + f_i far_i,   X <- g^n X + own
// with w_i = g^(n-1-i), f_i = g^(i+1) (states formed backwards: w_i = g^(i+1)). P and X are
// rounded to bf16 as the operands of a bf16 product must be (2^-8 of each term, as the output itself);
// scores, sums, weights and the state stay fp32.
//
// Heads alone do not fill the GPU when they are few, so a scan may be cut into segments, one CTA each: a first
// launch (kPieces) forms the own states of pieces of every segment but the last (smaller than segments, as
// it is launched without the last segment's share), and each segment's CTA sums those before it, decayed, in
// order. kFull does all of the above, forwards; kStates only forms the states, forwards or backwards, and
// writes the one that enters each chunk in bf16 for the kernel of the gradients (lla_linear_grad.cu).
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
constexpr int kMaxStages = 3;
constexpr int kWcBytes = 3 * kPanelBytes;
constexpr int kSmemMost = 232448 - 2048;  // 227 KB less the static part

// TMEM columns
// two buffers of scores (P takes the place of its scores: 32 keys in the first 16 of their 32 columns); own: the
// high part's product, then that of the middle and low parts
constexpr uint32_t kColS = 0, kColNear = 256, kColFar = 320, kColOwn = 384;

enum { kFull, kPieces, kStates };  // what a launch forms: see above

struct ScanParams {
    CUtensorMap map[4];
    LinTcScan scan[2];
    const float* log_a;
    float* seg;             // pieces' own states
    __nv_bfloat16* states;  // kStates: the entering states
    LinSeqs sq;
    int count, nseg, seg_chunks, npiece, piece_chunks, packed, batch;
};

// Warps: 0 and 2 TMA producers, 1 TMEM owner and MMA issuer, 4..11 P (every other block of 32 keys), 12..19 state
// (32 columns each), 20..23 write out, 24..31 split w o C. Warp w reaches TMEM lanes 32 (w % 4)..+31: rows of scores and out, rows of the state.
template <int kMode>
__global__ void __launch_bounds__(kScanThreads, 1) linear_scan_kernel(const __grid_constant__ ScanParams pr, int* err) {
    constexpr bool kStateOnly = kMode != kFull;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t qk_full[kMaxStages], v_full[kMaxStages], qk_free[kMaxStages], v_free[kMaxStages];
    __shared__ uint64_t scaled, own_full, own_read, x_ready, x_free, s_full[2], p_ready, o_full, o_read, drain;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int fail_sh;
    __shared__ float pw[132];    // g^n
    __shared__ __align__(16) float colw[32];  // weight of key c of an off-diagonal 32-key block
    __shared__ float diag[64];   // weight of key c for row r of a diagonal block, at 31 + r - c

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_dep_wait();    // the sequence table, the segments' states
    grid_dep_launch();
    // ---- which scan, 64 columns, segment, sequence and head
    int blk = blockIdx.x, si = 0;
    const int ncta = kMode == kPieces ? pr.npiece : pr.nseg;  // of one sequence, head and 64 columns
    while (si + 1 < pr.count && blk >= pr.batch * pr.sq.H * ncta * pr.scan[si].tiles)
        blk -= pr.batch * pr.sq.H * ncta * pr.scan[si++].tiles;
    const LinTcScan& sc = pr.scan[si];
    const int tile = blk % sc.tiles;
    blk /= sc.tiles;
    const int g = blk % ncta;
    blk /= ncta;
    const int h = blk % pr.sq.H;
    int b = blk / pr.sq.H, len = pr.sq.T, row0 = 0;
    if (pr.packed) {
        b = pr.sq.order[b];
        row0 = pr.sq.tab[b].x;
        len = pr.sq.tab[b].y;
        if (len < 0) return;
    }
    const int bh = b * pr.sq.H + h;
    const int z = pr.packed ? h : bh;  // outermost coordinate of the tensor maps
    const int nch = (len + kTile - 1) / kTile;
    const int have = nch <= pr.seg_chunks ? 1 : (nch + pr.seg_chunks - 1) / pr.seg_chunks;
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
    const int k_bytes = np * kPanelBytes;
    const int v_off = (kStateOnly ? 1 : 2) * k_bytes, stage_bytes = v_off + kPanelBytes;
    const int k_off = kStateOnly ? 0 : k_bytes;
    const int nst = (kStateOnly || np == 1) ? 3 : 2;
    uint8_t* wc = smem + nst * stage_bytes;
    uint8_t* xs = wc + kWcBytes;
    volatile int* fail = &fail_sh;

    if (tid == 0) {
        for (int s = 0; s < nst; s++) {
            mbar_init(&qk_full[s], 1);
            mbar_init(&v_full[s], 1);
            mbar_init(&qk_free[s], 1);
            mbar_init(&v_free[s], 1);
        }
        mbar_init(&scaled, 8);
        mbar_init(&own_full, 1);
        mbar_init(&own_read, 8);
        mbar_init(&x_ready, 8);
        mbar_init(&x_free, 1);
        mbar_init(&s_full[0], 1);
        mbar_init(&s_full[1], 1);
        mbar_init(&p_ready, 8);
        mbar_init(&o_full, 1);
        mbar_init(&o_read, 4);
        mbar_init(&drain, 1);
        fence_mbar_init();
        fail_sh = 0;
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
    // own states of the sequence's pieces, [64 columns][128 rows] each
    float* seg0 = pr.seg + (static_cast<int64_t>(sc.seg_base) +
                            static_cast<int64_t>(bh) * pr.npiece * sc.tiles + tile) * (kDepth * kTile);
    const int64_t seg_step = static_cast<int64_t>(sc.tiles) * (kDepth * kTile);
    if (kMode != kPieces && g > 0) {
        // the pieces before this segment, decayed to its start and summed in order
        float4 sum[2] = {};
        const int np_before = p0 / pr.piece_chunks;
#pragma unroll 2
        for (int gg = 0; gg < np_before; gg++) {
            const float f = gpow(la, before(p0) - before((gg + 1) * pr.piece_chunks));
            const float4* sg = reinterpret_cast<const float4*>(seg0 + gg * seg_step);
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const float4 y = sg[tid + i * kScanThreads];
                sum[i].x += f * y.x;
                sum[i].y += f * y.y;
                sum[i].z += f * y.z;
                sum[i].w += f * y.w;
            }
        }
        reinterpret_cast<float4*>(wc)[tid] = sum[0];
        reinterpret_cast<float4*>(wc)[tid + kScanThreads] = sum[1];
        __syncthreads();
    }
    auto fail_now = [&]() {
        if (atomicExch(&fail_sh, 1) == 0) record_error(err, kDevTimeout);
    };

    if (warp == 0 || warp == 2) {
        // a and b, and in a warp of its own c: its place is free earlier, and waited for longer
        if (elect_one()) {
            const bool is_c = warp == 2;
            uint64_t* full = is_c ? v_full : qk_full;
            uint64_t* free_ = is_c ? v_free : qk_free;
            int s = 0, sent = 0, t0 = row0 + chunk_of(0) * kTile;
            const int dt = rev ? -kTile : kTile;
            uint32_t ph = 1;
            uint8_t* st = smem;
            for (int j = 0; j < n; j++, t0 += dt) {
                if (j >= nst && !wait_one(&free_[s], ph, fail)) {
                    fail_now();
                    break;
                }
                if (is_c) {
                    mbar_expect_tx(&v_full[s], kPanelBytes);
                    tma_load_3d(st + v_off, &pr.map[sc.ic], &v_full[s], c0, t0, z);
                } else {
                    mbar_expect_tx(&qk_full[s], v_off);
                    for (int p = 0; p < np; p++) {
                        if (!kStateOnly) tma_load_3d(st + p * kPanelBytes, &pr.map[sc.ia], &qk_full[s], 64 * p, t0, z);
                        tma_load_3d(st + k_off + p * kPanelBytes, &pr.map[sc.ib], &qk_full[s], 64 * p, t0, z);
                    }
                }
                sent++;
                st += stage_bytes;
                if (++s == nst) {
                    s = 0;
                    st = smem;
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
            constexpr uint32_t kIdOwn2 = idesc_bf16(kTile, 2 * kDepth, 1, 1), kIdOwn1 = idesc_bf16(kTile, kDepth, 1, 1);
            // operands of the current stage and what a stage, a 16-column step of a K-major operand and a 16-row
            // step of an MN-major one (128) add to a descriptor's address field
            const uint64_t step = static_cast<uint64_t>(stage_bytes >> 4);
            const uint64_t a_first = sdesc(smem_u32(smem), 16, 1024), kmaj = sdesc(0, kPanelBytes, 1024) - sdesc(0, 16, 1024);
            const uint64_t w0 = sdesc(smem_u32(wc), kPanelBytes, 1024), x0 = sdesc(smem_u32(xs), kPanelBytes, 1024);
            const uint64_t to_b = static_cast<uint64_t>(k_off >> 4), to_c = static_cast<uint64_t>(v_off >> 4);
            auto kstep = [](int kk) { return static_cast<uint64_t>(((kk >> 2) * kPanelBytes + (kk & 3) * 32) >> 4); };
            auto scores = [&](uint64_t a, uint64_t* full, uint32_t ph, uint32_t buf) {
                if (!wait_one(full, ph, fail)) return false;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; kk++)
                    if (kk < ksteps) mma_bf16(tmem + kColS + buf * kTile, a + kstep(kk), a + to_b + kstep(kk), kIdS, kk > 0);
                if (ksteps > 4) {
#pragma unroll
                    for (int kk = 4; kk < 8; kk++)
                        if (kk < ksteps) mma_bf16(tmem + kColS + buf * kTile, a + kstep(kk), a + to_b + kstep(kk), kIdS, 1);
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
                ok = wait_one(&scaled, par, fail) && (!kStateOnly || wait_one(&qk_full[s], ph, fail)) &&
                     (j == 0 || wait_one(&own_read, par ^ 1u, fail));
                if (!ok) break;
                tc_fence_after();
                const uint64_t bt = a + to_b + kmaj;
#pragma unroll
                for (int kk = 0; kk < kTile / 16; kk++) mma_bf16(tmem + kColOwn, bt + 128u * kk, w0 + 128u * kk, kIdOwn2, kk > 0);
#pragma unroll
                for (int kk = 0; kk < kTile / 16; kk++)
                    mma_bf16(tmem + kColOwn + kDepth, bt + 128u * kk, w0 + 2 * (kPanelBytes >> 4) + 128u * kk, kIdOwn1, 1);
                mma_commit(&own_full);
                if (kStateOnly) {
                    mma_commit(&qk_free[s]);
                    mma_commit(&v_free[s]);  // the scale warps are done with c too
                } else {
                    ok = wait_one(&x_ready, par, fail) && (j == 0 || wait_one(&o_read, par ^ 1u, fail));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 8; kk++)
                        if (kk < ksteps) mma_bf16(tmem + kColFar, a + kstep(kk), x0 + 128u * kk, kIdX, kk > 0);
                    mma_commit(&x_free);
                    mma_commit(&qk_free[s]);
                    // the next chunk's scores, so that its P is built while this one's is multiplied
                    const uint64_t ct = a + to_c + kmaj;
                    const bool wrap = s + 1 == nst;
                    if (j + 1 < n)
                        ok = scores(wrap ? a_first : a + step, &qk_full[wrap ? 0 : s + 1], wrap ? ph ^ 1u : ph, par ^ 1u);
                    ok = ok && wait_one(&p_ready, par, fail);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; kk++)
                        mma_bf16_ta(tmem + kColNear, tmem + kColS + par * kTile + kk / 2 * 32 + kk % 2 * 8, ct + 128u * kk,
                                    kIdX, kk > 0);
                    mma_commit(&v_free[s]);
                    mma_commit(&o_full);
                }
                a += step;
                if (++s == nst) {
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
                uint32_t r[16];
                if (cb > w) {  // wholly ahead in time
#pragma unroll
                    for (int i = 0; i < 16; i++) r[i] = 0u;
                } else {
                    if (cb == w) {
                        float x[32];
                        tmem_ld32(cols + 32 * cb, x);
                        const float* dg = diag + 31 + lane;
#pragma unroll
                        for (int i = 0; i < 32; i++) {
                            const float f = dg[-i];
                            x[i] = f != 0.f ? x[i] * f : 0.f;  // masked: never the product with an infinity
                        }
#pragma unroll
                        for (int i = 0; i < 16; i++) r[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
                    } else {
                        const float rw = pw[32 * w + lane - 32 * cb - 31];
                        const f32x2 rw2 = pair2(rw, rw);
                        const ulonglong2* cw = reinterpret_cast<const ulonglong2*>(colw);
#pragma unroll
                        for (int hh = 0; hh < 2; hh++) {
                            uint32_t y[16];
                            tmem_ld16_issue(cols + 32 * cb + 16 * hh, y);
                            tmem_ld16_wait(y);
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                const ulonglong2 f = cw[4 * hh + i];
                                auto at = [&](int e) { return pair2(__uint_as_float(y[e]), __uint_as_float(y[e + 1])); };
                                r[8 * hh + 2 * i] = pack_bf16(mul2(mul2(at(4 * i), f.x), rw2));
                                r[8 * hh + 2 * i + 1] = pack_bf16(mul2(mul2(at(4 * i + 2), f.y), rw2));
                            }
                        }
                    }
                }
                tmem_st16_issue(cols + 32 * cb, r);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready);
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
                const float* sum = reinterpret_cast<const float*>(wc) + d;
#pragma unroll
                for (int c = 0; c < 32; c++) x[c] += sum[(cw + c) * kTile];
            }
#pragma unroll
            for (int c = 0; c < 16; c++) x2[c] = pair2(x[2 * c], x[2 * c + 1]);
        } else {
#pragma unroll
            for (int c = 0; c < 16; c++) x2[c] = 0ull;
        }
        auto put_x = [&]() {
            if (d < 64 * np) {
#pragma unroll
                for (int c = 0; c < 4; c++)
                    *reinterpret_cast<uint4*>(xs + sw128_off(d, cw / 8 + c)) =
                        make_uint4(pack_bf16(x2[4 * c]), pack_bf16(x2[4 * c + 1]), pack_bf16(x2[4 * c + 2]),
                                   pack_bf16(x2[4 * c + 3]));
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&x_ready);
        };
        if (kMode == kFull && n > 0) put_x();
        if (kMode == kStates) {  // the sum of the pieces is read
            __syncwarp();
            if (lane == 0) mbar_arrive(&x_ready);
        }
        bool ok = true;
        for (int j = 0; j < n; j++) {
            if (kMode == kStates && d < 64 * np) {
                // the entering state of this chunk, [128 rows][64 columns]
                __nv_bfloat16* to =
                    pr.states + ((static_cast<int64_t>(sc.states_base) + static_cast<int64_t>(bh) * nch + chunk_of(j)) *
                                     sc.tiles + tile) * (kTile * kDepth) + d * kDepth + cw;
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    uint32_t o[8];
#pragma unroll
                    for (int i = 0; i < 8; i++) o[i] = pack_bf16(x2[8 * c + i]);
                    store32(to + 16 * c, o, true, true);
                }
            }
            if (!wait_warp(&own_full, j & 1, fail)) {
                if (lane == 0) fail_now();
                ok = false;
                break;
            }
            tc_fence_after();
            const float gn = pw[rows_of(chunk_of(j))];
            f32x2 decay = pair2(gn, gn);
#pragma unroll 1
            for (int part = 1; part >= 0; part--) {  // the smaller first
                f32x2 y[8], u[8];
                tmem_ld16x2(lanes + kColOwn + part * kDepth + cw, lanes + kColOwn + part * kDepth + cw + 16, y, u);
#pragma unroll
                for (int c = 0; c < 8; c++) {
                    x2[c] = fma2(decay, x2[c], y[c]);
                    x2[c + 8] = fma2(decay, x2[c + 8], u[c]);
                }
                decay = pair2(1.f, 1.f);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&own_read);
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
#pragma unroll
                for (int c = 0; c < 16; c++) {
                    const float2 y = split2(x2[c]);
                    sg[(cw + 2 * c) * kTile] = y.x;
                    sg[(cw + 2 * c + 1) * kTile] = y.y;
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
        for (int j = 0; j < n; j++) {
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
    } else if (warp >= 24) {
        // thread: half a row of c, split before the products of the chunk before are done with the parts' place
        const int row = (warp & 3) * 32 + lane, h4 = (warp - 24) >> 2 << 2;
        bool ok = true;
        int s = 0;
        uint32_t ph = 0;
        uint8_t* st = smem;
        for (int j = 0; j < n; j++) {
            const int nr = rows_of(chunk_of(j));
            ok = wait_warp(&v_full[s], ph, fail);
            if (ok && nr < kTile) {
                // rows behind the sequence's end count nothing, whatever they hold
                ok = wait_warp(&qk_full[s], ph, fail);
                if (ok && row >= nr) {
                    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
                    for (int c = h4; c < h4 + 4; c++) {
                        const uint32_t off = sw128_off(row, c);
                        *reinterpret_cast<uint4*>(st + v_off + off) = zero;
                        for (int p = 0; p < np; p++) *reinterpret_cast<uint4*>(st + k_off + p * kPanelBytes + off) = zero;
                    }
                }
            }
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
            uint32_t p1[16], p2[16], p3[16];
#pragma unroll
            for (int c = 0; c < 4; c++) {
                const uint4 xv = *reinterpret_cast<const uint4*>(st + v_off + sw128_off(row, h4 + c));
                const uint32_t in[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    // three cuts of 8 bits: exact, 24 bits in all
                    const int e = 4 * c + q;
                    f32x2 f = mul2(pair2(__uint_as_float(in[q] << 16), __uint_as_float(in[q] & 0xffff0000u)), wt2);
                    p1[e] = cut(f);
                    f = less(f, p1[e]);
                    p2[e] = cut(f);
                    f = less(f, p2[e]);
                    p3[e] = cut(f);
                }
            }
            // the products of the chunk before, and at first the state warps' reading of the sum, are done with this place
            if (j > 0) ok = wait_warp(&own_full, (j - 1) & 1, fail);
            else if (kMode != kPieces) ok = wait_warp(&x_ready, 0, fail);
            if (!ok) break;
#pragma unroll
            for (int c = 0; c < 4; c++) {
                const uint32_t off = sw128_off(row, h4 + c);
                *reinterpret_cast<uint4*>(wc + off) = make_uint4(p1[4 * c], p1[4 * c + 1], p1[4 * c + 2], p1[4 * c + 3]);
                *reinterpret_cast<uint4*>(wc + kPanelBytes + off) =
                    make_uint4(p2[4 * c], p2[4 * c + 1], p2[4 * c + 2], p2[4 * c + 3]);
                *reinterpret_cast<uint4*>(wc + 2 * kPanelBytes + off) =
                    make_uint4(p3[4 * c], p3[4 * c + 1], p3[4 * c + 2], p3[4 * c + 3]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&scaled);
            st += stage_bytes;
            if (++s == nst) {
                s = 0;
                st = smem;
                ph ^= 1u;
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

int smem_bytes(bool state_only, int d1) {
    const int np = d1 > 64 ? 2 : 1;
    const int stage = ((state_only ? 1 : 2) * np + 1) * kPanelBytes;
    const int nst = (state_only || np == 1) ? 3 : 2;
    return nst * stage + kWcBytes + (state_only ? 0 : kPanelBytes) + 1024;
}

}  // namespace

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
    // Measured at d = 128 and 64: a chunk 2.1 us (1.2 where only the state is formed), a CTA's start and end 5 (4), the
    // second launch 3, a piece in a segment's sum 0.1.
    double best = 0;
    pl->nseg = 1;
    pl->seg_chunks = pl->piece_chunks = nch;
    pl->npiece = 0;
    for (int s = 1; s <= 64 && s <= nch; s++) {
        const int L = (nch + s - 1) / s;
        if ((nch + L - 1) / L != s) continue;  // the same cut as fewer segments
        const double main = cost(static_cast<double>(items) * s, L, 1.0, states ? 1.2 : 2.1, states ? 4.0 : 5.0);
        for (int r = 1; r <= 8; r *= 2) {  // pieces of a segment
            if (L % r != 0) break;
            const int P = (s - 1) * r;
            const double c = s == 1 ? main
                                    : main + cost(static_cast<double>(items) * P, L / r, (s - 1.0) / s, 1.2, 4.0) + 3.0 +
                                          0.1 * P;
            if (best == 0 || c < best) {
                best = c;
                pl->nseg = s;
                pl->seg_chunks = L;
                pl->npiece = P;
                pl->piece_chunks = L / r;
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
    pr.packed = packed;
    pr.batch = pl.batch;
    int base = 0, tiles = 0, d1 = 0;
    for (int i = 0; i < count; i++) {
        pr.scan[i] = scans[i];
        pr.scan[i].seg_base = base;
        base += pl.batch * sq.H * pl.npiece * scans[i].tiles;
        tiles += scans[i].tiles;
        if (scans[i].d1 > d1) d1 = scans[i].d1;
    }
    const unsigned per_seg = static_cast<unsigned>(pl.batch) * sq.H * tiles;
    if (pl.nseg > 1) {
        linear_scan_kernel<kPieces><<<per_seg * pl.npiece, kScanThreads, smem_bytes(true, d1), stream>>>(pr, err);
        note_launch(stream, "linear_scan_pieces");
    }
    const auto kern = states ? linear_scan_kernel<kStates> : linear_scan_kernel<kFull>;
    const int smem = smem_bytes(states != nullptr, d1);
    if (pl.nseg > 1) {
        const cudaError_t e = launch_pdl(kern, dim3(per_seg * pl.nseg), dim3(kScanThreads), smem, stream, pr, err);
        if (e != cudaSuccess) return e;
    } else {
        kern<<<per_seg, kScanThreads, smem, stream>>>(pr, err);
    }
    note_launch(stream, states ? "linear_scan_states" : "linear_scan");
    return cudaGetLastError();
}

}  // namespace lla
