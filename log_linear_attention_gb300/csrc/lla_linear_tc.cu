// Linear attention with one decay per head on tensor cores: bf16 rows, dk and dv multiples of 8.
//
// One kernel walks a scan (see lla_linear.cu: out_t = S_t^T a_t, S_t = g S_{t-1} + b_t c_t^T, forwards
// or backwards in time) over one (sequence, head, 64 columns of c) in chunks of 128 tokens. The state
// (d1 x 64, fp32) never leaves the registers of four warps. Per chunk, n valid rows:
//     scores  A B^T                      [128 x 128]  -> TMEM
//     own     B^T [hi | mid | lo]        [d1 x 192]   -> TMEM, w o C split into three bf16 parts, so that
//                                                     the state keeps the 24 bits of fp32
//     far     A X                        [128 x 64]   X = entering state, rounded to bf16
//     near    P C                        [128 x 64]   P = scores o g^|i-j|, bf16, read from TMEM
//     out_i = near_i + f_i far_i,   X <- g^n X + own
// with w_i = g^(n-1-i), f_i = g^(i+1) forwards and w_i = g^(i+1), f_i = g^(n-1-i) backwards. P and X are
// rounded to bf16 as the operands of a bf16 product must be (2^-8 of each term, as the output itself);
// scores, sums, weights and the state stay fp32.
//
// Heads alone do not fill the GPU when they are few, so a scan may be cut into segments: a first launch
// (kStateOnly) forms the own state of every segment but the last, and each segment's CTA joins those
// before it, decayed, in order.
//
// Rows of a chunk behind its sequence's end (another sequence's, when packed) are set to zero in shared
// memory before any product sums over them. Every wait is bounded; on overrun the kernel records
// LLA_ERR_TIMEOUT in the device error word, lets its own copies and MMAs land and returns.
#include <cmath>

#include "lla_linear.cuh"
#include "lla_tc_ptx.cuh"

namespace lla {
namespace {

constexpr int kScanThreads = 512;
constexpr int kMaxStages = 3;
constexpr int kDepth = 64;  // columns of c per CTA
constexpr int kWcBytes = 3 * kPanelBytes;
constexpr int kSmemMost = 232448 - 2048;  // 227 KB less the static part

// TMEM columns
constexpr uint32_t kColS = 0, kColP = 128, kColNear = 192, kColFar = 256, kColOwn = 320;

struct alignas(64) ScanParams {
    CUtensorMap map[4];
    LinTcScan scan[3];
    const float* log_a;
    float* seg;  // segments' own states
    LinSeqs sq;
    int count, nseg, seg_chunks, packed, batch;
};

__device__ __forceinline__ float gpow(float la, int n) { return n == 0 ? 1.f : expf(la * static_cast<float>(n)); }

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]: A's row i is lane i, two bf16 K elements per 32-bit column.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st16_issue(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Warps: 0 TMA producer, 1 TMEM owner and MMA issuer, 4..7 P, 8..11 state, 12..15 scale c and write out.
// Warp w reaches TMEM lanes 32 (w % 4)..+31: rows of scores and out, rows of the state.
template <bool kStateOnly>
__global__ void __launch_bounds__(kScanThreads, 1) linear_scan_kernel(const __grid_constant__ ScanParams pr, int* err) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t qk_full[kMaxStages], v_full[kMaxStages], qk_free[kMaxStages], v_free[kMaxStages];
    __shared__ uint64_t scaled, own_full, own_read, x_ready, x_free, s_full, p_ready, o_full, o_read, drain;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int fail_sh;
    __shared__ float pw[132];    // g^n
    __shared__ float colw[32];   // weight of key c of an off-diagonal 32-key block
    __shared__ float diag[64];   // weight of key c for row r of a diagonal block, at 31 + r - c

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_dep_wait();    // the sequence table, the segments' states
    grid_dep_launch();
    // ---- which scan, 64 columns, segment, sequence and head
    int blk = blockIdx.x, si = 0;
    const int nseg = kStateOnly ? pr.nseg - 1 : pr.nseg;
    while (si + 1 < pr.count && blk >= pr.batch * pr.sq.H * nseg * pr.scan[si].tiles)
        blk -= pr.batch * pr.sq.H * nseg * pr.scan[si++].tiles;
    const LinTcScan& sc = pr.scan[si];
    const int tile = blk % sc.tiles;
    blk /= sc.tiles;
    const int g = blk % nseg;
    blk /= nseg;
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
    if (g >= (kStateOnly ? have - 1 : have)) return;
    const int p0 = g * pr.seg_chunks;
    const int n = nch - p0 < pr.seg_chunks ? nch - p0 : pr.seg_chunks;  // chunks of this CTA
    const bool rev = sc.reverse != 0;
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
        mbar_init(&scaled, 4);
        mbar_init(&own_full, 1);
        mbar_init(&own_read, 4);
        mbar_init(&x_ready, 4);
        mbar_init(&x_free, 1);
        mbar_init(&s_full, 1);
        mbar_init(&p_ready, 4);
        mbar_init(&o_full, 1);
        mbar_init(&o_read, 4);
        mbar_init(&drain, 1);
        fence_mbar_init();
        fail_sh = 0;
    }
    if (warp == 1) tmem_alloc(&tmem_base_sh, 512);
    const float la = pr.log_a[h];
    if (tid >= 64 && tid < 64 + 129) pw[tid - 64] = gpow(la, tid - 64);
    if (tid >= 256 && tid < 288) colw[tid - 256] = gpow(la, rev ? tid - 256 : 31 - (tid - 256));
    if (tid >= 320 && tid < 383) {
        const int u = tid - 320 - 31;  // r - c
        diag[tid - 320] = rev ? (u <= 0 ? gpow(la, -u) : 0.f) : (u >= 0 ? gpow(la, u) : 0.f);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    auto fail_now = [&]() {
        if (atomicExch(&fail_sh, 1) == 0) record_error(err, kDevTimeout);
    };
    int sent_qk = 0, sent_v = 0;  // producer: copies issued

    if (warp == 0) {
        if (lane == 0) {
            for (int j = 0; j < n && !*fail; j++) {
                const int s = j % nst, t0 = row0 + chunk_of(j) * kTile;
                uint8_t* st = smem + s * stage_bytes;
                if (j >= nst && !mbar_wait(&qk_free[s], (j / nst - 1) & 1)) {
                    fail_now();
                    break;
                }
                mbar_expect_tx(&qk_full[s], v_off);
                for (int p = 0; p < np; p++) {
                    if (!kStateOnly) tma_load_3d(st + p * kPanelBytes, &pr.map[sc.ia], &qk_full[s], 64 * p, t0, z);
                    tma_load_3d(st + k_off + p * kPanelBytes, &pr.map[sc.ib], &qk_full[s], 64 * p, t0, z);
                }
                sent_qk++;
                if (j >= nst && !mbar_wait(&v_free[s], (j / nst - 1) & 1)) {
                    fail_now();
                    break;
                }
                mbar_expect_tx(&v_full[s], kPanelBytes);
                tma_load_3d(st + v_off, &pr.map[sc.ic], &v_full[s], c0, t0, z);
                sent_v++;
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t kIdS = idesc_bf16(kTile, kTile, 0, 0);    // A B^T, both K-major
            constexpr uint32_t kIdX = idesc_bf16(kTile, kDepth, 0, 1);   // A X and P C: B MN-major
            constexpr uint32_t kIdOwn = idesc_bf16(kTile, 3 * kDepth, 1, 1);
            const uint32_t base = smem_u32(smem), wcb = smem_u32(wc), xb = smem_u32(xs);
            auto scores = [&](int j) {
                const int s = j % nst;
                if (!mbar_wait(&qk_full[s], (j / nst) & 1)) return false;
                tc_fence_after();
                const uint32_t qb = base + s * stage_bytes, kb = qb + k_off;
                for (int kk = 0; kk < ksteps; kk++) {
                    const uint32_t off = (kk >> 2) * kPanelBytes + (kk & 3) * 32;
                    mma_bf16(tmem + kColS, sdesc(qb + off, 16, 1024), sdesc(kb + off, 16, 1024), kIdS, kk > 0);
                }
                mma_commit(&s_full);
                return true;
            };
            bool ok = true;
            if (!kStateOnly && n > 0) ok = scores(0);
            for (int j = 0; j < n && ok && !*fail; j++) {
                const int s = j % nst;
                const uint32_t sb = base + s * stage_bytes;
                ok = mbar_wait(&scaled, j & 1) && (!kStateOnly || mbar_wait(&qk_full[s], (j / nst) & 1)) &&
                     (j == 0 || mbar_wait(&own_read, (j - 1) & 1));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < kTile / 16; kk++)
                    mma_bf16(tmem + kColOwn, sdesc(sb + k_off + kk * 2048, kPanelBytes, 1024),
                             sdesc(wcb + kk * 2048, kPanelBytes, 1024), kIdOwn, kk > 0);
                mma_commit(&own_full);
                if (kStateOnly) {
                    mma_commit(&qk_free[s]);
                    mma_commit(&v_free[s]);  // the scale warps are done with c too
                    continue;
                }
                ok = mbar_wait(&x_ready, j & 1) && (j == 0 || mbar_wait(&o_read, (j - 1) & 1));
                if (!ok) break;
                tc_fence_after();
                for (int kk = 0; kk < ksteps; kk++) {
                    const uint32_t off = (kk >> 2) * kPanelBytes + (kk & 3) * 32;
                    mma_bf16(tmem + kColFar, sdesc(sb + off, 16, 1024), sdesc(xb + kk * 2048, kPanelBytes, 1024), kIdX,
                             kk > 0);
                }
                mma_commit(&x_free);
                mma_commit(&qk_free[s]);
                // P is built: the scores' columns are free for the next chunk
                ok = mbar_wait(&p_ready, j & 1);
                if (!ok) break;
                tc_fence_after();
                if (j + 1 < n) ok = scores(j + 1);
                if (!ok) break;
#pragma unroll
                for (int kk = 0; kk < kTile / 16; kk++)
                    mma_bf16_ta(tmem + kColNear, tmem + kColP + kk * 8, sdesc(sb + v_off + kk * 2048, kPanelBytes, 1024),
                                kIdX, kk > 0);
                mma_commit(&o_full);
                mma_commit(&v_free[s]);
            }
            if (!ok) fail_now();
            // every MMA issued above has completed before TMEM and shared memory go away
            mma_commit(&drain);
            if (!mbar_wait(&drain, 0)) fail_now();
        }
    } else if (warp >= 4 && warp < 8 && !kStateOnly) {
        const int w = warp & 3;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(w * 32) << 16);
        for (int j = 0; j < n; j++) {
            if (__any_sync(0xffffffffu, *fail != 0)) break;
            if (!warp_wait(&s_full, j & 1)) {
                if (lane == 0) fail_now();
                break;
            }
            tc_fence_after();
            bool ok = true;
#pragma unroll 1
            for (int cb = 0; cb < 4; cb++) {
                uint32_t r[16];
                if (rev ? cb < w : cb > w) {  // wholly on the other side of time
#pragma unroll
                    for (int i = 0; i < 16; i++) r[i] = 0u;
                } else {
                    float x[32];
                    tmem_ld32(lanes + kColS + 32 * cb, x);
                    if (cb == w) {
                        const float* dg = diag + 31 + lane;
#pragma unroll
                        for (int i = 0; i < 32; i++) {
                            const float f = dg[-i];
                            x[i] = f != 0.f ? x[i] * f : 0.f;  // masked: never the product with an infinity
                        }
                    } else {
                        const float rw = pw[rev ? 32 * cb - (32 * w + lane) : 32 * w + lane - 32 * cb - 31];
                        const float4* cw = reinterpret_cast<const float4*>(colw);
#pragma unroll
                        for (int i = 0; i < 8; i++) {
                            const float4 f = cw[i];
                            x[4 * i] *= f.x * rw;
                            x[4 * i + 1] *= f.y * rw;
                            x[4 * i + 2] *= f.z * rw;
                            x[4 * i + 3] *= f.w * rw;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 16; i++) r[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
                }
                // P C of the chunk before has read P
                if (cb == 0 && j > 0 && !warp_wait(&o_full, (j - 1) & 1)) {
                    ok = false;
                    break;
                }
                if (cb == 0) tc_fence_after();
                tmem_st16_issue(lanes + kColP + 16 * cb, r);
            }
            if (!ok) {
                if (lane == 0) fail_now();
                break;
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready);
        }
    } else if (warp >= 8 && warp < 12) {
        const int d = (warp & 3) * 32 + lane;  // row of the state
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const int64_t slot = (static_cast<int64_t>(sc.seg_base) + (static_cast<int64_t>(bh) * (pr.nseg - 1)) * sc.tiles) *
                             (kDepth * kTile);
        auto seg_at = [&](int gg) {
            return pr.seg + slot + (static_cast<int64_t>(gg) * sc.tiles + tile) * (kDepth * kTile) + d;
        };
        float x[kDepth];
#pragma unroll
        for (int c = 0; c < kDepth; c++) x[c] = 0.f;
        if (!kStateOnly) {
            if (sc.in && d < d1) {
                const float* in = sc.in + static_cast<int64_t>(sc.in_shared ? h : bh) * d1 * d2;
                const float f = gpow(la, before(p0));
                // rows of 4-column groups, or columns of the transpose
                if (sc.in_t) {
#pragma unroll
                    for (int c = 0; c < kDepth; c++)
                        if (c0 + c < d2) x[c] = f * in[static_cast<int64_t>(c0 + c) * d1 + d];
                } else {
#pragma unroll
                    for (int c = 0; c < kDepth; c += 4)
                        if (c0 + c < d2) {
                            const float4 y = *reinterpret_cast<const float4*>(in + static_cast<int64_t>(d) * d2 + c0 + c);
                            x[c] = f * y.x;
                            x[c + 1] = f * y.y;
                            x[c + 2] = f * y.z;
                            x[c + 3] = f * y.w;
                        }
                }
            }
            for (int gg = 0; gg < g; gg++) {
                const float f = gpow(la, before(p0) - before((gg + 1) * pr.seg_chunks));
                const float* sg = seg_at(gg);
#pragma unroll
                for (int c = 0; c < kDepth; c++) x[c] += f * sg[c * kTile];
            }
        }
        auto put_x = [&]() {
            if (d < 64 * np) {
#pragma unroll
                for (int c = 0; c < 8; c++)
                    *reinterpret_cast<uint4*>(xs + sw128_off(d, c)) =
                        make_uint4(pack_bf16(x[8 * c], x[8 * c + 1]), pack_bf16(x[8 * c + 2], x[8 * c + 3]),
                                   pack_bf16(x[8 * c + 4], x[8 * c + 5]), pack_bf16(x[8 * c + 6], x[8 * c + 7]));
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&x_ready);
        };
        if (!kStateOnly && n > 0) put_x();
        bool ok = true;
        for (int j = 0; j < n; j++) {
            if (__any_sync(0xffffffffu, *fail != 0)) {
                ok = false;
                break;
            }
            if (!warp_wait(&own_full, j & 1)) {
                if (lane == 0) fail_now();
                ok = false;
                break;
            }
            tc_fence_after();
            const float gn = pw[rows_of(chunk_of(j))];
#pragma unroll
            for (int c = 0; c < kDepth; c += 16) {
                uint32_t r[16];
                tmem_ld16_issue(lanes + kColOwn + c, r);
                tmem_ld16_wait(r);
#pragma unroll
                for (int i = 0; i < 16; i++) x[c + i] = gn * x[c + i] + __uint_as_float(r[i]);
                tmem_ld16_issue(lanes + kColOwn + kDepth + c, r);
                tmem_ld16_wait(r);
#pragma unroll
                for (int i = 0; i < 16; i++) x[c + i] += __uint_as_float(r[i]);
                tmem_ld16_issue(lanes + kColOwn + 2 * kDepth + c, r);
                tmem_ld16_wait(r);
#pragma unroll
                for (int i = 0; i < 16; i++) x[c + i] += __uint_as_float(r[i]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&own_read);
            if (!kStateOnly && j + 1 < n) {
                if (!warp_wait(&x_free, j & 1)) {
                    if (lane == 0) fail_now();
                    ok = false;
                    break;
                }
                put_x();
            }
        }
        if (ok) {
            if (kStateOnly) {
                float* sg = seg_at(g);
#pragma unroll
                for (int c = 0; c < kDepth; c++) sg[c * kTile] = x[c];
            } else if (sc.leave && g == have - 1 && d < d1) {
                float* o = sc.leave + (static_cast<int64_t>(bh) * d1 + d) * d2 + c0;
#pragma unroll
                for (int c = 0; c < kDepth; c += 4)
                    if (c0 + c < d2) *reinterpret_cast<float4*>(o + c) = make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]);
            }
        }
    } else if (warp >= 12) {
        const int quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        // out rows of chunk j
        auto write_out = [&](int j) {
            if (!warp_wait(&o_full, j & 1)) return false;
            tc_fence_after();
            const int ch = chunk_of(j), nr = rows_of(ch);
            const float f = row < nr ? pw[rev ? nr - 1 - row : row + 1] : 0.f;
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(sc.out) +
                                 ((pr.packed ? static_cast<int64_t>(h) * pr.sq.total + row0
                                             : static_cast<int64_t>(bh) * pr.sq.T) +
                                  static_cast<int64_t>(ch) * kTile) * d2 + c0;
            uint4 ch4[2][4];
#pragma unroll
            for (int hh = 0; hh < 2; hh++) {
                float a[32], y[32];
                tmem_ld32(lanes + kColNear + 32 * hh, a);
                tmem_ld32(lanes + kColFar + 32 * hh, y);
#pragma unroll
                for (int i = 0; i < 4; i++)
                    ch4[hh][i] = make_uint4(pack_bf16(a[8 * i] + f * y[8 * i], a[8 * i + 1] + f * y[8 * i + 1]),
                                            pack_bf16(a[8 * i + 2] + f * y[8 * i + 2], a[8 * i + 3] + f * y[8 * i + 3]),
                                            pack_bf16(a[8 * i + 4] + f * y[8 * i + 4], a[8 * i + 5] + f * y[8 * i + 5]),
                                            pack_bf16(a[8 * i + 6] + f * y[8 * i + 6], a[8 * i + 7] + f * y[8 * i + 7]));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_read);
#pragma unroll
            for (int hh = 0; hh < 2; hh++) {
                lane_group_transpose(ch4[hh], lane);
                const int col = 32 * hh + 8 * (lane & 3);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int r = quad * 32 + (lane & ~3) + i;
                    if (r < nr && c0 + col < d2)
                        *reinterpret_cast<uint4*>(out + static_cast<int64_t>(r) * d2 + col) = ch4[hh][i];
                }
            }
            return true;
        };
        bool ok = true;
        for (int j = 0; j < n && ok; j++) {
            if (__any_sync(0xffffffffu, *fail != 0)) break;
            const int s = j % nst, nr = rows_of(chunk_of(j));
            uint8_t* st = smem + s * stage_bytes;
            ok = warp_wait(&v_full[s], (j / nst) & 1) && (j == 0 || warp_wait(&own_full, (j - 1) & 1));
            if (ok && nr < kTile) {
                // rows behind the sequence's end count nothing, whatever they hold
                ok = warp_wait(&qk_full[s], (j / nst) & 1);
                if (ok && row >= nr) {
                    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
                    for (int c = 0; c < 8; c++) {
                        *reinterpret_cast<uint4*>(st + v_off + row * 128 + c * 16) = zero;
                        for (int p = 0; p < np; p++)
                            *reinterpret_cast<uint4*>(st + k_off + p * kPanelBytes + row * 128 + c * 16) = zero;
                    }
                }
            }
            if (!ok) break;
            const float wt = row < nr ? pw[rev ? row + 1 : nr - 1 - row] : 0.f;
#pragma unroll 2
            for (int c = 0; c < 8; c++) {
                const uint32_t off = sw128_off(row, c);
                const uint4 xv = *reinterpret_cast<const uint4*>(st + v_off + off);
                const uint32_t in[4] = {xv.x, xv.y, xv.z, xv.w};
                uint32_t p1[4], p2[4], p3[4];
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    float2 f = unpack_bf16(in[q]);
                    f.x *= wt;
                    f.y *= wt;
                    p1[q] = pack_bf16(f.x, f.y);
                    float2 t = unpack_bf16(p1[q]);
                    f.x -= t.x;
                    f.y -= t.y;
                    p2[q] = pack_bf16(f.x, f.y);
                    t = unpack_bf16(p2[q]);
                    p3[q] = pack_bf16(f.x - t.x, f.y - t.y);
                }
                *reinterpret_cast<uint4*>(wc + off) = make_uint4(p1[0], p1[1], p1[2], p1[3]);
                *reinterpret_cast<uint4*>(wc + kPanelBytes + off) = make_uint4(p2[0], p2[1], p2[2], p2[3]);
                *reinterpret_cast<uint4*>(wc + 2 * kPanelBytes + off) = make_uint4(p3[0], p3[1], p3[2], p3[3]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&scaled);
            if (!kStateOnly && j > 0) ok = write_out(j - 1);
        }
        if (ok && !kStateOnly && n > 0 && !__any_sync(0xffffffffu, *fail != 0)) ok = write_out(n - 1);
        if (!ok && lane == 0) fail_now();
    }

    __syncthreads();
    if (*fail && tid == 0) {
        // let the copies still in flight land before the shared memory goes away
        for (int i = sent_qk > nst ? sent_qk - nst : 0; i < sent_qk; i++) mbar_wait(&qk_full[i % nst], (i / nst) & 1);
        for (int i = sent_v > nst ? sent_v - nst : 0; i < sent_v; i++) mbar_wait(&v_full[i % nst], (i / nst) & 1);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// [z][rows][cols] bf16, box 64 columns x 128 rows of one z, 128-byte swizzle; columns and rows past
// the tensor's read as zero.
bool make_map_3d(CUtensorMap* m, const void* base, uint64_t z, uint64_t rows, uint64_t cols) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {cols, rows, z};
    cuuint64_t strides[2] = {cols * 2, rows * cols * 2};
    cuuint32_t box[3] = {64, 128, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) {
        cudaGetLastError();
        sms = 152;
    }
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

bool linear_tc_plan(LinTcPlan* pl, int batch, int H, int T, int64_t rows, int tiles) {
    if (T > (1 << 30) || rows / H > (1 << 30)) return false;  // token offsets are ints
    pl->batch = batch;
    const int64_t items = static_cast<int64_t>(batch) * H * tiles;
    const int nch = (T - 1) / kTile + 1;
    const int sms = sm_count();
    // chunks of all items (packed sequences: fewer than batch x nch)
    const double work = static_cast<double>(rows) / kTile * tiles;
    // segments: time in units of one chunk of the main kernel; a chunk of the state launch is about half of one,
    // a CTA's start and end about two, the extra launch about two
    double best = 0;
    pl->nseg = 1;
    for (int s = 1; s <= 64 && s <= nch; s++) {
        const int L = (nch + s - 1) / s;
        if ((nch + L - 1) / L != s) continue;  // the same cut as fewer segments
        auto waves = [&](double it, double share) {
            const double full = (it / sms > 1 ? std::ceil(it / sms) : 1.0) * (L + 2.0);
            const double spread = work * share / sms + L;  // ragged sequences: the longest item ends late
            return rows < static_cast<int64_t>(batch) * H * T && spread < full ? spread : full;
        };
        double c = waves(static_cast<double>(items) * s, 1.0);
        if (s > 1) c += 0.5 * waves(static_cast<double>(items) * (s - 1), (s - 1.0) / s) + 2.0;
        if (s == 1 || c < best) {
            best = c;
            pl->nseg = s;
        }
    }
    pl->seg_chunks = (nch + pl->nseg - 1) / pl->nseg;
    pl->seg_bytes = static_cast<size_t>(items) * (pl->nseg - 1) * kDepth * kTile * sizeof(float);
    return items * pl->nseg <= 0x7fffffff;
}

cudaError_t linear_tc_run(const LinTcPlan& pl, const LinTcMap* maps, int n_maps, const LinTcScan* scans, int count,
                          const LinSeqs& sq, const float* log_a, float* seg, int* err, cudaStream_t stream) {
    ScanParams pr = {};
    const bool packed = sq.tab != nullptr;
    for (int i = 0; i < n_maps; i++)
        if (!make_map_3d(&pr.map[i], maps[i].base, packed ? sq.H : static_cast<uint64_t>(pl.batch) * sq.H,
                         packed ? sq.total : sq.T, maps[i].cols))
            return cudaErrorInvalidValue;
    pr.log_a = log_a;
    pr.seg = seg;
    pr.sq = sq;
    pr.count = count;
    pr.nseg = pl.nseg;
    pr.seg_chunks = pl.seg_chunks;
    pr.packed = packed;
    pr.batch = pl.batch;
    int base = 0, tiles = 0, d1 = 0;
    for (int i = 0; i < count; i++) {
        pr.scan[i] = scans[i];
        pr.scan[i].tiles = (scans[i].d2 + kDepth - 1) / kDepth;
        pr.scan[i].seg_base = base;
        base += pl.batch * sq.H * (pl.nseg - 1) * pr.scan[i].tiles;
        tiles += pr.scan[i].tiles;
        if (scans[i].d1 > d1) d1 = scans[i].d1;
    }
    const unsigned per_seg = static_cast<unsigned>(pl.batch) * sq.H * tiles;
    cudaError_t e;
    if (pl.nseg > 1) {
        const int smem = smem_bytes(true, d1);
        e = cudaFuncSetAttribute(linear_scan_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost);
        if (e != cudaSuccess) return e;
        linear_scan_kernel<true><<<per_seg * (pl.nseg - 1), kScanThreads, smem, stream>>>(pr, err);
        note_launch(stream, "linear_scan_state");
    }
    const int smem = smem_bytes(false, d1);
    e = cudaFuncSetAttribute(linear_scan_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost);
    if (e != cudaSuccess) return e;
    if (pl.nseg > 1) {
        e = launch_pdl(linear_scan_kernel<false>, dim3(per_seg * pl.nseg), dim3(kScanThreads), smem, stream, pr, err);
        if (e != cudaSuccess) return e;
    } else {
        linear_scan_kernel<false><<<per_seg, kScanThreads, smem, stream>>>(pr, err);
    }
    note_launch(stream, "linear_scan");
    return cudaGetLastError();
}

}  // namespace lla
