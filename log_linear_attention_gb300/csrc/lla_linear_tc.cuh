// Building blocks of the tensor-core kernels of linear attention with one decay per head
// (lla_linear_tc.cu, lla_linear_grad.cu). In an unnamed namespace, as lla_tc_ptx.cuh.
#pragma once

#include "lla_linear.cuh"
#include "lla_tc_ptx.cuh"

namespace lla {
namespace {

constexpr int kDepth = 64;  // columns of c per CTA or item

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Pull one box of a tensor map into L2.
__device__ __forceinline__ void tma_prefetch_l2_3d(const CUtensorMap* map, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// Shared -> global: contiguous bytes (16-byte aligned, a multiple of 16); completion by the issuing thread's bulk groups.
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
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

// A shared-memory descriptor moved on: address and strides lie in the low word and do not carry out of it, so that one
// addition does (the thread that issues the MMAs is on the longest path of its kernels).
__device__ __forceinline__ uint64_t further(uint64_t desc, uint64_t by) {
    return (desc & 0xffffffff00000000ull) | (static_cast<uint32_t>(desc) + static_cast<uint32_t>(by));
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

__device__ __forceinline__ uint32_t pack_bf16(f32x2 x) {
    const float2 f = split2(x);
    return pack_bf16(f.x, f.y);
}

// 16 consecutive fp32 TMEM columns at each of two places, as pairs: both loads in flight, one wait.
__device__ __forceinline__ void tmem_ld16x2(uint32_t ta, uint32_t tb, f32x2* va, f32x2* vb) {
    uint32_t r[16], q[16];
    tmem_ld16_issue(ta, r);
    tmem_ld16_issue(tb, q);
    tmem_ld16_wait(r);
    tmem_ld16_wait(q);  // nothing is left to wait for: keeps the uses of q behind the wait
#pragma unroll
    for (int i = 0; i < 8; i++) {
        va[i] = pair2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
        vb[i] = pair2(__uint_as_float(q[2 * i]), __uint_as_float(q[2 * i + 1]));
    }
}

// x in two bf16 parts, two values at once: the first 8 bits cut off, the rest rounded.
__device__ __forceinline__ void split_pair(f32x2 x, uint32_t& hi, uint32_t& lo) {
    const float2 f = split2(x);
    hi = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
    lo = pack_bf16(fma2(pair2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)), pair2(-1.f, -1.f), x));
}

// P of this thread's row and one block of 32 keys, in place of its scores (fp32, 32 columns at `cols`): for every 16 keys
// eight columns of P's high parts and eight of its low ones, so that P keeps 16 bits and only the state and the output
// are rounded to bf16's eight.
// side 1: the keys lie in the row's reach, their weights colw[key] rw; 0: the diagonal block, weight diag[-key], 0 out of
// reach; -1: out of reach.
template <int kUnroll>
__device__ __forceinline__ void weigh_block(uint32_t cols, int side, const float* diag, const float* colw, float rw) {
    const f32x2 rw2 = pair2(rw, rw);
#pragma unroll(kUnroll)
    for (int half = 0; half < 2; half++) {
        uint32_t r[16];
        if (side < 0) {
#pragma unroll
            for (int i = 0; i < 16; i++) r[i] = 0u;
        } else {
            uint32_t y[16];
            tmem_ld16_issue(cols + 16 * half, y);
            tmem_ld16_wait(y);
            if (side == 0) {
                const float* dg = diag - 16 * half;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const float f = dg[-2 * i], g = dg[-2 * i - 1];
                    // out of reach: never the product with an infinity
                    split_pair(pair2(f != 0.f ? __uint_as_float(y[2 * i]) * f : 0.f,
                                     g != 0.f ? __uint_as_float(y[2 * i + 1]) * g : 0.f), r[i], r[8 + i]);
                }
            } else {
                const ulonglong2* cw = reinterpret_cast<const ulonglong2*>(colw + 16 * half);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const ulonglong2 f = cw[i];
                    split_pair(mul2(mul2(pair2(__uint_as_float(y[4 * i]), __uint_as_float(y[4 * i + 1])), f.x), rw2),
                               r[2 * i], r[8 + 2 * i]);
                    split_pair(mul2(mul2(pair2(__uint_as_float(y[4 * i + 2]), __uint_as_float(y[4 * i + 3])), f.y), rw2),
                               r[2 * i + 1], r[9 + 2 * i]);
                }
            }
        }
        tmem_st16_issue(cols + 16 * half, r);
    }
}

// One lane of a converged warp; code behind it counts as uniform, so descriptors stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Up to kTries tests of a barrier's phase, three instructions each: a test suspends the thread for some hundred
// cycles only, and two dozen waiting warps that did more between tests took most of the issue slots.
constexpr uint32_t kTries = 1024;
__device__ __forceinline__ bool mbar_try_many(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 i;\n\tmov.u32 i, %4;\n"
        "TRY:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "@p bra DONE;\n\t"
        "sub.u32 i, i, 1;\n\t"
        "setp.ne.u32 q, i, 0;\n\t"
        "@q bra TRY;\n"
        "DONE:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "n"(kSuspendNs), "n"(kTries)
        : "memory");
    return ok != 0;
}

// Bounded waits. They give up when another role has.
struct Bound {  // in shared memory
    long long cycles;
    int fail;  // set by the role that gave up first
};
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile Bound* to) {
    const long long start = clock64();
    while (!mbar_try_many(bar, parity)) {
        if (to->fail || clock64() - start > to->cycles) return false;
    }
    return true;
}
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, volatile Bound* to) {
    return mbar_try_many(bar, parity) || wait_long(bar, parity, to);
}
__device__ __noinline__ bool wait_long_warp(uint64_t* bar, uint32_t parity, volatile Bound* to) {
    const long long start = clock64();
    while (true) {
        const bool done = mbar_try_many(bar, parity);
        if (__all_sync(0xffffffffu, done)) return true;
        const bool late = to->fail || clock64() - start > to->cycles;
        if (__any_sync(0xffffffffu, late)) return false;
    }
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile Bound* to) {
    return __all_sync(0xffffffffu, mbar_try_many(bar, parity)) || wait_long_warp(bar, parity, to);
}

// 32 bytes of a global row in one store: a whole sector (16 bytes each where rows are not so aligned, `second` false
// where only the first 16 are the row's).
__device__ __forceinline__ void store32(__nv_bfloat16* to, const uint32_t (&o)[8], bool aligned, bool second) {
    if (aligned) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(o[0]), "r"(o[1]),
                     "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                     : "memory");
    } else {
        *reinterpret_cast<uint4*>(to) = make_uint4(o[0], o[1], o[2], o[3]);
        if (second) *reinterpret_cast<uint4*>(to + 8) = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// ------------------------------------------------------------------ host side

// [z][rows][cols] bf16, box 64 columns x box_rows rows of one z, 128-byte swizzle; columns and rows past
// the tensor's read as zero.
bool make_map_3d(CUtensorMap* m, const void* base, uint64_t z, uint64_t rows, uint64_t cols, uint32_t box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {cols, rows, z};
    cuuint64_t strides[2] = {cols * 2, rows * cols * 2};
    cuuint32_t box[3] = {64, box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace lla
