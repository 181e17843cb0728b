// The log-linear decode step of a batch over one shared prefix.
//
// Every sequence starts with the same P tokens. The Fenwick walk of P - 1 splits them into
// aligned blocks, each wholly inside one bucket of any later position t: the highest bit in which
// t and a position of the block differ lies above the block. So
//     o = sum_l lambda^(l) (own^(l))^T q + exp(D) sum_j lambda^(l(t, block j)) (prefix^(j))^T q,
// where own^(l) is bucket l restricted to positions >= P, prefix^(j) the prefix's state of block
// j decayed to P - 1, and D the sum of log_a over P..t. The prefix states are read once for the
// whole batch and never written; a sequence reads and writes only the buckets that hold own
// tokens. Bucket l >= 1 of position pos (bit l - 1 of pos set) is [(pos >> l) << l, + 2^(l-1)):
// it holds own tokens when its end is past P.
//
// Bound by the own states' bytes: 64 x 16 heads of 128 x 64, P = 30011, up to 4096 own tokens: 86 us for 492 MB, 85% of
// the copy rate, half of it writes. The prefix's kernel (20 us by itself) runs beside the own states' streams. The step on
// whole states (lla_decode_step) moves 621 MB there and takes 100 us.
#include <type_traits>

#include "lla_linear.cuh"
#include "lla_tc_ptx.cuh"

namespace lla {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxDk = 256;

// slot l is held at pos and has a position >= P
__device__ __forceinline__ bool own_held(int64_t pos, int64_t P, int l) {
    if (pos < P) return false;
    if (l == 0) return true;
    if (((pos >> (l - 1)) & 1) == 0) return false;
    return ((pos >> l) << l) + (int64_t(1) << (l - 1)) > P;
}

__device__ __forceinline__ void fma4(float4& o, float w, const float4& x) {
    o.x += w * x.x;
    o.y += w * x.y;
    o.z += w * x.z;
    o.w += w * x.w;
}

constexpr int kBatchTile = 32;  // sequences per CTA of the prefix kernel

// part[j][bh][x] = sum_i prefix[h][slot j][i][x] q[bh][i]. grid (held prefix slots, H, batch tiles): each
// slot is read once for kBatchTile sequences. Thread: four columns, kBatchTile DV4 / kThreads sequences.
template <typename T, int DV4>
__global__ void __launch_bounds__(kThreads) shared_prefix(const T* __restrict__ q, const float* __restrict__ prefix,
                                                          float* __restrict__ part, int64_t P, int B, int H, int dk,
                                                          int Lp) {
    constexpr int kGroups = kThreads / DV4;                                    // thread groups over the sequences
    constexpr int kSeq = kBatchTile / kGroups > 0 ? kBatchTile / kGroups : 1;  // sequences of a thread
    __shared__ float qs[kMaxDk][kBatchTile + 1];
    grid_dep_launch();
    const int j = blockIdx.x, h = blockIdx.y, b0 = blockIdx.z * kBatchTile, tid = threadIdx.x;
    int l = 0;  // the j-th held slot of the walk of P - 1
    for (int left = j; left > 0;) {
        l++;
        if (((P - 1) >> (l - 1)) & 1) left--;
    }
    const int nb = B - b0 < kBatchTile ? B - b0 : kBatchTile;
    for (int e = tid; e < kBatchTile * dk; e += kThreads) {
        const int b = e / dk, i = e - b * dk;
        qs[i][b] = b < nb ? load_f(q + (static_cast<int64_t>(b0 + b) * H + h) * dk + i) : 0.f;
    }
    __syncthreads();
    const int col4 = tid % DV4, g = tid / DV4;
    if (g * kSeq >= nb) return;
    const float4* S =
        reinterpret_cast<const float4*>(prefix) + (static_cast<int64_t>(h) * Lp + l) * dk * DV4 + col4;
    float4 o[kSeq];
#pragma unroll
    for (int u = 0; u < kSeq; u++) o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < dk; i0 += 8) {
        float4 x[8];
#pragma unroll
        for (int r = 0; r < 8; r++)
            if (i0 + r < dk) x[r] = S[static_cast<int64_t>(i0 + r) * DV4];
#pragma unroll
        for (int r = 0; r < 8; r++)
            if (i0 + r < dk) {
#pragma unroll
                for (int u = 0; u < kSeq; u++) fma4(o[u], qs[i0 + r][g * kSeq + u], x[r]);
            }
    }
#pragma unroll
    for (int u = 0; u < kSeq; u++) {
        const int b = g * kSeq + u;
        if (b < nb)
            reinterpret_cast<float4*>(part)[((static_cast<int64_t>(j) * B + b0 + b) * H + h) * DV4 + col4] = o[u];
    }
}

// One CTA per (b, h): the own buckets (carry, decay, read) and the prefix's parts. Level by level, four
// 16-byte loads of a thread in flight; each held state is read once and written once, past L2's retention.
// kOwnThreads: 256 where they hold all dk rows in one pass of four rows a thread, else 512 (64 x 16 heads of 128 x 64:
// 86 us against 89; 4 x 4 heads of 64 x 64: 6.9 against 6.5). The next level's loads issued ahead cost more registers
// than they give (101 us), two or eight rows a thread as much or more. `part` is written while this kernel already runs,
// so it is neither __restrict__ nor read through L1.
template <typename T, int DV4, int kOwnThreads>
__global__ void __launch_bounds__(kOwnThreads) shared_own(const T* __restrict__ q, const T* __restrict__ k,
                                                       const T* __restrict__ v, const float* __restrict__ log_a,
                                                       const float* __restrict__ lambda,
                                                       const float* part, float* __restrict__ decay,
                                                       float* __restrict__ states, const int64_t* __restrict__ tpos,
                                                       T* __restrict__ out, int64_t P, int B, int H, int dk, int Lmax,
                                                       int* err) {
    constexpr int DV = DV4 * 4;
    constexpr int kRows = kOwnThreads / DV4;
    constexpr int U = 4;  // rows of a thread in flight
    __shared__ float qs[kMaxDk], ks[kMaxDk], lam[40];
    constexpr int kGroups = kOwnThreads / DV;  // thread groups over the prefix's parts
    __shared__ float red[kOwnThreads / 32][DV], red_far[kGroups][DV], far_w[40];
    const int tid = threadIdx.x;
    const int64_t bh = blockIdx.x;
    const int b = static_cast<int>(bh / H);
    const int64_t t = tpos[b];
    if (t < P || t >= (int64_t(1) << (Lmax - 1))) {
        if (tid == 0) record_error(err, kDevBadInput);
        grid_dep_wait();  // with every sequence skipped too, this kernel ends after the one that writes the workspace
        return;
    }
    for (int x = tid; x < dk; x += kOwnThreads) {
        qs[x] = load_f(q + bh * dk + x);
        ks[x] = load_f(k + bh * dk + x);
    }
    for (int x = tid; x < Lmax; x += kOwnThreads) lam[x] = lambda[bh * Lmax + x];
    const float la = log_a[bh];
    const float D = (t > P ? decay[bh] : 0.f) + la;
    __syncthreads();
    if (tid == 0) decay[bh] = D;  // after every thread has read it

    const float a = expf(la);
    const int c = __ffsll(static_cast<long long>(t)) - 1;   // trailing zeros of t (t >= P >= 1)
    const int top = 64 - __clzll(static_cast<long long>(t));  // highest slot that t holds
    const int col4 = tid % DV4, row0 = tid / DV4;
    const int64_t msz4 = static_cast<int64_t>(dk) * DV4;
    float4* S = reinterpret_cast<float4*>(states) + bh * Lmax * msz4 + col4;
    const T* vp = v + bh * DV + col4 * 4;
    const float4 v4 = make_float4(load_f(vp), load_f(vp + 1), load_f(vp + 2), load_f(vp + 3));
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = row0; i0 < dk; i0 += U * kRows) {
        if (t > P) {
            float4 m[U];
#pragma unroll
            for (int r = 0; r < U; r++) m[r] = make_float4(0.f, 0.f, 0.f, 0.f);
            // the carry: slots 0..c of t - 1 into slot c + 1, its decay with the others' below
            for (int l = 0; l <= c; l++) {
                if (!own_held(t - 1, P, l)) continue;
                float4 x[U];
#pragma unroll
                for (int r = 0; r < U; r++)
                    if (i0 + r * kRows < dk) x[r] = __ldcs(S + l * msz4 + static_cast<int64_t>(i0 + r * kRows) * DV4);
#pragma unroll
                for (int r = 0; r < U; r++)
                    if (i0 + r * kRows < dk) fma4(m[r], 1.f, x[r]);
            }
            for (int l = c + 1; l <= top; l++) {
                if (l > c + 1) {  // a slot that both t - 1 and t hold
                    if (!own_held(t - 1, P, l)) continue;
#pragma unroll
                    for (int r = 0; r < U; r++)
                        if (i0 + r * kRows < dk) m[r] = __ldcs(S + l * msz4 + static_cast<int64_t>(i0 + r * kRows) * DV4);
                }
                const float ll = lam[l];
#pragma unroll
                for (int r = 0; r < U; r++) {
                    if (i0 + r * kRows < dk) {
                        m[r].x *= a; m[r].y *= a; m[r].z *= a; m[r].w *= a;
                        __stcs(S + l * msz4 + static_cast<int64_t>(i0 + r * kRows) * DV4, m[r]);
                        fma4(o, ll * qs[i0 + r * kRows], m[r]);
                    }
                }
            }
        }
        const float l0 = lam[0];
#pragma unroll
        for (int r = 0; r < U; r++) {
            const int i = i0 + r * kRows;
            if (i < dk) {
                const float ki = ks[i];
                const float4 x0 = make_float4(ki * v4.x, ki * v4.y, ki * v4.z, ki * v4.w);
                __stcs(S + static_cast<int64_t>(i) * DV4, x0);
                fma4(o, l0 * qs[i], x0);
            }
        }
    }
#pragma unroll
    for (int off = DV4; off < 32; off <<= 1) {
        o.x += __shfl_xor_sync(0xffffffffu, o.x, off);
        o.y += __shfl_xor_sync(0xffffffffu, o.y, off);
        o.z += __shfl_xor_sync(0xffffffffu, o.z, off);
        o.w += __shfl_xor_sync(0xffffffffu, o.w, off);
    }
    const int warp = tid >> 5, lane = tid & 31;
    if (lane < DV4) {
        red[warp][lane * 4 + 0] = o.x;
        red[warp][lane * 4 + 1] = o.y;
        red[warp][lane * 4 + 2] = o.z;
        red[warp][lane * 4 + 3] = o.w;
    }
    // the prefix block of slot l of the walk of P - 1 starts at ((P - 1) >> l) << l: its weight, at its place among the parts
    const int parts = 1 + __popcll(static_cast<unsigned long long>(P - 1));
    if (tid < 40 && (tid == 0 || ((P - 1) >> (tid - 1) & 1))) {
        const int64_t below = tid == 0 ? 0 : (int64_t(1) << (tid - 1)) - 1;
        const int j = tid == 0 ? 0 : 1 + __popcll(static_cast<unsigned long long>((P - 1) & below));
        far_w[j] = lam[64 - __clzll(static_cast<long long>(t ^ (((P - 1) >> tid) << tid)))];
    }
    grid_dep_wait();  // the prefix's parts (this kernel starts beside the one that forms them)
    __syncthreads();
    const int col = tid % DV, part0 = tid / DV;
    float far = 0.f;
#pragma unroll 4
    for (int j = part0; j < parts; j += kGroups)
        far += far_w[j] * __ldcg(part + (static_cast<int64_t>(j) * B * H + bh) * DV + col);
    red_far[part0][col] = far;
    __syncthreads();
    if (tid < DV) {
        float s = 0.f;
        far = 0.f;
#pragma unroll
        for (int w = 0; w < kOwnThreads / 32; w++) s += red[w][tid];
#pragma unroll
        for (int u = 0; u < kGroups; u++) far += red_far[u][tid];
        store_f(out + bh * DV + tid, s + expf(D) * far);
    }
}

int held_slots(int64_t prefix_len) {
    int n = 1;
    for (int64_t x = prefix_len - 1; x > 0; x &= x - 1) n++;
    return n;
}

template <typename T>
cudaError_t shared_t(const void* q, const void* k, const void* v, const float* log_a, const float* lambda,
                     const float* prefix, int64_t P, int Lp, float* decay, float* states, const int64_t* t, void* out,
                     float* part, int B, int H, int dk, int dv, int Lmax, int* err, cudaStream_t stream) {
    const T* qp = static_cast<const T*>(q);
    cudaError_t e = cudaSuccess;
    auto go = [&](auto pre, auto own, int own_threads) {
        pre<<<dim3(held_slots(P), H, (B + kBatchTile - 1) / kBatchTile), kThreads, 0, stream>>>(qp, prefix, part, P, B, H,
                                                                                              dk, Lp);
        note_launch(stream, "shared_prefix");
        e = launch_pdl(own, dim3(static_cast<unsigned>(B) * H), dim3(own_threads), 0, stream, qp,
                       static_cast<const T*>(k), static_cast<const T*>(v), log_a, lambda, static_cast<const float*>(part),
                       decay, states, t, static_cast<T*>(out), P, B, H, dk, Lmax, err);
        note_launch(stream, "shared_own");
    };
    auto pick = [&](auto dv4) {
        constexpr int DV4 = decltype(dv4)::value;
        if (dk <= 4 * (256 / DV4)) go(shared_prefix<T, DV4>, shared_own<T, DV4, 256>, 256);
        else go(shared_prefix<T, DV4>, shared_own<T, DV4, 512>, 512);
    };
    switch (dv) {
        case 16: pick(std::integral_constant<int, 4>()); break;
        case 32: pick(std::integral_constant<int, 8>()); break;
        case 64: pick(std::integral_constant<int, 16>()); break;
        default: pick(std::integral_constant<int, 32>()); break;
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t shared_workspace_bytes(int B, int H, int dv, int64_t prefix_len) {
    return static_cast<size_t>(held_slots(prefix_len)) * B * H * dv * sizeof(float);
}

cudaError_t decode_step_shared(int dtype, const void* q, const void* k, const void* v, const float* log_a,
                               const float* lambda, const float* prefix_states, int64_t prefix_len, int Lp,
                               float* prefix_decay, float* states, const int64_t* t, void* out, void* workspace,
                               int B, int H, int dk, int dv, int Lmax, int* err, cudaStream_t stream) {
    float* part = static_cast<float*>(workspace);
    if (dtype == 1)
        return shared_t<float>(q, k, v, log_a, lambda, prefix_states, prefix_len, Lp, prefix_decay, states, t, out,
                               part, B, H, dk, dv, Lmax, err, stream);
    return shared_t<__nv_bfloat16>(q, k, v, log_a, lambda, prefix_states, prefix_len, Lp, prefix_decay, states, t, out,
                                   part, B, H, dk, dv, Lmax, err, stream);
}

}  // namespace lla
