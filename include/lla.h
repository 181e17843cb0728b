/*
 * lla.h — C ABI of liblla.so: causal log-linear Mamba-2 attention on GB300 (sm_103a).
 *
 * The operator ("Log-Linear Attention", arXiv 2506.04761; gist.science pages in
 * Portuguese and French, §2 "Particionamento Hierarquico / Mascara Hierarquica"
 * and "Partitionnement par Arbre de Fenwick / Matrice de Masque Hierarchique"):
 *
 *     O = (Q K^T (.) M^S (.) M^H) V
 *     o_t = sum_{s<=t} lambda_t^(l(t,s)) * prod_{r=s+1..t} a_r * (q_t . k_s) * v_s
 *
 * M^S is the Mamba-2 semiseparable scalar-decay mask (a_r = exp(log_a_r) in
 * (0,1], exclusive of s so the diagonal is 1). M^H weights key s for query t
 * by lambda_t at the Fenwick level l(t,s) of s in t's prefix: l = 0 for s = t,
 * otherwise the bucket of size 2^(l-1) in the Fenwick decomposition of [0,t),
 * which equals 1 + floor(log2(t xor s)) with 0-indexed positions. A length-T
 * sequence uses L = bitlength(T-1) + 1 levels (7, 12, 14, 17 for T = 64, 2048,
 * 8192, 65536). There is no 1/sqrt(d) scale and no normalisation.
 *
 * Conventions for every entry point:
 *  - Tensors are dense, row-major (C-contiguous), batch-major: [B, H, ...].
 *  - q/k/v/out are bf16 (LLA_BF16) or fp32 (LLA_F32); log_a, lambda and decode
 *    states are always fp32; decode positions are int64.
 *  - Device pointers are caller-owned CUDA device memory on the current device.
 *    The library keeps no pointer after the call returns. Every pointer must be
 *    16-byte aligned.
 *  - `stream` is a cudaStream_t (NULL = legacy default stream). All work is
 *    enqueued asynchronously on it; outputs are valid once the stream reaches
 *    that point.
 *  - Return value: LLA_OK, or a negative lla_status. Argument errors are found
 *    on the host before anything is enqueued and leave all buffers untouched.
 *    Faults found by a kernel (an out-of-range decode position, a bounded wait
 *    that ran out) are recorded in a per-device error word and reported by
 *    lla_device_error(). No kernel traps and the library never exits.
 *  - The library keeps per-device state for the life of the process: the device
 *    address of its error word and of the lla_forward_noalloc scratch, looked up
 *    once, and a memory pool. Do not call it on a device after cudaDeviceReset()
 *    (or any teardown of that device's primary context) in the same process: the
 *    cached addresses would no longer be valid.
 */
#ifndef LLA_H
#define LLA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    LLA_OK = 0,
    LLA_ERR_INVALID_ARG = -1, /* null pointer, bad size, misaligned pointer */
    LLA_ERR_UNSUPPORTED = -2, /* valid operator, but a shape this build has no kernel for */
    LLA_ERR_CUDA = -3,        /* a CUDA runtime call or launch failed */
    LLA_ERR_TIMEOUT = -4,     /* a kernel's bounded wait ran out (device error word) */
    LLA_ERR_NOMEM = -5,       /* workspace allocation failed, or workspace too small */
    LLA_ERR_DEVICE = -6       /* a kernel rejected its device-side input (device error word) */
} lla_status;

typedef enum { LLA_BF16 = 0, LLA_F32 = 1 } lla_dtype;

/* Human-readable name of a status code (static string, never NULL). */
const char* lla_status_string(int status);

/* Number of Fenwick levels used by a length-T sequence: bitlength(T-1) + 1
 * (1 for T = 1, 0 for T <= 0). lambda's last dimension must equal this. */
int lla_num_levels(int64_t T);

/*
 * Chunk-parallel prefill (pages' "Chunk-scan" / "balayage par blocs": dense
 * intra-chunk work, hierarchical inter-chunk state passing, O(T log T)).
 *
 *   q      [B,H,T,dk]  dtype        queries
 *   k      [B,H,T,dk]  dtype        keys
 *   v      [B,H,T,dv]  dtype        values
 *   log_a  [B,H,T]     fp32         log of the Mamba-2 decay a_t (<= 0 expected;
 *                                   positive values are computed as given)
 *   lambda [B,H,T,L]   fp32         per-query, per-level weights, L = lla_num_levels(T)
 *   out    [B,H,T,dv]  dtype        written; must not overlap any input
 *   chunk  chunk length of the scan: 16, 32, 64 or 128, with T % chunk == 0.
 *          It sets how keys are grouped into inter-chunk states; the result is
 *          the same operator for every valid chunk (up to rounding order).
 *   dk, dv 1..128; the bf16 tensor-core path runs for dk in {64,128}, dv in {64,128},
 *          T % 128 == 0; other shapes run the fp32 SIMT path.
 *
 * Scratch: the call takes its workspace (inter-chunk states) from a
 * library-owned, stream-ordered memory pool on `stream` and returns it there.
 * Use lla_forward_ws to pass caller-owned workspace instead.
 */
int lla_forward(const void* q, const void* k, const void* v, const float* log_a, const float* lambda,
                void* out, int B, int H, int T, int dk, int dv, int chunk, void* stream, int dtype);

/*
 * lla_forward with HOST buffers (pinned for full copy bandwidth; pageable works,
 * slower): same arguments and layouts as lla_forward, but q, k, v, log_a, lambda
 * and out live in host memory (device or managed pointers: LLA_ERR_INVALID_ARG).
 * The B*H heads are split into up to eight groups; each group's inputs are copied
 * to the device on a library copy stream, its prefill runs on `stream`, and its
 * output is copied back on a second library stream, so copies of one group
 * overlap the kernels of the next. Device buffers come from the library pool.
 * The call returns after `out` is written (it synchronizes `stream`). Calls on
 * one device are serialized.
 */
int lla_forward_host(const void* q, const void* k, const void* v, const float* log_a, const float* lambda,
                     void* out, int B, int H, int T, int dk, int dv, int chunk, void* stream, int dtype);

/* Workspace bytes lla_forward_ws needs for these sizes (0 on invalid sizes). */
size_t lla_forward_workspace_size(int B, int H, int T, int dk, int dv, int chunk, int dtype);

/* lla_forward with caller-owned device workspace of at least
 * lla_forward_workspace_size(...) bytes, 256-byte aligned. The workspace holds
 * no state between calls; calls that share it must not overlap on the GPU.
 * Returns LLA_ERR_NOMEM if workspace_bytes is too small. */
int lla_forward_ws(const void* q, const void* k, const void* v, const float* log_a, const float* lambda,
                   void* out, int B, int H, int T, int dk, int dv, int chunk, void* stream, int dtype,
                   void* workspace, size_t workspace_bytes);

/*
 * lla_forward without any allocation, for callers that cannot call cudaMalloc
 * (a host that pre-sizes and owns every device allocation, or code that must
 * not grow the process's GPU footprint after start-up). "Log-Linear Attention"
 * describes no counterpart: this is a deployment variant of lla_forward with
 * identical arguments, results and kernels.
 *
 * Its scratch is a fixed, file-scope device array of LLA_NOALLOC_SCRATCH_BYTES
 * (32 MiB) that every GPU loading this library holds until the process exits.
 * Sizes whose workspace (lla_forward_workspace_size) exceeds it are rejected
 * with LLA_ERR_NOMEM before anything is enqueued. No cudaMalloc, cudaFree or
 * allocating library routine is called.
 *  - The first call on a device looks up that device's copy of the array; make
 *    that first call before capturing a stream into a CUDA graph. The address is
 *    kept for the life of the process (see the cudaDeviceReset note above).
 *  - Every call on a device shares the one array and leaves its contents
 *    behind; no part of it needs to start at zero (each call writes every
 *    scratch value before reading it). Calls whose work overlaps on the GPU
 *    (different streams, or graphs replayed concurrently) race on the array:
 *    serialise them.
 */
#define LLA_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)
int lla_forward_noalloc(const void* q, const void* k, const void* v, const float* log_a, const float* lambda,
                        void* out, int B, int H, int T, int dk, int dv, int chunk, void* stream, int dtype);

/*
 * Measurement aid: runs lla_forward once with a CUDA event recorded on `stream`
 * before the first kernel and after each kernel launch, waits for the last
 * event, and writes, in launch order, each kernel's elapsed device time in
 * milliseconds to kernel_ms[i] and its static name to kernel_names[i], for
 * i < cap. Returns the number of kernels the call launched (which may exceed
 * cap), or a negative lla_status. Synchronous; not meant for hot loops.
 */
int lla_forward_profile(const void* q, const void* k, const void* v, const float* log_a, const float* lambda,
                        void* out, int B, int H, int T, int dk, int dv, int chunk, void* stream, int dtype,
                        float* kernel_ms, const char** kernel_names, int cap);

/*
 * One recurrent decode step (pages' "Decodificacao" / "Inference": O(log T)
 * states S_t^(l), the new token updates the finest level and levels merge
 * along the Fenwick tree; O(log T) time and memory per step).
 *
 *   q, k   [B,H,dk]          dtype   the new token's query and key
 *   v      [B,H,dv]          dtype   its value
 *   log_a  [B,H]             fp32    log a_t of the new token
 *   lambda [B,H,Lmax]        fp32    lambda_t^(l) of the new token, l < Lmax
 *   fenwick_states [B,H,Lmax,dk,dv] fp32, read and written in place.
 *          Slot l holds bucket l of the Fenwick partition as
 *          sum_s prod_{r=s+1..pos} a_r k_s v_s^T, decayed to the last token
 *          `pos` already absorbed. On entry pos = t[b]-1 (nothing for t[b] = 0);
 *          on return pos = t[b]. Slots empty at `pos` (level l >= 1 with bit
 *          l-1 of pos clear) are never read and may hold anything.
 *   t      [B]               int64   device array: position of the new token per
 *          sequence (tokens 0..t-1 are in the states). Not modified: the caller
 *          advances it. Needs 0 <= t < 2^(Lmax-1); a sequence outside that range
 *          is skipped (its state and output untouched) and LLA_ERR_DEVICE is
 *          recorded in the device error word.
 *   out    [B,H,dv]          dtype   o_t = sum_l lambda_t^(l) S^(l)^T q_t (after the update)
 *   dk     1..256; dv in {16, 32, 64, 128}; Lmax in 1..40.
 */
int lla_decode_step(const void* q, const void* k, const void* v, const float* log_a, const float* lambda,
                    float* fenwick_states, const int64_t* t, void* out, void* stream,
                    int B, int H, int dk, int dv, int Lmax, int dtype);

/*
 * Prefill -> decode hand-off: the Fenwick state set after a prompt of T tokens,
 * i.e. what lla_decode_step expects on entry for the next position t = T.
 *
 *   k      [B,H,T,dk]  dtype   keys of the prompt
 *   v      [B,H,T,dv]  dtype   values
 *   log_a  [B,H,T]     fp32    log decays
 *   fenwick_states [B,H,Lmax,dk,dv] fp32, written for every sequence: slot 0 =
 *          k_{T-1} v_{T-1}^T, and each slot l >= 1 with bit l-1 of T-1 set = its
 *          Fenwick bucket of T-1's prefix, sum_s prod_{r=s+1..T-1} a_r k_s v_s^T.
 *          Slots empty at T-1 are left untouched. Needs Lmax >= bitlength(T-1) + 1.
 *   dk, dv 1..128.
 * Takes T fp32 values per (b, h) of scratch from the library's stream-ordered pool.
 * Tensor-core path (bf16, dk = 128): every held slot is written exactly once, its
 * pieces summed in a fixed order, so repeated calls give identical bits. The
 * CUDA-core path adds bucket pieces of at most 512 keys with fp32 atomics, so for
 * buckets of more than 1024 keys the last bits may vary between runs.
 */
int lla_prefill_state(const void* k, const void* v, const float* log_a, float* fenwick_states, int B, int H, int T,
                      int dk, int dv, int Lmax, void* stream, int dtype);

/*
 * Backward of lla_forward: gradients of L = sum over all elements of dout * out.
 * ("Log-Linear Attention", pt §2 "Mascara Hierarquica" / fr §2 "Matrice de
 * Masque Hierarchique" define the operator differentiated here; the pages name
 * the backward through lambda as needing its own kernels.)
 *
 *   q, k, v, log_a, lambda   the forward's inputs (same shapes, dtype, chunk rules)
 *   dout     [B,H,T,dv]  dtype   upstream gradient dL/dout
 *   dq, dk   [B,H,T,dk]  dtype   written
 *   dv       [B,H,T,dv]  dtype   written
 *   dlog_a   [B,H,T]     fp32    written
 *   dlambda  [B,H,T,L]   fp32    written (0 for levels with no key at that query)
 * The outputs must not overlap any input or each other. The forward's
 * intermediate states are recomputed, so no forward workspace is kept between
 * the calls. The chunk argument follows lla_forward. bf16 inputs with dk = 128,
 * dv = 64 and T % 128 == 0 run on tensor cores (128-token tiles, fp32
 * accumulation, bf16 operands); every other shape runs fp32 arithmetic on CUDA
 * cores with chunks of at most 64 (chunk 128 runs as 64: same operator,
 * different rounding order). Workspace comes from the same library-owned
 * stream-ordered pool as lla_forward. A kernel's bounded wait that runs out is
 * reported by lla_device_error as LLA_ERR_TIMEOUT. Errors: LLA_ERR_INVALID_ARG / LLA_ERR_UNSUPPORTED before any
 * launch, LLA_ERR_NOMEM if the pool cannot grow, LLA_ERR_CUDA on launch
 * failure.
 */
int lla_backward(const void* q, const void* k, const void* v, const float* log_a, const float* lambda,
                 const void* dout, void* dq, void* dk, void* dv, float* dlog_a, float* dlambda, int B, int H,
                 int T, int dk_, int dv_, int chunk, void* stream, int dtype);

/*
 * Packed variable-length sequences (no counterpart on the pages: a serving
 * layout for many prompts of different lengths in one call).
 *
 * Layout: every tensor is packed per head, [H, total_T, W] row-major; sequence
 * b owns rows cu_seqlens[b] .. cu_seqlens[b+1]-1 of every head, and its token
 * positions (hence its Fenwick levels) start at 0. cu_seqlens is DEVICE int32
 * [n_seq + 1], non-decreasing, cu_seqlens[0] >= 0, cu_seqlens[n_seq] <= total_T,
 * every length <= max_T. Lengths that break these rules are caught on the
 * device: that sequence is skipped and lla_device_error reports LLA_ERR_DEVICE.
 *
 * lla_forward_varlen: the prefill of every sequence.
 *   q, k [H,total_T,dk], v [H,total_T,dv] (dtype); log_a [H,total_T] fp32;
 *   lambda [H,total_T,L] fp32 with L = lla_num_levels(max_T); out [H,total_T,dv].
 *   bf16 with dv = 64 and dk in {64, 128}: the tensor-core prefill kernels walk
 *   every sequence's own 128-token tiles of the packed tensors (a sequence's
 *   last tile may end inside it; its rows past the end are neither read into
 *   the sequence's outputs nor written). Other shapes: the sequences are copied
 *   into a zero-padded [n_seq, H, Tpad] layout (Tpad = max_T rounded up to
 *   128) in pool workspace, run through the dense prefill kernels and copied
 *   back. Requires H * total_T < 2^31 for the tensor-core walk. chunk as in
 *   lla_forward.
 *
 * lla_prefill_state_varlen: the decode state set after every sequence, as
 * lla_prefill_state: fenwick_states [n_seq, H, Lmax, dk, dv] fp32 with
 * Lmax >= lla_num_levels(max_T); slots empty at a sequence's last position are
 * left untouched (an empty sequence touches none). bf16 with dk = 128 and
 * dv in {64, 128} runs the tensor-core hand-off over every sequence's own tile
 * range; other shapes run CUDA-core kernels.
 */
int lla_forward_varlen(const void* q, const void* k, const void* v, const float* log_a, const float* lambda,
                       void* out, const int32_t* cu_seqlens, int n_seq, int H, int total_T, int max_T, int dk, int dv,
                       int chunk, void* stream, int dtype);
int lla_prefill_state_varlen(const void* k, const void* v, const float* log_a, const int32_t* cu_seqlens,
                             float* fenwick_states, int n_seq, int H, int total_T, int max_T, int dk, int dv, int Lmax,
                             void* stream, int dtype);

/*
 * Log-linear Gated DeltaNet ("Log-Linear Attention", pt §2 "Generalizacao" and
 * fr §3 "Etudes de Cas": the hierarchical mask applied to Gated DeltaNet; the
 * base model is Gated DeltaNet's published gated delta rule):
 *
 *     o_t = sum_{s<=t} lambda_t^(l(t,s)) A[t,s] v_s,
 *     A[t,s] = beta_s k_s^T A_{s+1} A_{s+2} ... A_t q_t,
 *     A_r = exp(log_a_r) (I - beta_r k_r k_r^T),
 *
 * i.e. Gated DeltaNet's own attention matrix under the Fenwick mask M^H. In
 * recurrent form every held Fenwick bucket state S (dk x dv) evolves as
 * S <- A_t S, buckets merge on the lowbit carry as in lla_decode_step, and the
 * new token writes beta_t k_t v_t^T at level 0. Keys are expected L2-normalised
 * and beta in [0, 1] (the transition is then a contraction); other values are
 * computed as given.
 *
 * lla_gdn_forward: chunkwise prefill. Arguments as lla_forward, plus
 *   beta   [B,H,T]  fp32   delta-rule strength of every token.
 *   chunk  16, 32, 64 or 128 (128 runs as 64: same operator, different rounding
 *          order), T % chunk == 0; dk 1..128; dv a multiple of 16 up to 128.
 * All arithmetic is fp32 on CUDA cores. Workspace comes from the library's
 * stream-ordered pool: per head about (2 dk T + 2 (T / C) dk dv + dv T) floats.
 *
 * lla_gdn_decode_step: one recurrent step; arguments as lla_decode_step, plus
 *   beta   [B,H]    fp32   the new token's delta-rule strength.
 *   fenwick_states holds each bucket's state under the transitions above (the
 *   layout, emptiness and position rules of lla_decode_step apply unchanged).
 *   dk and dv in {16, 32, 64, 128}.
 */
int lla_gdn_forward(const void* q, const void* k, const void* v, const float* log_a, const float* beta,
                    const float* lambda, void* out, int B, int H, int T, int dk, int dv, int chunk, void* stream,
                    int dtype);
int lla_gdn_decode_step(const void* q, const void* k, const void* v, const float* log_a, const float* beta,
                        const float* lambda, float* fenwick_states, const int64_t* t, void* out, void* stream, int B,
                        int H, int dk, int dv, int Lmax, int dtype);
/* Measurement aid for lla_gdn_forward, as lla_forward_profile is for lla_forward. */
int lla_gdn_forward_profile(const void* q, const void* k, const void* v, const float* log_a, const float* beta,
                            const float* lambda, void* out, int B, int H, int T, int dk, int dv, int chunk,
                            void* stream, int dtype, float* kernel_ms, const char** kernel_names, int cap);

/*
 * Linear attention with one decay per head: the recurrence that the Fenwick hierarchy of
 * lla_forward is laid over, with one state and one constant decay for each head ("Log-Linear
 * Attention", pt section 2 / fr section 2 take gated linear attention as the base of the hierarchy):
 *
 *     S_t = g_h S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t,   g_h = exp(log_a_h),
 *
 * i.e. o_t = sum_{s<=t} g^(t-s) (q_t . k_s) v_s + g^(t+1) S_{-1}^T q_t. No scale, no normalisation.
 * With lambda = 1 at every level and log_a the same at every token, lla_forward computes the same.
 *
 *   log_a     [H]            fp32   log of each head's decay (<= 0 expected; -inf, a decay of 0, is
 *                                   valid; positive values are computed as given). A constant of the
 *                                   model: lla_linear_backward forms no gradient of it (for learned or
 *                                   per-token decays see lla_backward).
 *   state0    [B0,H,dk,dv]   fp32   S_{-1}, the state that the sequences go on from: B0 = 0 (state0
 *                                   NULL: zeros), 1 (one state for the whole batch, e.g. of a common
 *                                   prefix that was computed once) or B (one each).
 *   state_out [B,H,dk,dv]    fp32   written: S_{T-1}. NULL: not wanted.
 *   q, k [B,H,T,dk], v, out [B,H,T,dv]  dtype, as lla_forward; any T >= 1 (no chunk argument).
 *   Nothing that a call writes may overlap what it reads or writes besides (refused: LLA_ERR_INVALID_ARG),
 *   but for the states that a step updates in place. Prompts: B H (packed: n_seq H) up to 65535.
 *   dk, dv 1..128. bf16 with dk and dv multiples of 8 runs on tensor cores (128-token chunks, bf16
 *   operands, fp32 accumulation, states in fp32); every other shape runs fp32 arithmetic on CUDA
 *   cores. Sums are formed in a fixed order: repeated calls give identical bits.
 * Tokens are mixed in chunks of 128 (64 on CUDA cores): a chunk's tokens out of reach enter its
 * last product with weight 0. So an infinity or NaN in v may reach the other rows of its own chunk,
 * as well as every later row, in its own column; one in k or q obeys causality. Of the gradients,
 * the same goes for one in k and dq, one in q and dk (every earlier row), one in dout and dv (every
 * earlier row), and one in v obeys causality. An infinity may come out as NaN, in a state too. Rows
 * of other sequences (and, packed, rows of no sequence) are never mixed in.
 *
 * lla_linear_forward: prompts of one length.
 *
 * lla_linear_forward_varlen: packed sequences, layout and cu_seqlens rules as lla_forward_varlen:
 *   q, k [H,total_T,dk]; v, out [H,total_T,dv]; state0 [n0,H,dk,dv], n0 in {0, 1, n_seq};
 *   state_out [n_seq,H,dk,dv]. A sequence may be empty: its state_out is its state0 (or zeros).
 *   Rows of out that belong to no sequence are left as they were. A sequence whose bounds break the
 *   rules (cu_seqlens not rising, rows past total_T, more than max_T of them) is skipped, its rows and
 *   state_out left as they were, and lla_device_error reports LLA_ERR_DEVICE. max_T may be any bound of
 *   the lengths, but the cut into segments is made for a sequence of max_T tokens: the nearer it is
 *   to the longest, the faster the call.
 *
 * lla_linear_backward: gradients of sum(dout . out) + sum(dstate_out . state_out).
 *   dout       [B,H,T,dv]   dtype   upstream gradient of out
 *   dstate_out [B,H,dk,dv]  fp32    upstream gradient of state_out; NULL: zeros
 *   dq, dk [B,H,T,dk], dv [B,H,T,dv]  dtype, written
 *   dstate0    [B0,H,dk,dv] fp32    written (B0 = 1: summed over the batch in order); NULL: not wanted
 *   Nothing of the forward is kept: its states are formed again from k, v and state0.
 *
 * lla_linear_decode_step: one token of every sequence; state [B,H,dk,dv] fp32 is read and written in
 *   place (S_{t-1} on entry, S_t on return; what lla_linear_forward leaves in state_out). q, k
 *   [B,H,dk], v, out [B,H,dv] dtype.
 *
 * Workspace comes from the library's stream-ordered pool: at most 0.5 GiB for the pieces of a
 * tensor-core call (gradients keep 256 bytes for each row and 64 columns of v besides); on CUDA
 * cores the states of 64-token chunks, 1 GiB of them or one head's at a time. Errors:
 * LLA_ERR_INVALID_ARG / LLA_ERR_UNSUPPORTED before any launch, LLA_ERR_NOMEM if the pool cannot
 * grow, LLA_ERR_CUDA on a launch failure; a bounded wait that runs out is reported by
 * lla_device_error as LLA_ERR_TIMEOUT.
 */
int lla_linear_forward(const void* q, const void* k, const void* v, const float* log_a, const float* state0, void* out,
                       float* state_out, int B, int B0, int H, int T, int dk, int dv, void* stream, int dtype);
int lla_linear_forward_varlen(const void* q, const void* k, const void* v, const float* log_a, const float* state0,
                              void* out, float* state_out, const int32_t* cu_seqlens, int n_seq, int n0, int H,
                              int total_T, int max_T, int dk, int dv, void* stream, int dtype);
int lla_linear_backward(const void* q, const void* k, const void* v, const float* log_a, const float* state0,
                        const void* dout, const float* dstate_out, void* dq, void* dk, void* dv, float* dstate0, int B,
                        int B0, int H, int T, int dk_, int dv_, void* stream, int dtype);
int lla_linear_decode_step(const void* q, const void* k, const void* v, const float* log_a, float* state, void* out,
                           void* stream, int B, int H, int dk, int dv, int dtype);

/*
 * lla_decode_step for a batch whose sequences all start with the same prefix_len tokens (a system
 * prompt), whose Fenwick states are kept once per head instead of once per sequence. Every aligned
 * block of the prefix's Fenwick walk lies inside one bucket of any later position, so a step is
 *
 *     o_t = sum_l lambda_t^(l) (own^(l))^T q_t + exp(D_t) sum_j lambda_t^(l(t,j)) (prefix^(j))^T q_t
 *
 * with own^(l) the part of bucket l at positions >= prefix_len, j the walk's blocks, and D_t the sum
 * of log_a over the tokens prefix_len..t. The result is lla_decode_step's on the whole states.
 *
 *   q, k, v, log_a, lambda, t, out   as lla_decode_step; t[b] counts from the start of the prefix
 *   prefix_states [H,Lp,dk,dv] fp32  read only: what lla_prefill_state writes for the prefix (B = 1).
 *          Needs Lp >= lla_num_levels(prefix_len); slots that the prefix does not hold are not read.
 *   prefix_len    >= 1               tokens of the prefix (P)
 *   prefix_decay  [B,H]        fp32  D, read (not at t[b] = P, where it counts from 0) and written
 *   fenwick_states [B,H,Lmax,dk,dv] fp32, read and written in place: each sequence's own buckets. Slot
 *          l holds the part of bucket l at positions >= P. Slots without such positions are never read
 *          and may hold anything (so nothing is read at t[b] = P, and no initialisation is needed); a
 *          slot that the carry empties is left as it was.
 *   Needs prefix_len <= t < 2^(Lmax-1); a sequence outside that range is skipped (its states, decay
 *   and output untouched) and LLA_ERR_DEVICE is recorded in the device error word.
 *   After a prompt of n own tokens handled by lla_prefill_state on its own, the states are valid here
 *   where P is a multiple of a power of two >= n (then own levels do not depend on P).
 *   Nothing that is written may overlap another argument (refused: LLA_ERR_INVALID_ARG).
 *   dk 1..256; dv in {16, 32, 64, 128}; Lmax in 1..40. Workspace from the library's pool.
 */
int lla_decode_step_shared(const void* q, const void* k, const void* v, const float* log_a, const float* lambda,
                           const float* prefix_states, int64_t prefix_len, int Lp, float* prefix_decay,
                           float* fenwick_states, const int64_t* t, void* out, void* stream, int B, int H, int dk,
                           int dv, int Lmax, int dtype);

/*
 * The gated linear recurrence: a state per channel, every channel by itself, with a gate for each
 * token and channel (the vector-state layers that models mix with matrix-state ones):
 *
 *     h_t = exp(log_a_t) h_{t-1} + x_t,   h_{-1} = state0
 *
 * Gates of the input (1 - a_t, sqrt(1 - a_t^2) and the like) are the caller's, folded into x.
 *
 *   x, out    [B,T,D]   dtype       any T, D >= 1. Layers with heads: [B,H,T,d] is [B H,T,d], and
 *                                   [B,T,H,d] is [B,T,H d]; to the recurrence all channels are alike.
 *   log_a     [B,T,D]   gate_dtype  log of the gate (<= 0 expected; -inf, a gate of 0, is valid; positive
 *                                   values are computed as given, but where the product of some rows'
 *                                   gates overflows fp32 a NaN may come out). gate_dtype: LLA_F32, or dtype.
 *   state0    [B0,D]    fp32        h_{-1}: B0 = 0 (state0 NULL: zeros), 1 (one for the whole batch) or B.
 *   state_out [B,D]     fp32        written: h_{T-1} before its rounding to dtype. NULL: not wanted.
 * The recurrence is computed in fp32, sums in a fixed order: repeated calls give identical bits. Gates are
 * expf(log_a); those of lla_gated_forward(_varlen) with 16-bit log_a may be off by (1.3 |log_a| + 4) 2^-24 of
 * themselves (log_a's own step is 2^-8 of it), and are 0 below fp32's normal numbers. Channels
 * never mix; within one, an infinity or NaN reaches every later row of its sequence (gradients: every
 * earlier one) and no row of another.
 * Nothing that is written may overlap another argument (refused: LLA_ERR_INVALID_ARG).
 *
 * lla_gated_forward_varlen: packed sequences, x, log_a, out [total_T,D]; cu_seqlens device int32 [n_seq+1],
 *   non-decreasing, 0 <= cu_seqlens[0], cu_seqlens[n_seq] <= total_T. state0 [n0,D], n0 in {0, 1, n_seq};
 *   state_out [n_seq,D]. A sequence may be empty: its state_out is its state0 (or zeros). Rows of out that
 *   belong to no sequence are left as they were. Where cu_seqlens breaks these rules the call writes nothing
 *   and lla_device_error reports LLA_ERR_DEVICE.
 *
 * lla_gated_backward(_varlen): gradients of sum(dout . out) + sum(dstate_out . state_out).
 *   out        the forward's outputs as it left them (no x is needed: with F_t the gradient that reaches
 *              h_{t-1}, dlog_a_t = F_t h_{t-1}). In bf16 that h is the rounded one: dlog_a is exact for the
 *              outputs given, 2^-8 of each value from that of the unrounded states at most.
 *   dout       like out;  dstate_out [B,D] fp32, NULL: zeros
 *   dx         [B,T,D] dtype, dlog_a [B,T,D] gate_dtype: written (packed: 0 for rows of no sequence)
 *   dstate0    [B0,D] fp32, written (B0 = 1: summed over the batch in order); NULL: not wanted
 *
 * lla_gated_decode_step: one token of every sequence; x, log_a, out [B,D], state [B,D] fp32 read and written
 *   in place (h_{t-1} on entry, h_t on return; what the prompt left in state_out).
 *
 * Limits: rows x D up to 2^40, D up to 2^30; T (packed: total_T) up to 2^31 - 2^16. Workspace: only for dstate0 with B0 = 1
 * (B D floats, the library's pool). A bounded wait that runs out is reported by lla_device_error as
 * LLA_ERR_TIMEOUT. Fastest where rows of x and log_a are multiples of 16 bytes (copied by TMA); then where D is
 * a multiple of 4.
 */
int lla_gated_forward(const void* x, const void* log_a, const float* state0, void* out, float* state_out, int B, int B0,
                      int T, int D, void* stream, int dtype, int gate_dtype);
int lla_gated_forward_varlen(const void* x, const void* log_a, const float* state0, void* out, float* state_out,
                             const int32_t* cu_seqlens, int n_seq, int n0, int total_T, int D, void* stream, int dtype,
                             int gate_dtype);
int lla_gated_backward(const void* log_a, const void* out, const float* state0, const void* dout,
                       const float* dstate_out, void* dx, void* dlog_a, float* dstate0, int B, int B0, int T, int D,
                       void* stream, int dtype, int gate_dtype);
int lla_gated_backward_varlen(const void* log_a, const void* out, const float* state0, const void* dout,
                              const float* dstate_out, void* dx, void* dlog_a, float* dstate0,
                              const int32_t* cu_seqlens, int n_seq, int n0, int total_T, int D, void* stream, int dtype,
                              int gate_dtype);
int lla_gated_decode_step(const void* x, const void* log_a, float* state, void* out, void* stream, int B, int D,
                          int dtype, int gate_dtype);

/*
 * Drafted tokens (speculative decoding). A draft is a tree of N tokens: parent[i] < i is the node that node i
 * goes on from, or -1 for the last token that the states hold; -2 marks a place without a node (trees of
 * different sizes in one batch), which no node may name. A tree call computes the outputs of all nodes from
 * states that it only reads: what decode steps along each branch would give, with no copy of the states and
 * nothing to take back. A commit then appends the accepted tokens to the states in one pass: what a decode
 * step for each would leave.
 *
 *   parent [BP,N] int32, device: BP = 1 (one tree for the whole batch) or B. A sequence whose tree breaks the
 *          rules is skipped (its rows of out left as they were) and LLA_ERR_DEVICE is recorded. Rows of out of
 *          places without a node are left as they were, their inputs not used.
 *   count  [B] int32, device: accepted tokens of every sequence, 0 .. M (0: its states are left as they were).
 *   path   [B,M] int32, device: their node indexes in order (entries past count are not read; the same node
 *          twice is its token twice). NULL, with M = 0: the tokens 0 .. count-1, count <= N (a chain, or a
 *          few tokens at a time). A count or index out of range: that sequence is skipped, LLA_ERR_DEVICE.
 *   N, M 1..128.
 *
 * lla_decode_tree: node i at depth d_i (0 below parent -1) is the token at position t + d_i; its output is
 * lla_decode_step's after the nodes above it.
 *   q, k [B,H,N,dk], v, out [B,H,N,dv] dtype; log_a [B,H,N], lambda [B,H,N,Lmax] fp32
 *   fenwick_states [B,H,Lmax,dk,dv] fp32, read: tokens 0 .. t-1, as lla_decode_step takes them
 *   t [B] int64, device: needs 0 <= t and t + d_i < 2^(Lmax-1) (else skipped, LLA_ERR_DEVICE)
 * lla_decode_commit: the states after the accepted tokens t .. t + count - 1; t is not advanced. Slots that the
 *   last of them leaves empty stay as they were. Needs 0 <= t and t + count <= 2^(Lmax-1).
 * lla_linear_decode_tree, lla_linear_decode_commit: the same for lla_linear_decode_step; log_a [H] fp32,
 *   state [B,H,dk,dv] fp32.
 *   dk, dv 1..128; Lmax 1..40. Products with the states run on tensor cores: bf16 queries as they are, states
 *   in two bf16 parts (2^-16 of each element), fp32 calls in three parts of both; sums in fp32 in a fixed order
 *   (repeated calls give identical bits; a call of fewer heads may cut its sums otherwise). An infinity in the
 *   states, or a gate that is infinite in fp32, may come out as NaN; one in a node reaches only that node's and its
 *   descendants' outputs.
 * lla_gated_decode_tree, lla_gated_decode_commit: the same for lla_gated_decode_step; x, log_a, out [B,N,D],
 *   state [B,D] fp32; B up to 65535. (h of a node: exp(log_a_i) h_parent(i) + x_i.)
 *
 * Nothing that is written may overlap another argument (refused: LLA_ERR_INVALID_ARG). No workspace.
 */
int lla_decode_tree(const void* q, const void* k, const void* v, const float* log_a, const float* lambda,
                    const float* fenwick_states, const int64_t* t, const int32_t* parent, void* out, void* stream, int B,
                    int BP, int H, int N, int dk, int dv, int Lmax, int dtype);
int lla_decode_commit(const void* k, const void* v, const float* log_a, float* fenwick_states, const int64_t* t,
                      const int32_t* count, const int32_t* path, void* stream, int B, int H, int N, int M, int dk, int dv,
                      int Lmax, int dtype);
int lla_linear_decode_tree(const void* q, const void* k, const void* v, const float* log_a, const float* state,
                           const int32_t* parent, void* out, void* stream, int B, int BP, int H, int N, int dk, int dv,
                           int dtype);
int lla_linear_decode_commit(const void* k, const void* v, const float* log_a, float* state, const int32_t* count,
                             const int32_t* path, void* stream, int B, int H, int N, int M, int dk, int dv, int dtype);
int lla_gated_decode_tree(const void* x, const void* log_a, const float* state, const int32_t* parent, void* out,
                          void* stream, int B, int BP, int N, int D, int dtype, int gate_dtype);
int lla_gated_decode_commit(const void* x, const void* log_a, float* state, const int32_t* count, const int32_t* path,
                            void* stream, int B, int N, int M, int D, int dtype, int gate_dtype);

/*
 * Test hook for the failure path of the bounded waits (no counterpart on the
 * pages; not for production use). On the current device, for the tensor-core
 * prefill output kernel of dv = 64, the tensor-core kernels of linear
 * attention, the passes of the gated recurrence and the tree kernels whose states come by TMA (dv a
 * multiple of 4): limit_cycles > 0 bounds each of its pipeline
 * waits to that many SM cycles (<= 0 restores the default, about 2 s at the
 * maximum clock); hold != 0 makes its epilogue (where only states are formed,
 * the warps that hold the state) first wait on a barrier that nothing arrives
 * at, so that wait runs out. The kernel then records
 * LLA_ERR_TIMEOUT in the device error word, lets its own in-flight copies and
 * MMAs land (those drain waits keep the full bound), frees its tensor memory and
 * returns; the call's output is then undefined. Synchronous with the host; takes
 * effect for kernels launched afterwards. Returns LLA_OK or LLA_ERR_CUDA.
 */
int lla_debug_set_waits(int64_t limit_cycles, int hold);

/*
 * Reads and clears the device error word of the current device after
 * synchronising `stream`: LLA_OK if no kernel recorded a fault since the last
 * read, LLA_ERR_DEVICE for rejected device-side input, LLA_ERR_TIMEOUT for a
 * bounded wait that ran out, LLA_ERR_CUDA if the synchronisation itself failed.
 */
int lla_device_error(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LLA_H */
