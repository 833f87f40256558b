/*
 * moe_route.h -- C ABI of the GB300 (sm_103a) MoE routing library
 * (libmoe_route_gb300.so): route -> dispatch -> permute -> combine on one GPU.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - All tensor arguments are DEVICE pointers to row-major, contiguous
 *    buffers that the caller owns.  The library allocates and frees nothing,
 *    keeps no per-call state between calls and may be called from several
 *    host threads at once (each call only touches its own arguments).  Calls
 *    that may run at the same time on the GPU (other streams, other threads)
 *    must not share a dispatch workspace: it holds grid-barrier counters.
 *  - Every call is asynchronous on `stream` (a cudaStream_t; NULL = the
 *    legacy default stream) and never synchronises the host, so a sequence
 *    of calls can be captured into a CUDA graph.
 *  - Argument errors are found on the host before anything is launched; the
 *    call then returns a non-zero moe_status and launches nothing.  A failed
 *    launch returns MOE_ERR_CUDA.
 *  - Errors that only the device can see (an expert index outside [0,E), a
 *    bounded wait that ran out) are recorded in `status_word` (one int32 in
 *    device memory, may be NULL): the first error code is stored with an
 *    atomic compare-and-swap over 0, so the caller zeroes the word before the
 *    call and reads it after synchronising.  No kernel traps or asserts.
 *  - bf16 buffers are passed as `void*` (IEEE bfloat16 bit patterns).
 *  - Pointers must be 16-byte aligned; H must be a multiple of 8.
 *  - Cache use: outputs that fit in 5/8 of the GPU's L2 (the row copies,
 *    E4M3 codes and combine outputs) are stored with the default write-back
 *    policy, so that the kernel that reads them next finds them in L2; larger
 *    ones are streamed through it (evict-first).  The router leaves X in L2
 *    the same way when X fits, for the row copy that reads it again.
 *
 * Notation: N tokens, H hidden size, E experts, K experts per token,
 * slot s = n*K + k.  Limits: 1 <= E <= 256, 1 <= K <= min(E, 16),
 * N*K < 2^31, N >= 0 (N == 0 is a no-op that returns MOE_OK).
 */
#ifndef MOE_ROUTE_GB300_H
#define MOE_ROUTE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define MOE_API __attribute__((visibility("default")))
#else
#define MOE_API
#endif

/* Same object as cudaStream_t. */
typedef struct CUstream_st *moe_stream_t;

typedef enum moe_status {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,   /* a NULL required pointer, a size out of range */
    MOE_ERR_UNSUPPORTED = 2,   /* a valid request this build does not implement */
    MOE_ERR_MISALIGNED = 3,    /* a pointer not 16-byte aligned, H % 8 != 0 */
    MOE_ERR_WORKSPACE = 4,     /* workspace smaller than moe_dispatch_workspace_size() */
    MOE_ERR_CUDA = 5,          /* a CUDA runtime call or launch failed */
    MOE_ERR_TIMEOUT = 6,       /* (status_word only) a bounded device wait ran out */
    MOE_ERR_BAD_INDEX = 7,     /* (status_word only) topk_idx entry outside [0,E) */
    MOE_ERR_BAD_SCALE = 8      /* (status_word only) fp32 block scale not a power of two */
} moe_status;

/* Format of the E4M3 block scales (moe_dispatch_ex, moe_permute_ex). */
typedef enum moe_scale_format {
    MOE_SCALE_FP32 = 0,        /* fp32 [N*K, H/128]: the power-of-two scale s itself */
    MOE_SCALE_UE8M0 = 1        /* uint8 [N*K, H/128]: UE8M0 byte b, s = 2^(b - 127) */
} moe_scale_format;

/* Router implementation selector for moe_route_ex. */
typedef enum moe_route_algo {
    MOE_ROUTE_AUTO = 0,        /* tensor-core kernel where the shape allows it */
    MOE_ROUTE_TCGEN05 = 1,     /* tcgen05.mma + TMEM + TMA kernel (E % 8 == 0) */
    MOE_ROUTE_SIMT = 2         /* CUDA-core kernel, any E */
} moe_route_algo;

/*
 * moe_route -- the fused router.
 * Defined by the moe-engine page ("moe-engine：面向万卡集群的稀疏MoE训练基础设施"),
 * section 融合Triton路由内核: tokens @ gate_w -> softmax -> top-K -> renorm,
 * with K-round selection.  For every token n:
 *   L[e]   = sum_h X[n,h] * W_gate[h,e] (+ bias[e])    bf16 x bf16, fp32 accumulate
 *   p[e]   = softmax_e(L)[e]                          fp32
 *   idx    = the K experts with the largest logits, in descending order;
 *            equal logits go to the lower expert index; NaN counts as -inf
 *   w_k    = p[idx_k] / sum_j p[idx_j]  if renorm,  else  p[idx_k]
 * Arguments:
 *   X          bf16 [N,H]          token activations (read once)
 *   W_gate     bf16 [H,E]          gate weight, row-major ("tokens @ gate_w")
 *   bias       fp32 [E] or NULL    per-expert logit bias added before softmax
 *   topk_idx   int32 [N,K]         out: selected experts per token
 *   topk_w     fp32 [N,K]          out: routing weights
 *   status_word int32 [1] or NULL  device error word (MOE_ERR_TIMEOUT)
 * Errors: MOE_ERR_INVALID_ARG (NULL X/W_gate/outputs with N > 0, E or K out
 * of range), MOE_ERR_MISALIGNED, MOE_ERR_CUDA.
 */
MOE_API moe_status moe_route(const void *X, const void *W_gate, const float *bias,
                     int64_t N, int H, int E, int K, int renorm,
                     int32_t *topk_idx, float *topk_w, int32_t *status_word,
                     moe_stream_t stream);

/* moe_route with an explicit implementation; MOE_ERR_UNSUPPORTED if the
 * requested kernel cannot take this shape (MOE_ROUTE_TCGEN05 needs E % 8 == 0
 * and a GPU of compute capability 10.x). */
MOE_API moe_status moe_route_ex(const void *X, const void *W_gate, const float *bias,
                        int64_t N, int H, int E, int K, int renorm,
                        int32_t *topk_idx, float *topk_w, int32_t *status_word,
                        int algo, moe_stream_t stream);

/*
 * moe_route_stats -- moe_route_ex with the router statistics of the
 * moe-engine page (section 专家负载均衡) taken in the same pass:
 *   lse[n]           = log(sum_e exp(L[n,e]))   fp32 [N] or NULL: the per-token
 *                      logsumexp a z-loss squares (-inf for a token whose
 *                      logits are all -inf or NaN)
 *   expert_counts[e] = #{(n,k) : topk_idx[n,k] == e}   int32 [E] or NULL:
 *                      the expert histogram, counted in the router's epilogue
 *                      (the same values moe_dispatch writes)
 * expert_counts is overwritten (set to zero on `stream`, then accumulated by
 * the kernel).  Other arguments, layout and errors as moe_route_ex.
 */
MOE_API moe_status moe_route_stats(const void *X, const void *W_gate, const float *bias,
                           int64_t N, int H, int E, int K, int renorm,
                           int32_t *topk_idx, float *topk_w, float *lse,
                           int32_t *expert_counts, int32_t *status_word,
                           int algo, moe_stream_t stream);

/*
 * moe_load_stats -- expert-load statistics from the counts (and optionally the
 * logsumexp values) of moe_route_stats, in one small kernel:
 *   stats[0] = max_e counts[e] / mean              (imbalance ratio)
 *   stats[1] = P95(counts) / mean, P95 by linear interpolation between the
 *              sorted counts at position 0.95 * (E - 1)
 *   stats[2] = z_coef * (1/N) * sum_n lse[n]^2      (0 if lse is NULL or N == 0)
 *   stats[3] = mean = sum_e counts[e] / E
 * The ratios are 0 when every count is 0.  The sum of lse^2 is deterministic:
 * each of 1024 threads sums a fixed set of the squares in a fixed order in
 * Kahan-compensated fp32, and the 1024 per-thread sums are then added in fp64
 * in a fixed order; the count sums are exact integers.  counts int32 [E]
 * (1 <= E <= 256), lse fp32 [N] or NULL, stats fp32 [4] (all device memory).
 * Errors: MOE_ERR_INVALID_ARG (NULL counts or stats, E out of range, N < 0),
 * MOE_ERR_MISALIGNED, MOE_ERR_CUDA.
 */
MOE_API moe_status moe_load_stats(const int32_t *expert_counts, int E, const float *lse, int64_t N,
                          float z_coef, float *stats, moe_stream_t stream);

/* Bytes of device workspace moe_dispatch needs for these sizes (0 means the
 * workspace pointer may be NULL). */
MOE_API size_t moe_dispatch_workspace_size(int64_t N, int E, int K);

/*
 * moe_dispatch -- counting-sort dispatch into an expert-contiguous buffer.
 * Defined by the PithTrain page ("一万行Python构建MoE训练栈：解构4D并行、
 * DualPipeV调度与FP8算子"), §8.2 O(n) counting sort 替代 O(n log n) argsort
 * (bincount with private histograms -> prefix sum -> scatter with
 * expand_idx), specialised to one GPU (no expert-parallel ranks, no
 * all-to-all), and by the moe-engine page's conservation check
 * sum(dispatch_cnt) == N*K (section 实验结果与性能数据 / Token守恒验证).
 *   expert_counts[e]  = #{slots s : topk_idx[s] == e}
 *   expert_offsets[e] = sum_{e' < e} expert_counts[e'],  expert_offsets[E] = N*K
 *   row_map[s]        = the row of slot s in the expert-contiguous buffer;
 *                       rows are ordered by (expert, s): the stable argsort
 *                       of the slots by expert
 *   src_slot[r]       = the slot whose row is r (inverse of row_map)
 * and, when X is given, the row permute of moe_permute below.
 * Arguments:
 *   topk_idx        int32 [N,K]     expert ids (from moe_route or the caller)
 *   X               bf16 [N,H] or NULL   NULL: metadata only
 *   expert_counts   int32 [E]       out
 *   expert_offsets  int32 [E+1]     out
 *   row_map         int32 [N*K]     out
 *   src_slot        int32 [N*K] or NULL   out
 *   X_perm          bf16 [N*K,H] or NULL  out (needs X)
 *   X_fp8           uint8 [N*K,H] or NULL out, E4M3 codes (needs X, H % 128 == 0)
 *   X_scale         fp32 [N*K,H/128] or NULL  out, with X_fp8
 *   status_word     int32 [1] or NULL  device error word (MOE_ERR_BAD_INDEX)
 *   workspace       device scratch of moe_dispatch_workspace_size() bytes
 * An index outside [0,E) is reported in status_word; the outputs are then
 * unspecified but every write stays inside the buffers described above.
 * Launches: with a workspace, one cooperative launch counts, scans, scatters
 * and copies the rows; when the row copy moves 256 MiB or more (X read once
 * plus the rows written) the copy runs as a second launch of the permute
 * kernel instead.  Without a workspace: one cluster launch for the metadata,
 * then the permute kernel.
 */
MOE_API moe_status moe_dispatch(const int32_t *topk_idx, const void *X,
                        int64_t N, int H, int E, int K,
                        int32_t *expert_counts, int32_t *expert_offsets,
                        int32_t *row_map, int32_t *src_slot,
                        void *X_perm, void *X_fp8, float *X_scale,
                        int32_t *status_word,
                        void *workspace, size_t workspace_bytes,
                        moe_stream_t stream);

/*
 * moe_dispatch_ex -- moe_dispatch with a choice of block-scale format for the
 * E4M3 copy.  The PithTrain page (§7.2 架构感知的量化核, _compute_fp8_scale)
 * gives two branches of the scale rule: fp32 scales (the bit rule quoted at
 * moe_permute below) and, on Blackwell, E8M0 scales -- the same fp32 product
 * t = fl32(max(amax, 1e-4) * fl32(1/448)) converted with round-toward-+inf to
 * an unsigned 8-bit exponent (cvt.rp.satfinite.ue8m0x2.f32).  Both give the
 * same power-of-two s and hence the same E4M3 codes; MOE_SCALE_UE8M0 stores
 * one byte b per block (s = 2^(b - 127)) instead of a float.
 *   X_scale      fp32 [N*K, H/128] (MOE_SCALE_FP32, 4-byte aligned) or
 *                uint8 [N*K, H/128] (MOE_SCALE_UE8M0), with X_fp8; or NULL
 *   scale_format a moe_scale_format; anything else is MOE_ERR_INVALID_ARG
 * Every other argument, and the errors, as moe_dispatch.
 */
MOE_API moe_status moe_dispatch_ex(const int32_t *topk_idx, const void *X,
                           int64_t N, int H, int E, int K,
                           int32_t *expert_counts, int32_t *expert_offsets,
                           int32_t *row_map, int32_t *src_slot,
                           void *X_perm, void *X_fp8, void *X_scale, int scale_format,
                           int32_t *status_word,
                           void *workspace, size_t workspace_bytes,
                           moe_stream_t stream);

/*
 * moe_route_dispatch -- moe_route_ex (MOE_ROUTE_AUTO) followed by
 * moe_dispatch_ex of its own top-K ids with a bf16 row copy: the router of the
 * moe-engine page (融合Triton路由内核) and the counting sort of the PithTrain
 * page (§8.2), with the same outputs as the two calls.  Where the tensor-core
 * router runs in its split-K mode (few tokens: every CTA resident at once) the
 * whole path is ONE cooperative launch: each CTA, after its top-K epilogue,
 * counts its own slots, a bounded grid barrier follows, and every CTA then
 * forms the offsets, writes row_map for its slots and copies its tokens' rows
 * (from L2, where the router just streamed them).  Otherwise (a row copy of
 * more than 64 MiB included), or where the cooperative launch is refused, the
 * two calls run one after the other.
 *   X, W_gate, bias, renorm, topk_idx, topk_w   as moe_route
 *   expert_counts, expert_offsets, row_map, src_slot   as moe_dispatch
 *   X_perm       bf16 [N*K, H], 16-byte aligned, or NULL (metadata only)
 *   workspace    at least moe_dispatch_workspace_size(N, E, K) bytes, 256-byte
 *                aligned, zero before the first call (left zero by every call
 *                that did not time out)
 *   launches     host int or NULL: out, the number of kernels this call launched
 * Errors: those of moe_route_ex and moe_dispatch_ex; MOE_ERR_WORKSPACE when the
 * workspace is missing or too small.  The status word receives MOE_ERR_TIMEOUT
 * if the grid barrier ran out (the workspace must then be zeroed before it is
 * used again).  A split-K launch whose clusters were dropped (a profiler may run
 * a cooperative cluster launch that way) still gives the same outputs: each CTA
 * then takes the whole H range of its tile and touches no other CTA's memory.
 * The one launch is cooperative.  With the environment variable
 * MOE_FUSED_LAUNCH=noncooperative (read once per process) it is launched
 * without that attribute, for profilers that run cooperative cluster launches
 * without clusters; every CTA is then still resident at once on an otherwise
 * idle GPU (the launch is planned as one wave), but that is not guaranteed.
 */
MOE_API moe_status moe_route_dispatch(const void *X, const void *W_gate, const float *bias,
                              int64_t N, int H, int E, int K, int renorm,
                              int32_t *topk_idx, float *topk_w,
                              int32_t *expert_counts, int32_t *expert_offsets,
                              int32_t *row_map, int32_t *src_slot, void *X_perm,
                              int32_t *status_word, void *workspace, size_t workspace_bytes,
                              int *launches, moe_stream_t stream);

/*
 * moe_dispatch_ep -- expert-parallel dispatch metadata with token
 * deduplication for the tokens of one GPU: the metadata of
 * fused_dedup_prepare_dispatch on the PithTrain page (§8.2 O(n) counting sort
 * 替代 O(n log n) argsort: counts per expert and per EP rank, prefix sums,
 * send metadata, dedup scatter, counting sort, expand_idx).  The all-to-all
 * that moves the rows between GPUs is not part of this library.
 * The E experts are split over R = ep_size ranks, P = E / R consecutive
 * experts each (rank(e) = e / P).  A token is sent to a rank once, however
 * many of its K experts live there.
 *   expert_counts, expert_offsets, row_map   as moe_dispatch (int32 [E], [E+1], [N*K])
 *   rank_counts[r]    int32 [R]: tokens sent to rank r (deduplicated)
 *   rank_offsets[r]   int32 [R+1]: exclusive prefix, rank_offsets[R] = send rows
 *   send_token[row]   int32 [N*min(K,R)]: the token of send row `row`; rows are
 *                     ordered by (rank, token)
 *   slot_send_row[s]  int32 [N*K]: the send row carrying the token of slot s to
 *                     the rank of its expert
 *   expand_idx[q]     int32 [N*K]: for row q of the expert-contiguous order
 *                     (slot s), the index of s's token among its rank's send
 *                     rows: slot_send_row[s] - rank_offsets[rank(topk_idx[s])]
 *                     (what the receiving rank gathers its expert rows by)
 *   send_meta         int32 [R, P+1]: per rank, the dedup token count, then the
 *                     slot count of each of its P experts
 *   X_send            bf16 [N*min(K,R), H] or NULL: X_send[row] = X[send_token[row]]
 *                     (needs X)
 *   workspace         as moe_dispatch (moe_dispatch_workspace_size(N, E, K) bytes)
 * Three launches on `stream`.  Errors: as moe_dispatch; MOE_ERR_INVALID_ARG
 * if ep_size < 1, ep_size > E or E % ep_size != 0; MOE_ERR_UNSUPPORTED beyond
 * the one-launch dispatch's size limit (the workspace is required).  An expert
 * index outside [0,E) is reported in status_word; its slot gets no rows.
 */
MOE_API moe_status moe_dispatch_ep(const int32_t *topk_idx, const void *X,
                           int64_t N, int H, int E, int K, int ep_size,
                           int32_t *expert_counts, int32_t *expert_offsets, int32_t *row_map,
                           int32_t *rank_counts, int32_t *rank_offsets,
                           int32_t *send_token, int32_t *slot_send_row, int32_t *expand_idx,
                           int32_t *send_meta, void *X_send, int32_t *status_word,
                           void *workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * moe_dispatch_noalloc -- moe_dispatch without a caller-provided workspace.
 * The pages have no counterpart: this is a convenience of this library for
 * callers that cannot allocate device memory when they dispatch -- engines that
 * fix their whole device-memory plan up front and forbid later allocation,
 * code running where cudaMalloc would block or synchronise the device, or C
 * callers with no device allocator of their own.  The inputs and outputs are
 * still the caller's (same meaning as in moe_dispatch); the scratch is a
 * 1 MiB + 256 B array compiled into the library, which every GPU that loads
 * the library holds until the process exits.  The call allocates and frees
 * nothing.
 *  - The first call on each device looks up the array's device address
 *    (with that device current) and caches it; make that first call before
 *    any stream capture.
 *  - Every call clears the array's barrier counters on `stream` and then uses
 *    the whole array: calls that may overlap on the GPU (other streams, other
 *    host threads) race on it and must be serialised by the caller.
 *  - Limit: the launch takes C = min(N, number of SMs) CTAs, each with
 *    ceil(N / C) tokens, and a CTA holds at most 16384 slots, so the call
 *    needs ceil(N / C) * K <= 16384 (on a 152-SM GB300 with K = 3: up to
 *    N = 830072); larger calls return MOE_ERR_UNSUPPORTED and launch nothing.
 *  - Every argument check of moe_dispatch runs on the host before any CUDA
 *    call: a rejected call queues nothing on `stream`.
 */
MOE_API moe_status moe_dispatch_noalloc(const int32_t *topk_idx, const void *X,
                                int64_t N, int H, int E, int K,
                                int32_t *expert_counts, int32_t *expert_offsets,
                                int32_t *row_map, int32_t *src_slot,
                                void *X_perm, void *X_fp8, float *X_scale,
                                int32_t *status_word, moe_stream_t stream);

/*
 * moe_permute -- the row permute of the dispatch, on its own.
 * The gathered_tokens input of forward_mlp on the PithTrain page
 * (§6.1 模型协议先行): X_perm[row_map[n*K+k], :] = X[n, :].
 * With X_fp8/X_scale (H % 128 == 0) every 1x128 block of X[n,:] is also
 * quantised with the power-of-two scale of §7.2 架构感知的量化核
 * (_compute_fp8_scale, fp32-scale branch):
 *   s = pow2ceil(fl32(max(amax, 1e-4) * fl32(1/448))),  q = E4M3_rn_satfinite(x / s)
 * and q, s are written for every destination row of the token.
 * row_map must be a permutation of [0, N*K) (as moe_dispatch writes it);
 * rows outside [0, N*K) are skipped and reported as MOE_ERR_BAD_INDEX.
 * X_perm may be NULL when only the E4M3 copy is wanted.
 */
MOE_API moe_status moe_permute(const void *X, const int32_t *row_map,
                       int64_t N, int H, int K,
                       void *X_perm, void *X_fp8, float *X_scale,
                       int32_t *status_word, moe_stream_t stream);

/* moe_permute with a choice of block-scale format (see moe_dispatch_ex). */
MOE_API moe_status moe_permute_ex(const void *X, const int32_t *row_map,
                          int64_t N, int H, int K,
                          void *X_perm, void *X_fp8, void *X_scale, int scale_format,
                          int32_t *status_word, moe_stream_t stream);

/*
 * moe_combine -- weighted gather back to token order.
 * The weighted part of forward_aggregate on the PithTrain page (§6.1
 * 模型协议先行, "weighted expert output"):
 *   out[n,:] = sum_{k=0}^{K-1} topk_w[n,k] * Y[row_map[n*K+k], :]
 * accumulated in fp32 in k order and rounded to bf16 (nearest even).
 * Arguments: Y bf16 [N*K,H] (expert outputs in the expert-contiguous order),
 * row_map int32 [N*K], topk_w fp32 [N,K], out bf16 [N,H].
 * Rows outside [0, N*K) contribute nothing and are reported as
 * MOE_ERR_BAD_INDEX in status_word.
 */
MOE_API moe_status moe_combine(const void *Y, const int32_t *row_map, const float *topk_w,
                       int64_t N, int H, int K, void *out,
                       int32_t *status_word, moe_stream_t stream);

/*
 * moe_combine_residual -- moe_combine plus the residual connection: the whole
 * of forward_aggregate on the PithTrain page (§6.1 模型协议先行, "weighted
 * expert output + residual connection"), fused into the same pass:
 *   out[n,:] = sum_{k=0}^{K-1} topk_w[n,k] * Y[row_map[n*K+k], :] + residual[n,:]
 * with the weighted sum accumulated in fp32 in k order, the residual added in
 * fp32, and one rounding to bf16 (nearest even).
 * Arguments: as moe_combine, plus residual bf16 [N,H] (required, 16-byte
 * aligned).  out may be the residual buffer itself (in-place update of the
 * residual stream); any other overlap of out with Y or residual is undefined.
 * Errors: as moe_combine; a NULL residual with N > 0 is MOE_ERR_INVALID_ARG.
 */
MOE_API moe_status moe_combine_residual(const void *Y, const int32_t *row_map, const float *topk_w,
                                const void *residual, int64_t N, int H, int K, void *out,
                                int32_t *status_word, moe_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * The experts: what runs between dispatch and combine.
 *
 * E4M3 operands carry one power-of-two scale per block, as moe_dispatch_ex writes
 * them: 1x128 blocks for rows ([R, C/128]), 128x128 blocks for weights
 * ([E, ceil(rows/128), ceil(cols/128)], the last blocks cut at the edges), in
 * either moe_scale_format.  A value is code * scale.  An fp32 scale that is not a
 * positive normal power of two is reported as MOE_ERR_BAD_SCALE in status_word
 * (its exponent is used).  A NaN code, and UE8M0's NaN 255, give NaN results.  The
 * quantisers leave NaNs out of a block's maximum and write them as NaN codes; a block
 * with an infinity gets the largest scale, NaN codes for the infinities and zeros.
 * expert_offsets is moe_dispatch's: int32 [E+1], the rows of expert e are
 * [offsets[e], offsets[e+1]); a group may be empty.  NULL with E = 1 means one group
 * of all R rows (a plain product).  A group that is not inside [0, R] or runs
 * backwards is treated as empty and reported as MOE_ERR_BAD_INDEX; no access leaves
 * the buffers.  All calls need a GPU of compute capability 10.x
 * (MOE_ERR_UNSUPPORTED elsewhere).
 * ---------------------------------------------------------------------------
 */

/*
 * moe_quantize_weight -- E4M3 weights from bf16 ones:
 *   s = pow2ceil(fl32(max(amax of the 128x128 block, 1e-4) * fl32(1/448)))
 *   W_fp8 = E4M3_rn_satfinite(W / s)
 *   W bf16 [E, rows, cols], W_fp8 uint8 [E, rows, cols], W_scale as above
 * E in 1..256, rows in 1..2^22, cols % 8 == 0.  One launch.
 */
MOE_API moe_status moe_quantize_weight(const void *W, int E, int rows, int cols, void *W_fp8, void *W_scale,
                               int scale_format, moe_stream_t stream);

/*
 * moe_expert_gemm -- the experts' products, rows times weights (W is [E, rows, cols]):
 *   transpose == 0:  Y[r, m] = sum_k x[r,k] W[e(r), m, k]    x [R, cols], Y [R, rows]
 *   transpose != 0:  Y[r, k] = sum_m x[r,m] W[e(r), m, k]    x [R, rows], Y [R, cols]
 * (the second is the gradient with respect to the first one's x).  fp32
 * accumulation over the whole reduction in the tensor cores, which cut where they add
 * (2^18 positive products: 3e-4 of their sum), one rounding to bf16.
 *   X_fp8 uint8 [R, red], X_scale [R, red/128], W_fp8 uint8 [E, rows, cols], W_scale
 *   Y bf16; rows of no group are left as they are
 * The reduction (cols, or rows when transposed) is a multiple of 128, the other
 * side of 16, both at most 2^18.  R == 0 is a no-op.  One launch.
 * Errors: MOE_ERR_INVALID_ARG (sizes, NULLs, expert_offsets NULL with E > 1),
 * MOE_ERR_MISALIGNED, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA.
 */
MOE_API moe_status moe_expert_gemm(const void *X_fp8, const void *X_scale, int x_scale_format,
                           const void *W_fp8, const void *W_scale, int w_scale_format,
                           const int32_t *expert_offsets, int64_t R, int E, int rows, int cols, int transpose,
                           void *Y, int32_t *status_word, moe_stream_t stream);

/*
 * moe_expert_wgrad -- the weight gradient of moe_expert_gemm (transpose == 0), from
 * the E4M3 rows that went into it:
 *   dW[e, m, k] = add[e, m, k] + sum_{r in group e} dY[r, m] * x[r, k]
 *   dY bf16 [R, rows], X_fp8 uint8 [R, cols], X_scale [R, cols/128]
 *   add fp32 [E, rows, cols] or NULL (nothing is added); may be dW itself when that is fp32
 *   dW  fp32 (dw_bf16 == 0) or bf16 [E, rows, cols]; an empty group gives add, or zeros
 * x is a bf16 number exactly (an E4M3 value times a power of two), the products are
 * accumulated in fp32: segments of 2048 rows (bf16 result: 16384) in the tensor cores,
 * which cut where they add, the segments of a longer group rounding to nearest.
 * rows % 8 == 0, cols % 128 == 0, both at most 2^18.  One launch.
 */
MOE_API moe_status moe_expert_wgrad(const void *dY, const void *X_fp8, const void *X_scale, int x_scale_format,
                            const int32_t *expert_offsets, int64_t R, int E, int rows, int cols,
                            const float *add, void *dW, int dw_bf16, int32_t *status_word, moe_stream_t stream);

/*
 * moe_swiglu -- the gated activation between the two products:
 *   GU bf16 [R, 2I]: gate columns, then up columns;  a = g / (1 + exp(-g)) * u
 *   A_fp8 uint8 [R, I], A_scale [R, I/128]: a in E4M3 (the rule of moe_permute)
 *   GU_fp8 uint8 [R, 2I], GU_scale [R, 2I/128], or both NULL: GU in E4M3, the
 *   checkpoint that moe_swiglu_backward reads instead of GU
 * I % 128 == 0, I <= 2^20, R * I / 128 < 2^36.  One launch.
 */
MOE_API moe_status moe_swiglu(const void *GU, int64_t R, int I, void *A_fp8, void *A_scale,
                      void *GU_fp8, void *GU_scale, int scale_format, moe_stream_t stream);

/*
 * moe_swiglu_backward -- its gradient, from the E4M3 checkpoint:
 *   s = 1 / (1 + exp(-g));  dg = da u s (1 + g (1 - s));  du = da g s
 *   dA bf16 [R, I], GU_fp8 and GU_scale (gu_scale_format) as moe_swiglu wrote them
 *   dGU bf16 [R, 2I] or NULL (what moe_expert_wgrad reads)
 *   dGU_fp8, dGU_scale (scale_format) or both NULL (what the transposed
 *   moe_expert_gemm reads); quantised from the unrounded gradient
 * One of the two outputs is required.  One launch.
 */
MOE_API moe_status moe_swiglu_backward(const void *dA, const void *GU_fp8, const void *GU_scale, int gu_scale_format,
                               int64_t R, int I, void *dGU, void *dGU_fp8, void *dGU_scale, int scale_format,
                               int32_t *status_word, moe_stream_t stream);

/*
 * moe_expert_swiglu -- both projections, the activation and their product in one launch:
 *   gu[r] = x[r] W1[e(r)]^T (fp32: g, then u);  a = g / (1 + exp(-g)) * u
 *   X_fp8 uint8 [R, H], X_scale [R, H/128]; W1_fp8 uint8 [E, 2I, H] (gate rows, then up rows), W1_scale
 *   A_fp8, A_scale; GU_fp8, GU_scale or both NULL: as moe_swiglu writes them (scale_format)
 * What moe_expert_gemm and moe_swiglu compute, without the bf16 rounding between them: both outputs are
 * quantised from the products' fp32 sums, and no bf16 row is written.  Rows of no group are left as they are.
 * H % 128 == 0, I % 128 == 0, H <= 2^18, I <= 2^17.  R == 0 is a no-op.
 * Errors: as moe_expert_gemm.
 */
MOE_API moe_status moe_expert_swiglu(const void *X_fp8, const void *X_scale, int x_scale_format,
                             const void *W1_fp8, const void *W1_scale, int w_scale_format,
                             const int32_t *expert_offsets, int64_t R, int E, int H, int I,
                             void *A_fp8, void *A_scale, void *GU_fp8, void *GU_scale, int scale_format,
                             int32_t *status_word, moe_stream_t stream);

/*
 * moe_expert_swiglu_backward -- the down projection's input gradient joined with the activation's:
 *   da[r] = dy[r] W2[e(r)] (fp32);  dg, du of da as in moe_swiglu_backward
 *   dY_fp8 uint8 [R, H], dY_scale [R, H/128] (dy_scale_format); W2_fp8 uint8 [E, H, I], W2_scale
 *   GU_fp8, GU_scale (gu_scale_format): the checkpoint of moe_expert_swiglu or moe_swiglu
 *   dGU, or dGU_fp8 and dGU_scale (scale_format), or all three: as moe_swiglu_backward writes them
 * What moe_expert_gemm (transposed) and moe_swiglu_backward compute, without the bf16 rounding of da between
 * them.  Sizes, rows of no group, errors: as moe_expert_swiglu.  One launch.
 */
MOE_API moe_status moe_expert_swiglu_backward(const void *dY_fp8, const void *dY_scale, int dy_scale_format,
                             const void *W2_fp8, const void *W2_scale, int w_scale_format,
                             const int32_t *expert_offsets, const void *GU_fp8, const void *GU_scale,
                             int gu_scale_format, int64_t R, int E, int H, int I,
                             void *dGU, void *dGU_fp8, void *dGU_scale, int scale_format,
                             int32_t *status_word, moe_stream_t stream);

/* Bytes of device workspace moe_layer needs. */
MOE_API size_t moe_layer_workspace_size(int N, int H, int I, int E, int K);

/*
 * moe_layer -- the whole layer for a few tokens (N <= 64) in one cooperative launch:
 *   topk_idx, topk_w   as moe_route_ex(X, W_gate, bias, renorm)
 *   gu  = W1[e] q(x) (fp32);  a = g / (1 + exp(-g)) * u;  y = W2[e] q(a) (fp32)
 *   out = sum_k topk_w[n,k] y_k (+ residual), one rounding to bf16
 * with q the E4M3 rounding with 1x128 scales of moe_permute: what dispatch (E4M3),
 * moe_expert_gemm, moe_swiglu, moe_expert_gemm and combine compute, without the bf16
 * roundings between them.  The weights of every expert that is chosen are read once.
 *   X bf16 [N,H], W_gate bf16 [H,E], bias fp32 [E] or NULL
 *   W1_fp8 uint8 [E, 2I, H] (gate rows, then up rows), W1_scale [E, 2I/128, H/128]
 *   W2_fp8 uint8 [E, H, I], W2_scale [E, H/128, I/128]; both in scale_format
 *   residual bf16 [N,H] or NULL (may be out)
 *   topk_idx int32 [N,K], topk_w fp32 [N,K], out bf16 [N,H]: outputs
 *   workspace  moe_layer_workspace_size() bytes, 256-byte aligned; its first
 *              256 + 4 * (E + 128) * (I/128) bytes zero before the first call with these E and I
 *              (every call leaves them zero).  Calls that may overlap need their own.
 *              A call captured into a graph keeps the address: the buffer has to live as long as
 *              the graph, and a clearing that was captured has happened only once that graph ran.
 * H % 128 == 0, I % 128 == 0, both <= 65536, 1 <= K <= min(E, 16), E <= 256.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_MISALIGNED, MOE_ERR_WORKSPACE,
 * MOE_ERR_UNSUPPORTED (N > 64), MOE_ERR_CUDA; status_word: MOE_ERR_TIMEOUT, MOE_ERR_BAD_SCALE.
 */
MOE_API moe_status moe_layer(const void *X, const void *W_gate, const float *bias,
                     const void *W1_fp8, const void *W1_scale, const void *W2_fp8, const void *W2_scale,
                     int scale_format, const void *residual, int N, int H, int I, int E, int K, int renorm,
                     int32_t *topk_idx, float *topk_w, void *out, int32_t *status_word,
                     void *workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * The norms around the experts.  Both need a GPU of compute capability 10.x
 * (MOE_ERR_UNSUPPORTED elsewhere).
 * ---------------------------------------------------------------------------
 */
typedef enum moe_grad_type { MOE_GRAD_FP32 = 0, MOE_GRAD_BF16 = 1 } moe_grad_type;

/*
 * moe_rms_norm -- the norm in front of the router, with the residual stream's addition:
 *   s = bf16(x + residual) (x itself without a residual);  rstd = 1 / sqrt(mean of s^2 + eps)
 *   y = s * rstd * weight
 *   X, residual bf16 [N, H] (residual may be NULL), weight [H] (weight_type: a moe_grad_type), 0 < eps <= 1
 *   S bf16 [N, H]: with a residual, and only then; may be the residual or X
 *   Y bf16 [N, H] or NULL (may be X, but not S): what moe_route and moe_dispatch read
 *   Y_fp8 uint8 [N, H], Y_scale [N, H/128] (scale_format) or both NULL (H % 128 == 0): y in E4M3 by the
 *   rule of moe_permute, quantised from the unrounded y, for products of all rows (a shared expert)
 *   rstd fp32 [N] or NULL: what moe_rms_norm_backward reads
 * Y or Y_fp8 is required.  The mean is summed in fp32: a row whose sum of squares leaves its range gives zeros
 * (rows of values beyond 1e17 or so).  H % 8 == 0, 8 <= H <= 16384, N < 2^31.  One launch.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_MISALIGNED, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA.
 */
MOE_API moe_status moe_rms_norm(const void *X, const void *residual, const void *weight, int weight_type, float eps,
                             int64_t N, int H, void *S, void *Y, void *Y_fp8, void *Y_scale, int scale_format,
                             float *rstd, moe_stream_t stream);

/* Bytes of device workspace moe_rms_norm_backward needs (0 for sizes it does not take). */
MOE_API size_t moe_rms_norm_backward_workspace_size(int64_t N, int H);

/*
 * moe_rms_norm_backward -- its gradient:
 *   xh = s * rstd;  d = dy * weight;  dx = rstd * (d - xh * mean of d xh) + dS
 *   dweight[h] = add[h] + sum_n dy[n,h] * xh[n,h]
 *   dY bf16 [N, H]; S bf16 [N, H] and rstd fp32 [N] as moe_rms_norm left them (S is X without a residual)
 *   dS bf16 [N, H] or NULL: the gradient that reaches s through the residual stream
 *   add fp32 [H] or NULL, may be dweight
 *   dX bf16 [N, H] (the gradient of x and of the residual alike); may be dY, S or dS
 *   dweight fp32 [H], summed in fp32 in an order that depends on N and H alone
 *   workspace  moe_rms_norm_backward_workspace_size() bytes, 16-byte aligned, in any state; calls that
 *              may overlap need their own
 * A row with rstd 0 (its squares left fp32) gives dS to dX, or zeros, and nothing to dweight.  Infinities and NaNs reach
 * their own row of dX, and dweight.
 * N == 0 writes dweight (add, or zeros).  Sizes as moe_rms_norm.  Two launches.
 * Errors: as moe_rms_norm, and MOE_ERR_WORKSPACE; status_word: MOE_ERR_TIMEOUT.
 */
MOE_API moe_status moe_rms_norm_backward(const void *dY, const void *S, const void *weight, int weight_type,
                             const float *rstd, const void *dS, const float *add, int64_t N, int H,
                             void *dX, float *dweight, int32_t *status_word,
                             void *workspace, size_t workspace_bytes, moe_stream_t stream);

/* Bytes of device workspace moe_grad_norm and moe_clip_grad_norm need for n tensors. */
MOE_API size_t moe_grad_norm_workspace_size(int n);

/*
 * moe_grad_norm -- the 2-norm of n tensors together: norm = sqrt(sum of g^2), fp32 [1].
 *   grads   HOST array of n device pointers, aligned to their elements only
 *   sizes   HOST array: elements of each (0 allowed, the pointer is then not looked at), 2^44 bytes at most
 *           together, counted as four an element
 *   types   HOST array: the moe_grad_type of each
 *   workspace  moe_grad_norm_workspace_size(n) bytes, 16-byte aligned, in any state; calls that may
 *              overlap need their own
 * The host arrays are read during the call only.  Squares are added in fp32 for up to 65 values and in 64 bits
 * beyond (also where a square would leave the range of fp32), in an order that depends on the list alone; NaNs and
 * infinities propagate.  n == 0 gives 0.  A launch for each 1024 tensors (one up to 128) and one more.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_MISALIGNED, MOE_ERR_WORKSPACE, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA.
 */
MOE_API moe_status moe_grad_norm(const void *const *grads, const int64_t *sizes, const int *types, int n,
                             float *norm, void *workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * moe_clip_grad_norm -- the tensors scaled down to a largest norm, which the host never sees:
 *   out[i] = grads[i] * c,  c = min(1, max_norm / (norm + 1e-6)) rounded to fp32,  norm as moe_grad_norm
 *   out   HOST array of n device pointers of the same types, or NULL: in place (nothing is written if c is 1).
 *         out[i] may be grads[i]; any other overlap, and a tensor that is listed twice, is undefined
 *   max_norm >= 0
 * If norm is infinite or NaN (a value is, or the norm of finite ones is beyond fp32), c is 1.
 * Errors: as moe_grad_norm.
 */
MOE_API moe_status moe_clip_grad_norm(const void *const *grads, void *const *out, const int64_t *sizes,
                             const int *types, int n, double max_norm, float *norm,
                             void *workspace, size_t workspace_bytes, moe_stream_t stream);

/* A static, human-readable name for a status code. */
MOE_API const char *moe_status_string(moe_status status);

/* ABI version of this header (bumped on any signature change). */
MOE_API int moe_abi_version(void);
#define MOE_ABI_VERSION 1

#ifdef __cplusplus
}
#endif

#endif /* MOE_ROUTE_GB300_H */
