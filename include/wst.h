/*
 * wst.h -- C ABI of libwst: persistent, warp-specialized bf16 contractions
 * for NVIDIA GB300 (sm_103a).
 *
 * The first three operations, each one hand-written CUDA kernel behind one call
 * (the declarations below hold the others: norm-fused GEMMs, IKBO attention,
 * expert parallelism, mixture-of-experts routing and its gradients, 8-bit
 * products with block scales, the operators of a decoding step):
 *
 *   wst_gemm_bf16            dense (optionally strided-batched) GEMM with an
 *                            optional fused bias / bias+SiLU epilogue.
 *                            Source: "How We Built TLX: A Hardware-Native GPU
 *                            Compiler for Production ML at Scale" (Meta
 *                            Engineering), section "Introducing TLX": the
 *                            tiled matmul C = A.B with an fp32 accumulator,
 *                            restructured into a TMA producer, a single MMA
 *                            issuer accumulating in tensor memory, and an
 *                            epilogue that stores the tile; the fused
 *                            epilogue follows "Five key areas" (model-aware
 *                            kernel fusion).
 *   wst_grouped_gemm_bf16    one GEMM per group (mixture-of-experts expert
 *                            matmuls) over variable, device-resident row
 *                            offsets.  Source: same page, "TLX in
 *                            Production" and "Case Study 3: Distributed
 *                            Grouped GEMM for LLM Pretraining".
 *   wst_ikbo_linear_compress in-kernel-broadcast linear compression,
 *                            Y[c] = W . concat(U[user(c)], Cf[c]), with the
 *                            user part W_u.U[u] computed once per user and
 *                            broadcast inside the kernel.  Source: same page,
 *                            "Case Study 2: In-Kernel Broadcast Optimization
 *                            for RecSys" and "TLX Provides a Building Block
 *                            for the Final Stage of This Optimization"
 *                            (matmul decomposition, a persistent
 *                            warp-specialized kernel in which user and
 *                            candidate GEMMs share one buffer ring, and
 *                            tile-level release/acquire across CTAs).
 *
 * Conventions shared by every call
 * --------------------------------
 *  - All matrix pointers are DEVICE pointers to memory the caller owns and
 *    keeps alive until the work on `stream` has finished.  The library never
 *    allocates or frees device memory and never falls back to the CPU; the
 *    only device memory it keeps is the fixed scratch array of
 *    wst_ikbo_linear_compress_noalloc.
 *  - `stream` is a cudaStream_t (NULL = the legacy default stream).  Every
 *    call is asynchronous: it validates its arguments on the host, enqueues
 *    its kernel (a few calls: two) on `stream`, and returns.
 *  - bf16 is IEEE-style bfloat16; accumulation is fp32; bf16 outputs are
 *    rounded to nearest even.
 *  - Alignment: every matrix pointer is 16-byte aligned and every leading
 *    dimension / batch stride, in bytes, is a multiple of 16 (the tensor
 *    memory accelerator's rule).  Otherwise WST_ERR_ALIGNMENT.
 *  - `workspace` is a caller-owned device buffer of at least
 *    wst_workspace_size(...) bytes, zero-filled once before first use (for
 *    example with wst_workspace_init).  It carries the device error word and,
 *    for IKBO, the per-user partial products and their ready flags.  One
 *    workspace may serve different operations one after another, but must not
 *    be used by two calls that can run at the same time.
 *  - Errors found on the host are returned before anything is enqueued.
 *    Errors found on the device (a bounded wait that ran out, inconsistent
 *    device offsets, a row index out of range in wst_permute_rows) are
 *    latched in the workspace; wst_sync_status reads and clears them.  No
 *    call aborts, traps or throws.
 */
#ifndef WST_H_
#define WST_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  WST_OK = 0,
  WST_ERR_INVALID_ARG = 1,  /* a size, pointer, stride or enum is out of range   */
  WST_ERR_ALIGNMENT = 2,    /* pointer / stride breaks the 16-byte rule          */
  WST_ERR_UNSUPPORTED = 3,  /* valid request this build does not implement        */
  WST_ERR_CUDA = 4,         /* a CUDA runtime/driver call failed (see message)    */
  WST_ERR_TIMEOUT = 5,      /* a device-side bounded wait ran out                 */
  WST_ERR_BAD_OFFSETS = 6   /* device offsets break their operation's rule       */
} wst_status;

typedef enum { WST_F32 = 0, WST_BF16 = 1 } wst_dtype;

/* 8-bit floating point: e4m3 (largest 448, no infinity) and e5m2 (largest 57344). */
typedef enum { WST_E4M3 = 0, WST_E5M2 = 1 } wst_fp8;

typedef enum {
  WST_EPI_NONE = 0,      /* C = A.B^T                                   */
  WST_EPI_BIAS = 1,      /* C = A.B^T + bias[n]                         */
  WST_EPI_BIAS_SILU = 2, /* C = SiLU(A.B^T + bias[n]), SiLU(x)=x/(1+e^-x) */
  WST_EPI_BIAS_GELU = 3  /* C = GELU(A.B^T + bias[n]), GELU(x)=x*Phi(x), Phi the standard
                            normal distribution function (exact erf form) */
} wst_epilogue;

/*
 * Process-wide tuning options.  They choose between equivalent schedules of
 * the same computation (the results are bitwise equal); the pages have no
 * counterpart.  A value applies to every later call on every thread of the
 * process; set options between calls, not while another thread is calling.
 * (WST_OPT_NORM_STATS alone changes the order of a sum; see below.)
 *   WST_OPT_GROUPED_SCHEDULE  tile schedule of wst_grouped_gemm_bf16:
 *                             WST_SCHED_STATIC (default: persistent CTA pairs
 *                             walk the tiles in a fixed order) or
 *                             WST_SCHED_CLC (one CTA pair per tile launched,
 *                             running pairs take unstarted pairs' tiles by
 *                             hardware cluster launch control).
 *   WST_OPT_DENSE_CTA_GROUP   tile shape of the dense, batched and
 *                             norm-fused GEMMs: 0 automatic (default: CTA
 *                             pairs on 256-row tiles when M > 128 and
 *                             K > 512, else one CTA per 128-row tile), 1
 *                             always one CTA per 128-row tile, 2 always CTA
 *                             pairs.
 *   WST_OPT_IKBO_SCHEDULE     candidate schedule of the IKBO linear
 *                             compression (both entry points):
 *                             WST_SCHED_STATIC (default: a persistent grid,
 *                             each CTA's user items, then one contiguous
 *                             candidate range balanced on the host) or
 *                             WST_SCHED_CLC (one CTA per user item and per
 *                             16-candidate chunk launched; running CTAs take
 *                             over unstarted ones by hardware cluster launch
 *                             control).
 *   WST_OPT_NORM_STATS        where wst_gemm_rmsnorm_bf16 and
 *                             wst_gemm_layernorm_bf16 take the row
 *                             statistics: WST_NORM_STATS_AUTO (default: a
 *                             separate pass over A when N > 2048 (RMSNorm)
 *                             or N > 512 (LayerNorm) and the workspace
 *                             holds the statistics, else in the GEMM), WST_NORM_STATS_FUSED (always gathered
 *                             in the GEMM from the A tiles in shared memory)
 *                             or WST_NORM_STATS_PASS (always the separate
 *                             pass; a workspace smaller than
 *                             wst_gemm_norm_workspace_size() is then
 *                             WST_ERR_INVALID_ARG).  The two forms sum in a
 *                             different order: results agree to rounding,
 *                             not bitwise.
 * wst_set_option returns WST_ERR_INVALID_ARG for an unknown option or value.
 */
typedef enum {
  WST_OPT_GROUPED_SCHEDULE = 0,
  WST_OPT_DENSE_CTA_GROUP = 1,
  WST_OPT_IKBO_SCHEDULE = 2,
  WST_OPT_NORM_STATS = 3
} wst_option;

typedef enum { WST_SCHED_STATIC = 0, WST_SCHED_CLC = 1 } wst_schedule;
typedef enum {
  WST_NORM_STATS_AUTO = 0,
  WST_NORM_STATS_FUSED = 1,
  WST_NORM_STATS_PASS = 2
} wst_norm_stats;

wst_status wst_set_option(wst_option opt, int value);
/* Current value of an option in *value (WST_ERR_INVALID_ARG if unknown). */
wst_status wst_get_option(wst_option opt, int* value);

/* Bytes of workspace a call needs.  GEMM and grouped GEMM need
 * wst_workspace_size(0, 0, 0); IKBO needs wst_workspace_size(num_users, O, D). */
size_t wst_workspace_size(int num_users, int O, int D);

/* Zero-fill `bytes` of `workspace` on `stream` (asynchronous). */
wst_status wst_workspace_init(void* workspace, size_t bytes, void* stream);

/*
 * Dense / strided-batched GEMM.  For b in [0,batch), m in [0,M), n in [0,N):
 *   C[b][m][n] = epi( sum_k A[b][m][k] * B[b][n][k] (+ bias[b][n]) )
 *   A     bf16, element (b,m,k) at A + b*strideA + m*lda + k   (row-major M x K)
 *   B     bf16, element (b,n,k) at B + b*strideB + n*ldb + k   (N x K, K
 *         contiguous: the column-major K x N operand)
 *   bias  bf16, element (b,n) at bias + b*strideBias + n; NULL unless epi>0;
 *         strideBias 0 shares one bias row across the batch
 *   C     c_type, element (b,m,n) at C + b*strideC + m*ldc + n
 *   Strides are in ELEMENTS.  strideA / strideB may be 0 (operand shared by
 *   the whole batch); strideC must be 0 only when batch == 1.
 * Requires batch >= 1, M, N, K >= 1, lda >= K, ldb >= K, ldc >= N.
 */
wst_status wst_gemm_bf16(int batch, int M, int N, int K,
                         const void* A, long lda, long strideA,
                         const void* B, long ldb, long strideB,
                         const void* bias, long strideBias,
                         void* C, long ldc, long strideC, wst_dtype c_type,
                         wst_epilogue epi, void* workspace, void* stream);

/*
 * GEMM on RMS-normalised rows of A (normalisation fused into the GEMM).  Same
 * arguments, layouts and rules as wst_gemm_bf16, plus eps >= 0:
 *   r[b][m]    = 1 / sqrt( (1/K) sum_k A[b][m][k]^2 + eps )
 *   C[b][m][n] = epi( r[b][m] * sum_k A[b][m][k] * B[b][n][k] (+ bias[b][n]) )
 * i.e. y = RMSNorm(x) W^T (+ b) with the norm's learned per-feature scale
 * folded into B by the caller.  The normalised A is never formed: r is
 * applied to the fp32 accumulators in the GEMM's epilogue.  The row
 * statistics come either from the A tiles as they stream through shared
 * memory (A read from HBM once; every 256-column tile of N recomputes them)
 * or from a separate pass over A into the workspace (one more read of A,
 * the GEMM then runs without the statistics warps); WST_OPT_NORM_STATS
 * chooses, by default the pass when N > 2048 and workspace_bytes >=
 * wst_gemm_norm_workspace_size(batch, M, N, strideA, strideB, 0).
 * workspace: 16-byte aligned, at least 256 bytes (the status header).
 * Source: the TLX write-up ("How We Built TLX: A Hardware-Native GPU Compiler
 * for Production ML at Scale", companion work on norm fusion into GEMMs, and
 * "Five key areas": model-aware fusion); the pages give no formula, this is
 * the plainest RMSNorm reading.  Runs on 256 x 256 CTA-pair tiles when
 * M > 128 and K > 512, else on single-CTA 128 x 256 tiles.
 */
wst_status wst_gemm_rmsnorm_bf16(int batch, int M, int N, int K,
                                 const void* A, long lda, long strideA,
                                 const void* B, long ldb, long strideB, float eps,
                                 const void* bias, long strideBias,
                                 void* C, long ldc, long strideC, wst_dtype c_type,
                                 wst_epilogue epi, void* workspace, size_t workspace_bytes,
                                 void* stream);

/*
 * GEMM on LayerNorm-normalised rows of A.  Same arguments, layouts and rules
 * as wst_gemm_rmsnorm_bf16, with
 *   mu[b][m]   = (1/K) sum_k A[b][m][k]
 *   var[b][m]  = (1/K) sum_k (A[b][m][k] - mu[b][m])^2      (biased)
 *   C[b][m][n] = epi( sum_k (A[b][m][k] - mu) / sqrt(var + eps) * B[b][n][k]
 *                     (+ bias[b][n]) )
 * i.e. y = LayerNorm(x) W^T (+ b), the norm's per-feature scale folded into B
 * and its shift into bias by the caller.  Computed as
 *   r (A.B^T)[m][n] - r mu s[n],   r = 1/sqrt(var + eps),  s[n] = sum_k B[n][k],
 * a first kernel writing the column sums s (fp32) into the workspace.  The
 * statistics are shifted-data sums in fp32 about the row's first element c
 * (mu = c + E[d], var = E[d^2] - E[d]^2 with d = A - c, clamped at 0), taken
 * from the A tiles in the GEMM or by a separate pass over A, as for
 * wst_gemm_rmsnorm_bf16 (WST_OPT_NORM_STATS; by default the pass when N >
 * 512 and workspace_bytes >= wst_gemm_norm_workspace_size(batch, M, N,
 * strideA, strideB, 1)).
 * workspace: 16-byte aligned, at least wst_gemm_layernorm_workspace_size(
 * batch, N, strideB) bytes (workspace_bytes says how many were given;
 * smaller returns WST_ERR_INVALID_ARG).  Two or three kernel launches on
 * `stream`.
 * Source: the same TLX norm-fusion item as wst_gemm_rmsnorm_bf16 (the pages
 * name LayerNorm and RMSNorm without formulas); standard LayerNorm reading.
 */
wst_status wst_gemm_layernorm_bf16(int batch, int M, int N, int K,
                                   const void* A, long lda, long strideA,
                                   const void* B, long ldb, long strideB, float eps,
                                   const void* bias, long strideBias,
                                   void* C, long ldc, long strideC, wst_dtype c_type,
                                   wst_epilogue epi, void* workspace, size_t workspace_bytes,
                                   void* stream);

/* Workspace bytes wst_gemm_layernorm_bf16 needs: the status header plus
 * batch (1 when strideB == 0) rows of N fp32 column sums, each padded to a
 * multiple of 4 floats. */
size_t wst_gemm_layernorm_workspace_size(int batch, int N, long strideB);

/* Workspace bytes with which the norm GEMMs (layernorm != 0: LayerNorm) can
 * take the row statistics from a separate pass: the header, the LayerNorm
 * column sums, then 8 bytes (r, r*mu as two fp32) per row of A (batch * M
 * rows; M when batch == 1 or strideA == 0), 16-byte aligned.  0 for
 * invalid sizes. */
size_t wst_gemm_norm_workspace_size(int batch, int M, int N, long strideA, long strideB,
                                    int layernorm);

/*
 * Grouped GEMM over G groups sharing N and K.  d_offsets is a DEVICE int32
 * array of G+1 entries, non-decreasing, d_offsets[0] = 0, d_offsets[G] <=
 * M_total; group g owns rows [d_offsets[g], d_offsets[g+1]) of A and C
 * (empty groups allowed; rows behind the last group belong to none, as where
 * wst_moe_plan had pairs without an expert):
 *   C[m][n] = epi( sum_k A[m][k] * B[g][n][k] (+ bias[g][n]) ),  m in group g
 *   A     bf16 [M_total][K] row-major, leading dimension lda
 *   B     bf16, element (g,n,k) at B + g*strideB_group + n*ldb + k
 *   bias  bf16, element (g,n) at bias + g*strideBias + n, or NULL (epi == 0)
 *   C     c_type [M_total][N], leading dimension ldc.  Rows outside every
 *         group are never written.
 * Offsets that break the rule are detected on the device: the kernel clamps
 * them into [0, M_total] (so no access leaves the buffers) and latches
 * WST_ERR_BAD_OFFSETS for wst_sync_status.
 */
wst_status wst_grouped_gemm_bf16(int G, int M_total, int N, int K,
                                 const void* A, long lda,
                                 const void* B, long ldb, long strideB_group,
                                 const int* d_offsets,
                                 const void* bias, long strideBias,
                                 void* C, long ldc, wst_dtype c_type,
                                 wst_epilogue epi, void* workspace, void* stream);

/*
 * Expert parallelism: the grouped GEMM's experts spread over the R ranks
 * (GPUs) of a node ("How We Built TLX: A Hardware-Native GPU Compiler for
 * Production ML at Scale", "Case Study 3: Distributed Grouped GEMM for LLM
 * Pretraining" and "TLX in Production": the distributed grouped GEMM of
 * mixture-of-experts pretraining).  G experts, G divisible by R; rank r owns
 * experts [r*G/R, (r+1)*G/R).  A token t routed to k experts forms the pairs
 * p = t*k + s (s < k).  One layer on a rank:
 *   1. wst_ep_dispatch_plan on the rank's routing table (host);
 *   2. exchange the per-(rank, local expert) counts (an all-to-all);
 *   3. wst_permute_rows gathers the token rows of the pairs in send order;
 *   4. all-to-all of the rows (send_counts out, the received counts in);
 *   5. wst_ep_receive_plan orders the received rows by local expert;
 *      wst_permute_rows gathers them, wst_grouped_gemm_bf16 multiplies them
 *      by the rank's experts (group offsets from the plan);
 *   6. wst_permute_rows scatters the products back to received order, the
 *      reverse all-to-all returns them, and wst_permute_rows scatters them
 *      to their pairs.
 * The exchanges are the caller's collectives (for example NCCL); the plans
 * are host functions and need no GPU.
 *
 * wst_ep_dispatch_plan: HOST arrays.
 *   routing            int32 [num_tokens][top_k], expert ids in [0, num_experts)
 *   send_counts        out int32 [world_size]: pairs sent to each rank
 *   send_group_counts  out int32 [num_experts]: pairs per expert (entry
 *                      r*G/R + j: rank r's local expert j)
 *   send_pairs         out int32 [num_tokens*top_k]: the pair carried by each
 *                      send row, ordered by destination rank, then local
 *                      expert, then pair id
 * Returns WST_ERR_INVALID_ARG for a bad size, an expert id out of range or
 * num_experts not divisible by world_size.
 */
wst_status wst_ep_dispatch_plan(int num_tokens, int top_k, const int* routing, int num_experts,
                                int world_size, int* send_counts, int* send_group_counts,
                                int* send_pairs);

/*
 * wst_ep_receive_plan: HOST arrays.  Rows arrive from the world_size ranks
 * in source order, each source's block ordered by local expert, with
 * recv_group_counts[s][e] rows from source s for local expert e.
 *   group_offsets  out int32 [experts_per_rank+1]: the grouped GEMM's offsets
 *                  of the expert-major order
 *   expert_rows    out int32 [total received rows]: expert-major row i is
 *                  received row expert_rows[i] (local expert e, then source s)
 */
wst_status wst_ep_receive_plan(int world_size, int experts_per_rank, const int* recv_group_counts,
                               int* group_offsets, int* expert_rows);

/*
 * Row permutation on the GPU: for i < n_rows,
 *   dst row (d_dst_index ? d_dst_index[i] : i) = src row (d_src_index ? d_src_index[i] : i).
 * src, dst: DEVICE pointers, rows of row_bytes bytes at src_stride /
 * dst_stride bytes apart (row_bytes and strides multiples of 16, pointers
 * 16-byte aligned); the index arrays are DEVICE int32 (or NULL), and the
 * source / destination hold n_src_rows / n_dst_rows rows.  An index of -1 (no
 * row: what wst_moe_plan leaves behind the last one) skips the row; another
 * outside them skips it and latches WST_ERR_INVALID_ARG in `workspace` (a
 * zero-filled workspace of at least wst_workspace_size(0, 0, 0) bytes) for
 * wst_sync_status.  Asynchronous on `stream`.
 */
wst_status wst_permute_rows(int n_rows, size_t row_bytes, const void* src, size_t src_stride,
                            const int* d_src_index, int n_src_rows, void* dst, size_t dst_stride,
                            const int* d_dst_index, int n_dst_rows, void* workspace, void* stream);

/*
 * Mixture-of-experts routing on the GPU: the router in front of the grouped
 * GEMM, the plan of its rows, and the sum of its results per token.  One layer:
 *   wst_moe_route -> wst_moe_plan -> wst_permute_rows by row_token (or
 *   wst_quantize_fp8_dispatch by position) -> wst_grouped_gemm_bf16 (or
 *   wst_grouped_gemm_fp8) -> wst_moe_combine,
 * all on device arrays, without a copy to the host, so the whole layer can be
 * captured in a CUDA graph.  The gradients: wst_moe_combine_backward,
 * wst_grouped_gemm_wgrad_bf16 for the weights, wst_grouped_gemm_bf16 with the
 * transposed weights for the rows, wst_moe_combine without weights to add the
 * rows' gradients per token, wst_moe_route_backward.
 *
 * These entry points (and the 8-bit ones below) also require their operands on
 * the calling thread's current device (else WST_ERR_INVALID_ARG).
 *
 * wst_moe_route: for each of T tokens, with x its E logits (logits_type, rows
 * `ld` elements apart, aligned to their elements only):
 *   x <= -3e38 (-inf, or a mask of the type's lowest value): the expert is off
 *   s_e = exp(x_e) / sum over the live experts of exp(x)   (WST_SCORE_SOFTMAX)
 *         or 1 / (1 + exp(-x_e))                           (WST_SCORE_SIGMOID)
 *   v_e = s_e + bias[e]      (bias fp32 [E] or NULL; it takes part in the
 *                            choice, not in the weights; -inf: expert off)
 *   groups > 1: the experts form `groups` equal consecutive groups; a group's
 *         score is the sum of its group_best (1 or 2) largest v; the
 *         top_groups groups with the largest scores stay
 *   experts[t][i], i < top_k: the experts with the largest v, in descending
 *         order of v; ties (of experts and of groups) go to the lower index
 *   weights[t][i] = scale * s_i / (renorm ? sum of the chosen s : 1)
 * Slots for which no live expert is left get expert -1 and weight 0 (a row
 * with every expert off gets nothing else).  A NaN ranks above every number,
 * as in torch.topk, and shows in the weights.  Without a bias the experts are
 * ranked by their logits (and groups by their largest, for group_best 1);
 * otherwise as if the scores were computed in 64 bits.
 * Limits: E <= 1024, top_k <= 16, groups <= 32, T < 2^31 - 1024 (also for the
 * gradient), else WST_ERR_UNSUPPORTED; T * top_k is below 2^31 - 2^20.
 */
typedef enum { WST_SCORE_SOFTMAX = 0, WST_SCORE_SIGMOID = 1 } wst_score;

wst_status wst_moe_route(int T, int E, int top_k, const void* logits, long ld, wst_dtype logits_type,
                         wst_score score, const float* bias, int groups, int top_groups,
                         int group_best, int renorm, float scale, int* experts, float* weights,
                         void* stream);

/* Gradient of wst_moe_route's weights with respect to the logits:
 *   dlogits[t][e] = sum_i dweights[t][i] d weights[t][i] / d logits[t][e],
 * the choice of the experts held fixed.  `experts` as wst_moe_route left it
 * (other ids outside [0, E) count as -1: no gradient; an expert in two slots
 * gets the sum of both).  dlogits: logits_type, rows `ldd` apart, every one of
 * its T x E elements is written; it may be the logits array itself. */
wst_status wst_moe_route_backward(int T, int E, int top_k, const void* logits, long ld,
                                  wst_dtype logits_type, wst_score score, int renorm, float scale,
                                  const int* experts, const float* dweights, void* dlogits, long ldd,
                                  void* stream);

/* The rows of the grouped product: a stable sort of the pairs p = t * top_k + i
 * by experts[p].  All arrays DEVICE int32.
 *   offsets    out [num_experts + 1]: rows of expert e are [offsets[e], offsets[e+1])
 *   row_pair   out [num_tokens * top_k]: the pair of each row, pair ids
 *              ascending inside an expert; -1 behind the last row
 *   row_token  out, same shape: the pair's token (row_pair / top_k); -1 behind
 *   position   out [num_tokens][top_k]: the row of each pair; -1 without one
 * A pair with expert -1 gets no row; so does one with another id outside
 * [0, num_experts), which also latches WST_ERR_INVALID_ARG in the workspace.
 * workspace: zero-filled once, wst_moe_plan_workspace_size(...) bytes.
 * num_experts <= 1024, else WST_ERR_UNSUPPORTED. */
wst_status wst_moe_plan(int num_tokens, int top_k, const int* experts, int num_experts, int* offsets,
                        int* row_pair, int* row_token, int* position, void* workspace,
                        size_t workspace_bytes, void* stream);

/* Workspace bytes wst_moe_plan needs for num_pairs = num_tokens * top_k pairs
 * (0 for invalid sizes). */
size_t wst_moe_plan_workspace_size(int num_pairs, int num_experts);

/* The weighted sum of each token's rows:
 *   out[t][n] = sum_i w[t][i] * y[position[t][i]][n]      (i ascending, in fp32)
 *   y         y_type [n_rows][N], rows ldy elements apart
 *   position  DEVICE int32 [T][top_k]; a negative entry adds nothing; one of
 *             n_rows or more adds nothing and latches WST_ERR_INVALID_ARG
 *   weights   fp32 [T][top_k], or NULL: all 1
 *   out       out_type [T][N], rows ldo apart; every token is written (0 where
 *             it has no row); it must not overlap y
 * Rows are 16-byte aligned; N is arbitrary.  top_k <= 32, N < 2^31 - 8192, T <
 * 2^31 - 1024 (also for the gradients), else WST_ERR_UNSUPPORTED. */
wst_status wst_moe_combine(int T, int top_k, int N, const void* y, long ldy, wst_dtype y_type,
                           int n_rows, const int* position, const float* weights, void* out, long ldo,
                           wst_dtype out_type, void* workspace, void* stream);

/* Gradients of wst_moe_combine for dout (out_type [T][N]):
 *   dy[position[t][i]][n] = w[t][i] * dout[t][n]     (y_type; NULL: not wanted)
 *   dweights[t][i] = sum_n dout[t][n] * y[position[t][i]][n]   (fp32; NULL: not
 *                    wanted, y is then not read and may be NULL; 0 for a pair
 *                    without a row)
 * Rows of dy that no pair names are left as they were; a row that two pairs
 * name gets one of the two values (wst_moe_plan names each row once).  dy must
 * not overlap dout or y. */
wst_status wst_moe_combine_backward(int T, int top_k, int N, const void* dout, long ldo,
                                    wst_dtype out_type, const void* y, long ldy, wst_dtype y_type,
                                    int n_rows, const int* position, const float* weights, void* dy,
                                    long lddy, float* dweights, void* workspace, void* stream);

/*
 * Quantisation to 8 bits with one fp32 scale for each block of 128 values:
 *   amax  = max |x| over the block, at least 2^-100
 *   scale = amax * (1/largest), or with pow2 the smallest power of two with
 *           amax <= largest * scale
 *   q     = round to nearest even of x * (1/scale)         (x ~ q * scale)
 * all in fp32.  A block with a NaN or an infinity gets it as its scale.
 * x: x_type [M][K] per batch entry.  Modes (element (i,j) of q at q + i*ldq + j,
 * of the scales at scales + i*lds + j):
 *   WST_FP8_ROWS      blocks 1 x 128: q [M][K], scales [ceil(K/128)][M]
 *                     (block-major: the scales of one K block are consecutive)
 *   WST_FP8_COLS      blocks 128 x 1, transposed: q [K][M], scales [ceil(M/128)][K]
 *                     (the ROWS form of x transposed)
 *   WST_FP8_BLOCKS    blocks 128 x 128: q [M][K], scales [ceil(M/128)][ceil(K/128)]
 *   WST_FP8_BLOCKS_T  the same blocks transposed: q [K][M], scales
 *                     [ceil(K/128)][ceil(M/128)]
 * A last block is what is left of its row or column.  x and q are 16-byte
 * aligned with leading dimensions and batch strides of whole 16 bytes.  M <=
 * 65535 * 128 in every mode (the modes with 128-row blocks use a grid dimension
 * per block; longer inputs go in parts), else WST_ERR_UNSUPPORTED.
 */
typedef enum {
  WST_FP8_ROWS = 0,
  WST_FP8_COLS = 1,
  WST_FP8_BLOCKS = 2,
  WST_FP8_BLOCKS_T = 3
} wst_fp8_mode;

wst_status wst_quantize_fp8(wst_fp8_mode mode, int batch, int M, int K, const void* x, long ldx,
                            long strideX, wst_dtype x_type, void* q, long ldq, long strideQ,
                            wst_fp8 q_type, float* scales, long lds, long strideS, int pow2,
                            void* stream);

/* WST_FP8_ROWS of each row m of x, stored to the rows position[m][c], c <
 * copies, of q [n_rows][K] and the scales [ceil(K/128)][n_rows]: the tokens'
 * rows of a grouped product (position as wst_moe_plan leaves it).  A negative
 * entry is skipped, one of n_rows or more is skipped and latches
 * WST_ERR_INVALID_ARG.  Rows that no entry names are left as they were; a row
 * that two entries name gets either of the two. */
wst_status wst_quantize_fp8_dispatch(int M, int K, int copies, const void* x, long ldx,
                                     wst_dtype x_type, const int* position, int n_rows, void* q,
                                     long ldq, wst_fp8 q_type, float* scales, long lds, int pow2,
                                     void* workspace, void* stream);

/*
 * Product of 8-bit matrices with block scales.  For m < M, n < N:
 *   C[m][n] = epi( sum_b sA(m,b) sB(n,b) sum_{k in block b} A[m][k] B[n][k] (+ bias[n]) ),
 * blocks of 128 along K (the last one what is left).
 *   A       a_type [M][K], leading dimension lda
 *   scaleA  fp32, sA(m,b) at scaleA + b*ldsa + m      (WST_FP8_ROWS of the rows)
 *   B       b_type [N][K], leading dimension ldb
 *   scaleB  fp32; b_scaling WST_FP8_ROWS: sB(n,b) at scaleB + b*ldsb + n;
 *           WST_FP8_BLOCKS: sB(n,b) at scaleB + (n/128)*ldsb + b
 *   bias    bf16 [N], NULL unless epi > 0
 *   C       c_type [M][N], leading dimension ldc; M may be 0
 * The products of a block accumulate in the tensor core; the blocks are scaled
 * (by sA sB, itself an fp32 product that has to be finite) and added in fp32.
 * A training step's other products are the same call: dA = dC . B with B
 * quantised as WST_FP8_BLOCKS_T, dB = dC^T . A with both quantised as
 * WST_FP8_COLS (b_scaling WST_FP8_ROWS).
 * a_type and b_type may differ.  A, B, C are 16-byte aligned with leading
 * dimensions of whole 16 bytes.
 * workspace: at least the 256-byte header, zero-filled once.  With
 * wst_gemm_fp8_workspace_size() bytes the K loops of a product with few tiles
 * (a step of a few tokens) are split over the idle SMs and their fp32 sums
 * added in a fixed order; smaller ones run whole tiles.  After
 * WST_ERR_TIMEOUT call wst_sync_status before using the workspace again.
 */
wst_status wst_gemm_fp8(int M, int N, int K, const void* A, long lda, wst_fp8 a_type,
                        const float* scaleA, long ldsa, const void* B, long ldb, wst_fp8 b_type,
                        const float* scaleB, long ldsb, wst_fp8_mode b_scaling, const void* bias, void* C,
                        long ldc, wst_dtype c_type, wst_epilogue epi, void* workspace,
                        size_t workspace_bytes, void* stream);

/* The same for G groups of rows: rows [d_offsets[g], d_offsets[g+1]) of A and C
 * with B + g*strideB_group, scaleB + g*strideSB_group and bias + g*strideBias
 * (offsets as in wst_grouped_gemm_bf16: rows behind the last group are left as
 * they were). */
wst_status wst_grouped_gemm_fp8(int G, int M_total, int N, int K, const void* A, long lda, wst_fp8 a_type,
                                const float* scaleA, long ldsa, const void* B, long ldb,
                                long strideB_group, wst_fp8 b_type, const float* scaleB, long ldsb,
                                long strideSB_group, wst_fp8_mode b_scaling, const int* d_offsets,
                                const void* bias, long strideBias, void* C, long ldc, wst_dtype c_type,
                                wst_epilogue epi, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes with which the 8-bit products split their K loops. */
size_t wst_gemm_fp8_workspace_size(void);

/*
 * Weight gradient of the grouped GEMM: for every group g, n < N, k < K
 *   dB[g][n][k] = sum_{m in group g} dC[m][n] * A[m][k]        (fp32 accumulation)
 * or, with accumulate != 0, that added to what dB holds (rounded once to
 * db_type each time).  An empty group's gradient is 0 (or adds nothing).
 *   dC  bf16 [M_total][N], leading dimension lddc
 *   A   bf16 [M_total][K], leading dimension lda
 *   dB  db_type, element (g,n,k) at dB + g*stride_dB + n*lddb + k; it must not
 *       overlap dC or A
 * d_offsets as in wst_grouped_gemm_bf16; rows behind the last group belong to
 * no gradient (whatever they hold).  Pointers 16-byte aligned, leading
 * dimensions and strides multiples of 16 bytes.  (The gradient of the rows is wst_grouped_gemm_bf16 of dC with the
 * weights transposed.)
 */
wst_status wst_grouped_gemm_wgrad_bf16(int G, int M_total, int N, int K, const void* dC, long lddc,
                                       const void* A, long lda, const int* d_offsets, void* dB,
                                       long lddb, long stride_dB, wst_dtype db_type, int accumulate,
                                       void* workspace, void* stream);

/*
 * IKBO linear compression.  Candidates of user u are [off[u], off[u+1]) of
 * the DEVICE int32 array d_user_offsets (num_users+1 entries, non-decreasing,
 * from 0 to num_cand).  For every candidate c of user u:
 *   Y[c][o][d] = sum_{f<Du} W[o][f] U[u][f][d] + sum_{f<Dc} W[o][Du+f] Cf[c][f][d]
 *   U   bf16 [num_users][Du][D]   (d contiguous)
 *   Cf  bf16 [num_cand][Dc][D]    (d contiguous)
 *   W   bf16 [O][Du+Dc]           (user columns first)
 *   Y   fp32 [num_cand][O][D]     (d contiguous)
 * The user part P[u] = W[:, :Du].U[u] is computed once per user per call
 * into the workspace and added to each of that user's candidates inside the
 * kernel; the broadcast user features are never materialised.
 * This build supports D == 128, O a multiple of 32 up to 256, Du and Dc
 * multiples of 8 with Du + Dc <= 512 (else WST_ERR_UNSUPPORTED).  The
 * kernel is a cooperative launch: all of its CTAs are resident at once.
 */
wst_status wst_ikbo_linear_compress(int num_users, int num_cand, int Du, int Dc,
                                    int D, int O,
                                    const void* U, const void* Cf, const void* W,
                                    const int* d_user_offsets,
                                    void* Y, void* workspace, void* stream);

/*
 * Allocation-free form of wst_ikbo_linear_compress (the pages have no
 * counterpart; this is a library convenience).  For callers that cannot
 * allocate device memory when they call -- code under a fixed memory budget,
 * behind an allocator it must not bypass, or inside a host framework that
 * owns every allocation -- the per-user partial products, ready flags and
 * error word live in a device array inside the library instead of a
 * caller-owned workspace.  Same arguments and results as
 * wst_ikbo_linear_compress, minus the workspace, plus:
 *   d_status  optional DEVICE int32 (NULL to skip) that receives this call's
 *             device-side status (0, WST_ERR_TIMEOUT or WST_ERR_BAD_OFFSETS)
 *             once the call's work on `stream` has run.
 * Limits and behaviour:
 *  - The array holds 4 MiB on every GPU that loads the library, until the
 *    process exits; wst_workspace_size(num_users, O, D) must not exceed it
 *    (64 users at O = 32, D = 128 need about 1 MiB).  Larger requests return
 *    WST_ERR_INVALID_ARG before anything is enqueued.
 *  - The call allocates and frees nothing.  Its first call on a device (and
 *    the first after a cudaDeviceReset, which gives the device a new
 *    context) looks up the array's device address with cudaGetSymbolAddress
 *    and caches it for that context; make that first call before any stream
 *    capture.  If it comes while `stream` is being captured, the call returns
 *    WST_ERR_UNSUPPORTED and enqueues nothing.
 *  - Every call on a device shares the one array and clears its header and
 *    flags at the start: calls that can overlap on the GPU (other streams,
 *    other host threads) race and must be serialised by the caller.
 */
wst_status wst_ikbo_linear_compress_noalloc(int num_users, int num_cand, int Du, int Dc,
                                            int D, int O,
                                            const void* U, const void* Cf, const void* W,
                                            const int* d_user_offsets, void* Y,
                                            int* d_status, void* stream);

/*
 * IKBO attention ("How We Built TLX: A Hardware-Native GPU Compiler for
 * Production ML at Scale", Case Study 2, which names an IKBO form of
 * FlashAttention whose key/value reads are shared by the candidates of one
 * user; the pages give no formula, and the reading implemented is below).
 * Candidates of user u are [off[u], off[u+1]) of the DEVICE int32 array
 * d_user_offsets (num_users+1 entries, non-decreasing, from 0 to num_cand);
 * candidate c owns the Lq query rows [c*Lq, (c+1)*Lq).  For every query row r
 * of a candidate of user u and every head h:
 *   O[r][h][:] = sum_j softmax_j(scale * Q[r][h][:] . K[u][j][h][:]) V[u][j][h][:]
 * over all Lkv context rows j of user u (no mask).
 *   Q   bf16 [num_cand*Lq][H][Dh]    (Dh contiguous)
 *   K   bf16 [num_users][Lkv][H][Dh]
 *   V   bf16 [num_users][Lkv][H][Dh]
 *   O   o_type [num_cand*Lq][H][Dh]  (fp32 or bf16)
 *   scale  any finite float (1/sqrt(Dh) is the usual choice)
 * The query rows of all candidates of a user are processed together in
 * 128-row tiles, so each user's K/V is read once per tile and per head, not
 * once per candidate.  The probabilities are rounded to bf16 before the
 * product with V; row maxima, sums and the output accumulate in fp32.
 * This build supports Dh == 128 (else WST_ERR_UNSUPPORTED) and needs
 * num_cand*Lq < 2^31.  Offsets that break the rule are clamped into range on
 * the device and latched as WST_ERR_BAD_OFFSETS.
 * workspace: 16-byte aligned, zero-filled once (wst_workspace_init) and
 * then reused; `workspace_bytes` says how large it is.  With at least
 * wst_ikbo_attention_workspace_size() bytes the items (user, head, 128-row
 * query tile) of the last partial wave of the persistent grid are split by
 * key blocks over all CTAs and their partial results merged through the
 * workspace (so the result of a split item is summed in another order);
 * with less (at least the 256-byte error-word header) whole items only.
 * One call at a time per workspace.
 */
wst_status wst_ikbo_attention_bf16(int num_users, int num_cand, int Lq, int H, int Dh, int Lkv,
                                   const void* Q, const void* K, const void* V,
                                   const int* d_user_offsets, float scale,
                                   void* O, wst_dtype o_type, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* Workspace bytes for wst_ikbo_attention_bf16's split schedule (header,
 * per-CTA flags and one partial O/m/l slot per CTA, for up to 256 CTAs). */
size_t wst_ikbo_attention_workspace_size(void);

/*
 * One step of decoding: new keys and values into a paged cache, attention of a
 * step's tokens over it, products of few rows with 4-bit weights.
 *
 * A paged cache holds the keys (and, in an array of its own with the same
 * strides, the values) of all sequences, bf16, in num_pages pages of page_size
 * tokens:
 *   element (page, token, head, d) at base + page*page_stride + token*token_stride
 *                                     + head*head_stride + d
 * so [page][token][head][d] and [page][head][token][d] are both possible, and
 * keys and values may share pages.  Pointers are 16-byte aligned, strides (in
 * elements) multiples of 16 bytes.  Slot s is token s % page_size of page
 * s / page_size.
 *
 * wst_cache_append_bf16: for every token t < T with slots[t] >= 0
 *   q_out[t][h] = R(q[t][h]),  slot of k_cache [h] = R(k[t][h]),
 *   slot of v_cache [h] = v[t][h]
 * R turns rot/2 pairs of the first rot components by positions[t]*inv_freq[j]
 * (radians, reduced by whole turns in 64-bit integers: off by at most
 * |position * inv_freq| 2^-52 + 2^-30, 5e-7 at position 2^31 and inv_freq 1, and by
 * fp32's rounding of what is left), pair j being components (j, j + rot/2)
 * (WST_ROPE_HALVES) or (2j, 2j + 1) (WST_ROPE_PAIRS):
 *   (a, b) -> (a cos - b sin, b cos + a sin)
 * in fp32, rounded once to bf16; the other components are copied.
 *   q, k, v    x_type, element (t,h,d) at x + t*ldx + h*Dh + d; q may be NULL
 *              (H and q_out are then not looked at)
 *   positions  DEVICE int32 [T]; inv_freq DEVICE fp32 [rot/2], finite (both may
 *              be NULL when rot == 0)
 *   slots      DEVICE int32 [T]; a token with a negative slot is skipped: its
 *              q_out is left as it was; one of num_pages*page_size or more is
 *              skipped and latches WST_ERR_INVALID_ARG; of two tokens with one
 *              slot either is stored, perhaps in parts
 *   q_out      bf16, rows ldqo apart; it may be q itself (bf16, ldqo == ldq),
 *              and must not overlap the other inputs or outputs
 * Dh and rot are multiples of 16, Dh <= 256, else WST_ERR_UNSUPPORTED.
 */
typedef enum { WST_ROPE_HALVES = 0, WST_ROPE_PAIRS = 1 } wst_rope;

wst_status wst_cache_append_bf16(int T, int H, int Hkv, int Dh, int rot, wst_rope style, const void* q, long ldq,
                                 const void* k, long ldk, const void* v, long ldv, wst_dtype x_type,
                                 const int* positions, const float* inv_freq, const int* slots, void* q_out,
                                 long ldqo, void* k_cache, void* v_cache, int num_pages, int page_size,
                                 long page_stride, long token_stride, long head_stride, void* workspace,
                                 void* stream);

/*
 * Attention of a step's tokens over a paged cache that holds them already.
 * Sequence b < B has the tokens [off[b], off[b+1]) of Q (n_b of them) behind
 * context[b] cached ones; its key j is token j % page_size of page
 * page_table[b][j / page_size], its i-th token being key context[b] + i.
 * For token t = off[b] + i, head h and key head h / (H / Hkv):
 *   O[t][h][:] = sum_j p_j V[j][:],  p = softmax of scale * Q[t][h][:] . K[j][:]
 * over the keys j that token t sees: all of the context, and of the new tokens
 * those whose bit is set in its mask (new token d: bit d % 32 of mask[t][d / 32]),
 * or with mask NULL those up to itself (a chain; one token sees everything).  A
 * token that sees no key gets zeros.  Scores are fp32 (a larger one is infinite); a key
 * that scores -inf weighs nothing, and a row of nothing else is zeros as well.  Keys that
 * a token does not see take no part, whatever they hold (NaN or infinities in them or in
 * the rest of a page included).
 *   Q       bf16, element (t,h,d) at Q + t*ldq + h*Dh + d
 *   d_q_offsets  DEVICE int32 [B+1], from 0, non-decreasing, at most T: rows behind
 *           the last sequence are left as they were; d_context DEVICE int32 [B]
 *   mask    DEVICE int32 [T][mask_words], rows ldm apart, or NULL
 *   k_cache, v_cache  as wst_cache_append_bf16 leaves them
 *   page_table  DEVICE int32 [B][max_pages], rows ldt apart; only the entries of a
 *           sequence's keys are read
 *   scale   finite, of at most 2e38
 *   O       o_type, element (t,h,d) at O + t*ldo + h*Dh + d; it must not overlap the
 *           inputs
 * The probabilities enter the product with V as bf16 (as three bf16, good to 2^-24,
 * where O is fp32); row maxima, sums and the output accumulate in fp32, where O is bf16 up
 * to 65,536 keys at a time as the tensor core adds, which cuts off (up to 2^-11 of O).
 * After a tree is verified, two calls of wst_permute_rows move the accepted tokens'
 * rows of a cache together: into an array of their own and back behind the context
 * (a row's new place may be another's old one).  A row is a token's heads where they
 * follow one another ([page][token][head]); in a cache of [page][head][token] every
 * head of a token is a row of its own.
 * Supported: Dh 64 and 128, H / Hkv <= 128, page_size 8, 16, 32, 64 or a multiple of
 * 128, max_pages * page_size <= 2^30, T <= 2^30, B <= 2^29 (else
 * WST_ERR_UNSUPPORTED).
 * Offsets, lengths or masks that break the rules (also context[b] + n_b above
 * max_pages * page_size, or n_b above 32 * mask_words) are clamped and latch
 * WST_ERR_BAD_OFFSETS; a page outside the cache reads as zeros and latches
 * WST_ERR_INVALID_ARG.
 * workspace: at least the 256-byte header, zero-filled once.  With
 * wst_tree_attention_workspace_size() bytes sequences are cut so that every SM gets
 * the same share of all keys (the pieces are added in a fixed order, by a second
 * kernel); smaller ones give whole (sequence, key head, 128 query rows) to an SM.
 */
wst_status wst_tree_attention_bf16(int B, int T, int H, int Hkv, int Dh, const void* Q, long ldq,
                                   const int* d_q_offsets, const int* d_context, const int* mask, int mask_words,
                                   long ldm, const void* k_cache, const void* v_cache, int num_pages, int page_size,
                                   long page_stride, long token_stride, long head_stride, const int* page_table,
                                   int max_pages, long ldt, float scale, void* O, long ldo, wst_dtype o_type,
                                   void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes with which wst_tree_attention_bf16 cuts sequences. */
size_t wst_tree_attention_workspace_size(void);

/*
 * Product of bf16 rows with 4-bit weights that have one scale for every
 * `group` consecutive k.  For m < M, n < N:
 *   C[m][n] = epi( sum_b s[b][n] sum_{k in group b} A[m][k] (w[n][k] - 8) (+ bias[n]) )
 *   A       bf16 [M][K], leading dimension lda; M may be 0
 *   W       4-bit numbers w in 0..15, two a byte: w[n][k] is the low (k even) or
 *           high (k odd) half of byte W + n*ldw + k/2 (ldw in bytes)
 *   scales  bf16, s[b][n] at scales + b*lds + n, b < ceil(K/group)
 *   bias    bf16 [N], NULL unless epi > 0
 *   C       c_type [M][N], leading dimension ldc
 * group is 32, 64 or 128, sizes below 2^31 - 1024, else WST_ERR_UNSUPPORTED (also
 * where the tiles' blocks of 256 k exceed 2^31); K is arbitrary (a last group is
 * what is left).  The weights are exact in bf16; products accumulate in fp32
 * inside a group, the groups are scaled and added in fp32.  Pointers are 16-byte
 * aligned, leading dimensions and strides multiples of 16 bytes.  Meant for the
 * few rows of a decoding step: every 32 rows read the weights once.
 * workspace: at least the 256-byte header, zero-filled once.  With
 * wst_gemm_w4_workspace_size() bytes the K loops are cut so that every SM gets
 * the same share (the pieces of a tile are added in a fixed order); smaller ones
 * run whole tiles.
 */
wst_status wst_gemm_w4(int M, int N, int K, const void* A, long lda, const void* W, long ldw, const void* scales,
                       long lds, int group, const void* bias, void* C, long ldc, wst_dtype c_type,
                       wst_epilogue epi, void* workspace, size_t workspace_bytes, void* stream);

/* The same for G groups of rows: rows [d_offsets[g], d_offsets[g+1]) of A and C
 * with W + g*strideW_group (bytes), scales + g*strideS_group and
 * bias + g*strideBias (offsets as in wst_grouped_gemm_bf16: rows behind the last
 * group are left as they were). */
wst_status wst_grouped_gemm_w4(int G, int M_total, int N, int K, const void* A, long lda, const void* W, long ldw,
                               long strideW_group, const void* scales, long lds, long strideS_group, int group,
                               const int* d_offsets, const void* bias, long strideBias, void* C, long ldc,
                               wst_dtype c_type, wst_epilogue epi, void* workspace, size_t workspace_bytes,
                               void* stream);

/* Workspace bytes with which the 4-bit products cut their K loops. */
size_t wst_gemm_w4_workspace_size(void);

/* Rows of a tile (8, 16 or 32: a form of the kernel each) that a 4-bit product of these
 * sizes takes on num_sms SMs; G 0: wst_gemm_w4.  0 for sizes out of range. */
int wst_gemm_w4_tile_rows(int G, int M, int N, int K, int num_sms);

/* Synchronize `stream`, then return and clear the first device-side error
 * latched in `workspace` (WST_OK if none). */
wst_status wst_sync_status(void* workspace, void* stream);

/* Static description of a status code. */
const char* wst_status_string(wst_status s);

/* Text of the last host-side error on the calling thread ("" if none). */
const char* wst_last_error(void);

/* Library version string. */
const char* wst_version(void);

#ifdef __cplusplus
}
#endif

#endif /* WST_H_ */
