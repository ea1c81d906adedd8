/*
 * pgg.h -- C ABI of the GB300 (sm_103a) fused MoE permute + grouped-matmul
 * backward, input gradient only.
 *
 * Operation (page "MoeInitRoutingGroupedMatmulGrad design", section
 * "数学定义和公式", element-wise gradient formula):
 *
 *     d_x[b, k] = sum_{i : batch(i) = b} sum_n gradY[i, n] * weight[g(i), k, n]
 *
 *   gradY  [M, N]     upstream gradient d_y in expanded (expert-sorted) order,
 *                     M = batch * topK                       (section "输入输出")
 *   weight [G, K, N]  expert weights, same dtype as gradY     (section "输入输出")
 *   g(i)              expert whose block of rows holds row i; block g has
 *                     groupList[g] rows (counts, not a cumulative sum; a count
 *                     of 0 is an empty expert)         (sections "输入输出", "约束")
 *   batch(i)          original_pos(i) / topK, original_pos = b * topK + j
 *                     (section "数学定义和公式", Step 2)
 *   expandedRowIdx    int64 [L], L == M. rowIdxType 0 (gather form): entry i is
 *                     the original position of expanded row i. rowIdxType 1
 *                     (scatter form): entry p is the expanded row of original
 *                     position p                 (section "输入输出", note 1)
 *   out               FP32 [batch, K], always FP32 whatever the input dtype
 *                     (section "输入输出", note 2; section 2.6.2)
 *
 * The [M, K] intermediate d_y @ weight^T is never materialised (section 1.1).
 * The result is bitwise identical from run to run: the topK contributions to
 * each out element are added in increasing expanded-row order (section 2.4.1
 * asks for deterministic computation).
 *
 * Conventions shared by every call below:
 *   - All tensors are dense and row-major. Device pointers are addresses in the
 *     current CUDA device's memory; the caller owns every buffer and keeps it
 *     alive until the work on `stream` has finished. The library allocates no
 *     memory and keeps no state between calls except per-device cached device
 *     attributes and the test hooks at the end of this file.
 *   - Calls only enqueue work on `stream` (NULL = legacy default stream) and
 *     never synchronise. Inputs are not modified.
 *   - Every kernel except the one that resets the workspace header (the first
 *     of a routing or index-validation stage) is launched with programmatic
 *     stream serialization: its CTAs may be scheduled while the previous
 *     kernel in the stream (the library's own, or the caller's) drains, and it
 *     waits for that kernel's completion before it reads any memory, so stream
 *     order is kept exactly.
 *   - Host-detected errors are returned synchronously and nothing is enqueued.
 *   - Device-detected errors (bad index, groupList sum, not a permutation,
 *     a wait that ran out) are written to the status word, the first uint32 of
 *     the workspace: 0 means success, otherwise one of PGG_ERR_INDEX ..
 *     PGG_ERR_TIMEOUT. Read it after the stream has finished. When routing
 *     validation fails, `out` is zero-filled instead of computed.
 *   - Alignment: gradY and weight must be aligned to their element size,
 *     out to 4 bytes, expandedRowIdx and groupList to 8 bytes, and the
 *     workspace to 256 bytes; otherwise PGG_ERR_ALIGN. Any N and K are
 *     accepted. When N * sizeof(dtype) is a multiple of 16 bytes and gradY
 *     and weight are 16-byte aligned, the grouped GEMM runs on the tensor
 *     cores with its operands streamed by the tensor-memory-access unit,
 *     which needs both. Otherwise, for 16-bit dtypes with an even N and
 *     gradY and weight 4-byte aligned, it still runs on the tensor cores,
 *     with the operands copied 4 bytes at a time by gather warps (plan
 *     variant 5; same tiles, same bits as variant 0 where both apply). In
 *     every other case (fp32 rows that are not a multiple of 16 bytes, odd
 *     N, 2-byte aligned pointers) it runs on the FP32 pipes (plan variant
 *     3), with the same ordered scatter-add and the same determinism. For
 *     the same call the tensor-core and FP32-pipe paths may differ in the
 *     last bits of the GEMM sums, never from run to run.
 */
#ifndef PGG_H
#define PGG_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st* pgg_stream_t;

/* Input dtype of gradY and weight (section "输入输出": FLOAT / FLOAT16 / BF16). */
typedef enum { PGG_F32 = 0, PGG_F16 = 1, PGG_BF16 = 2 } pgg_dtype;

typedef enum {
  PGG_OK = 0,
  PGG_ERR_NULL = 1,      /* a required pointer is NULL */
  PGG_ERR_SHAPE = 2,     /* sizes violate the constraint table (L != M, M != batch*topK, ...) */
  PGG_ERR_ATTR = 3,      /* topK <= 0, batch <= 0, or rowIdxType not in {0, 1} */
  PGG_ERR_DTYPE = 4,     /* dtype not in pgg_dtype */
  PGG_ERR_WORKSPACE = 5, /* workspace smaller than pgg_dx_workspace_size reports */
  PGG_ERR_CUDA = 6,      /* a CUDA runtime/driver call failed (launch, tensor map, device query) */
  PGG_ERR_ALIGN = 7,     /* pointer or row-stride alignment, see above */
  /* device-detected, written to the status word: */
  PGG_ERR_INDEX = 16,    /* an expandedRowIdx entry outside [0, M) */
  PGG_ERR_GROUPSUM = 17, /* a negative groupList entry, or sum(groupList) != M */
  PGG_ERR_NOT_PERM = 18, /* expandedRowIdx is not a permutation of [0, M) */
  PGG_ERR_TIMEOUT = 19,  /* a bounded wait inside a kernel ran out (no hang; result invalid) */
  PGG_ERR_CHECK = 20     /* checked build only (libpgg_checks.so, compiled with -DPGG_CHECKS):
                            a device bounds check on an index read from the routing tables
                            failed; the access was kept in bounds, the result is invalid */
} pgg_status;

/*
 * Workspace bytes pgg_dx_execute needs for these sizes (the two-phase
 * get-workspace-size / execute convention of section 2.2.2). Pure host code:
 * no CUDA call. Arguments as for pgg_dx_execute; L is the length of
 * expandedRowIdx. The figure grows as 12*M + 4*batch*ceil(K/128) bytes plus a
 * few KB; it is independent of N and never holds an [M, K] array.
 * Returns PGG_OK and writes *workspace_bytes, or a host error code.
 */
int pgg_dx_workspace_size(int64_t M, int64_t N, int64_t K, int64_t G, int64_t L,
                          int64_t batch, int64_t topK, int rowIdxType, pgg_dtype dtype,
                          size_t* workspace_bytes);

/*
 * Computes out[batch, K] (FP32, fully overwritten) from gradY, weight,
 * expandedRowIdx and groupList as defined at the top of this file.
 *
 *   gradY          device, [M, N] of `dtype`
 *   weight         device, [G, K, N] of `dtype`
 *   expandedRowIdx device, int64 [L], L == M, form selected by rowIdxType
 *   groupList      device, int64 [G], per-expert row counts (sum must be M)
 *   M, N, K, G     sizes; M == batch * topK, all >= 1, M < 2^31
 *   batch, topK    attributes (section "约束": both > 0)
 *   rowIdxType     0 gather form, 1 scatter form
 *   workspace      device scratch of at least pgg_dx_workspace_size bytes,
 *                  256-byte aligned, contents on entry irrelevant; holds the
 *                  status word at offset 0 after the call
 *   out            device, FP32 [batch, K]
 *   stream         CUDA stream the work is enqueued on
 *
 * Equivalent to pgg_dx_route_prep followed by pgg_dx_grouped_gemm on the same
 * workspace and stream.
 */
int pgg_dx_execute(const void* gradY, const void* weight, const int64_t* expandedRowIdx,
                   const int64_t* groupList, int64_t M, int64_t N, int64_t K, int64_t G,
                   int64_t L, int64_t batch, int64_t topK, int rowIdxType, pgg_dtype dtype,
                   void* workspace, size_t workspace_bytes, float* out, pgg_stream_t stream);

/*
 * First stage of pgg_dx_execute, exposed so that each stage can be timed on
 * its own: validates the routing on the device (writing the status word),
 * builds the per-expert row offsets (exclusive scan of groupList), the list
 * of row blocks that skips empty experts, the inverse of expandedRowIdx and,
 * per expanded row, its token and its rank among that token's rows; resets
 * the scatter-add tickets. Same arguments and errors as pgg_dx_execute,
 * without the value tensors and `out`.
 */
int pgg_dx_route_prep(const int64_t* expandedRowIdx, const int64_t* groupList, int64_t M,
                      int64_t N, int64_t K, int64_t G, int64_t L, int64_t batch, int64_t topK,
                      int rowIdxType, pgg_dtype dtype, void* workspace, size_t workspace_bytes,
                      pgg_stream_t stream);

/*
 * Second stage of pgg_dx_execute: the persistent grouped-GEMM kernel with the
 * fused, ordered scatter-add into out. Requires a pgg_dx_route_prep with the
 * same sizes, routing and workspace earlier on the same stream (or otherwise
 * ordered before it). If the status word is non-zero on entry the kernel
 * zero-fills out and returns. Same arguments and errors as pgg_dx_execute.
 */
int pgg_dx_grouped_gemm(const void* gradY, const void* weight, const int64_t* expandedRowIdx,
                        const int64_t* groupList, int64_t M, int64_t N, int64_t K, int64_t G,
                        int64_t L, int64_t batch, int64_t topK, int rowIdxType, pgg_dtype dtype,
                        void* workspace, size_t workspace_bytes, float* out,
                        pgg_stream_t stream);

/* How pgg_dx_execute will run a problem of these sizes (host only, no CUDA call). */
typedef struct {
  int32_t variant;          /* 0 = wide row blocks on CTA pairs (tensor-bound), 1 = narrow row
                               blocks (weight streaming), 2 = wide row blocks on single CTAs,
                               3 = FP32-pipe kernel (rows of N * sizeof(dtype) bytes that are
                               not a multiple of 16), 4 = owner kernel (each CTA pair owns a
                               block of d_x: few experts per token, 16-bit dtypes; falls back
                               to variant 0 when an expert's rows are not in increasing original
                               position), 5 = variant 0 with its operands copied by gather
                               warps (16-bit rows of an even length that is not a multiple of
                               8 elements); pgg_dx_execute also takes variant 5 (4-byte aligned,
                               16-bit, even N) or else 3 when gradY or weight is not 16-byte
                               aligned */
  int32_t rows_per_block;   /* expanded rows per tile: the MMA N extent (variant 4: tokens per
                               slab) */
  int32_t k_per_block;      /* output columns per CTA and tile (128; a CTA pair covers 256) */
  int32_t stages;           /* shared-memory pipeline depth */
  int32_t k_blocks;         /* ceil(K / k_per_block) */
  int32_t band_k_blocks;    /* k-blocks per band of the tile order */
  int64_t max_row_blocks;   /* upper bound on row blocks: ceil(M/rows_per_block) + G */
  size_t workspace_bytes;   /* as pgg_dx_workspace_size */
  int32_t threads;          /* threads per CTA of the grouped-GEMM kernel */
  int32_t smem_bytes;       /* dynamic shared memory per CTA */
  int32_t cta_pair;         /* 1: clusters of two CTAs share each tile (tcgen05 cta_group::2) */
} pgg_plan_info;

int pgg_dx_plan(int64_t M, int64_t N, int64_t K, int64_t G, int64_t L, int64_t batch,
                int64_t topK, int rowIdxType, pgg_dtype dtype, pgg_plan_info* info);

/* Human-readable name of a pgg_status code (static string). */
const char* pgg_status_string(int status);

/*
 * Test hooks (process-wide; not needed in normal use).
 * pgg_debug_set_wait_limit_ns: time limit of every bounded wait inside the
 *   kernels (default 2e9 ns). 0 restores the default.
 * pgg_debug_set_ticket_bias: added to the ticket count each ordered
 *   scatter-add waits for; a positive bias makes every wait of a row with
 *   rank > 0 run out, which exercises the PGG_ERR_TIMEOUT path. 0 = off.
 * pgg_debug_force_variant: -1 = automatic (default), 0 .. 5 = force the
 *   variant reported by pgg_dx_plan (2, 4 and 5 exist for the 16-bit dtypes
 *   only, 5 for an even N only; rows that are not a multiple of 16 bytes
 *   take variant 5 when they can, else 3). The 4-bit products take 0 (many
 *   rows an expert), 1 (codes streamed) and 3 where their sizes allow them.
 * pgg_debug_set_band_k_blocks: k-blocks per band of the tile order (0 =
 *   automatic). The result does not depend on it, bit for bit: only the time
 *   order of the tiles changes, never the order of the additions.
 * pgg_debug_set_hold_release: non-zero makes the epilogue of the owner d_x
 *   variant, of the forward and of the weight-gradient kernels withhold its
 *   first release of an accumulator, so that the MMA thread's bounded wait
 *   for it runs out: exercises PGG_ERR_TIMEOUT in those kernels (every CTA
 *   role gives up, drains its copies and MMAs and frees tensor memory). A CTA
 *   pair with fewer than three tiles never waits for that release. 0 = off.
 */
void pgg_debug_set_wait_limit_ns(uint64_t ns);
void pgg_debug_set_ticket_bias(uint32_t bias);
void pgg_debug_force_variant(int variant);
void pgg_debug_set_band_k_blocks(int k_blocks);
void pgg_debug_set_hold_release(int hold);

/*
 * pgg_dx_execute for callers that cannot allocate device memory. (The pages
 * have no counterpart of this call; it is a service of this library.)
 *
 * Who needs it: code that has no allocator at hand when the gradient is due
 * -- a plugin inside a framework that owns all device memory, a serving or
 * real-time runtime that reserved HBM up front and forbids cudaMalloc later,
 * plain C code without an allocator handle. Such a caller passes the same
 * inputs and `out` as to pgg_dx_execute, but no workspace: the call uses a
 * fixed 8 MiB scratch array that the library's CUDA module reserves on every
 * device that loads the library, held until the process exits. It calls no
 * cudaMalloc, cudaFree or other allocating routine.
 *
 *   status  optional device pointer (may be NULL); after the work on `stream`
 *           has finished it holds the device-detected status word that
 *           pgg_dx_execute would have left at the start of its workspace.
 *
 * Returns PGG_ERR_WORKSPACE when pgg_dx_workspace_size for these sizes exceeds
 * 8 MiB (8388608 bytes; e.g. M = 108000, K = 7168 needs 4.3 MB), and
 * otherwise what pgg_dx_execute returns.
 *
 * Each call looks up the scratch array's device address (cudaGetSymbolAddress)
 * on the current device, so the address stays valid after cudaDeviceReset;
 * only a call made while `stream` is being captured reuses the address that
 * the previous call on the device looked up, so make the first call on a
 * device before any stream capture on it. Every call on a device shares the one
 * array, and each call re-initialises what it needs, so leftover contents from
 * the previous call do no harm -- but two calls whose work overlaps on the GPU
 * (for example on two streams without ordering between them) race on the
 * array and give wrong results. Order such calls on one stream.
 */
int pgg_dx_execute_static_scratch(const void* gradY, const void* weight,
                                  const int64_t* expandedRowIdx, const int64_t* groupList,
                                  int64_t M, int64_t N, int64_t K, int64_t G, int64_t L,
                                  int64_t batch, int64_t topK, int rowIdxType, pgg_dtype dtype,
                                  float* out, uint32_t* status, pgg_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Weight gradient (the companion operator; page "MoeInitRoutingGroupedMatmulGrad
 * design", section 1.2 "为何不计算 d_weight", item 3: a separate grouped matmul
 * expanded_x^T @ d_y per expert; section 1.1: the forward's MoeInitRouting
 * lays out the token rows by expert, expanded_x[i] = x[batch(i)]):
 *
 *     dweight[g, k, n] = sum_{expanded rows i of expert g} x[batch(i), k] * gradY[i, n]
 *
 *   x              device, [batch, K] of `dtype`: the forward input in original
 *                  token order. expanded_x is never materialised: its rows are
 *                  gathered from x by token. (A caller that kept expanded_x
 *                  [M, K] instead passes it as x with batch = M, topK = 1 and
 *                  expandedRowIdx = 0 .. M-1, groupList unchanged.)
 *   gradY          device, [M, N] of `dtype`, expanded order
 *   expandedRowIdx, groupList, M, N, K, G, L, batch, topK, rowIdxType, dtype:
 *                  as for pgg_dx_execute
 *   out_dtype      dtype of dweight: `dtype` (the page sizes d_weight in the
 *                  input precision) or PGG_F32; else PGG_ERR_DTYPE. Accumulation
 *                  is always FP32; a 16-bit output is rounded to nearest even.
 *   workspace      at least pgg_dw_workspace_size bytes, 256-byte aligned;
 *                  status word at offset 0 as for pgg_dx_execute
 *   dweight        device, [G, K, N] of out_dtype, fully overwritten; an expert
 *                  with no rows gets zeros; zero-filled when the routing
 *                  validation fails
 *
 * Each element is produced by one tile with a fixed order of additions (the
 * expert's rows in increasing order, in MMA blocks of 16), so the result is
 * bitwise repeatable. Runs on the tensor cores when dtype is 16-bit, K and N
 * are multiples of 8 and x, gradY, dweight are 16-byte aligned (variant 0);
 * also on the tensor cores, with the gradY rows copied 4 bytes at a time by
 * the gather warps and dweight written with 4-byte stores, when N is even but
 * not a multiple of 8 (or gradY / dweight are only 4-byte aligned) while K is
 * a multiple of 8 and x is 16-byte aligned (variant 5); otherwise on the FP32
 * pipes (variant 3, also forced by pgg_debug_force_variant(3)). Alignment: x
 * and gradY aligned to their element size, dweight to its element size.
 */
int pgg_dw_workspace_size(int64_t M, int64_t N, int64_t K, int64_t G, int64_t L,
                          int64_t batch, int64_t topK, int rowIdxType, pgg_dtype dtype,
                          size_t* workspace_bytes);

int pgg_dw_execute(const void* x, const void* gradY, const int64_t* expandedRowIdx,
                   const int64_t* groupList, int64_t M, int64_t N, int64_t K, int64_t G,
                   int64_t L, int64_t batch, int64_t topK, int rowIdxType, pgg_dtype dtype,
                   pgg_dtype out_dtype, void* workspace, size_t workspace_bytes, void* dweight,
                   pgg_stream_t stream);

/*
 * Second stage of pgg_dw_execute, exposed so that the kernel can be timed on
 * its own: the weight-gradient kernel alone, on a workspace prepared by
 * pgg_dx_route_prep with the same sizes and routing (the routing step is the
 * same for both gradients). Same arguments and errors as pgg_dw_execute.
 */
int pgg_dw_grouped_gemm(const void* x, const void* gradY, const int64_t* expandedRowIdx,
                        const int64_t* groupList, int64_t M, int64_t N, int64_t K, int64_t G,
                        int64_t L, int64_t batch, int64_t topK, int rowIdxType, pgg_dtype dtype,
                        pgg_dtype out_dtype, void* workspace, size_t workspace_bytes,
                        void* dweight, pgg_stream_t stream);

/*
 * How pgg_dw_execute runs these sizes with 16-byte aligned pointers: variant 0
 * (tensor cores: k_per_block = 128 output rows, 256 output columns, 64
 * reduction rows per stage), 5 (the same with the gradY rows gathered by
 * warps: N even, not a multiple of 8) or 3 (FP32 pipes: 64 rows, 128
 * columns, 32 rows per step); k_blocks and band_k_blocks hold the k and n
 * blocks per expert.
 */
int pgg_dw_plan(int64_t M, int64_t N, int64_t K, int64_t G, int64_t L, int64_t batch,
                int64_t topK, int rowIdxType, pgg_dtype dtype, pgg_plan_info* info);

/*
 * ---------------------------------------------------------------------------
 * Forward (the operation these are the gradients of; page
 * "MoeInitRoutingGroupedMatmulGrad design", sections 1.1 and 1.2, forward
 * chain: MoeInitRouting(x) -> expanded_x, GroupedMatmul(expanded_x, weight)
 * -> y):
 *
 *     y[i, n] = sum_k x[batch(i), k] * weight[g(i), k, n]      (i in expanded order)
 *
 *   x              device, [batch, K] of `dtype`, original token order; the rows
 *                  of expanded_x are gathered from it by the routing, never
 *                  materialised
 *   weight         device, [G, K, N] of `dtype`
 *   expandedRowIdx, groupList, M, N, K, G, L, batch, topK, rowIdxType, dtype:
 *                  as for pgg_dx_execute
 *   out_dtype      dtype of y: `dtype` or PGG_F32 (else PGG_ERR_DTYPE); FP32
 *                  accumulation, one round-to-nearest-even for 16-bit outputs
 *   workspace      at least pgg_fwd_workspace_size bytes, 256-byte aligned;
 *                  status word at offset 0 as for pgg_dx_execute
 *   y              device, [M, N] of out_dtype, expanded order, fully
 *                  overwritten; zero-filled when the routing validation fails
 *
 * Each element is one dot product over k in a fixed order: bitwise
 * repeatable. Tensor cores when dtype is 16-bit, K and N are multiples of 8
 * and x, weight, y are 16-byte aligned (variant 0); also on the tensor cores,
 * with the weight rows copied 4 bytes at a time by the gather warps and y
 * written with 4-byte stores, when N is even but not a multiple of 8 (or
 * weight / y are only 4-byte aligned) while K is a multiple of 8 and x is
 * 16-byte aligned (variant 5); otherwise the FP32 pipes (variant 3, also forced
 * by pgg_debug_force_variant(3)). x and weight aligned to their element size,
 * y to its element size.
 */
int pgg_fwd_workspace_size(int64_t M, int64_t N, int64_t K, int64_t G, int64_t L,
                           int64_t batch, int64_t topK, int rowIdxType, pgg_dtype dtype,
                           size_t* workspace_bytes);

int pgg_fwd_execute(const void* x, const void* weight, const int64_t* expandedRowIdx,
                    const int64_t* groupList, int64_t M, int64_t N, int64_t K, int64_t G,
                    int64_t L, int64_t batch, int64_t topK, int rowIdxType, pgg_dtype dtype,
                    pgg_dtype out_dtype, void* workspace, size_t workspace_bytes, void* y,
                    pgg_stream_t stream);

/*
 * The two stages of pgg_fwd_execute, exposed so that each can be timed on its
 * own: the routing step (validation, expert offsets, row blocks of up to 256
 * rows, tokens) and the forward kernel on the workspace it prepared. Same
 * arguments and errors as pgg_fwd_execute (the routing step without the value
 * tensors and y).
 */
int pgg_fwd_route_prep(const int64_t* expandedRowIdx, const int64_t* groupList, int64_t M,
                       int64_t N, int64_t K, int64_t G, int64_t L, int64_t batch, int64_t topK,
                       int rowIdxType, pgg_dtype dtype, void* workspace, size_t workspace_bytes,
                       pgg_stream_t stream);

int pgg_fwd_grouped_gemm(const void* x, const void* weight, const int64_t* expandedRowIdx,
                         const int64_t* groupList, int64_t M, int64_t N, int64_t K, int64_t G,
                         int64_t L, int64_t batch, int64_t topK, int rowIdxType, pgg_dtype dtype,
                         pgg_dtype out_dtype, void* workspace, size_t workspace_bytes, void* y,
                         pgg_stream_t stream);

/*
 * How pgg_fwd_execute runs these sizes with 16-byte aligned pointers: variant
 * 0 (tensor cores on CTA pairs: row blocks of rows_per_block = 256 expanded
 * rows x 256 n, k_per_block = 64 per stage), 5 (the same with the weight rows
 * gathered by warps: N even, not a multiple of 8) or 3 (FP32 pipes: 64 rows x
 * 128 n, 32 k per step; also when x holds 64 GiB or more, batch * K / 8 >=
 * 2^32 - 1, since the tensor-core kernel addresses x rows with 32-bit offsets
 * in 16-byte units); band_k_blocks holds the n blocks per row block.
 */
int pgg_fwd_plan(int64_t M, int64_t N, int64_t K, int64_t G, int64_t L, int64_t batch,
                 int64_t topK, int rowIdxType, pgg_dtype dtype, pgg_plan_info* info);

/*
 * ---------------------------------------------------------------------------
 * Probs-weighted unpermute backward (page "NPU DeepSeek-V3.2-Exp TileLang
 * operator practice", section moe_token_unpermute_grad). For the combine that
 * follows the expert matmul, out[b] = sum_j prob[b, j] * permuted[row(b, j)]:
 *
 *     perm_grad[row(b, j), h] = d_out[b, h] * prob[b, j]        (prob = 1 when probs is NULL)
 *     probs_grad[b, j]        = sum_h d_out[b, h] * permuted[row(b, j), h]
 *
 * with row(b, j) the expanded row of original position b * topK + j, read from
 * expandedRowIdx in the rowIdxType form (0 gather, 1 scatter, as above). No
 * experts are involved. perm_grad is the gradY of pgg_dx_execute and
 * pgg_dw_execute.
 *
 *   permuted       device, [M, H] of `dtype` (may be NULL when probs is NULL)
 *   d_out          device, [batch, H] of `dtype`
 *   probs          device, [batch, topK] of `dtype`, or NULL (plain scatter copy)
 *   probs_grad_dtype  `dtype` or PGG_F32 (the dot products accumulate in FP32)
 *   workspace      pgg_unpermute_grad_workspace_size bytes, 256-byte aligned;
 *                  status word at offset 0 (PGG_ERR_INDEX / PGG_ERR_NOT_PERM
 *                  zero-fill both outputs)
 *   perm_grad      device, [M, H] of `dtype`, fully overwritten
 *   probs_grad     device, [batch, topK], required with probs
 *
 * perm_grad is d_out * prob rounded once to `dtype`; each probs_grad is one
 * FP32 sum in a fixed order: bitwise repeatable. All pointers aligned to their
 * element size; 16-byte vector access when H * sizeof(dtype) is a multiple of
 * 16 and the row pointers are 16-byte aligned.
 */
int pgg_unpermute_grad_workspace_size(int64_t M, int64_t batch, int64_t topK,
                                      size_t* workspace_bytes);

int pgg_unpermute_grad(const void* permuted, const void* d_out, const void* probs,
                       const int64_t* expandedRowIdx, int64_t M, int64_t H, int64_t batch,
                       int64_t topK, int rowIdxType, pgg_dtype dtype, pgg_dtype probs_grad_dtype,
                       void* workspace, size_t workspace_bytes, void* perm_grad, void* probs_grad,
                       pgg_stream_t stream);

/*
 * The same call in two stream-ordered stages, for callers that validate the
 * routing once and apply it to several tensors, and for timing the kernel
 * alone. pgg_unpermute_grad is exactly prep followed by apply.
 *   pgg_unpermute_grad_prep   index validation and the inverse map, into the
 *                             workspace (status word at offset 0).
 *   pgg_unpermute_grad_apply  the unpermute kernel; reads the workspace that a
 *                             prep of the same expandedRowIdx (same M, batch,
 *                             topK, rowIdxType) filled earlier on the stream.
 *                             Its arguments and checks are those of
 *                             pgg_unpermute_grad.
 */
int pgg_unpermute_grad_prep(const int64_t* expandedRowIdx, int64_t M, int64_t batch, int64_t topK,
                            int rowIdxType, void* workspace, size_t workspace_bytes,
                            pgg_stream_t stream);

int pgg_unpermute_grad_apply(const void* permuted, const void* d_out, const void* probs,
                             const int64_t* expandedRowIdx, int64_t M, int64_t H, int64_t batch,
                             int64_t topK, int rowIdxType, pgg_dtype dtype,
                             pgg_dtype probs_grad_dtype, void* workspace, size_t workspace_bytes,
                             void* perm_grad, void* probs_grad, pgg_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Router: the top-k choice of experts from router logits, the routing weights,
 * and the expanded order that the grouped products of this file read.
 *
 *     s          = softmax(logits[b]) over all G experts, or sigmoid(logits[b])
 *     key[b, e]  = logits[b, e] + bias[e], or with PGG_BIAS_ON_SCORE s[e] + bias[e]
 *                  (bias takes part in the choice only)
 *     experts[b] = the topK largest keys in decreasing order, the lowest index
 *                  first among equals
 *     probs[b,j] = scale * s[experts[b,j]], or with `renormalize`
 *                  scale * s[experts[b,j]] / sum over the chosen of s
 *     expandedRowIdx, groupList: the pairs p = b * topK + j sorted by
 *                  (experts[b,j], p), in the rowIdxType form, and the experts' counts
 *
 *   score    pgg_score, with PGG_BIAS_ON_SCORE added where the bias was learnt
 *            for the scores (a selection bias that balances the experts' load
 *            without an auxiliary loss is). Without a bias the choice goes by
 *            the logits either way.
 *   logits   device, [batch, G] of `dtype`; -inf masks an expert (weight 0, its key
 *            -inf with any finite bias). A token whose experts are all masked takes
 *            the lowest indices; where the chosen scores are all 0 in fp32 the
 *            weights are 0. A NaN key sorts below every other, so that the order
 *            stays valid. Scores follow IEEE arithmetic: a softmax over a NaN or a
 *            +inf is NaN, so are all of the token's weights; a sigmoid is NaN for a
 *            NaN alone (renormalised: all weights, if that one is chosen).
 *   bias     device, fp32 [G], or NULL
 *   G <= 1024, topK <= min(G, 32), else PGG_ERR_SHAPE
 *   workspace at least pgg_route_workspace_size bytes, 256-byte aligned; the
 *            status word at offset 0 is 0 after the call
 *   probs    device, fp32 [batch, topK];  experts device, int64 [batch, topK]
 *   expandedRowIdx device, int64 [batch * topK];  groupList device, int64 [G]
 *
 * Weights are computed in fp32; the order depends on no atomic's order.
 */
typedef enum {
  PGG_SCORE_SOFTMAX = 0,
  PGG_SCORE_SIGMOID = 1,
  PGG_BIAS_ON_SCORE = 16 /* added to one of them, pgg_route_execute only */
} pgg_score;

int pgg_route_workspace_size(int64_t batch, int64_t G, int64_t topK, size_t* workspace_bytes);

int pgg_route_execute(const void* logits, const float* bias, int64_t batch, int64_t G,
                      int64_t topK, int rowIdxType, pgg_dtype dtype, pgg_score score,
                      int renormalize, float scale, void* workspace, size_t workspace_bytes,
                      float* probs, int64_t* experts, int64_t* expandedRowIdx,
                      int64_t* groupList, pgg_stream_t stream);

/*
 * Gradient of probs for the logits (bias gets none: the choice is piecewise
 * constant). d_logits [batch, G] of `dtype` is written whole; needs no
 * workspace. A token whose `experts` hold an index outside [0, G) or one
 * twice gets NaN. Only the plain softmax reads more than the chosen logits.
 * d_logits may be logits itself; another overlap is not allowed.
 */
int pgg_route_grad(const float* d_probs, const void* logits, const int64_t* experts,
                   int64_t batch, int64_t G, int64_t topK, pgg_dtype dtype, pgg_score score,
                   int renormalize, float scale, void* d_logits, pgg_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Gated expert product (the first half of an expert's feed-forward part):
 *
 *     [gate | up][i, :] = x[batch(i), :] weight[g(i), :, :]
 *     h[i, f] = prob * silu(gate[i, f]) * up[i, f],  silu(t) = t / (1 + exp(-t))
 *
 * with prob = probs[original position of row i], or 1 when probs is NULL. The
 * second half with the weighted combination of a token's experts is
 * pgg_dx_execute(h, w_down [G, H, F]), whose output is [batch, H].
 *
 *   x        device, [batch, K] of `dtype`, original token order
 *   weight   device, [G, K, 2F] of `dtype`: F gate columns, then F up columns
 *   probs    device, fp32 [batch, topK], or NULL
 *   expandedRowIdx, groupList, M, G, L, batch, topK, rowIdxType: as for
 *            pgg_dx_execute
 *   h        device, [M, F] of `dtype`, expanded order
 *   gate_up  device, [M, 2F] of `dtype` (what pgg_swiglu_grad reads), or NULL
 *   workspace at least pgg_swiglu_workspace_size bytes, 256-byte aligned; status
 *            word at offset 0. When the routing is not valid both outputs are
 *            zero-filled.
 *
 * Accumulation, activation and weight are fp32; each output is rounded once.
 * Bitwise repeatable.
 */
int pgg_swiglu_workspace_size(int64_t M, int64_t F, int64_t K, int64_t G, int64_t L,
                              int64_t batch, int64_t topK, int rowIdxType, pgg_dtype dtype,
                              size_t* workspace_bytes);

int pgg_swiglu_execute(const void* x, const void* weight, const int64_t* expandedRowIdx,
                       const int64_t* groupList, const float* probs, int64_t M, int64_t F,
                       int64_t K, int64_t G, int64_t L, int64_t batch, int64_t topK,
                       int rowIdxType, pgg_dtype dtype, void* workspace, size_t workspace_bytes,
                       void* h, void* gate_up, pgg_stream_t stream);

/*
 * How pgg_swiglu_execute runs these sizes with 16-byte aligned tensors (16-bit
 * dtypes with K and F multiples of 8, else, and for other tensors, variant 3):
 * variant 0 (tensor cores, row blocks of up to 256 rows on CTA pairs), 1
 * (tensor cores, row blocks of up to 16 .. 128 rows, the weight streamed: few
 * rows per expert) or 3 (FP32 pipes: any dtype, size and alignment). The
 * fields not named here are 0. Host only, no CUDA call.
 */
int pgg_swiglu_plan(int64_t M, int64_t F, int64_t K, int64_t G, int64_t L, int64_t batch,
                    int64_t topK, int rowIdxType, pgg_dtype dtype, pgg_plan_info* info);

/*
 * Gradient of the gate, from d_h and the kept gate_up:
 *
 *     d_up = prob d_h silu(gate);  d_gate = prob d_h up silu'(gate)
 *     d_probs[original position of i] = sum over f of d_h silu(gate) up
 *     h = prob silu(gate) up
 *
 * d_gate_up [M, 2F] is the gradY of pgg_dx_execute and pgg_dw_execute with the
 * gate's weight; h [M, F] that of pgg_dw_execute with the down projection's.
 *   probs    fp32 [batch, topK] or NULL;  d_probs fp32 [batch, topK] or NULL
 *            (not without probs: PGG_ERR_NULL);  h may be NULL
 *   workspace pgg_swiglu_grad_workspace_size bytes, 256-byte aligned; status word
 *            at offset 0 (an index that is not a permutation zero-fills the outputs)
 */
int pgg_swiglu_grad_workspace_size(int64_t M, int64_t batch, int64_t topK,
                                   size_t* workspace_bytes);

int pgg_swiglu_grad(const void* d_h, const void* gate_up, const float* probs,
                    const int64_t* expandedRowIdx, int64_t M, int64_t F, int64_t batch,
                    int64_t topK, int rowIdxType, pgg_dtype dtype, void* workspace,
                    size_t workspace_bytes, void* d_gate_up, float* d_probs, void* h,
                    pgg_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * A shared projection with one low-rank adapter per token:
 *
 *     y[t, :] = x[t, :] weight + scale[ad] (x[t, :] a[ad]) b[ad]^T,  ad = adapter[t]
 *
 *   x        device, [T, K] of `dtype`;  weight device, [K, N] of `dtype`
 *   a        device, [A, K, R] of `dtype`;  b device, [A, N, R] of `dtype` (the
 *            rank is innermost in both); an adapter of a smaller rank is stored
 *            with zero columns
 *   adapter  device, int64 [T], -1 = no adapter; another value outside [0, A)
 *            sets PGG_ERR_INDEX and zero-fills the outputs
 *   scale    device, fp32 [A], or NULL (1)
 *   A <= 1023, R <= 256, T < 2^30, else PGG_ERR_SHAPE
 *   workspace at least pgg_adapters_workspace_size bytes, 256-byte aligned; status
 *            word at offset 0
 *   y        device, [T, N] of `dtype`
 *
 * Tokens may be in any order. Sums are fp32, the low-rank row scale x a among them:
 * it enters the second product in fp32, or as the sum of two values of `dtype`
 * (2^-16 of it is lost in bf16, 2^-21 in fp16, where it may reach 131008), and y is
 * rounded once. What one adapter's weights hold (infinities, NaN) does not reach
 * the tokens of another. No output may overlap an input.
 */
int pgg_adapters_workspace_size(int64_t T, int64_t K, int64_t N, int64_t R, int64_t A,
                                pgg_dtype dtype, size_t* workspace_bytes);

int pgg_adapters_execute(const void* x, const void* weight, const void* a, const void* b,
                         const int64_t* adapter, const float* scale, int64_t T, int64_t K,
                         int64_t N, int64_t R, int64_t A, pgg_dtype dtype, void* workspace,
                         size_t workspace_bytes, void* y, pgg_stream_t stream);

/*
 * How pgg_adapters_execute runs these sizes with 16-byte aligned tensors:
 * variant 0 (tensor cores, tokens sorted by adapter, blocks of 256), 1 (tensor
 * cores, blocks of up to 64 tokens in the caller's order, the weight streamed
 * and the low-rank part on the FP32 pipes) or 3 (FP32 pipes); rows_per_block is
 * that of the projection, max_row_blocks counts the low-rank rows' blocks.
 */
int pgg_adapters_plan(int64_t T, int64_t K, int64_t N, int64_t R, int64_t A, pgg_dtype dtype,
                      pgg_plan_info* info);

/*
 * Its gradient with the projection frozen:
 *
 *     v = scale (d_y b[ad]),  d_x = d_y weight^T + v a[ad]^T  [T, K], may be NULL
 *     d_a[ad] = sum over its tokens of x^T v                  [A, K, R]
 *     d_b[ad] = sum over its tokens of d_y^T (scale x a[ad])  [A, N, R]
 *
 * all of `dtype`; an adapter without tokens gets zeros. Sums are fp32. v and
 * u = scale x a[ad] enter the second products as the sums of two values of `dtype`
 * (as in the forward) where 16-bit tensors have widths that are multiples of 8 and
 * are 16-byte aligned, else rounded once to `dtype`. No output may overlap an
 * input: d_x, d_a and d_b are written side by side.
 */
int pgg_adapters_grad_workspace_size(int64_t T, int64_t K, int64_t N, int64_t R, int64_t A,
                                     pgg_dtype dtype, size_t* workspace_bytes);

int pgg_adapters_grad(const void* d_y, const void* x, const void* weight, const void* a,
                      const void* b, const int64_t* adapter, const float* scale, int64_t T,
                      int64_t K, int64_t N, int64_t R, int64_t A, pgg_dtype dtype,
                      void* workspace, size_t workspace_bytes, void* d_x, void* d_a, void* d_b,
                      pgg_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Products with 4-bit expert weights (serving): the forward, the gated product
 * and the down projection with the combination, with weights
 *
 *     w[g, n, k] = scale[g, n, k / groupSize] (code[g, n, k] - zero[g, n, k / groupSize])
 *
 *     PGG_W4_ROWS      out[i, n] = sum_k x[batch(i), k] w[g(i), n, k]          [M, N]
 *     PGG_W4_GATED     out[i, f] = prob silu(gate) up, gate = column f, up = column N + f of
 *                      the same product                                        [M, N]
 *     PGG_W4_COMBINED  out[b, n] = sum over the rows i of token b of
 *                      sum_k x[i, k] w[g(i), n, k], as pgg_dx_execute          [batch, N]
 *
 *   x        device, of `dtype`: [batch, K] in token order; combined: [M, K] in
 *            expanded order
 *   codes    device, uint8 [G, C, ceil(K / 2)], C = N (gated: 2 N): byte j of a
 *            column holds code k = 2 j in its lower half and k = 2 j + 1 in its
 *            upper (which is not used where K is odd and ends there)
 *   scales   device, [G, C, ceil(K / groupSize)] of scale_dtype, `dtype` or PGG_F32
 *   zeros    device, uint8 of the same shape (0 .. 255; codes are 0 .. 15), or NULL: 8
 *   expandedRowIdx, groupList, M, G, L, batch, topK, rowIdxType: as for
 *            pgg_dx_execute
 *   probs    gated: device, fp32 [batch, topK], or NULL (1); else NULL
 *   groupSize at least 1; the last group of a column may be shorter
 *   out_dtype rows: `dtype` or PGG_F32; gated: `dtype`; combined: PGG_F32
 *   workspace at least pgg_w4_workspace_size bytes, 256-byte aligned; status word
 *            at offset 0. When the routing is not valid the output is zero-filled.
 *
 * Sums are fp32, and each output is rounded once. The weights are not rounded to
 * 16 bits. Few rows an expert multiply x with the codes and then a group's fp32 sum
 * with its scale. fp32 x, and K or groupSize that is no multiple of 32, form each
 * weight in fp32. Many rows an expert multiply with the weight as one fp16 number
 * where that is exact (bf16 scales, no zeros) and as the sum of two (22 bits)
 * otherwise, and bring the weights of a column to fp16's range by a power of two: a
 * weight there is off by up to (|code - zero| + 1) 2^-35 of its column's largest
 * scale (with zeros above 16 up to 2^-31). In all of them a 16-bit x is brought to
 * fp16's range a row at a time and keeps its bits but for what lies below 2^-35 of
 * the row's largest value. Bitwise repeatable.
 *
 * A row of x with infinities or NaN gives what the sums of its weights times these
 * give, +-inf or NaN. A scale that is not finite leaves no result of its
 * column finite, whether +-inf or NaN.
 */
typedef enum { PGG_W4_ROWS = 0, PGG_W4_GATED = 1, PGG_W4_COMBINED = 2 } pgg_w4_product;

int pgg_w4_workspace_size(pgg_w4_product product, int64_t M, int64_t N, int64_t K, int64_t G,
                          int64_t L, int64_t batch, int64_t topK, int rowIdxType,
                          int64_t groupSize, pgg_dtype dtype, size_t* workspace_bytes);

int pgg_w4_execute(pgg_w4_product product, const void* x, const uint8_t* codes,
                   const void* scales, const uint8_t* zeros, const int64_t* expandedRowIdx,
                   const int64_t* groupList, const float* probs, int64_t M, int64_t N, int64_t K,
                   int64_t G, int64_t L, int64_t batch, int64_t topK, int rowIdxType,
                   int64_t groupSize, pgg_dtype dtype, pgg_dtype scale_dtype, pgg_dtype out_dtype,
                   void* workspace, size_t workspace_bytes, void* out, pgg_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * The norms before and after a block, with its gate and residual scale, in one
 * pass: what stands between the block's output y and the next block's input h.
 *
 *     n = N_post(y),  r = residual_scale x + gate n,  h = N_pre(r)
 *     N(v) = (v - mean) / sqrt(var + eps) (weight_offset + weight) + bias    PGG_NORM_LAYER
 *     N(v) = v / sqrt(mean of v^2 + eps) (weight_offset + weight)            PGG_NORM_RMS
 *     N(v) = v                                                               PGG_NORM_NONE
 *
 *   x        device, [T, H] of `dtype`: the residual stream before the block
 *   y        device, [T, H] of y_dtype, `dtype` or PGG_F32 (what pgg_dx_execute
 *            leaves), or NULL: r = residual_scale x (then post and gate_kind are none)
 *   gate     device, of param_dtype, as gate_kind says; NULL for PGG_GATE_NONE
 *   post_weight, post_bias, pre_weight, pre_bias
 *            device, [H] of param_dtype, each may be NULL (the factor is then 1, the
 *            bias 0); none without a norm, no bias with PGG_NORM_RMS: PGG_ERR_ATTR
 *   param_dtype `dtype` or PGG_F32
 *   r, h     device, [T, H] of `dtype`; r may be NULL, h is NULL exactly if pre is
 *            PGG_NORM_NONE, one of them is written
 *
 * All in fp32, the pre norm on r before r is rounded. No device-detected errors.
 * r may be x; another overlap of outputs and inputs is not allowed.
 */
typedef enum { PGG_NORM_NONE = 0, PGG_NORM_RMS = 1, PGG_NORM_LAYER = 2 } pgg_norm;

/* Shape of the gate: [H], [T] or [T, H]. */
typedef enum {
  PGG_GATE_NONE = 0,
  PGG_GATE_CHANNEL = 1,
  PGG_GATE_TOKEN = 2,
  PGG_GATE_FULL = 3
} pgg_gate;

int pgg_block_norm(const void* x, const void* y, const void* gate, const void* post_weight,
                   const void* post_bias, const void* pre_weight, const void* pre_bias, int64_t T,
                   int64_t H, pgg_dtype dtype, pgg_dtype y_dtype, pgg_dtype param_dtype,
                   pgg_norm post, pgg_norm pre, pgg_gate gate_kind, float residual_scale,
                   float weight_offset, float eps, void* r, void* h, pgg_stream_t stream);

/*
 * Its gradient, from d_r (the gradient of r by its later uses) and d_h, the kept
 * r and y:
 *
 *     g = d_r + N_pre'(d_h at r),  d_x = residual_scale g
 *     d_gate = g n, summed over what the gate was broadcast over
 *     d_y = N_post'(g gate at y), and the sums over rows for weights and biases
 *
 *   d_r      device, [T, H] of `dtype`, or NULL (0); d_h: [T, H] of dh_dtype,
 *            `dtype` or PGG_F32; NULL exactly if pre is PGG_NORM_NONE
 *   r        device, [T, H] of `dtype`, NULL exactly if pre is PGG_NORM_NONE
 *   d_x      device, [T, H] of `dtype`;  d_y the same, NULL exactly if y is
 *   d_gate   fp32 [H] or [T]; for PGG_GATE_FULL [T, H] of param_dtype; NULL
 *            exactly if gate is
 *   d_post_weight, d_post_bias, d_pre_weight, d_pre_bias
 *            device, fp32 [H], each may be NULL; not without its parameter
 *   workspace at least pgg_block_norm_grad_workspace_size bytes, 256-byte aligned;
 *            the status word at offset 0 is 0 after the call
 *
 * Sums over rows are fp32, in an order that depends on the sizes alone. d_x may
 * be d_r; another overlap of outputs and inputs is not allowed.
 */
int pgg_block_norm_grad_workspace_size(int64_t T, int64_t H, size_t* workspace_bytes);

int pgg_block_norm_grad(const void* d_r, const void* d_h, const void* r, const void* y,
                        const void* gate, const void* post_weight, const void* post_bias,
                        const void* pre_weight, const void* pre_bias, int64_t T, int64_t H,
                        pgg_dtype dtype, pgg_dtype y_dtype, pgg_dtype dh_dtype,
                        pgg_dtype param_dtype, pgg_norm post, pgg_norm pre, pgg_gate gate_kind,
                        float residual_scale, float weight_offset, float eps, void* workspace,
                        size_t workspace_bytes, void* d_x, void* d_y, void* d_gate,
                        float* d_post_weight, float* d_post_bias, float* d_pre_weight,
                        float* d_pre_bias, pgg_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * The global norm of a list of gradients, and the gradients clipped to it:
 *
 *     norm = |scale| sqrt(sum over all tensors of g^2)
 *     out  = g c,  c = scale min(1, max_norm / (norm + eps))
 *
 *   count    number of tensors, 0 or more
 *   grads    host array of count device pointers (NULL where a size is 0)
 *   sizes    host array: elements of each, 0 or more;  dtypes: host array
 *   scale    multiplies every gradient (1 / the loss scale, 1 / accumulated steps)
 *   max_norm 0 or more (may be infinite); eps 0 or more
 *   norm     device, fp32
 *   out      host array of device pointers; out[i] has the dtype of grads[i]. It is
 *            grads[i] itself or overlaps no gradient, and overlaps no other output
 *            (one tensor twice in the list, say): else PGG_ERR_ATTR
 *   workspace at least pgg_clip_workspace_size bytes, 256-byte aligned; the status
 *            word at offset 0 is 0 after the call
 *
 * The host arrays are read during the call only. A norm that is not finite clips
 * nothing: c = scale, and the caller sees it in `norm`. Where c is 1 a gradient
 * that is its own output is not written. Squares are summed in fp32 and fp64;
 * neither their sum nor a small gradient's square leaves the range.
 */
int pgg_clip_workspace_size(int64_t count, size_t* workspace_bytes);

int pgg_grad_norm(int64_t count, const void* const* grads, const int64_t* sizes,
                  const pgg_dtype* dtypes, float scale, void* workspace, size_t workspace_bytes,
                  float* norm, pgg_stream_t stream);

int pgg_clip_grads(int64_t count, const void* const* grads, const int64_t* sizes,
                   const pgg_dtype* dtypes, float max_norm, float eps, float scale,
                   void* workspace, size_t workspace_bytes, float* norm, void* const* out,
                   pgg_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PGG_H */
