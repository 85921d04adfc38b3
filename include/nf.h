/*
 * nf.h -- C ABI of the GB300 (sm_103a) inner-persistent row-normalization
 * library (libnf.so).
 *
 * What the library computes, and where the operations come from:
 *   - Fused residual add + RMSNorm forward, in place: the RMSNormAdd
 *     benchmark with in-place update semantics in "optimize inner persistent
 *     scheduler for static fusion" (NVIDIA/Fuser PR #5281), changes
 *     walkthrough, test_rmsnorm_add_fwd.py entry.
 *   - RMSNorm forward and LayerNorm forward: "TMA inner persistent
 *     scheduler" (NVIDIA/Fuser PR #5587), description (RMS norm and layer
 *     norm, with a workspace).
 *   - LayerNorm backward as a combined per-row (inner) and across-rows
 *     (outer) reduction: "Llu/ln bwd" (NVIDIA/Fuser PR #207), title and the
 *     discussion, which names the layer norm backward as the special case of
 *     a grid-parallel normalization reducing both within and across rows.
 *   - The other variants that discussion lists: grid-parallel inner
 *     normalization (rows longer than one CTA: the cluster and split
 *     families) and outer normalization (nf_outer_norm_*); and the
 *     backward passes of RMSNorm and of the fused residual add.
 * The pages name the operations but print no formulas; each function below
 * states the textbook definition it implements.
 *
 * Beside the pages' operations stand the operators at the two ends of the
 * row stream that the norms work on, and its 8-bit form: the norms with an
 * 8-bit output (nf_rmsnorm_q8, nf_fused_add_rmsnorm_q8), the embedding lookup
 * and its gradient (nf_embedding_*), and log probabilities of given tokens
 * with their gradient (nf_token_logprob_*).  Between a block's norm and its
 * attention stand the operators on heads, short rows that a projection's
 * output is cut into: their rotation by position (nf_rope_*), their RMSNorm
 * with that rotation (nf_qk_rmsnorm_rope_*) and the step that appends keys and
 * values to a paged cache (nf_kv_append).  All of these follow the conventions
 * below except where they say otherwise; nf_set_path does not concern them.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Layout.   Activations are row-major, contiguous [rows, hidden] arrays of
 *           bf16 (IEEE binary32 with the low 16 mantissa bits dropped),
 *           row stride = hidden.  Weight, gamma and beta are [hidden] bf16.
 *           mean/rstd are [rows] fp32; dgamma/dbeta are [hidden] fp32.
 * Pointers. Every data pointer is a DEVICE pointer on the current CUDA
 *           device (or managed memory).  bf16 pointers, dgamma, dbeta and
 *           the workspace must be 16-byte aligned; mean/rstd 4-byte
 *           aligned.  Null pointers are accepted only when rows == 0.
 * hidden.   The compiled sizes 1024, 2048, 4096, 5120, 8192, 12288 get
 *           kernels specialized per size.  Any other multiple of 8 up to
 *           32768 (forward ops) or 16384 (backward ops) runs on the
 *           runtime-hidden kernels (NF_PATH_DYNAMIC); longer rows, up to
 *           262144 (forward) or 131072 (backward), run on the grid-parallel
 *           cluster kernels (NF_PATH_CLUSTER), which split one row over a
 *           cluster of 2, 4 or 8 CTAs; longer still, up to
 *           NF_SPLIT_MAX_HIDDEN, on the split kernels (NF_PATH_SPLIT), which
 *           spread a row over any number of CTAs, or, for up to 8 rows that
 *           fit on chip, the grid kernels (NF_PATH_GRID), which hold the
 *           rows in shared memory across one grid barrier; both need a
 *           workspace (the forward ops then take the _ws entry points).
 *           Other values (not a positive multiple of 8, or longer) return
 *           NF_ERR_UNSUPPORTED_HIDDEN.
 * rows.     Any value >= 0; rows == 0 returns NF_OK without launching.
 * eps.      Finite and > 0.
 * Stream.   Work is enqueued on `stream` (NULL = the legacy default
 *           stream) and the call returns without synchronizing.
 * Ownership.The caller owns every buffer (workspaces included); the
 *           library allocates no device memory.  It caches, per device, the
 *           SM count and the address of its device status word.
 * Launches. Kernels are launched as programmatic dependents of the work
 *           ahead of them on the stream; each waits for that work to
 *           complete before it touches memory, so stream order holds for
 *           every caller, and the calls can be captured into CUDA graphs.
 *           The first call of an entry point on a device sets kernel
 *           attributes (cudaFuncSetAttribute) and caches device state, so
 *           make that first call outside a stream capture.
 * Errors.   Argument checks happen before any launch and return a status;
 *           a failed launch returns NF_ERR_CUDA.  Nothing is thrown across
 *           the ABI.  A kernel that gives up on a bounded wait records
 *           NF_ERR_TIMEOUT in the device status word (read it with
 *           nf_get_device_status) and returns without trapping.
 * Aliasing. Outputs may not partially overlap inputs or each other; the
 *           only aliasing allowed is stated per function.
 * Results.  Accumulation is fp32; results are bit-identical from run to
 *           run on the same device (every reduction has a fixed order).
 */
#ifndef NF_H_
#define NF_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    NF_OK = 0,
    NF_ERR_INVALID_ARG = 1,         /* null pointer, rows < 0, bad eps, bad overlap */
    NF_ERR_UNSUPPORTED_HIDDEN = 2,  /* hidden not in the compiled set */
    NF_ERR_MISALIGNED = 3,          /* pointer alignment rule broken */
    NF_ERR_WORKSPACE_TOO_SMALL = 4, /* workspace_bytes below the queried size */
    NF_ERR_CUDA = 5,                /* a CUDA runtime call or launch failed */
    NF_ERR_TIMEOUT = 6,             /* a kernel gave up on a bounded wait */
    NF_ERR_UNSUPPORTED_PATH = 7     /* forced path not built for this op/size */
} nf_status;

/* = cudaStream_t.  NULL is the legacy default stream. */
typedef struct CUstream_st* nf_stream;

/* Kernel families.  NF_PATH_AUTO lets the library choose from rows, hidden
 * and the SM count; the others force one family (for tests and ablations).
 *   REG     -- row resident in registers, 128-bit loads, one row per group
 *              of threads ("optimize inner persistent scheduler for static
 *              fusion": static hidden size, warp-multiple block size).
 *   CLUSTER -- one row split across a thread-block cluster, partial sums
 *              exchanged through distributed shared memory: the small-batch
 *              idea of the same page (more SMs per row), and the
 *              grid-parallel inner normalization "Llu/ln bwd" lists as
 *              missing (rows longer than one CTA holds; any hidden, forward
 *              and backward).
 *   BULK    -- a producer warp stages rows into a shared-memory ring with
 *              bulk asynchronous copies; consumer warps read 128-bit vectors
 *              from shared memory; registers move from producer to
 *              consumers ("TMA inner persistent scheduler").
 *   DYNAMIC -- the hidden size is a runtime argument (any multiple of 8 up
 *              to 32768 forward, 16384 backward); a thread owns at most
 *              four 16-byte vectors of a row, a compile-time bound ("TMA
 *              inner persistent scheduler": dynamic block dimensions).  The
 *              backward, and the RMSNorm / LayerNorm forward on rows of one
 *              warp, stream the next row through a per-thread copy ring in
 *              shared memory (nf_plan_query reports its bytes).  The only
 *              family for hidden sizes outside the compiled set.
 *   SPLIT   -- one row cut into 8192-element chunks, one CTA per (chunk,
 *              row), the row statistics passed through a caller workspace
 *              in global memory: grid-parallel inner normalization across
 *              any number of CTAs ("Llu/ln bwd"), for rows longer than a
 *              cluster holds (any multiple of 8 up to NF_SPLIT_MAX_HIDDEN).
 *              Forward calls on this family need a workspace: use the _ws
 *              entry points and nf_workspace_size.
 *   GRID    -- the split family's rows held on chip: one cooperative launch
 *              of one 512-thread CTA per SM; CTA c keeps its slice of
 *              ceil(hidden / 8 / SMs) vectors of EVERY row in shared memory,
 *              the CTAs exchange the per-row partial sums through the
 *              workspace across one grid barrier (a bounded wait: if it runs
 *              out the kernel records NF_ERR_TIMEOUT in the device status
 *              word and returns), and every CTA adds them in the same fixed
 *              order.  Each input row is read from memory once (the
 *              backward reads dy a second time, from L2), and a column's
 *              every row is in one CTA, so the backward writes
 *              dgamma / dbeta (dw) directly.  For 1 to 8 rows whose slices
 *              fit (rows * ceil(hidden / 8 / SMs) * 16 bytes within about
 *              226 KB): on GB300 up to 4 rows of 4194304 or 8 of 2097152.
 *              The automatic choice takes it wherever the split family
 *              would run and the rows fit, except for the RMSNorm backward
 *              (the split family's apply pass measured faster there).
 *              Forward calls need a workspace, as for SPLIT.  The fused op normalizes the residual as
 *              stored (bf16), the literal reading of the in-place update;
 *              the other families normalize the fp32 sum (both are within
 *              the stated tolerance of the exact result).                   */
typedef enum {
    NF_PATH_AUTO = 0,
    NF_PATH_REG = 1,
    NF_PATH_CLUSTER = 2,
    NF_PATH_BULK = 3,
    NF_PATH_DYNAMIC = 4,
    NF_PATH_SPLIT = 5,
    NF_PATH_GRID = 6
} nf_path;

/* Longest row any family handles (the split family). */
#define NF_SPLIT_MAX_HIDDEN (1LL << 26)

/* Operation ids for nf_plan_query. */
typedef enum {
    NF_OP_FUSED_ADD_RMSNORM = 0,
    NF_OP_RMSNORM_FWD = 1,
    NF_OP_LAYERNORM_FWD = 2,
    NF_OP_LAYERNORM_BWD = 3,
    NF_OP_RMSNORM_BWD = 4
} nf_op;

/* A launch plan, as chosen for (op, rows, hidden) on the current device. */
typedef struct {
    int32_t path;            /* nf_path actually used (never AUTO) */
    int32_t grid;            /* CTAs in the main launch */
    int32_t block;           /* threads per CTA */
    int32_t cluster;         /* CTAs per cluster (1 = none) */
    int32_t rows_per_cta;    /* rows a CTA computes at once (bulk: consumer row groups) */
    int32_t smem_bytes;      /* dynamic shared memory per CTA */
    int32_t launches;        /* kernel launches per call */
    int32_t partials;        /* column-partial slots (backward ops), else 0 */
} nf_plan;

/* Fused residual add + RMSNorm forward, in place.  For each row r:
 *     s_j          = x[r][j] + residual[r][j]          (fp32)
 *     residual[r][j] <- bf16(s_j)
 *     x[r][j]       <- bf16( s_j * rsqrt(mean_k(s_k^2) + eps) * weight[j] )
 * The normalization reads the unrounded fp32 sum s.  x and residual are
 * both read and written; they must not overlap each other, and weight must
 * not overlap either. */
nf_status nf_fused_add_rmsnorm(void* x, void* residual, const void* weight,
                               int64_t rows, int64_t hidden, float eps, nf_stream stream);

/* Bytes of workspace `op` needs for (rows, hidden) on the current device,
 * enough under every kernel family (so nf_set_path cannot make it short).
 * For the forward ops it is nonzero only because the split family (rows
 * longer than a cluster holds, or forced) keeps per-row partial statistics
 * there: rows * (8 * chunks + 8) bytes, chunks = ceil(hidden / 8192).  For
 * the backward ops it equals nf_layernorm_bwd_workspace_size /
 * nf_rmsnorm_bwd_workspace_size.  0 when rows == 0, hidden is unsupported,
 * op is unknown or the device cannot be queried. */
size_t nf_workspace_size(nf_op op, int64_t rows, int64_t hidden);

/* The forward entry points with a caller workspace (16-byte aligned, at
 * least nf_workspace_size(op, rows, hidden) bytes, contents irrelevant, not
 * overlapping any argument).  They behave exactly as the plain calls; the
 * workspace is used only when the plan is the split family (automatic
 * beyond the runtime-hidden limits, or forced).  Without a workspace (the
 * plain calls, or NULL here) an automatic split plan runs on the cluster
 * family instead where that holds the row (hidden <= 262144); longer rows,
 * or a forced split, return NF_ERR_WORKSPACE_TOO_SMALL. */
nf_status nf_fused_add_rmsnorm_ws(void* x, void* residual, const void* weight, int64_t rows,
                                  int64_t hidden, float eps, void* workspace,
                                  size_t workspace_bytes, nf_stream stream);

/* RMSNorm forward:  y[r][j] = bf16( x[r][j] * rsqrt(mean_k(x[r][k]^2) + eps) * weight[j] ).
 * y may be x itself (in place); any other overlap is rejected. */
nf_status nf_rmsnorm_fwd(void* y, const void* x, const void* weight,
                         int64_t rows, int64_t hidden, float eps, nf_stream stream);
nf_status nf_rmsnorm_fwd_ws(void* y, const void* x, const void* weight, int64_t rows,
                            int64_t hidden, float eps, void* workspace, size_t workspace_bytes,
                            nf_stream stream);

/* LayerNorm forward with biased variance:
 *     mean[r] = (1/H) sum_j x[r][j]
 *     var     = (1/H) sum_j (x[r][j] - mean[r])^2        (two passes over the resident row)
 *     rstd[r] = rsqrt(var + eps)
 *     y[r][j] = bf16( (x[r][j] - mean[r]) * rstd[r] * gamma[j] + beta[j] )
 * mean and rstd (fp32, [rows]) are the values a backward pass needs; either
 * may be NULL to skip it.  y may be x itself. */
nf_status nf_layernorm_fwd(void* y, float* mean, float* rstd, const void* x,
                           const void* gamma, const void* beta,
                           int64_t rows, int64_t hidden, float eps, nf_stream stream);
nf_status nf_layernorm_fwd_ws(void* y, float* mean, float* rstd, const void* x,
                              const void* gamma, const void* beta, int64_t rows, int64_t hidden,
                              float eps, void* workspace, size_t workspace_bytes,
                              nf_stream stream);

/* Bytes of workspace nf_layernorm_bwd needs for (rows, hidden) on the
 * current device, under any kernel family (0 when rows == 0 or hidden is
 * unsupported).  The value depends on the device's SM count, so query it
 * on the device that runs the call.  Returns 0 also if the device cannot
 * be queried. */
size_t nf_layernorm_bwd_workspace_size(int64_t rows, int64_t hidden);

/* LayerNorm backward.  With xhat = (x - mean) * rstd and g = dy * gamma:
 *   inner (per row):   dx[r][j] = bf16( rstd[r] * ( g_j - mean_k(g_k) - xhat_j * mean_k(g_k * xhat_k) ) )
 *   outer (per column): dgamma[j] = sum_r dy[r][j] * xhat[r][j],  dbeta[j] = sum_r dy[r][j]
 * mean/rstd are the forward's saved values (eps is folded into rstd, so
 * none is passed).  dgamma/dbeta are overwritten, not accumulated.  The
 * column sums go through `workspace` in two stages -- per-CTA partials,
 * then a fixed-order sum -- so they are deterministic.  workspace is a
 * caller-owned device buffer, 16-byte aligned, of at least
 * nf_layernorm_bwd_workspace_size(rows, hidden) bytes; its contents on
 * entry do not matter.  dx may be dy or x itself (exact alias).  With
 * rows == 0 nothing is read and dgamma/dbeta, where not NULL, are set to 0
 * (an empty column sum). */
nf_status nf_layernorm_bwd(void* dx, float* dgamma, float* dbeta,
                           const void* dy, const void* x, const float* mean, const float* rstd,
                           const void* gamma, int64_t rows, int64_t hidden,
                           void* workspace, size_t workspace_bytes, nf_stream stream);

/* Bytes of workspace nf_rmsnorm_bwd needs for (rows, hidden) on the current
 * device, under any kernel family (same rules as the LayerNorm query). */
size_t nf_rmsnorm_bwd_workspace_size(int64_t rows, int64_t hidden);

/* RMSNorm backward (the RMS counterpart of the combined inner + outer
 * reduction of "Llu/ln bwd"; "TMA inner persistent scheduler": RMS norm
 * with a workspace).  For y = x * rstd * w with
 * rstd = rsqrt(mean_k(x_k^2) + eps), g = dy * w and xhat = x * rstd:
 *   inner (per row):    dx[r][j] = bf16( rstd * ( g_j - xhat_j * mean_k(g_k * xhat_k) ) )
 *   outer (per column): dw[j]    = sum_r dy[r][j] * xhat[r][j]          (fp32, overwritten)
 * rstd is recomputed from x inside the kernel (one more sum in the same
 * row reduction, no extra memory traffic), so the forward need not save
 * it; pass the forward's eps.  The column sums go through `workspace` in
 * two fixed-order stages (deterministic).  dx may be dy or x itself.
 * rows == 0 sets dw (if not NULL) to 0.  Same pointer, alignment and
 * workspace rules as nf_layernorm_bwd. */
nf_status nf_rmsnorm_bwd(void* dx, float* dw, const void* dy, const void* x, const void* weight,
                         int64_t rows, int64_t hidden, float eps, void* workspace,
                         size_t workspace_bytes, nf_stream stream);

/* Fused residual-add + RMSNorm backward ("optimize inner persistent
 * scheduler for static fusion" pairs the fused add + RMSNorm forward with
 * in-place residual semantics; this is its gradient).  The forward left
 * s = x + residual in `residual` and y = s * rstd(s) * w in x.  Given the
 * gradient dy of y and, optionally, dres of the residual stream s:
 *   rstd   = rsqrt(mean_j(s_j^2) + eps)     (recomputed from the saved s)
 *   dx     = bf16( rstd * (g - s * rstd^2 * mean_j(g * s)) + dres ),  g = dy * w
 *   dw[j]  = sum_r dy[r][j] * s[r][j] * rstd[r]                      (fp32)
 * dx is the gradient of both forward inputs (x and residual).  dres may be
 * NULL (no residual-stream gradient); dx may be exactly dy, dres or
 * residual (in place).  Same hidden sizes, workspace (see
 * nf_rmsnorm_bwd_workspace_size), alignment and error rules as
 * nf_rmsnorm_bwd; dres, if given, must be 16-byte aligned. */
nf_status nf_fused_add_rmsnorm_bwd(void* dx, float* dw, const void* dy, const void* dres,
                                   const void* residual, const void* weight, int64_t rows,
                                   int64_t hidden, float eps, void* workspace,
                                   size_t workspace_bytes, nf_stream stream);

/* Size of the fixed scratch area nf_layernorm_bwd_noalloc uses. */
#define NF_LAYERNORM_BWD_NOALLOC_SCRATCH_BYTES (16u << 20)

/* LayerNorm backward that allocates nothing and takes no workspace.  The
 * source pages have no counterpart to this call; it is an addition of this
 * library for callers that cannot call cudaMalloc where they run the
 * backward pass (code inside a region where the framework's caching
 * allocator must not be entered, plugins that only receive pre-allocated
 * buffers, latency-critical paths that cannot take cudaMalloc's implicit
 * synchronization).  Same arguments, results and rules as nf_layernorm_bwd
 * minus the workspace: the column partials go to a fixed
 * NF_LAYERNORM_BWD_NOALLOC_SCRATCH_BYTES area of static device memory
 * inside the library (held by every GPU that loads the library until the
 * process exits).  Argument errors return what nf_layernorm_bwd returns, in
 * the same order, before the area is looked at.  A size whose partials need
 * more than the area under the plan the call runs returns
 * NF_ERR_WORKSPACE_TOO_SMALL before anything is launched.  At the compiled
 * sizes the largest need is hidden 12288 (one slot of 2 * 12288 fp32 per
 * SM: 14.25 MiB on a 152-SM GPU, so a part with more than 170 SMs refuses
 * it); the runtime-hidden sizes near 16384 and the split family's very long
 * rows can need more and are refused.  The first call on each device looks
 * up the area's device address (cudaGetSymbolAddress, with that device
 * current) and caches it; make that first call before any stream capture.
 * cudaDeviceReset ends the context that owns the area, so a process that
 * resets a device must not call this entry point on that device again.
 * Every call shares the one area, which keeps the last call's contents
 * (nothing needs clearing: every partial is written before it is read);
 * calls that overlap on the GPU -- on different streams or from different
 * host threads -- race on it, so serialize them. */
nf_status nf_layernorm_bwd_noalloc(void* dx, float* dgamma, float* dbeta, const void* dy,
                                   const void* x, const float* mean, const float* rstd,
                                   const void* gamma, int64_t rows, int64_t hidden,
                                   nf_stream stream);

/* Largest hidden size of the operators with an 8-bit output. */
#define NF_Q8_MAX_HIDDEN 32768

/* 8-bit formats.  E4M3: 3 mantissa bits, largest value 448.  INT8: two's
 * complement, -127 to 127. */
typedef enum { NF_Q8_E4M3 = 0, NF_Q8_INT8 = 1 } nf_q8_format;

/* RMSNorm forward, and the fused residual add + RMSNorm, with an 8-bit
 * output and its scales: the normalized rows as a product in 8 bits reads
 * them.  The source pages have no counterpart; the operator is
 * nf_rmsnorm_fwd / nf_fused_add_rmsnorm with the quantization of its output
 * in the same pass.  For each row r:
 *     s_j      = x[r][j]                                  (nf_rmsnorm_q8)
 *     s_j      = x[r][j] + residual[r][j]; residual[r][j] <- bf16(s_j)   (fused)
 *     y_j      = s_j * rsqrt(mean_k(s_k^2) + eps) * weight[j]            (fp32)
 *     scale    = max(max_j |y_j| / Q, 2^-100),  Q = 448 (E4M3) or 127 (INT8)
 *     q[r][j]  = y_j / scale, rounded to nearest, ties to even
 * so q * scale stands for y.  group = 0: one scale per row, scale is [rows]
 * fp32.  group = 128: one scale per 128 columns (the last group may be
 * shorter), scale is [rows, ceil(hidden / 128)] fp32.  y is not rounded to
 * bf16 before it is quantized.  A scale whose largest |y| is not finite, or
 * whose largest |s_j * weight[j]| is not finite in fp32 (max |y| is found as
 * that maximum times the rsqrt), is not finite either, and its q are 0; a row whose sum of squares is not
 * finite in fp32 (a NaN, an infinity, magnitudes beyond about 1e19) has NaN
 * for every scale.  x is only read; nothing may overlap.  q: [rows, hidden]
 * bytes, 8-byte aligned; scale 4-byte aligned.  hidden: a multiple of 8 up
 * to NF_Q8_MAX_HIDDEN.  rows == 0 returns NF_OK.  No workspace. */
nf_status nf_rmsnorm_q8(void* q, float* scale, const void* x, const void* weight, int64_t rows,
                        int64_t hidden, float eps, nf_q8_format format, int64_t group,
                        nf_stream stream);
nf_status nf_fused_add_rmsnorm_q8(void* q, float* scale, const void* x, void* residual,
                                  const void* weight, int64_t rows, int64_t hidden, float eps,
                                  nf_q8_format format, int64_t group, nf_stream stream);

/* Element types of the operators that take more than one. */
typedef enum { NF_BF16 = 0, NF_F32 = 1 } nf_dtype;

/* Embedding lookup with scaling, the rows a residual stream starts from:
 *     y[i][j] = bf16( scale * table[ids[i]][j] ),   i < tokens, j < hidden
 * An id outside [0, vocab) (padding) gives a row of zeros.  ids: int32
 * (id_bytes 4) or int64 (id_bytes 8).  table: [vocab, hidden] bf16, y:
 * [tokens, hidden] bf16.  hidden: a multiple of 8 up to 2^20; tokens below
 * 2^31; vocab 1 to 2^30; scale finite.  y overlaps nothing. */
nf_status nf_embedding_fwd(void* y, const void* ids, int32_t id_bytes, const void* table, int64_t tokens,
                           int64_t vocab, int64_t hidden, float scale, nf_stream stream);

/* Gradient of the lookup, by sorted tokens:
 *     g[v][j] = scale * sum over { i : ids[i] = v } of dy[i][j]          (fp32)
 *     dtable = g (accumulate 0: every row is written, those without tokens
 *     with zeros), or dtable += g (accumulate 1: only rows with tokens are
 *     touched).  Ids outside [0, vocab) contribute nothing.
 * dtable: [vocab, hidden], NF_F32 or NF_BF16; a bf16 element is rounded
 * once, at the end.  Sums added to fp32 elements are added in L2, where a
 * result below 2^-126 becomes 0.  The order of every sum is fixed: an id's
 * tokens are cut into pieces, each piece is summed in token order, and the
 * pieces' sums are added in a fixed grouping.  So results are deterministic;
 * where the cuts fall depends on all ids, the sizes and the device's SM count.
 * All but small calls sort the tokens by id in the workspace (16-byte aligned,
 * at least nf_embedding_bwd_workspace_size(tokens, hidden) bytes on the device
 * that runs the call, asked for in small calls too; contents irrelevant).  How
 * many ids coincide changes neither the launches nor the workspace.  Sizes as
 * for the lookup.
 * Nothing may overlap.  tokens == 0 reads nothing (dy, ids and workspace may
 * be NULL) and, with accumulate 0, writes zeros. */
size_t nf_embedding_bwd_workspace_size(int64_t tokens, int64_t hidden);
nf_status nf_embedding_bwd(void* dtable, nf_dtype dtable_type, int32_t accumulate, const void* dy,
                           const void* ids, int32_t id_bytes, int64_t tokens, int64_t vocab, int64_t hidden,
                           float scale, void* workspace, size_t workspace_bytes, nf_stream stream);

/* Largest number of alternatives nf_token_logprob_fwd returns. */
#define NF_TOP_MAX 32

/* Log probabilities of given tokens, with entropy and top alternatives.  For
 * each row of logits l (rows of `vocab` elements, `stride` elements apart,
 * NF_BF16 or NF_F32) at a temperature T, with m = max_j l_j and
 * d_j = (l_j - m) / T:
 *     log S      = log sum_j exp(d_j)
 *     logprob    = d_t - log S,  t = targets[r]      (0 where t is outside [0, vocab))
 *     entropy    = log S - sum_j exp(d_j) d_j / S
 *     stats[r]   = (m, log S), what the gradient needs
 *     top_*[r]   = the `top` most probable tokens, the most probable first and
 *                  the lower id first among equals (0 and -0 are equal):
 *                  their log probability and id
 * Entries of -infinity are masked: probability 0, never an alternative; where
 * fewer than `top` entries are left the rest hold (-infinity, -1).  A row with
 * every entry masked has stats (-inf, -inf), entropy 0, logprob -inf (0 where
 * t is outside).  A row with a NaN or +infinity has NaN for every value but
 * m, and ids of -1.  logprob, entropy: [rows] fp32; stats: [rows, 2] fp32,
 * 8-byte aligned; top_logprob: [rows, top] fp32; top_ids: [rows, top] int64;
 * top 0 to NF_TOP_MAX (0: both may be NULL).  targets: int32 (id_bytes 4) or
 * int64 (id_bytes 8).  logits need the alignment of an element only.  vocab 1
 * to 2^30, stride >= vocab, T from 2^-64 to 2^64.  Elements behind a row's
 * vocab are not read.  Nothing may overlap.  rows == 0 returns NF_OK.  No
 * workspace. */
nf_status nf_token_logprob_fwd(float* logprob, float* entropy, float* stats, float* top_logprob,
                               int64_t* top_ids, const void* logits, nf_dtype type, int64_t stride,
                               const void* targets, int32_t id_bytes, int64_t rows, int64_t vocab,
                               float temperature, int32_t top, nf_stream stream);

/* Gradient of logprob and entropy with respect to the logits.  With
 * p_j = exp(d_j - log S) from the forward's stats, g = d_logprob[r] (taken as
 * 0 where t is outside [0, vocab)) and h = d_entropy[r] (NULL: 0):
 *     dlogits[r][j] = ( g (1[j = t] - p_j) - h p_j (log p_j + entropy[r]) ) / T
 * in the logits' type, rows `dstride` elements apart; elements behind a row's
 * vocab are left as they are.  A row with every entry masked gets zeros.
 * entropy is the forward's, and may be NULL where d_entropy is.  dlogits may
 * be the logits themselves (same pointer and stride); nothing else may
 * overlap it, from its first element to its last (rows of one matrix between
 * the rows of the other count as an overlap).  Sizes as for the forward. */
nf_status nf_token_logprob_bwd(void* dlogits, int64_t dstride, const void* logits, nf_dtype type,
                               int64_t stride, const void* targets, int32_t id_bytes, const float* stats,
                               const float* entropy, const float* d_logprob, const float* d_entropy,
                               int64_t rows, int64_t vocab, float temperature, nf_stream stream);

/* ---- Operators on attention heads ----------------------------------------
 * A row is one head of one token: head_dim elements (1 to NF_HEAD_MAX_DIM,
 * else NF_ERR_UNSUPPORTED_HIDDEN), contiguous.  A set of heads (queries, keys
 * or values of a batch) is described by its first element and its strides, so
 * that views of a projection's output, and orders other than [batch, tokens,
 * heads, head_dim], need no copy.  Pointers need the alignment of an element.
 * Rows whose pointers and strides are multiples of 16 bytes, of at most 64
 * 16-byte vectors, and whose rotated part (in the half layout each half of it)
 * is whole vectors run on vector kernels; others run element by element on
 * slower ones.  Strides are not negative.  The rows of an output are apart: in
 * the order of its strides, each dimension steps over the ones inside it.  An
 * output overlaps nothing but where it says so; sets whose rows lie between
 * one another's (the queries and keys of one projection) do not overlap.  Sets
 * of three strides each that 256 steps do not tell apart count as overlapping.
 * batch * tokens * heads, over all sets of a call, is below 2^31.  Types:
 * NF_BF16 and NF_F32, one for a call, its weights included.                   */
#define NF_HEAD_MAX_DIM 512

typedef struct {
    void* data;           /* batch 0, token 0, head 0, element 0; inputs are only read */
    int64_t batch_stride; /* in elements */
    int64_t token_stride;
    int64_t head_stride;
    int32_t heads;        /* 1 to 2^20 */
} nf_heads;

/* Which elements of a head are a pair i, i < dim / 2. */
typedef enum {
    NF_ROPE_HALF = 0,        /* i and i + dim / 2 */
    NF_ROPE_INTERLEAVED = 1  /* 2i and 2i + 1     */
} nf_rope_layout;

/* The rotation of a call.  The first `dim` elements of a head (even, 0 to
 * head_dim; 0: none) are pairs (a, b), which a token at position p turns by
 * t_i = p * f_i:
 *     a' = magnitude * (a cos t_i - b sin t_i)
 *     b' = magnitude * (b cos t_i + a sin t_i)
 * The elements behind are left as they are.  The frequencies f_i come as
 * rates: the share of a turn per position, f_i / (2 pi), modulo 1 and in units
 * of 2^-64 (nf_rope_rates makes them).  The 64-bit product rate * p is then the
 * angle modulo a turn with no reduction of large angles: it is off by p * 2^-65
 * turns at most, the rates' own rounding p times.  Its sine and cosine are
 * within 2^-22 of their values, however small these are.  Positions are any
 * integers, negative ones too. */
typedef struct {
    const uint64_t* rates;  /* device, [dim / 2] */
    int32_t dim;
    nf_rope_layout layout;
    float magnitude;        /* finite; 1 unless the context's scaling asks for another */
    const void* positions;  /* device, of token t of batch b: [b * position_stride + t] */
    int32_t position_bytes; /* 4 (int32) or 8 (int64) */
    int64_t position_stride;/* 0: every batch has the same positions */
} nf_rope;

/* Scalings of the frequencies f_i = base^(-2i / dim) for contexts longer than
 * those of training by `factor` (>= 1):
 *   NF_ROPE_PLAIN   none (factor and the rest are ignored)
 *   NF_ROPE_LINEAR  f_i / factor (position interpolation)
 *   NF_ROPE_NTK     the base is base * factor^(dim / (dim - 2)), so that the
 *                   slowest pair alone is slowed by the factor (dim >= 4)
 *   NF_ROPE_PARTS   pairs that turn `high` times or more within `length`
 *                   positions (the context of training) keep f_i, those that
 *                   turn `low` times or less take f_i / factor, and those
 *                   between a mixture linear in their number of turns
 *                   ("YaRN", section 3.2; it suggests the magnitude
 *                   0.1 ln(factor) + 1) */
typedef enum { NF_ROPE_PLAIN = 0, NF_ROPE_LINEAR = 1, NF_ROPE_NTK = 2, NF_ROPE_PARTS = 3 } nf_rope_scaling;

/* Host only: writes dim / 2 rates to host memory, each the nearest to its
 * frequency's share of a turn.  dim even, 2 to
 * NF_HEAD_MAX_DIM; base > 1, factor >= 1, length > 0, 0 <= low < high, all
 * finite (those that the scaling uses). */
nf_status nf_rope_rates(uint64_t* rates, int32_t dim, double base, nf_rope_scaling scaling, double factor,
                        double length, double low, double high);
/* The same from given frequencies, in radians per position (finite, below
 * 2^20 in magnitude; negative ones turn the other way). */
nf_status nf_rope_rates_of(uint64_t* rates, const double* frequencies, int32_t count);

/* Queries and keys turned by their tokens' positions (k_out and k may both be
 * NULL).  nf_rope_bwd is the gradient for q and k, given that of the turned
 * ones: the same pairs turned back, times the magnitude.  An output may be its
 * own input (same pointer and strides).  Computed in fp32, rounded once. */
nf_status nf_rope_fwd(const nf_heads* q_out, const nf_heads* q, const nf_heads* k_out, const nf_heads* k,
                      nf_dtype type, int64_t batch, int64_t tokens, int64_t head_dim, const nf_rope* rope,
                      nf_stream stream);
nf_status nf_rope_bwd(const nf_heads* dq, const nf_heads* dq_out, const nf_heads* dk, const nf_heads* dk_out,
                      nf_dtype type, int64_t batch, int64_t tokens, int64_t head_dim, const nf_rope* rope,
                      nf_stream stream);

/* RMSNorm of each query and key head, with the rotation in the same pass:
 *     n   = x * rsqrt(mean(x^2) + eps) * weight
 *     out = the pairs of n turned, the rest of n
 * computed in fp32, rounded once.  The weights are [head_dim], one for all
 * query heads and one for all key heads.  rope may be NULL (no rotation), and
 * so may k_out, k and k_weight.  An output may be its own input. */
nf_status nf_qk_rmsnorm_rope_fwd(const nf_heads* q_out, const nf_heads* q, const void* q_weight,
                                 const nf_heads* k_out, const nf_heads* k, const void* k_weight, nf_dtype type,
                                 int64_t batch, int64_t tokens, int64_t head_dim, float eps,
                                 const nf_rope* rope, nf_stream stream);

/* Its gradient.  dq_out and dk_out are the gradients of the outputs.  With g
 * the pairs of dq_out turned back, xhat = x * rsqrt(mean(x^2) + eps):
 *     dq       = rstd * (g * weight - xhat * mean(g * weight * xhat))
 *     dq_weight = sum over batch, tokens and heads of g * xhat   ([head_dim] fp32)
 * and so for the keys.  dq may be dq_out or q itself (same pointer and
 * strides), dk likewise.  workspace: 4-byte aligned, at least
 * nf_qk_rmsnorm_rope_bwd_workspace_size(head_dim) bytes on the device that
 * runs the call; contents irrelevant, and no call that overlaps this one on the
 * GPU may use it.  The order of every sum is fixed.  With
 * batch * tokens == 0 the weights' gradients are written with zeros. */
size_t nf_qk_rmsnorm_rope_bwd_workspace_size(int64_t head_dim);
nf_status nf_qk_rmsnorm_rope_bwd(const nf_heads* dq, float* dq_weight, const nf_heads* dq_out, const nf_heads* q,
                                 const void* q_weight, const nf_heads* dk, float* dk_weight,
                                 const nf_heads* dk_out, const nf_heads* k, const void* k_weight, nf_dtype type,
                                 int64_t batch, int64_t tokens, int64_t head_dim, float eps, const nf_rope* rope,
                                 void* workspace, size_t workspace_bytes, nf_stream stream);

/* A paged cache of keys or values: `pages` pages of `page_size` slots, a slot
 * with a row for each head.  In the rows' own type, or in 8 bits with a scale
 * (fp32) for each row: q * scale stands for the row. */
typedef enum { NF_CACHE_SAME = 0, NF_CACHE_E4M3 = 1, NF_CACHE_INT8 = 2 } nf_cache_type;
typedef struct {
    void* data;
    int64_t page_stride, slot_stride, head_stride;  /* in elements */
    float* scale;                                   /* 8-bit caches; else ignored */
    int64_t scale_page_stride, scale_slot_stride, scale_head_stride;
} nf_pages;

/* Appends the keys and values of new tokens to a paged cache; the queries of
 * the same tokens may be prepared in the same launch.  For each token i of
 * `tokens`:
 *   - its sequence s: with starts ([seqs + 1] int32, rising from 0), the one
 *     with starts[s] <= i < starts[s + 1] (sequences without new tokens have
 *     starts[s] == starts[s + 1]); with starts NULL, one token per sequence, s = i
 *   - its place p = past[s] + i - starts[s], past ([seqs] int32) the tokens
 *     that the sequence has in the cache before the call
 *   - its page table[s * table_stride + p / page_size], its slot p % page_size
 * k (normalized with k_weight and eps unless that is NULL, then turned by the
 * token's angles) goes to k_cache, v, as it is, to v_cache; q (likewise, with
 * q_weight) to q_out, which may be q itself.  The position that turns a token
 * is rope->positions[i], or p where that is NULL.  A token of no sequence (i
 * behind starts[seqs] or, without starts, behind seqs), or of one with past <
 * 0, is padding: nothing of it is written.  A token whose place lies behind
 * max_pages pages, or whose page is outside [0, pages), is not stored; its q is
 * written all the same.  Nothing else in the caches is touched.  Where two
 * tokens of a call share a slot (tables that share a page to be written), what
 * that slot holds is not defined.
 * 8-bit rows: scale = max(max|y| / Q, 2^-100), Q = 448 (E4M3) or 127 (INT8),
 * q = y / scale rounded to nearest, ties to even; y is not rounded to the rows'
 * type before.  A row with a NaN or an infinity has scale NaN and q 0.
 * q_out and q may both be NULL.  table is [seqs, max_pages] int32; seqs up to
 * 2^30. */
nf_status nf_kv_append(const nf_pages* k_cache, const nf_pages* v_cache, nf_cache_type cache_type, int64_t pages,
                       int32_t page_size, const nf_heads* k, const nf_heads* v, const void* k_weight,
                       const nf_heads* q_out, const nf_heads* q, const void* q_weight, nf_dtype type,
                       int64_t tokens, int64_t seqs, int64_t head_dim, const int32_t* starts,
                       const int32_t* past, const int32_t* table, int64_t table_stride, int32_t max_pages,
                       float eps, const nf_rope* rope, nf_stream stream);

/* Outer normalization: the statistics run down the columns, over the rows
 * (batch normalization of a [rows, hidden] matrix in training mode; the
 * "Llu/ln bwd" discussion lists block- and grid-parallel outer
 * normalization among the normalization variants).  For each column j:
 *     mean[j] = (1/R) sum_r x[r][j]
 *     var_j   = (1/R) sum_r (x[r][j] - mean[j])^2          (biased)
 *     rstd[j] = rsqrt(var_j + eps)
 *     y[r][j] = bf16( (x[r][j] - mean[j]) * rstd[j] * gamma[j] + beta[j] )
 * hidden: any multiple of 8 (no compiled-size restriction); rows >= 0
 * (rows == 0 writes nothing).  mean/rstd ([hidden] fp32) may be NULL.  The
 * per-column statistics are merged from row stripes in a fixed order
 * (Chan's pairwise formula), so results are deterministic.  workspace:
 * caller-owned, 16-byte aligned, at least
 * nf_outer_norm_workspace_size(rows, hidden) bytes, contents irrelevant.
 * y may be x itself.  Two forms: three streaming launches (statistics per
 * row stripe, a merge per column, the apply pass), the default; and, with
 * nf_set_path(NF_PATH_GRID), one cooperative launch that keeps each CTA's
 * row stripe on chip band of columns by band and merges across bounded grid
 * barriers (reads x once, but measured slower; NF_ERR_UNSUPPORTED_PATH when
 * a stripe of rows / SMs rows does not fit two band buffers of 16 vectors). */
size_t nf_outer_norm_workspace_size(int64_t rows, int64_t hidden);
nf_status nf_outer_norm_fwd(void* y, float* mean, float* rstd, const void* x, const void* gamma,
                            const void* beta, int64_t rows, int64_t hidden, float eps,
                            void* workspace, size_t workspace_bytes, nf_stream stream);

/* Outer normalization backward (saved per-column mean/rstd).  With
 * xhat = (x - mean[j]) * rstd[j] and g = dy * gamma[j]:
 *   dx[r][j]  = bf16( rstd[j] * ( g - (1/R) sum_s g[s][j] - xhat * (1/R) sum_s g[s][j] xhat[s][j] ) )
 *   dgamma[j] = sum_r dy[r][j] * xhat[r][j],  dbeta[j] = sum_r dy[r][j]   (fp32, overwritten)
 * The column sums go through `workspace` and the fixed-order column
 * reduction.  dx may be dy or x itself.  rows == 0 sets dgamma/dbeta (if
 * not NULL) to 0.  Same pointer and workspace rules as the forward. */
nf_status nf_outer_norm_bwd(void* dx, float* dgamma, float* dbeta, const void* dy, const void* x,
                            const float* mean, const float* rstd, const void* gamma, int64_t rows,
                            int64_t hidden, void* workspace, size_t workspace_bytes,
                            nf_stream stream);

/* Force a kernel family for every later call in this process (NF_PATH_AUTO
 * restores the library's choice).  A call whose op/size has no kernel of the
 * forced family returns NF_ERR_UNSUPPORTED_PATH.  Not thread-safe with
 * respect to calls in flight on other host threads; meant for tests and
 * ablations. */
nf_status nf_set_path(nf_path path);

/* The plan a call of `op` with (rows, hidden) would use now on the current
 * device, without launching anything. */
nf_status nf_plan_query(nf_op op, int64_t rows, int64_t hidden, nf_plan* out);

/* Pure host planning, no CUDA call: the plan for (op, rows, hidden) on a
 * device with `sm_count` SMs under the kernel-family choice `path`
 * (NF_PATH_AUTO = the library's own rule).  nf_plan_query and every entry
 * point use exactly this function with the device's SM count and the
 * nf_set_path setting.  Returns NF_ERR_UNSUPPORTED_HIDDEN,
 * NF_ERR_UNSUPPORTED_PATH or NF_ERR_INVALID_ARG (rows < 0, sm_count < 1,
 * unknown op or path, out == NULL) without touching *out. */
nf_status nf_plan_compute(nf_op op, int64_t rows, int64_t hidden, int32_t sm_count,
                          nf_path path, nf_plan* out);

/* Copy the device status word of the current device to the host after the
 * work queued on `stream` finishes (this synchronizes `stream`), reset it to
 * NF_OK, and return the copied value (NF_OK or NF_ERR_TIMEOUT), or
 * NF_ERR_CUDA if the copy itself fails. */
nf_status nf_get_device_status(nf_stream stream);

/* Test hook for the bounded-wait machinery: launch one CTA that waits on a
 * shared-memory barrier which nothing completes, giving up after
 * `timeout_ns` nanoseconds (clamped to [1e3, 1e9]).  The kernel records
 * NF_ERR_TIMEOUT in the device status word and returns normally; the
 * context stays usable. */
nf_status nf_selftest_wait_timeout(int64_t timeout_ns, nf_stream stream);

/* Test hook for the grid family's barrier: launch two cooperative CTAs that
 * wait at the grid barrier for a third CTA that does not exist, giving up
 * after `timeout_ns` nanoseconds (clamped to [1e3, 1e9]).  `workspace`: 16
 * bytes of device memory, 16-byte aligned, for the arrival counter (zeroed
 * on `stream` first).  The kernel records NF_ERR_TIMEOUT in the device
 * status word and returns normally.  NF_ERR_INVALID_ARG (null) or
 * NF_ERR_MISALIGNED before launching anything. */
nf_status nf_selftest_grid_timeout(void* workspace, int64_t timeout_ns, nf_stream stream);

/* Measurement hook: the launch floor set beside small-batch timings.
 * kind 0 launches one 32-thread CTA that only waits for the previous
 * kernel in the stream and exits (launched as a programmatic dependent,
 * like every operation's kernels); dst, src and bytes are ignored.  kind 1
 * copies `bytes` bytes (a positive multiple of 16) from src to dst
 * (16-byte aligned device pointers, not overlapping) with 256-thread CTAs
 * holding 4 16-byte vectors per thread, launched the same way: the
 * simplest kernel that moves a small-batch call's bytes.  Returns
 * NF_ERR_INVALID_ARG (unknown kind, bad size, null or overlapping
 * buffers) or NF_ERR_MISALIGNED before launching anything. */
nf_status nf_selftest_floor(int32_t kind, void* dst, const void* src, int64_t bytes,
                            nf_stream stream);

/* Human-readable name of a status code (static string, never NULL). */
const char* nf_status_string(nf_status status);

/* Library version string (static). */
const char* nf_version(void);

#ifdef __cplusplus
}
#endif

#endif /* NF_H_ */
