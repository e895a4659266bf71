/*
 * solattn.h -- C ABI of libsolattn, a B200 (sm_100a) implementation of the
 * Sol-Attn forward attention operator.
 *
 * Sol-Attn ("Sol-Attn: Accelerating Video Generation Inference via On-the-Fly
 * Attention Sparsification", abstract and paperlayer summary §3 Methodology)
 * runs one online-softmax pass over key/value blocks. For every query block it
 * scores each key block with a proxy taken from the mean-pooled Q and K blocks,
 * keeps the block for exact attention only if the proxy clears a threshold set
 * relative to the running maximum, and folds every dropped block back in as one
 * pseudo-key that carries the block's mean V ("approximate correction" by
 * proxy-score reuse). The proxy map is never written to memory.
 *
 * Definitions used here (the pages leave these open; this library fixes them):
 *   q_i, k_j, v_j  means of Q, K, V over the VALID rows of query block i /
 *                  key block j (a ragged last block divides by its row count n_j)
 *   s_ij           = q_i . k_j / sqrt(d)                          (block proxy)
 *   visit order    query block i visits key blocks (j0 + t) mod nKB,
 *                  t = 0..nKB-1, with j0 = min(floor(i*Bq/Bk), nKB-1)
 *   threshold      M = max of the proxies visited so far (current included);
 *                  the visited block is kept iff s_ij >= M - tau
 *   output row r   keep_correct: [sum_kept sum_c e^{s_rc} v_c + sum_dropped n_j e^{s_ij} v_j]
 *                               / [sum_kept sum_c e^{s_rc} + sum_dropped n_j e^{s_ij}]
 *                  keep_drop:    the same without the dropped terms
 *                  dense:        every block kept (plain softmax attention)
 *   with s_rc = q_r . k_c / sqrt(d).
 * These are the definitions of solattn_forward. solattn_forward_gaussian and
 * solattn_forward_ex add the pages' query-dependent Gaussian threshold, sink tokens and
 * the token-to-block correction; each is defined where it is declared below.
 *
 * Data layout: q, k, v and out are contiguous row-major bf16 [B][H][N][d]
 * (token index n = (t*Y + y)*X + x for a (t, y, x) patch grid, t-major).
 * Pooled buffers are contiguous fp32 [B][H][nB][d].
 *
 * Threading: every entry point that takes a stream enqueues work on that
 * CUDA stream (cudaStream_t passed as void*, NULL = legacy default stream)
 * and returns without waiting, except solattn_get_status and
 * solattn_forward_host, which synchronise the stream.
 *
 * Ownership: the caller allocates and owns every buffer (inputs, output,
 * statistics, workspace). The library allocates no memory at run time. Its one
 * device-memory holding is the static scratch of solattn_forward_noalloc
 * (SOLATTN_NOALLOC_SCRATCH_BYTES), a module-scope device array that exists on
 * every GPU where the library's module is loaded, for the life of the process.
 * solattn_forward_host also keeps, per device, two non-blocking copy streams and
 * a few events, created at its first call there and kept for the process.
 */
#ifndef SOLATTN_H
#define SOLATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Routing / correction mode. */
typedef enum {
  SOLATTN_DENSE = 0,        /* every key block kept: plain softmax attention        */
  SOLATTN_KEEP_DROP = 1,    /* dropped blocks discarded ("keep-or-drop")             */
  SOLATTN_KEEP_CORRECT = 2  /* dropped blocks re-enter as proxy-weighted pseudo-keys */
} solattn_mode;

/* Status codes. Argument errors are returned before any device work is queued. */
typedef enum {
  SOLATTN_OK = 0,
  SOLATTN_EINVAL = -1,       /* null, misaligned or other-GPU pointer, N/B/H < 1, bad mode, tau < 0 or NaN */
  SOLATTN_EUNSUPPORTED = -2, /* d or Bq/Bk not in {64,128}, nKB > 1024, B*H > 65535, no sm_100 device */
  SOLATTN_ECUDA = -3,        /* a CUDA runtime or driver call failed                          */
  SOLATTN_ETIMEOUT = -4,     /* a device-side wait ran past its limit (reported by get_status) */
  SOLATTN_EWORKSPACE = -5,   /* workspace pointer null/misaligned or smaller than required     */
  SOLATTN_EBOUNDS = -6,      /* a device-side bounds check failed (libsolattn_debug.so only:
                                the build with -DSOLATTN_DEBUG; reported by get_status)        */
  SOLATTN_ETABLE = -7        /* a sequence length or page number on the device lies outside the
                                call's buffers (reported by get_status)                        */
} solattn_status;

/* Per-call statistics (device pointers). */
typedef struct {
  /* [B*H] int64: sum over query blocks i of |K_i| (kept key blocks) for each
   * (b, h). Required. Overwritten by every solattn_forward call; in dense mode
   * it is nQB*nKB. */
  int64_t *kept_per_head;
  /* Optional (NULL to skip): [B*H][nQB][ceil(nKB/32)] uint32 keep bit-mask,
   * bit (j & 31) of word (j >> 5) set iff query block i keeps key block j.
   * Overwritten for every valid query block. For tests; off the timed path. */
  uint32_t *keep_mask;
} solattn_stats;

/* Largest number of key blocks per head (nKB = ceil(N/Bk)) a call accepts. */
#define SOLATTN_MAX_KEY_BLOCKS 1024

/*
 * Bytes of device workspace solattn_forward needs for this shape: a small
 * header (work counter, device status word), the pooled q, k, v blocks in fp32,
 * an fp16 copy of v, the work schedule, the keep bits and correction records of
 * the routing pass, and what the Gaussian threshold and the token-to-block
 * correction need. Returns 0 for an unsupported or invalid shape.
 */
size_t solattn_workspace_size(int B, int H, int N, int d, int Bq, int Bk);

/*
 * Mean-pool one bf16 tensor x [B][H][N][d] over blocks of `blk` rows into
 * xbar [B][H][ceil(N/blk)][d] fp32 (ragged last block: mean over its valid
 * rows). Step "mean pooling of each query and key block" (paperlayer summary
 * §2 Preliminaries; §3 Methodology, "pooled keys and summed values").
 * x must be 16-byte aligned, xbar 16-byte aligned. blk in {64,128}, d in {64,128}.
 * Returns SOLATTN_OK or an error code; asynchronous on `stream`.
 */
int solattn_pool(const void *x, float *xbar, int B, int H, int N, int d, int blk,
                 void *stream);

/*
 * The Sol-Attn forward operator (one fused pass per query tile: routing,
 * exact attention on kept blocks, correction for dropped blocks; abstract and
 * paperlayer summary §3 Methodology, "Unified execution").
 *
 *   q, k, v    device, bf16 [B][H][N][d], 16-byte aligned. The P.V product runs in
 *              fp16 (on an fp16 copy of v made by the pooling pass), so entries of v
 *              must lie in the fp16 range, |v| <= 65504; larger ones become inf.
 *   out        device, bf16 [B][H][N][d], 16-byte aligned (written)
 *   B, H, N    batch, heads, tokens (>= 1); nKB = ceil(N/Bk) <= SOLATTN_MAX_KEY_BLOCKS
 *   d          head dim, 64 or 128
 *   Bq, Bk     query / key block sizes, each 64 or 128
 *   tau        threshold offset in logit units, >= 0; +INFINITY keeps every block;
 *              ignored in dense mode
 *   mode       a solattn_mode
 *   stats      required; stats->kept_per_head device [B*H] int64
 *   workspace  device, 256-byte aligned, >= solattn_workspace_size(...) bytes;
 *              must not be used by another call that runs at the same time
 *   stream     cudaStream_t (as void*)
 *
 * Every device pointer must belong to the current device (cudaGetDevice): one that
 * belongs to another GPU is rejected with SOLATTN_EINVAL. The buffers' sizes cannot be
 * checked here; the caller guarantees the sizes stated above.
 *
 * Returns SOLATTN_OK once the work is queued (errors inside the kernels are
 * reported by solattn_get_status), or an error code with nothing queued.
 */
int solattn_forward(const void *q, const void *k, const void *v, void *out,
                    int B, int H, int N, int d, int Bq, int Bk, float tau, int mode,
                    const solattn_stats *stats, void *workspace, size_t ws_bytes,
                    void *stream);

/*
 * solattn_forward plus two CUDA events (cudaEvent_t as void*, either may be NULL)
 * recorded on `stream` immediately before and after the attention kernel, so a
 * caller can time that kernel alone inside a timed region. Same arguments,
 * results and errors as solattn_forward.
 */
int solattn_forward_events(const void *q, const void *k, const void *v, void *out,
                           int B, int H, int N, int d, int Bq, int Bk, float tau, int mode,
                           const solattn_stats *stats, void *workspace, size_t ws_bytes,
                           void *stream, void *ev_attn_begin, void *ev_attn_end);

/*
 * Size of the library's static device scratch used by solattn_forward_noalloc
 * (64 MiB, held on every GPU that loads the library until the process exits).
 */
#define SOLATTN_NOALLOC_SCRATCH_BYTES (64u << 20)

/*
 * solattn_forward for callers that cannot allocate device memory. The paper has no
 * counterpart to this entry point; it is an interface convenience of this library.
 *
 * Who needs it: code that receives only its input and output buffers and a stream
 * (plugin interfaces of inference runtimes, callbacks that run while the host
 * framework's allocator is locked, processes with a fixed device-memory budget where
 * a late cudaMalloc fails or synchronises the whole device) cannot provide the
 * workspace solattn_forward asks for. This entry point takes the same arguments minus
 * the workspace and calls no allocating routine (no cudaMalloc, cudaFree or library
 * allocator); its scratch is a static device array of SOLATTN_NOALLOC_SCRATCH_BYTES.
 *
 *   - The first call on a device looks up that array's device address
 *     (cudaGetSymbolAddress) with the device current, and later calls on that device
 *     reuse it; make this first call before any stream capture. cudaDeviceReset
 *     unloads the module and may move the array: do not call this entry point on a
 *     device after resetting it in the same process.
 *   - Shapes whose solattn_workspace_size(...) exceeds SOLATTN_NOALLOC_SCRATCH_BYTES
 *     are rejected with SOLATTN_EWORKSPACE before any device work.
 *   - Every call on a device uses the same scratch, which keeps the previous call's
 *     contents; the call clears what must start at zero (work counter, status word)
 *     on its stream. Calls that overlap on the GPU (on different streams, or from
 *     different threads) race on the scratch and give wrong results: serialise them.
 *   - Device-side wait timeouts are recorded in the static scratch and are not
 *     reported to the caller; use solattn_forward and solattn_get_status when that
 *     status is needed.
 * Arguments, results and the other errors are those of solattn_forward.
 */
int solattn_forward_noalloc(const void *q, const void *k, const void *v, void *out,
                            int B, int H, int N, int d, int Bq, int Bk, float tau, int mode,
                            const solattn_stats *stats, void *stream);

/* Variant of the Gaussian threshold's variance estimate. */
typedef enum {
  SOLATTN_GAUSS_EXACT = 0,  /* full pooled-key covariance: sigma_i^2 = q_i^T Cov[K] q_i / d      */
  SOLATTN_GAUSS_DIAG = 1    /* its diagonal only: sigma_i^2 = sum_e q_ie^2 Cov[K]_ee / d          */
} solattn_gauss_variant;

/*
 * solattn_forward with the pages' query-dependent Gaussian threshold in place of the
 * running-maximum rule ("Sol-Attn: Accelerating Video Generation Inference via
 * On-the-Fly Attention Sparsification", paperlayer summary §2, Figure 2: a threshold from
 * the proxy-logit mean, standard deviation and a standardized offset beta; §3
 * "Dynamic threshold routing": mean and variance from the pooled keys' first and second
 * moments, one shared cutoff; appendix "Diagonal threshold estimator").
 *
 *   theta_i  = q_i . E[K] / sqrt(d) + beta * sigma_i, with E and Cov taken over the key
 *              blocks' pooled rows k_j (equal weight, 1/nKB), sigma_i as in `variant`
 *   keep     iff s_ij >= theta_i; the block with query block i's largest proxy (lowest
 *              index on ties) is always kept, so no exact set is empty
 *   output   as solattn_forward for `mode` (dense ignores beta)
 *
 * beta may be +-infinity (-inf keeps every block, +inf only each row's top block).
 * Errors: beta NaN or an unknown variant -> SOLATTN_EINVAL; otherwise as
 * solattn_forward. The workspace is the same (solattn_workspace_size).
 */
int solattn_forward_gaussian(const void *q, const void *k, const void *v, void *out,
                             int B, int H, int N, int d, int Bq, int Bk, float beta, int variant,
                             int mode, const solattn_stats *stats, void *workspace, size_t ws_bytes,
                             void *stream);

/* Routing rule of solattn_forward_ex. */
typedef enum {
  SOLATTN_RULE_RUNNING_MAX = 0,  /* keep iff s_ij >= M - tau (solattn_forward)                 */
  SOLATTN_RULE_GAUSS_EXACT = 1,  /* keep iff s_ij >= theta_i, exact covariance (solattn_forward_gaussian) */
  SOLATTN_RULE_GAUSS_DIAG = 2    /* the same with the diagonal covariance                       */
} solattn_rule;

/* Routing options of solattn_forward_ex. */
typedef struct {
  int rule;    /* solattn_rule                                                          */
  float tau;   /* running-max rule: tau >= 0 (+infinity keeps every block)              */
  float beta;  /* Gaussian rules: standardized offset (not NaN; +-infinity allowed)     */
  int n_sink;  /* leading key tokens kept as sinks: 0 <= n_sink <= N                    */
  int correction; /* keep_correct only: SOLATTN_CORR_BLOCK (0) or SOLATTN_CORR_TOKEN (1)   */
} solattn_route;

/* Correction of solattn_forward_ex in keep_correct mode. */
typedef enum {
  SOLATTN_CORR_BLOCK = 0,  /* dropped block j enters query block i with the block proxy s_ij     */
  SOLATTN_CORR_TOKEN = 1   /* it enters row r with the token-to-block logit q_r . k_j / sqrt(d)   */
} solattn_correction;

/*
 * The forward operator with every routing option. Sinks: the text key-value tokens that
 * the pages keep in the exact branch for every query ("Sol-Attn: Accelerating Video
 * Generation Inference via On-the-Fly Attention Sparsification", paperlayer summary,
 * App. A Additional Experimental Details). This library takes them to be the first
 * n_sink key tokens (a prefix of the [B][H][N][d] layout): every key block that holds
 * one of them, ceil(n_sink / Bk) blocks, is kept by every query block under either rule
 * and is never folded into the correction. The proxies of sink blocks still enter the
 * running maximum, so the other keep decisions do not change; under a Gaussian rule the
 * top-block guard applies only to a query block that would otherwise keep nothing.
 * Token-to-block correction (keep_correct, correction = SOLATTN_CORR_TOKEN): the pages
 * fuse routing and correction through a token-to-block score tile ("Unified execution",
 * paperlayer summary §3). Each row r then meets every block j its query block dropped as
 * one pseudo-key: logit q_r . k_j / sqrt(d) (pooled key k_j), weight n_j, value v_j,
 * inside the same online softmax as the exact blocks (computed on the tensor cores over
 * the head's pooled keys, with the kept blocks masked out).
 * With n_sink = 0 and the block correction, rule RUNNING_MAX equals solattn_forward and
 * the Gaussian rules equal solattn_forward_gaussian.
 * Errors: route NULL, an unknown rule, tau < 0 or NaN (running max), beta NaN (Gaussian),
 * n_sink outside [0, N] or an unknown correction -> SOLATTN_EINVAL; otherwise as
 * solattn_forward.
 */
int solattn_forward_ex(const void *q, const void *k, const void *v, void *out,
                       int B, int H, int N, int d, int Bq, int Bk, const solattn_route *route,
                       int mode, const solattn_stats *stats, void *workspace, size_t ws_bytes,
                       void *stream);

/*
 * The routing stage on its own, for the routing-overhead measurement ("Sol-Attn:
 * Accelerating Video Generation Inference via On-the-Fly Attention Sparsification",
 * paperlayer summary §4 Experiments, "Efficient On-the-Fly Sparsification": routing that
 * consumes proxy scores on chip, against top-k and top-p routing, which materialise the
 * proxy map and traverse its rows; §2 Block-Sparse Attention). The three routers read the
 * same pooled blocks and write keep bits in the layout of solattn_stats.keep_mask:
 *
 *   qbar, kbar  device fp32 [B][H][nQB][d] and [B][H][nKB][d] (block means, as written by
 *               solattn_pool with blk = Bq and Bk), 16-byte aligned
 *   keep_mask   device u32 [B][H][nQB][ceil(nKB/32)], written
 *   proxy_map   device fp32 scratch of solattn_proxy_map_bytes(...) bytes (map_bytes), which
 *               the top-k and top-p routers fill with s_ij = q_i . k_j / sqrt(d)
 *
 * solattn_route_keep: the running-maximum rule of solattn_forward (same visit order, same
 *   tau), computed as the forward kernel's router does, with no proxy leaving the chip.
 * solattn_route_topk: keeps the min(k, nKB) key blocks with the largest proxies of every
 *   query block (ties: lower block index). k >= 1.
 * solattn_route_topp: ranks the key blocks of a query block by mass n_j e^{s_ij} (n_j valid
 *   keys of block j; ties: lower index) and keeps the shortest prefix whose share of the
 *   row's total mass reaches p (a block is kept iff the mass ranked before it is below
 *   p times the total). 0 < p <= 1.
 * The readings of top-k and top-p are this library's (the pages name the rules only).
 * Errors: null or misaligned pointers, tau < 0 or NaN, k < 1, p outside (0, 1] ->
 * SOLATTN_EINVAL; a short proxy_map -> SOLATTN_EWORKSPACE; otherwise as solattn_forward.
 * Asynchronous on `stream`.
 */
int solattn_route_keep(const float *qbar, const float *kbar, int B, int H, int N, int d, int Bq, int Bk,
                       float tau, uint32_t *keep_mask, void *stream);
size_t solattn_proxy_map_bytes(int B, int H, int N, int Bq, int Bk);
int solattn_route_topk(const float *qbar, const float *kbar, int B, int H, int N, int d, int Bq, int Bk,
                       int k, float *proxy_map, size_t map_bytes, uint32_t *keep_mask, void *stream);
int solattn_route_topp(const float *qbar, const float *kbar, int B, int H, int N, int d, int Bq, int Bk,
                       float p, float *proxy_map, size_t map_bytes, uint32_t *keep_mask, void *stream);

/*
 * Synchronise `stream` and read the device status word of `workspace`
 * (SOLATTN_OK, or SOLATTN_ETIMEOUT if a bounded device-side wait gave up).
 */
int solattn_get_status(const void *workspace, void *stream);

/* Bytes of device scratch solattn_forward_host needs (device copies of q, k,
 * v, out, the per-head counts, per-chunk status words and the forward
 * workspace). 0 if invalid. */
size_t solattn_host_workspace_size(int B, int H, int N, int d, int Bq, int Bk);

/*
 * End-to-end call on HOST buffers: copies q, k, v (bf16 [B][H][N][d], host) to
 * the device scratch, runs the forward operator (running-max rule, `tau`,
 * `mode` as in solattn_forward), copies the bf16 output to `out` and the
 * per-head kept counts to `kept_per_head` (host int64 [B*H], may be NULL),
 * synchronises `stream` and returns the first non-zero device status, else
 * SOLATTN_OK.
 * The (b, h) heads are independent, so the call is a pipeline over up to 16
 * chunks of consecutive heads: the upload of one chunk and the download of the
 * one before overlap the forward of the chunk between them. Uploads and
 * downloads run on the library's copy streams for this device, the forward on
 * `stream`; the result equals that of one solattn_forward over all heads.
 * Copies overlap only from page-locked (pinned) host memory.
 * dev_scratch: device, 256-byte aligned, >= solattn_host_workspace_size(...).
 * Calls on one device are serialised (they share the copy streams). On an error
 * the call waits for the copies it issued before returning.
 */
int solattn_forward_host(const void *q, const void *k, const void *v, void *out,
                         int B, int H, int N, int d, int Bq, int Bk, float tau, int mode,
                         int64_t *kept_per_head, void *dev_scratch, size_t scratch_bytes,
                         void *stream);

/*
 * Self-test of the device watchdog: launches one block that waits on a
 * barrier nobody completes, with a limit of `limit_ns` nanoseconds, and
 * stores the resulting status (SOLATTN_ETIMEOUT when the watchdog works) in
 * the workspace status word. Read it with solattn_get_status.
 */
int solattn_watchdog_selftest(void *workspace, size_t ws_bytes, uint64_t limit_ns,
                              void *stream);

/*
 * Self-test of the software exp2 the softmax evaluates on the FMA pipe for part of
 * its exponentials: y[i] = 2^x[i] for n device floats (x, y device pointers).
 * Lets a test compare it with exp2 within its stated bound (relative error 7.5e-5
 * for x >= -125; smaller inputs are clamped to -125).
 */
int solattn_selftest_exp2(const float *x, float *y, int n, void *stream);

/*
 * ---------------------------------------------------------------------------------------
 * Dense attention beside the operator: to an encoder's states, and over a paged cache.
 *
 * A diffusion transformer's block attends its own tokens (solattn_forward) and, with the
 * same heads, the states of a text or image encoder; a streaming generator attends a cache
 * of earlier frames. These entry points compute plain softmax attention (no routing)
 * for those two, in bf16 or fp16, with shared key heads and strided tensors, and write and
 * read the cache, in 16 bits or quantised to 8. They are inference operators, as the rest
 * of the library: no gradients.
 *
 * Common to all of them:
 *   dtype      solattn_dtype of the 16-bit tensors
 *   H, Hkv     query heads and key heads; Hkv divides H, query head h uses key head h / (H/Hkv)
 *   d          64 or 128; the logits are scaled by 1/sqrt(d)
 *   strides    in elements; the d elements of a row are contiguous, every stride is a
 *              multiple of 8 elements (16 for 8-bit pages) and every base address of 16 bytes.
 *              Inputs may overlap or repeat (stride 0); outputs may not
 *   empty rows a query that sees no key gives a row of zeros
 *   rounding   the probabilities (8-bit pages: times the value's scale) are rounded to the product's 16-bit type,
 *              bf16, or fp16 for fp16 and 8-bit pages: off by at most 2^-8 (2^-11) of their value, or in fp16 by 2^-25 of the row's
 *              largest where they are below 2^-14 of it. Sums and outputs are in 32 bits until the last rounding, with
 *              probabilities of up to 2^15 before it: bf16 values from 2^112 up may overflow. Scales of 8-bit pages may be
 *              negative or zero; those of values count from 2^-100 to 2^100 in magnitude
 *   masked     keys and values behind a sequence's length are not used, whatever they hold.
 *              Keys that only LATER queries see (causal) must have finite values (v)
 *   lengths    cu and len are device data and unknown to the host. Values outside the
 *              buffers are cut to them and page numbers outside the cache read as zeros (writes are
 *              dropped); either is recorded as SOLATTN_ETABLE in the workspace's status word
 *   workspace  device, 256-byte aligned, of the size that the size function gives; its first 256 bytes must be
 *              zero before its first use. The status word keeps the first error until the
 *              caller clears it (the binding's calls without a workspace take one of their own, so nobody sees its status). Not to be used by two calls that may run at the same time
 *   errors     as solattn_forward; nothing is queued on an error
 * ---------------------------------------------------------------------------------------
 */
typedef enum {
  SOLATTN_BF16 = 0,
  SOLATTN_FP16 = 1
} solattn_dtype;

/* A [B][heads][n][d] tensor. A tensor of packed rows [n][heads][d] has stride_b = 0. */
typedef struct {
  void *ptr;
  int64_t stride_b, stride_h, stride_n;
} solattn_view;

/* What the pages of a cache hold. */
typedef enum {
  SOLATTN_CACHE_16 = 0,    /* rows in the calls' 16-bit dtype                                */
  SOLATTN_CACHE_INT8 = 1,  /* int8 codes, one fp32 scale for each row of d: x = code * scale */
  SOLATTN_CACHE_E4M3 = 2   /* the same with e4m3 codes                                       */
} solattn_cache_kind;

/*
 * A cache: k and v are [num_pages][Hkv][page][d] views (stride_b of a page, stride_h of a
 * head in it, stride_n of a row), k_scale and v_scale contiguous fp32 [num_pages][Hkv][page]
 * (8-bit kinds only). page is 16, 32, 64 or 128 tokens.
 */
typedef struct {
  solattn_view k, v;
  float *k_scale, *v_scale;
  int num_pages, Hkv, page, d, kind;
} solattn_cache;

/*
 * The sequences of a call over a cache. Sequence b has len[b] tokens in the cache; position
 * j of it is row j % page of page table[b * width + j / page]. Its NEW tokens, the last
 * n_b = cu[b+1] - cu[b] of them, are rows cu[b] .. cu[b+1] - 1 of the packed tensors.
 * Table entries behind a sequence's last page are not read. Two sequences may share pages
 * that no call writes.
 */
typedef struct {
  const int32_t *table; /* device [B][width]                                                  */
  const int32_t *cu;    /* device [B+1], ascending from 0, at most total                      */
  const int32_t *len;   /* device [B], n_b <= len[b] <= width * page                          */
  int B, width, total;  /* total: rows of the packed tensors (those behind cu[B] are left alone) */
} solattn_seqs;

/*
 * Attention of q [B][H][Nq][d] to k, v [B][Hkv][Nk][d]: sequence b's queries see its first
 * key_len[b] keys (device int32 [B], or NULL: all Nk). Nq and Nk may be 0 or more.
 */
size_t solattn_cross_workspace_size(int B, int H, int Hkv, int Nq, int Nk, int d);
int solattn_cross(const solattn_view *q, const solattn_view *k, const solattn_view *v, const solattn_view *out,
                  const int32_t *key_len, int B, int H, int Hkv, int Nq, int Nk, int d, int dtype,
                  void *workspace, size_t ws_bytes, void *stream);

/*
 * Attention of the new tokens q [total][H][d] (packed; stride_b ignored) over the cache,
 * which already holds them. causal = 0: every new token sees its whole sequence; 1: up to its own position.
 * max_new: the largest n_b the caller expects; it chooses the kernel only, and a larger n_b
 * is computed all the same.
 */
size_t solattn_paged_workspace_size(int B, int H, int Hkv, int total, int d);
int solattn_paged_forward(const solattn_view *q, const solattn_view *out, const solattn_cache *cache,
                          const solattn_seqs *seqs, int H, int max_new, int causal, int dtype, void *workspace,
                          size_t ws_bytes, void *stream);

/*
 * Writes the new tokens' keys and values [total][Hkv][d] into their pages. 8-bit kinds:
 * scale = fl(max|x| / TOP) and code = nearest(x TOP / max|x|), ties to even, TOP = 127
 * (int8) or 448 (e4m3); a row of zeros has scale 0, a row with an infinity or NaN has scale
 * NaN. Where two new tokens share a page's row (pages shared by two sequences) the row's codes and scale are
 * pieces of either, in no particular order. Lengths out of range are cut as the attention cuts them; tokens in front of
 * their sequence's first position are not written. status: device, 256-byte aligned, 256 bytes, zero before first use
 * (any workspace of the calls above serves).
 */
int solattn_cache_append(const solattn_cache *cache, const solattn_view *new_k, const solattn_view *new_v,
                         const solattn_seqs *seqs, int dtype, void *status, void *stream);

/* Reads the new tokens' rows back into k_out and v_out [total][Hkv][d]: code * scale, rounded
 * once. Rows whose page is outside the cache are left as they were. */
int solattn_cache_read(const solattn_cache *cache, const solattn_seqs *seqs, const solattn_view *k_out,
                       const solattn_view *v_out, int dtype, void *status, void *stream);

/* Static description of a status code. */
const char *solattn_strerror(int status);

#ifdef __cplusplus
}
#endif

#endif /* SOLATTN_H */
