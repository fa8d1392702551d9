/*
 * asffn.h -- C ABI of libasffn.so: activation-sparse FFN decode on B200 (sm_100a).
 *
 * The operations follow the problem statement of the pages on PowerInfer-style
 * neuron-level sparse inference:
 *   - predict(x) -> active index list: the online neuron predictor
 *     ("PowerInfer Guide: Exploiting Activation Sparsity for LLM AI", section 3
 *     "Adaptive Online Neuron Predictors", predictor equation and the Step 2
 *     predictor module), read as the 2-layer MLP of the "PowerInfer_x64" page
 *     ("Prediction and Caching"): h = ReLU(W1 x + b1), z = W2 h + b2,
 *     neuron k active iff sigmoid(z_k) > tau (strict), i.e. z_k > logit(tau).
 *   - sparse_ffn(x, idx) -> y: the neuron-aware sparse operator (PowerInfer
 *     Guide, section 4 "Neuron-Aware Sparse GPU Operators", and the FFN
 *     equation of "The Hidden Inefficiency") evaluated only for listed neurons.
 *   - activation counts + hot permutation: the offline profiler and hot/cold
 *     split (PowerInfer Guide, Step 1), used to store hot rows first.
 *
 * Conventions shared by every call:
 *   - All pointers named "device" are CUDA device pointers owned by the caller;
 *     the library never allocates or frees device memory and never keeps a
 *     pointer after a call returns (the descriptor structs are read at call
 *     time only).
 *   - Calls that take a stream enqueue work on it and return without
 *     synchronising (except asf_read_error).  Launch failures return
 *     ASF_ERR_CUDA; no call terminates the process.
 *   - Arguments are validated on the host before any launch; a call that
 *     returns an error has enqueued nothing.
 *   - Checks that need device data (an index outside [0, n), count > n) cannot
 *     be done on the host: the kernel skips the offending item and records the
 *     fault in the workspace error word, read with asf_read_error.
 *   - Weights, x and y must be 16-byte aligned; d and r must be multiples of 8
 *     (fp16) or 4 (fp32).  x has the weight dtype; y is always fp32.
 *   - Accumulation is fp32 throughout.
 */
#ifndef ASFFN_H
#define ASFFN_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define ASF_API __attribute__((visibility("default")))
#else
#define ASF_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* cudaStream_t; NULL means the legacy default stream. */
typedef struct CUstream_st *asf_stream_t;

typedef enum {
  ASF_OK = 0,
  ASF_ERR_INVALID_ARG = 1,  /* null pointer, bad size, tau outside (0,1), ... */
  ASF_ERR_MISALIGNED = 2,   /* a pointer or row length breaks the alignment rule */
  ASF_ERR_UNSUPPORTED = 3,  /* dtype/activation/batch combination not built */
  ASF_ERR_CUDA = 4,         /* a CUDA runtime call or launch failed */
  ASF_ERR_DEVICE_INDEX = 5, /* device saw idx outside [0, n) or count > n */
  ASF_ERR_TIMEOUT = 6,      /* a bounded device-side wait gave up */
  ASF_ERR_WORKSPACE = 7     /* workspace missing, misaligned or too small */
} asf_status;

typedef enum { ASF_F32 = 0, ASF_F16 = 1 } asf_dtype;

/* ASF_ACT_RELU : y = W_down ReLU(W_up x + b)                  (up + down)
 * ASF_ACT_REGLU: y = W_down (ReLU(W_gate x + b) * (W_up x))   (gate, up, down) */
typedef enum { ASF_ACT_RELU = 0, ASF_ACT_REGLU = 1 } asf_act;

#define ASF_MAX_BATCH 32

/* Two-layer predictor, borrowed device pointers.  Row-major. */
typedef struct {
  int32_t d;          /* input width (hidden size) */
  int32_t r;          /* predictor hidden width */
  int32_t n;          /* number of FFN neurons (d_ffn) */
  asf_dtype wdtype;   /* dtype of W1, W2 and of x */
  const void *W1;     /* [r][d] */
  const float *b1;    /* [r] */
  const void *W2;     /* [n][r] */
  const float *b2;    /* [n] */
} asf_predictor;

/* One FFN layer, borrowed device pointers.  Row k of every matrix belongs to
 * neuron k in storage order (after any hot permutation). */
typedef struct {
  int32_t d;          /* hidden size */
  int32_t n;          /* number of neurons */
  asf_dtype wdtype;   /* dtype of Wg, Wu, WdT and of x */
  asf_act act;
  const void *Wg;     /* [n][d] gate rows (REGLU), NULL for RELU */
  const void *Wu;     /* [n][d] up rows */
  const void *WdT;    /* [n][d] W_down transposed: row k = column k of W_down */
  const float *bias;  /* [n] bias of the ReLU input: gate (REGLU) or up (RELU) */
  int32_t hot_rows;   /* rows 0..hot_rows-1 are active for most tokens (hot neurons stored
                         first by the offline permutation); asf_sparse_ffn prefetches them
                         into L2 while the list is still being predicted.  0 = no hint.
                         Affects speed only, never results. */
  int32_t row_stride; /* elements between consecutive rows of Wg/Wu/WdT; 0 means d.  With
                         row_stride = m*d and Wu = Wg + d, WdT = Wu + d (REGLU; for RELU
                         WdT = Wu + d) the layer is in the neuron-major packed layout
                         (gate|up|down of a neuron contiguous, see asf_gather_rows), and the
                         sparse FFN fetches each neuron with one bulk copy. */
  const void *l2_next[2];      /* optional L2 prefetch hint: up to two device ranges that are
                                  read soon after this call (for example the next layer's
                                  predictor W1 and W2).  The call's last kernel pulls them into
                                  L2 while it waits for the sparse FFN, whose row stream does
                                  not keep HBM busy on its own.  Each non-NULL range must be
                                  16-byte aligned and mapped for l2_next_bytes[i] bytes (the
                                  tail below a multiple of 16 is skipped).  NULL / 0 = none.
                                  Affects speed only, never results. */
  int64_t l2_next_bytes[2];
} asf_ffn;

/* Bytes of device workspace needed by asf_predict / asf_sparse_ffn /
 * asf_dense_ffn / asf_activation_counts for batches up to max_batch.  Either
 * descriptor may be NULL; with both, the size also serves
 * asf_predict_sparse_ffn (the two scratch areas side by side).  Returns 0 on
 * invalid arguments. */
ASF_API size_t asf_workspace_bytes(const asf_predictor *pred, const asf_ffn *ffn, int32_t max_batch);

/* Zero a freshly allocated workspace (256-byte aligned device buffer).  Must be
 * called once before first use; afterwards every call leaves the workspace's
 * counters at zero again.  One workspace serves one stream at a time. */
ASF_API asf_status asf_workspace_init(void *ws, size_t ws_bytes, asf_stream_t stream);

/* Online predictor for B tokens (1 <= B <= ASF_MAX_BATCH).
 *   x     device [B][d], wdtype
 *   tau   threshold on sigmoid(z), 0 < tau < 1
 *   idx   device int32 [n]: on completion idx[0..count) holds the ascending
 *         storage indices of the neurons predicted active for at least one of
 *         the B tokens (the union); entries past count are left untouched
 *   count device int32 [1]
 * Stays on the device: no host synchronisation. */
ASF_API asf_status asf_predict(const asf_predictor *pred, const void *x, int32_t B, float tau,
                       int32_t *idx, int32_t *count, void *ws, size_t ws_bytes,
                       asf_stream_t stream);

/* Sparse FFN over an index list, every token over the same list.
 *   x     device [B][d], wdtype
 *   idx   device int32 [n]; the first *count entries are used (any order,
 *         duplicates are summed twice); entries outside [0, n) are skipped and
 *         flagged
 *   count device int32 [1], 0 <= *count <= n (larger is clamped and flagged)
 *   y     device fp32 [B][d], overwritten: y_b = sum_j a_{idx_j, b} WdT[idx_j]
 *         with a = ReLU(gate + bias) * up  (REGLU)  or  ReLU(up + bias)  (RELU) */
ASF_API asf_status asf_sparse_ffn(const asf_ffn *ffn, const void *x, int32_t B, const int32_t *idx,
                          const int32_t *count, float *y, void *ws, size_t ws_bytes,
                          asf_stream_t stream);

/* One layer of the decode path in one call: asf_predict followed by
 * asf_sparse_ffn over the predicted list (the predictor-then-sparse-operator
 * flow of the PowerInfer Guide, Step 2 predictor module feeding the Step 3
 * sparse FFN, and the PowerInfer_x64 page's "Prediction and Caching"), with
 * the same results (idx, count and y bit for bit).  For B <= 4 the sparse FFN kernel ranks the predictor's
 * union mask itself, so no separate compaction kernel or index-list round
 * trip sits between the two; larger batches run the two calls' kernels.
 *   pred, ffn   descriptors of the same layer: equal d, n and wdtype
 *   x, B, tau   as for asf_predict
 *   idx, count  outputs as for asf_predict (the list the FFN used)
 *   y           output as for asf_sparse_ffn
 *   ws          at least asf_workspace_bytes(pred, ffn, B) bytes */
ASF_API asf_status asf_predict_sparse_ffn(const asf_predictor *pred, const asf_ffn *ffn, const void *x,
                                          int32_t B, float tau, int32_t *idx, int32_t *count, float *y,
                                          void *ws, size_t ws_bytes, asf_stream_t stream);

/* The same layer in two halves, for callers that put other work or timing
 * events between the predictor and the sparse FFN.  Called in this order on
 * one stream with identical arguments, _begin then _end enqueue exactly the
 * kernels of asf_predict_sparse_ffn and give the same idx, count and y bit for
 * bit.  _begin runs the predictor and leaves its result (the union mask, or
 * for B > 8 the list itself) in the workspace; _end compacts the mask when
 * needed and runs the sparse FFN.  Nothing else may use the workspace between
 * the two.  Arguments, validation and errors as for asf_predict_sparse_ffn. */
ASF_API asf_status asf_predict_sparse_ffn_begin(const asf_predictor *pred, const asf_ffn *ffn, const void *x,
                                                int32_t B, float tau, int32_t *idx, int32_t *count, float *y,
                                                void *ws, size_t ws_bytes, asf_stream_t stream);
ASF_API asf_status asf_predict_sparse_ffn_end(const asf_predictor *pred, const asf_ffn *ffn, const void *x,
                                              int32_t B, float tau, int32_t *idx, int32_t *count, float *y,
                                              void *ws, size_t ws_bytes, asf_stream_t stream);

/* Dense FFN over all n neurons (the unsparsified reference, same kernels with an
 * implicit identity index list).  Arguments as asf_sparse_ffn. */
ASF_API asf_status asf_dense_ffn(const asf_ffn *ffn, const void *x, int32_t B, float *y, void *ws,
                         size_t ws_bytes, asf_stream_t stream);

/* Offline profiler: counts[k] += number of the T tokens of x (device [T][d])
 * whose ReLU input (gate + bias for REGLU, up + bias for RELU) is > 0.
 * counts: device int64 [n], accumulated so calibration can be chunked. */
ASF_API asf_status asf_activation_counts(const asf_ffn *ffn, const void *x, int32_t T, int64_t *counts,
                                 void *ws, size_t ws_bytes, asf_stream_t stream);

/* Strided row gather on the device: dst row i (at dst + i*dst_stride bytes) =
 * src row p (at src + p*src_stride bytes) with p = perm[i] (p = i when perm is
 * NULL), row_bytes each, for i < n_rows; rows with p outside [0, src_rows) are
 * skipped.  With dst_stride = m*d*s and dst offsets 0, d*s, 2*d*s it builds the
 * neuron-major packed layout of asf_ffn (and applies a hot permutation in the
 * same pass).  Source and destination ranges must not overlap. */
ASF_API asf_status asf_gather_rows(const void *src, int64_t src_stride, int32_t src_rows, void *dst,
                                   int64_t dst_stride, int32_t n_rows, int64_t row_bytes,
                                   const int32_t *perm, asf_stream_t stream);

/* Host-side, synchronous: perm = neuron ids in descending count order, equal
 * counts in ascending id order.  counts: host int64 [n]; perm_out: host int32 [n]. */
ASF_API asf_status asf_hot_permutation(const int64_t *counts, int32_t n, int32_t *perm_out);

/* Row gather on the device: dst row i = src row perm[i], for i < n_rows.
 * src, dst: device [n_rows][row_bytes], distinct buffers; perm: device int32
 * [n_rows] with values in [0, n_rows) (out-of-range rows are skipped). */
ASF_API asf_status asf_permute_rows(const void *src, void *dst, int32_t n_rows, int64_t row_bytes,
                            const int32_t *perm, asf_stream_t stream);

/* Sparse FFN that allocates nothing and needs no workspace.
 *
 * No counterpart in the paper: this is a deployment convenience.  Some
 * callers cannot allocate device memory where they run the FFN -- for example
 * a plugin inside a host framework that owns every device allocation through
 * its own pool, or a latency-critical path that cannot afford the implicit
 * device synchronisation of cudaMalloc.  This call computes exactly what
 * asf_sparse_ffn computes (same kernels, same summation order, so the same y
 * bit for bit), but takes its scratch from a file-scope device array of
 * ASF_NOALLOC_SCRATCH_BYTES inside the library, which every GPU that loads the
 * library holds until the process exits.
 *
 *   ffn, x, B, idx, count, y   as for asf_sparse_ffn
 *   fault   optional device int32: if not NULL, it receives the raw fault bits
 *           of this call (0 = none; bit 0 = index out of range, bit 1 = timeout)
 *
 * Size limit.  The call needs 4096 bytes of counters plus the scratch of
 * asf_sparse_ffn: for B <= 4, G * B * d * 4 bytes of per-CTA partial sums with
 * G = min(SM count, 256) (148 on B200); for larger B, n * B * 4 bytes of
 * activations plus the down projection's S * B * d * 4 bytes of split sums
 * (S <= 64 splits of the index list).  Shapes that need more than
 * ASF_NOALLOC_SCRATCH_BYTES return ASF_ERR_UNSUPPORTED without enqueuing
 * anything.  On B200 the 32 MiB array covers every layer with d <= 12288 and
 * n <= 49152 at every batch up to ASF_MAX_BATCH; the largest need among them,
 * d = 12288 at B = 4, is 29.1 MB.
 *
 * The first call on each device looks up the array's device address for the
 * current device (cudaGetSymbolAddress) and keeps it for the life of the
 * process; make that first call before any stream capture.  The kept address
 * is not valid across cudaDeviceReset (the library's module is reloaded in the
 * new context): do not use this call after resetting a device.  Each call
 * clears the array's counters and fault word on `stream` before its kernels
 * run.  All calls share the one array: calls that can overlap on the GPU
 * (other streams, other threads) race and must be serialised by the caller.
 * No device memory is allocated or freed, directly or by a library routine. */
#define ASF_NOALLOC_SCRATCH_BYTES (32u << 20)
ASF_API asf_status asf_sparse_ffn_noalloc(const asf_ffn *ffn, const void *x, int32_t B, const int32_t *idx,
                                          const int32_t *count, float *y, int32_t *fault, asf_stream_t stream);

/* ---------------------------------------------------------------------------
 * 4-bit weights with group scales.
 *
 * The pages run their models at 4 bits ("PowerInfer Guide", the hardware
 * sizing table); these calls are the sparse FFN, a dense product and the
 * format between them.  A row of k weights is stored as
 *
 *   kp / 2 bytes of codes (kp = k rounded up to a multiple of 128), then one
 *   fp16 scale per group of 32, 64 or 128 weights, zero padded:
 *   asf_w4_row_bytes(k, group) bytes, a multiple of 16.
 *
 * Weight i is (code_i - 8) * scale[i / group], 0 <= code_i <= 15; weights past
 * k have code 8.  In each block of 128 weights (16 little-endian 32-bit words)
 * word 4t+j (t, j in 0..3) holds weights 32j+8t .. 32j+8t+7, and weight 2p+h of
 * a word is the nibble at bit 16h+4p.  Rows are plain bytes: asf_gather_rows
 * and asf_permute_rows move them.
 *
 * No weight is rounded on its way through a product: sums run in fp32, scales
 * multiply fp32 sums.  x is fp16 or fp32 (an fp32 x enters exactly; it must be
 * finite and below 2^117, since a group's sum is formed before its scale).  A
 * token's result does not depend on the call's other tokens' values. */
#define ASF_W4_MAX_K 65536
#define ASF_W4_MAX_ROWS (1 << 30)    /* rows of a matrix, neurons of a layer */

typedef struct {
  int32_t rows, k;      /* weights are [rows][k]; k a multiple of 8, at most ASF_W4_MAX_K */
  int32_t group;        /* 32, 64 or 128 */
  const void *data;     /* device, 16-byte aligned; written by asf_w4_quantize only */
  int64_t row_stride;   /* bytes between rows: a multiple of 16, >= asf_w4_row_bytes(k, group) */
} asf_w4_matrix;

/* One FFN layer of 4-bit rows, neuron by neuron: gate | up | down rows (REGLU)
 * or up | down rows (RELU) of a neuron one after the other, each
 * asf_w4_row_bytes(d, group) bytes, the down row being a column of W_down. */
typedef struct {
  int32_t d, n;
  int32_t group;
  asf_act act;
  const void *data;        /* device, 16-byte aligned */
  int64_t neuron_stride;   /* bytes between neurons: a multiple of 16, >= 3 (REGLU) or 2 (RELU) rows */
  const float *bias;       /* device [n] */
} asf_w4_ffn;

/* Bytes of one row, or 0 for a k or group that the format does not have. */
ASF_API int64_t asf_w4_row_bytes(int32_t k, int32_t group);

/* Rows [rows][k] (fp16 or fp32, contiguous, 16-byte aligned, apart from the
 * matrix) to 4 bits, into mat->data: per group scale = fp16(max |w| / 7), code = clamp(round half to
 * even(w / scale), -8, 7) + 8, evaluated in fp32; a group of scale 0 gets code
 * 8.  A group with a NaN, an infinity or a scale past fp16's range gets the
 * scale NaN, so that no product over it looks sound. */
ASF_API asf_status asf_w4_quantize(const void *src, asf_dtype dtype, const asf_w4_matrix *mat, asf_stream_t stream);

/* The weights back as contiguous [rows][k] fp16 (rounded once) or fp32 (exact),
 * apart from the matrix. */
ASF_API asf_status asf_w4_dequantize(const asf_w4_matrix *mat, void *dst, asf_dtype dtype, asf_stream_t stream);

/* Workspace bytes of asf_w4_matmul / asf_w4_sparse_ffn for batches up to
 * max_batch (either descriptor may be NULL; with both, enough for each of the
 * calls in turn).  0 on invalid arguments.  asf_workspace_init zeroes it once. */
ASF_API size_t asf_w4_workspace_bytes(const asf_w4_matrix *mat, const asf_w4_ffn *ffn, int32_t max_batch);

/* y[b][i] = act(sum_k w[i][k] x[b][k] + bias[i]) for 1 <= B <= ASF_MAX_BATCH tokens.
 *   x     device [B][k] in xdtype, 16-byte aligned
 *   bias  device fp32 [rows], or NULL
 *   relu  0: none, 1: max(., 0)
 *   y     device [B][rows] in ydtype (fp16: the fp32 sum rounded once), overwritten;
 *         must not overlap x */
ASF_API asf_status asf_w4_matmul(const asf_w4_matrix *mat, const void *x, asf_dtype xdtype, int32_t B,
                                 const float *bias, int32_t relu, void *y, asf_dtype ydtype, void *ws,
                                 size_t ws_bytes, asf_stream_t stream);

/* asf_sparse_ffn over 4-bit rows: x [B][d] in xdtype, idx/count/y as there;
 * idx and count both NULL runs all n neurons (asf_dense_ffn).  The activations
 * between the two products are fp32; with its scale, one enters the second
 * product in 22 bits (16 where it is 2^20 below its token's largest).  An
 * activation that passes fp32's range, by itself or times a group's scale, is an
 * infinity: its token's y is infinite, with the signs of the down weights, and NaN
 * where such a weight is 0. */
ASF_API asf_status asf_w4_sparse_ffn(const asf_w4_ffn *ffn, const void *x, asf_dtype xdtype, int32_t B,
                                     const int32_t *idx, const int32_t *count, float *y, void *ws, size_t ws_bytes,
                                     asf_stream_t stream);

/* ---------------------------------------------------------------------------
 * Adapters: low-rank corrections of a 4-bit matrix, of which each token of a call
 * uses its own, or none, beside the product that all of them share. */
#define ASF_MAX_LORA_RANK 256

typedef struct {
  int32_t adapters, rank;  /* rank a multiple of 8, at most ASF_MAX_LORA_RANK (pad with zeros) */
  int32_t k, rows;         /* of the matrix */
  asf_dtype dtype;         /* of A and B, and of x */
  const void *A;           /* device [adapters][rank][k], 16-byte aligned */
  const void *B;           /* device [adapters][rows][rank], 16-byte aligned */
  const float *scale;      /* device fp32 [adapters], or NULL: 1 */
} asf_lora;

/* Workspace bytes of asf_w4_matmul_lora for batches up to max_batch (enough for
 * asf_w4_matmul on the same matrix, too).  0 on invalid arguments. */
ASF_API size_t asf_w4_lora_workspace_bytes(const asf_w4_matrix *mat, const asf_lora *lora, int32_t max_batch);

/* y[b] = act(W x[b] + bias + scale[a] B[a] (A[a] x[b])), a = which[b]
 *   which  device int32 [batch]: a token's adapter, negative for none; one from
 *          `adapters` on counts as none and is flagged
 * All else as for asf_w4_matmul, with x in the adapters' dtype.  Everything between x
 * and y is fp32, y is rounded once, and a token's result does not depend on the call's
 * other tokens, nor on their adapters; the adapter's share not on their number either
 * (the product's sums are split by it). */
ASF_API asf_status asf_w4_matmul_lora(const asf_w4_matrix *mat, const asf_lora *lora, const int32_t *which, const void *x,
                                      asf_dtype xdtype, int32_t batch, const float *bias, int32_t relu, void *y,
                                      asf_dtype ydtype, void *ws, size_t ws_bytes, asf_stream_t stream);

/* ---------------------------------------------------------------------------
 * Tree attention: the attention step in front of the predictor (PowerInfer_x64
 * page: attention, then predictor, then the sparse operators) for the tokens
 * of one call, over a paged key/value cache in fp16.
 *
 * R requests share the call's T tokens (1 <= R, T <= ASF_MAX_BATCH): tokens
 * begin[r] .. begin[r+1]-1 are request r's (none is allowed), tokens outside
 * every range take no part.  Request r has lens[r] keys in the cache; its i-th
 * token of the call is at position lens[r] + i.  With one token a request this
 * is plain decoding; several are a tree of drafted tokens, of which token t
 * sees every key before lens[r] and, of the call's tokens, those of its own
 * request whose bit is set in anc[t] (bit j: token j of the call; a token sees
 * itself only through its own bit).  A token that sees nothing gets zeros, and
 * what it does not see, NaN or not, does not reach it.
 *
 * Position p of request r is row p % page of page table[r * max_pages + p / page].
 * After a tree is verified, its accepted tokens are appended again, in order,
 * with lens unchanged; then lens grows.
 *
 * table, lens and begin are device memory.  What the host cannot check (a page
 * outside [0, pages), begin not ascending within 0..T, a negative length, a
 * position past max_pages * page) is skipped, as a key that nobody sees or a
 * row that is not written, and recorded in the workspace error word. */
#define ASF_MAX_KV_HEADS 1024
#define ASF_MAX_HEAD_GROUP 128       /* query heads of a kv head */
#define ASF_MAX_KEYS (1 << 30)       /* most of max_pages * page */

typedef struct {
  int32_t pages, page;               /* pages, and tokens in each */
  int32_t heads, head_dim;           /* kv heads; head_dim a multiple of 8, at most 128 */
  void *k, *v;                       /* device fp16, 16-byte aligned, one layout for both */
  /* elements, multiples of 8; token_stride, and the others where there are
   * several pages or heads, at least head_dim */
  int64_t page_stride, token_stride, head_stride;
} asf_kv_cache;

/* Workspace bytes of asf_tree_attention for up to R requests and T tokens with
 * q_heads query heads.  0 on invalid arguments. */
ASF_API size_t asf_attention_workspace_bytes(const asf_kv_cache *cache, int32_t q_heads, int32_t R, int32_t T);

/* Writes the tokens' keys and values (device fp16 [T][heads][head_dim], 16-byte
 * aligned; rows of the cache only where the call does not write) at their positions.  ws: at least 4096 bytes, for the error word. */
ASF_API asf_status asf_kv_append(const asf_kv_cache *cache, const int32_t *table, int32_t max_pages, int32_t R,
                                 const int32_t *lens, const int32_t *begin, int32_t T, const void *k, const void *v,
                                 void *ws, size_t ws_bytes, asf_stream_t stream);

/* o[t][h] = sum over the keys p that t sees of softmax_p(scale q[t][h] . k_p) v_p,
 * query head h reading kv head h / (q_heads / heads).
 *   q, o  device fp16 [T][q_heads][head_dim], 16-byte aligned, without overlap
 *   anc   device 32-bit masks [T] */
ASF_API asf_status asf_tree_attention(const asf_kv_cache *cache, const int32_t *table, int32_t max_pages, int32_t R,
                                      const int32_t *lens, const int32_t *begin, int32_t T, int32_t q_heads,
                                      const void *q, const int32_t *anc, float scale, void *o, void *ws,
                                      size_t ws_bytes, asf_stream_t stream);

/* asf_tree_attention, and for each key the attention weight that it received:
 * scores (device fp32 [R][heads][S], request by request, by position) gains, for every
 * key before lens[r], the sum over request r's tokens and the kv head's query heads of
 * softmax_p; the positions of the call's own tokens are set to their sums, whatever
 * was there.  Every token of the call counts, and nothing takes its weight off again:
 * the call is for tokens that stay.  Drafts are attended with asf_tree_attention; once
 * their tree is verified, the accepted tokens, appended again, go through this call by
 * themselves, lens as it was and each seeing those before it and itself, which leaves
 * the scores of decoding them one by one and nothing of the other drafts.  Positions
 * from lens[r] + the request's tokens on, and requests without tokens, stay as they
 * are.  S has to cover the positions seen: those from S on are skipped and flagged.
 * scores is apart from q and o.  o is asf_tree_attention's, bit for bit.
 * The workspace may hold every row's scores, 4 bytes for each token, query head and
 * position that the table has room for, up to 512 MB; it is needed during the call
 * alone, so that calls one after the other share it. */
ASF_API size_t asf_attention_scored_workspace_bytes(const asf_kv_cache *cache, int32_t q_heads, int32_t R, int32_t T,
                                                    int32_t max_pages);
ASF_API asf_status asf_tree_attention_scored(const asf_kv_cache *cache, const int32_t *table, int32_t max_pages, int32_t R,
                                             const int32_t *lens, const int32_t *begin, int32_t T, int32_t q_heads,
                                             const void *q, const int32_t *anc, float scale, void *o, float *scores,
                                             int32_t S, void *ws, size_t ws_bytes, asf_stream_t stream);

/* ---------------------------------------------------------------------------
 * Eviction: requests whose caches have grown too long keep `keep` of their keys, the
 * same number for each kv head, but each head its own: the first `first` and the last
 * `recent` positions, and of those between the ones with the largest scores (as
 * asf_tree_attention_scored adds them up; equal scores: the lower position; NaN is
 * below everything).  A request of at most `keep` keys keeps all.  What stays keeps its
 * order, and moves to the pages of table_out, from its position 0 on:
 *   lens_out    device int32 [R]: min(lens[r], keep)
 *   kept        device int32 [R][heads][keep]: the old positions, ascending
 *   scores_out  device fp32 [R][heads][S_out], S_out >= keep: their scores
 * and of the cache the rows of table_out's pages; past lens_out[r] everything stays
 * as it is, and so do table's pages, which may be shared with other requests and are
 * the caller's to reuse once the call has run.  Pages of table_out are pages of no
 * table, and listed once.  first + recent <= keep.  scores as there ([R][heads][S]).
 * Rows are moved with their bits: turned keys stay turned by their first positions, so
 * new tokens' positions (asf_rotary_append's pos) go on from the old length.
 *
 * Bad pages, lengths below 0 or past S or the table, and kept keys past table_out
 * are skipped, clamped and flagged as for asf_tree_attention.  ws: at least 4096
 * bytes, for the error word.  Outputs are apart from inputs and from one another, from
 * the cache as asf_rotary_append's. */
ASF_API asf_status asf_kv_evict(const asf_kv_cache *cache, const int32_t *table, int32_t max_pages, int32_t R,
                                const int32_t *lens, const float *scores, int32_t S, int32_t keep, int32_t first,
                                int32_t recent, const int32_t *table_out, int32_t max_pages_out, int32_t *lens_out,
                                float *scores_out, int32_t S_out, int32_t *kept, void *ws, size_t ws_bytes,
                                asf_stream_t stream);

/* ---------------------------------------------------------------------------
 * Rotary positions: queries and keys are turned before they meet in tree
 * attention.  Of a head's head_dim columns the first rot_dim are turned in pairs,
 * the others pass bit for bit: pair j of a token at position p, (u, w), becomes
 * scale (u cos a - w sin a, w cos a + u sin a) with a = p f_j, where pair j is
 * columns j and j + rot_dim / 2 (ASF_ROTARY_HALF) or 2j and 2j + 1
 * (ASF_ROTARY_PAIRS).  Computed in fp32 and rounded once; the angle, modulo a
 * turn, in whole numbers, so that it is as exact at position 2^31 as at 1.
 * Positions are any int32 values; -p turns back what p has turned. */
#define ASF_MAX_ROTARY_DIM 512
#define ASF_MAX_ROTARY_HEADS 65535
#define ASF_ROTARY_HALF 0
#define ASF_ROTARY_PAIRS 1

typedef struct {
  int32_t head_dim, rot_dim;   /* rot_dim even, at most head_dim */
  int32_t layout;              /* ASF_ROTARY_HALF or ASF_ROTARY_PAIRS */
  float scale;                 /* of cos and sin: 1, or what asf_rotary_frequencies says */
  const uint64_t *turns;       /* device [rot_dim / 2], 8-byte aligned: f_j in 2^-64 turns, see asf_rotary_turns */
} asf_rotary;

/* Host: the usual frequencies, radians per position, and the scale that goes with
 * them.  f_j = base^(-2j / rot_dim), and for contexts `factor` (>= 1) times as long
 *   ASF_ROTARY_LINEAR  f_j / factor
 *   ASF_ROTARY_NTK     of the base base * factor^(rot_dim / (rot_dim - 2)), as
 *                      which the slowest pair is LINEAR's and the fastest PLAIN's
 *   ASF_ROTARY_YARN    "YaRN: Efficient Context Window Extension of Large Language
 *                      Models": f_j (1 - m_j) + m_j f_j / factor, m_j rising from 0
 *                      to 1 between the (rounded) pairs that make 32 turns and one
 *                      turn in the `original` context; scale 1 + 0.1 ln(factor)
 * freq_out: host double [rot_dim / 2].  factor and original are read by the
 * scalings that name them. */
#define ASF_ROTARY_PLAIN 0
#define ASF_ROTARY_LINEAR 1
#define ASF_ROTARY_NTK 2
#define ASF_ROTARY_YARN 3
ASF_API asf_status asf_rotary_frequencies(int32_t rot_dim, double base, int32_t scaling, double factor, double original,
                                          double *freq_out, float *scale_out);

/* Host: freq [n] (radians per position, below 2^100 in size) as turns modulo 1, in
 * units of 2^-64, rounded to the nearest. */
ASF_API asf_status asf_rotary_turns(const double *freq, int32_t n, uint64_t *turns_out);

/* y = x turned, [T][heads][head_dim] each in dtype, T any positive number: token t's
 * head h starts t * token_stride + h * head_stride elements from x or y.
 *   x, y    16-byte aligned, strides not negative and multiples of 16 bytes, head_dim
 *           too; y's heads do not meet.  y is x (same strides), or apart from it
 *           from first to last byte
 *   pos     device int32 [T] */
ASF_API asf_status asf_rotary_apply(const asf_rotary *rot, const void *x, asf_dtype dtype, int32_t T, int32_t heads,
                                    int64_t x_token_stride, int64_t x_head_stride, const int32_t *pos, void *y,
                                    int64_t y_token_stride, int64_t y_head_stride, asf_stream_t stream);

/* asf_kv_append with the turn in front of it, in one launch: the tokens' keys go to
 * the cache turned, their values as they are, and q_out [T][q_heads][head_dim]
 * (contiguous) becomes q turned.  q, k and v are fp16, their heads contiguous, their
 * tokens q_stride, k_stride and v_stride elements apart (multiples of 8, at least a
 * token's width): slices of one joint projection.  Tokens outside every range take no
 * part.  q_out may be q where q is contiguous, else it is apart from q, k and v; and from
 * the cache, from the first to the last byte of its keys and of its values.
 *   pos    device int32 [T], the tokens' positions: not lens[r] + i where tokens of a
 *          tree are alternatives, or where keys have been evicted
 * Everything else, and errors, as for asf_kv_append. */
ASF_API asf_status asf_rotary_append(const asf_rotary *rot, const asf_kv_cache *cache, const int32_t *table,
                                     int32_t max_pages, int32_t R, const int32_t *lens, const int32_t *begin, int32_t T,
                                     const int32_t *pos, int32_t q_heads, const void *q, int64_t q_stride, void *q_out,
                                     const void *k, int64_t k_stride, const void *v, int64_t v_stride, void *ws,
                                     size_t ws_bytes, asf_stream_t stream);

/* ---------------------------------------------------------------------------
 * Neuron-sharded layer across GPUs (the layer + neuron partitioning of the
 * "PowerInfer_x64" page's multi-GPU coordination): rank r holds the predictor
 * rows and FFN rows of its own neurons, and the ranks' partial outputs are
 * summed.  Here the sum is part of the layer's last kernel: each rank reduces
 * its own per-CTA partials, publishes the result in its own buffer, and reads
 * the other ranks' published results directly over peer memory (NVLink /
 * NVSwitch), adding all ranks in rank order -- so every rank gets the same y,
 * bit for bit, with no separate collective launch.
 *
 * Every pointer below is a device pointer valid on the calling rank's GPU:
 * its own buffers, and the other ranks' buffers mapped into this process
 * (CUDA IPC handles opened with peer access).  The buffers are owned by the
 * caller and reused by every call; a rank must make the same sequence of
 * calls (same B each time) as every other rank of the group.
 */
#define ASF_MAX_PEERS 8
typedef struct {
  int32_t world;                   /* ranks in the group, 1..ASF_MAX_PEERS */
  int32_t rank;                    /* this rank (0 when one process emulates all ranks) */
  int32_t max_batch;               /* B the buffers were sized for, <= ASF_MAX_BATCH */
  int32_t d;                       /* hidden size */
  float *pub[ASF_MAX_PEERS];       /* rank r's publication buffer: 2 * max_batch * d fp32 */
  uint32_t *flag[ASF_MAX_PEERS];   /* rank r's flag words: ceil(d/32) * max_batch uint32 */
  uint32_t *epoch;                 /* this rank's call counters: ceil(d/32) * max_batch uint32
                                      (times world when one process emulates all ranks);
                                      zero them, and every flag word, once before the first call */
} asf_peer_group;

/* One layer of a neuron-sharded model on this rank: as asf_predict_sparse_ffn
 * over this rank's predictor and FFN rows (idx and count are local storage
 * indices), except that y receives the sum over all ranks of their partial
 * outputs, exchanged through grp.  A peer that does not publish within 200 ms
 * makes the call record ASF_ERR_TIMEOUT in the workspace error word; its share
 * is then missing from y. */
ASF_API asf_status asf_predict_sparse_ffn_exchange(const asf_predictor *pred, const asf_ffn *ffn, const void *x,
                                                   int32_t B, float tau, int32_t *idx, int32_t *count, float *y,
                                                   void *ws, size_t ws_bytes, const asf_peer_group *grp,
                                                   asf_stream_t stream);

/* The exchange on its own: y = sum over ranks r (in rank order) of the sum
 * over g < G (in order) of rank r's part[g][B][d] (fp32).  With
 * local_ranks == 1 the call is this rank's part of the exchange; with
 * local_ranks == grp->world one process holds every rank's partials (rank r
 * at part + r * part_rank_stride, its y at y + r * y_rank_stride, its
 * counters at grp->epoch + r * ceil(d/32) * max_batch) and runs all ranks in
 * one cooperative launch on its GPU (testing the exchange without several
 * GPUs; ASF_ERR_UNSUPPORTED if the ranks' blocks cannot all be resident).
 * 1 <= G <= 256.  ws: a workspace (at least 4096 bytes) for the error word. */
ASF_API asf_status asf_reduce_exchange(const float *part, int64_t part_rank_stride, int32_t G, int32_t B, int32_t d,
                                       const asf_peer_group *grp, int32_t local_ranks, float *y,
                                       int64_t y_rank_stride, void *ws, size_t ws_bytes, asf_stream_t stream);

/* Test hook for the failure path of the bounded device waits (no counterpart
 * in the pages).  Process-wide; read when a call enqueues its kernels.
 *   ASF_INJECT_NONE                 normal operation (the default)
 *   ASF_INJECT_WITHHOLD_FFN_COPIES  in the one-kernel sparse FFN (B <= 4),
 *       CTA 0's producer issues none of its row copies, so that CTA's bounded
 *       wait for its first row runs out (after 200 ms): the kernel records
 *       ASF_ERR_TIMEOUT in the workspace error word, skips that CTA's rows and
 *       returns.  y is then incomplete.  No memory is touched out of bounds,
 *       nothing hangs and the CUDA context stays usable; the next call on the
 *       same workspace (after asf_read_error) runs normally.
 * Returns ASF_ERR_INVALID_ARG for any other mode. */
#define ASF_INJECT_NONE 0
#define ASF_INJECT_WITHHOLD_FFN_COPIES 1
ASF_API asf_status asf_set_fault_injection(int32_t mode);

/* Wait for the stream, then return (in *host_out) and clear the device error
 * word: 0, or the asf_status of the first device-side fault recorded. */
ASF_API asf_status asf_read_error(void *ws, int32_t *host_out, asf_stream_t stream);

/* Static description of a status code. */
ASF_API const char *asf_status_string(asf_status s);

/* ABI version: major * 100 + minor (1.02: asf_ffn.hot_rows, asf_ffn.row_stride, asf_gather_rows;
 * 1.03: asf_ffn.l2_next; 1.04: asf_predict_sparse_ffn; 1.05: asf_sparse_ffn_noalloc;
 * 1.06: asf_predict_sparse_ffn_begin / _end, asf_set_fault_injection, asf_peer_group,
 * asf_predict_sparse_ffn_exchange, asf_reduce_exchange). */
ASF_API int32_t asf_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ASFFN_H */
