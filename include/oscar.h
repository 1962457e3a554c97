/*
 * oscar.h - C ABI of the OSCAR two-bit rotated KV-cache decode path for GB300
 * (sm_103a).
 *
 * Method (three web pages about one paper, cited by title and section):
 *   [GIST]  gist.science, "OSCAR: Offline Spectral Covariance-Aware Rotation
 *           for 2-bit KV Cache Quantization", Technical summary 2.1, 2.2 A
 *           (offline calibration), 2.2 B (online serving).
 *   [ZAKER] myzaker.com OSCAR article, parts "OSCAR 把旋转对准 attention"
 *           (rotation) and "从离线校准到在线推理的 pipeline" (token pool,
 *           demotion kernel, INT2 decode, online-softmax merge).
 *
 * Conventions shared by every call:
 *   - Row vectors: a rotated key is k~ = k . R with R = U . H_Had . P_br.
 *   - head_dim d = 128, 16 tokens per page; a (token, KV head, K|V) vector
 *     of 128 rotated channels is quantised in groups of g consecutive
 *     channels (g = 128 by default; 64 or 32 per layer, for K and V apart,
 *     see quant_group_k / quant_group_v), each with an fp16 scale and zero.
 *     Smaller groups are where the bit-reversal P_br of R matters: it
 *     interleaves high- and low-variance channels across the groups
 *     ([GIST] 2.2 A; [ZAKER] "OSCAR 把旋转对准 attention").
 *   - bfloat16 data is passed as uint16_t bit patterns.
 *   - All device memory is allocated and freed by the caller.  The library
 *     keeps no state besides cached device attributes; calls on different
 *     streams may run concurrently when they touch disjoint memory.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Device
 *     calls are asynchronous; every argument is validated on the host before
 *     any launch, and a rejected call launches nothing.
 *   - Device-side faults the host cannot see in advance (page ids outside the
 *     pool, lengths above their capacity, an expired bounded wait) never trap:
 *     the kernel skips the offending access and ORs a bit into the optional
 *     device status word `dev_status` (see OSCAR_DEV_*).
 *   - No C++ exception crosses this boundary.
 *
 * Page pool layout (this library's format; the pages fix only "paged KV",
 * "4 codes per byte" and "scale/zero point"), with G_K = 128 / g_K and
 * G_V = 128 / g_V groups per vector.  A block of one (page p, KV head h)
 * has 1024 + 64 (G_K + G_V) bytes (1152 with one group each,
 * OSCAR_BLOCK_BYTES) and sits at byte (p * n_kv_heads + h) * block:
 *   [0, 512)     K code rows: token slot t, code byte l at 32 t + l;
 *   [512, 1024)  V code rows, the two tokens of a slot pair interleaved by
 *                16-bit halves: token slot t, code byte l at
 *                512 + 64 (t / 2) + 4 (l / 2) + 2 (t % 2) + (l % 2);
 *   [1024, ...)  token slot t: its G_K K (scale, zero) fp16 pairs, then its
 *                G_V V pairs, at 1024 + 4 (G_K + G_V) t.
 *   Code byte l of a token row holds code positions 4l .. 4l+3 (bits
 *   2 (c % 4)); position c holds rotated channel c when G = 1.  When G > 1
 *   it holds channel
 *     K: c = 32 t + 8 e + j (t, e < 4, j < 8):  (j / J) g + (j % J) 16 + 4 t + e,
 *     V: c = 16 a + 8 e + m (a < 8, e < 2, m < 8): (m / M) g + (m % M) 16 + 2 a + e,
 *   with J = M = 8 / G, so that each tensor-core operand tile of the decode
 *   kernel draws on one group.  Group q is rotated channels [q g, (q+1) g).
 *   Logical history position x of request b lives in page
 *   page_table[b][x / 16], slot x % 16.
 */
#ifndef OSCAR_H_
#define OSCAR_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define OSCAR_ABI_VERSION 4

#define OSCAR_HEAD_DIM 128
#define OSCAR_PAGE_TOKENS 16
#define OSCAR_BLOCK_BYTES 1152

typedef int32_t oscar_status;
enum {
  OSCAR_OK = 0,
  OSCAR_ERR_INVALID_ARG = 1,     /* null pointer, bad dimension or length     */
  OSCAR_ERR_ALIGNMENT = 2,       /* a pointer misses its required alignment  */
  OSCAR_ERR_WORKSPACE = 3,       /* workspace missing or too small            */
  OSCAR_ERR_CUDA = 4,            /* a CUDA runtime call or launch failed      */
  OSCAR_ERR_NO_CONVERGENCE = 5,  /* the host eigensolver did not converge     */
  OSCAR_ERR_UNSUPPORTED = 6,     /* a valid but unimplemented configuration   */
  OSCAR_ERR_FILE = 7             /* a file missing, unreadable, truncated or   */
                                 /* failing its format or checksum check       */
};

/* Bits a kernel ORs into *dev_status (never cleared by the library). */
#define OSCAR_DEV_PAGE_BOUNDS 0x1   /* a page id outside [0, n_pages): skipped  */
#define OSCAR_DEV_LENGTH 0x2        /* a length above its capacity: clamped     */
#define OSCAR_DEV_TIMEOUT 0x4       /* a bounded wait expired: work abandoned   */

/* Human-readable name of a status code (static string, never NULL). */
const char* oscar_status_string(oscar_status s);

/* OSCAR_ABI_VERSION of the loaded library. */
int32_t oscar_abi_version(void);

/*
 * oscar_set_page_wait_limit - the decode kernel's time budget for a warp's
 * scan of its INT2 pages, which also bounds each wait for a page copy to
 * land.  A warp past it gives up the rest of its pages, sets
 * OSCAR_DEV_TIMEOUT in dev_status, and the call's output must not be used.
 * limit_ns <= 0 restores the default (1 s, far beyond any scan).  Returns
 * the previous limit.  Copies already issued are still waited for (up to
 * 1 s each) before a CTA exits, and the workspace stays ready for the next
 * call.  A stalled copy is the only way this path runs in normal use; a
 * short limit makes it run on purpose (tests of the failure path).
 * Process-wide, read when a decode call is issued.  Host-only.
 */
int64_t oscar_set_page_wait_limit(int64_t limit_ns);

/*
 * One attention layer's cache: a three-segment token pool, BF16 sink (64
 * tokens) | INT2 history (paged) | BF16 recent window (256-slot ring).
 * [ZAKER] pipeline part; [GIST] 2.2 B (hybrid-precision paged layout).
 * Pointers are device pointers unless marked host.  The struct itself is
 * read on the host during the call only; it may be reused or freed after.
 */
typedef struct oscar_layer_desc {
  int32_t batch;              /* B >= 1                                        */
  int32_t n_q_heads;          /* H_q, a multiple of n_kv_heads                */
  int32_t n_kv_heads;         /* H_kv >= 1; GQA group g = H_q / H_kv in {4, 8} */
  int32_t head_dim;           /* must be 128                                   */
  int32_t sink_cap;           /* sink capacity in tokens (64 on the pages)     */
  int32_t recent_cap;         /* recent ring capacity (256 on the pages)       */
  int32_t max_pages_per_seq;  /* row length of page_table                      */
  int32_t max_hist;           /* host upper bound on every hist_len[b]         */
  int64_t n_pages;            /* physical pages in the pool                    */
  float tau_k;                /* clip threshold of this layer's keys, > 0      */
  float tau_v;                /* clip threshold of this layer's values, > 0    */
  uint8_t* pages;             /* pool, 128-byte aligned (layout above)         */
  const int32_t* page_table;  /* [B][max_pages_per_seq] physical page ids      */
  const int32_t* hist_len;    /* [B] INT2 history length of each request       */
  const uint16_t* sink_k;     /* [B][sink_cap][H_kv][d] bf16, 16-byte aligned  */
  const uint16_t* sink_v;     /* same layout                                   */
  const int32_t* sink_len;    /* [B] valid sink tokens (slots 0..len-1)        */
  uint16_t* recent_k;         /* [B][recent_cap][H_kv][d] bf16 ring            */
  uint16_t* recent_v;         /* same layout                                   */
  const int32_t* recent_len;  /* [B] valid recent tokens                       */
  const int32_t* recent_start;/* [B] ring slot of the oldest recent token      */
  const float* r_k;           /* [H_kv][d][d] row-major R_K, k~ = k . R_K      */
  const float* r_v;           /* [H_kv][d][d] row-major R_V                    */
  int32_t* dev_status;        /* optional device word for OSCAR_DEV_* bits     */
  int32_t quant_group_k;      /* K quantisation group g_K: 32, 64 or 128 (0 = 128) */
  int32_t quant_group_v;      /* V quantisation group g_V: 32, 64 or 128 (0 = 128) */
  int32_t codebook;           /* 0: uniform levels 0..3; 1: levels_k / levels_v  */
  float levels_k[4];          /* codebook 1: K levels l_0 < .. < l_3 (fp16 values) */
  float levels_v[4];          /* codebook 1: V levels                          */
} oscar_layer_desc;

/*
 * Codebook levels (desc->levels_k / levels_v, used when desc->codebook = 1):
 * four fp16 values 0 <= l_0 < l_1 < l_2 < l_3 <= 3 in the normalised domain
 * u = (x - zero) / scale, where the group's (scale, zero) are those of the
 * uniform codec; a value dequantises to zero + scale * l[code].  Levels that
 * are not fp16 values, not increasing or outside [0, 3] are rejected with
 * OSCAR_ERR_INVALID_ARG.  Levels 0, 1, 2, 3 give the uniform codes except
 * at exact ties u = 1.5 (lower level here, round-half-even there).
 */

/* Bytes of one (page, KV head) block for groups g_k, g_v (0 = 128); 0 for
 * any other value.  Host-only. */
int64_t oscar_block_bytes(int32_t quant_group_k, int32_t quant_group_v);

/*
 * oscar_build_rotation - the fixed rotation of one (layer, KV head) from
 * calibration rows.  [GIST] 2.1 and 2.2 A; [ZAKER] "OSCAR 把旋转对准 attention".
 *
 *   C = x^T x / n over the n rows of x (host, row-major [n][d], float64):
 *   post-RoPE queries of the KV head's query group for R_K (C_Q), or rows of
 *   S.V (see oscar_score_weighted_rows) for R_V (C_S).  U = eigenvectors of C
 *   by descending eigenvalue, each column's largest-|entry| made positive
 *   (ties: lowest index).  r_out = U . H . P_br with the orthonormal Sylvester
 *   Hadamard H and the bit-reversal permutation P_br.
 *
 *   d must be a power of two in [2, 1024]; n >= 1.  r_out (host, [d][d]
 *   row-major) is written; eigvals_out (host, [d], nullable) receives the
 *   eigenvalues in the same order.  Host-only, synchronous, thread-safe.
 *   Returns OSCAR_ERR_NO_CONVERGENCE if the eigensolver does not converge.
 */
oscar_status oscar_build_rotation(const double* x, int64_t n, int32_t d,
                                  double* r_out, double* eigvals_out);

/*
 * oscar_build_canalized_rotation - the block-diagonal rotation of the OScaR
 * variant.  [CSDN] section 四.2 (channels split into groups, each rotated
 * within the group; no inversion, no iteration).
 *
 *   r_out (host, [d][d] row-major, float64) = I_(d/block) (x) H_block, with
 *   H_block the orthonormal Sylvester Hadamard of size block.  The variant's
 *   per-token scaling is carried by the per-token (scale, zero) of this
 *   codec, so the rotation is the whole difference; the demotion and decode
 *   calls take it like any R.  d and block powers of two, 1 <= block <= d
 *   <= 1024.  Host-only, synchronous, thread-safe.
 */
oscar_status oscar_build_canalized_rotation(int32_t d, int32_t block, double* r_out);

/*
 * oscar_build_rotation_from_covariance - as oscar_build_rotation, from a
 * covariance computed elsewhere (for instance by oscar_covariance on the
 * device): c (host, [d][d] row-major, float64) is symmetrised as
 * (c + c^T) / 2 and decomposed; r_out = U . H . P_br, eigvals_out (nullable)
 * as in oscar_build_rotation.  OSCAR_ERR_INVALID_ARG for non-finite entries.
 * Host-only, synchronous, thread-safe.
 */
oscar_status oscar_build_rotation_from_covariance(const double* c, int32_t d, double* r_out,
                                                  double* eigvals_out);

/*
 * oscar_covariance - calibration covariance on the device.  [GIST] 2.1 and
 * 2.2 A (C_Q = Q^T Q over calibration queries for R_K, C_S = (S V)^T (S V)
 * for R_V, both divided by the number of rows).
 *
 *   c_out (device, [d][d] row-major, fp32) = X^T X / n over the n rows of x
 *   (device, bf16, row r at x + r * ld, d = 128 values each).  Products of
 *   bf16 values are exact in fp32; sums are fp32 over at most 2048 rows,
 *   then over those partials in a fixed order (the result does not depend
 *   on scheduling).  If workspace is NULL the required size is written to
 *   *workspace_bytes and nothing runs; otherwise the call is asynchronous on
 *   `stream`.  x 16-byte aligned, ld a multiple of 8, c_out 16-byte and the
 *   workspace 256-byte aligned (OSCAR_ERR_ALIGNMENT); d must be 128.
 */
oscar_status oscar_covariance(const uint16_t* x, int64_t n, int32_t d, int64_t ld, float* c_out,
                              void* workspace, size_t* workspace_bytes, void* stream);

/*
 * oscar_value_covariance - the score-weighted value covariance on the
 * device.  [GIST] 2.1 and 2.2 A (C_S = (1/N) V^T S^T S V, S = row-softmax of
 * the calibration scores).
 *
 *   c_out (device, [d][d] row-major, fp32) = (S V)^T (S V) / n_q with
 *   S = row-softmax(q k^T / sqrt(d)), over device bf16 rows q [n_q], k and
 *   v [n_k] (row r at base + r * ld, d = 128 values each).  The rows of S V
 *   are formed in fp32 (exact bf16 products in Q K^T, an fp32 softmax, P
 *   split into two bf16 parts against the bf16 values), then their
 *   covariance as fp32 partials of 256 rows added in a fixed order.  If
 *   workspace is NULL the required size is written to *workspace_bytes and
 *   nothing runs; otherwise asynchronous on `stream`.  q, k, v 16-byte
 *   aligned, ld a multiple of 8, c_out 16-byte and workspace 256-byte
 *   aligned (OSCAR_ERR_ALIGNMENT); n_q, n_k >= 1 and d = 128.
 */
oscar_status oscar_value_covariance(const uint16_t* q, int64_t n_q, const uint16_t* k, const uint16_t* v,
                                    int64_t n_k, int32_t d, int64_t ld, float* c_out, void* workspace,
                                    size_t* workspace_bytes, void* stream);

/*
 * oscar_score_weighted_rows - rows of S.V for the value covariance
 * C_S = (1/N) V^T S^T S V.  [GIST] 2.1 and 2.2 A.
 *
 *   S = row-softmax(q k^T * scale) with q [n_q][d], k and v [n_k][d] (host,
 *   row-major, float64); out [n_q][d] = S . v.  scale is normally 1/sqrt(d).
 *   Host-only, synchronous.
 */
oscar_status oscar_score_weighted_rows(const double* q, int64_t n_q, const double* k,
                                       const double* v, int64_t n_k, int32_t d,
                                       double scale, double* out);

/*
 * oscar_clip_threshold - per-layer clip threshold from rotated calibration
 * activations.  [GIST] 2.2 A (thresholds estimated from the rotated
 * calibration activations); the estimator is this library's choice:
 *
 *   tau = nearest-rank `quantile` of |acts[h] . r[h]| over every element of
 *   every head h < n_heads (acts [n_heads][rows][d], r [n_heads][d][d], host,
 *   float64).  0 < quantile <= 1.  Writes *tau_out.  Host-only.
 */
oscar_status oscar_clip_threshold(const double* acts, int64_t rows, int32_t n_heads,
                                  int32_t d, const double* r, double quantile,
                                  double* tau_out);

/*
 * oscar_fit_codebook - the Lloyd-Max codebook of one layer's K or V from
 * calibration rows.  [ZAKER] "OSCAR 把旋转对准 attention", closing part (the
 * code repo combines the rotation with a Lloyd-Max codebook); the fit is this
 * library's reading:
 *
 *   For every row of x [n][d] (host float64, d = 128) and its head's
 *   rotation r [d][d]: x~ = clamp(x . r, -tau, tau); scale = fp16((max -
 *   min) / 3), zero = fp16(min) (round to nearest even); rows with scale 0
 *   are skipped; u = (x~ - zero) / scale for each channel.  Lloyd's iteration
 *   over all u from levels {0, 1, 2, 3}: thresholds at the midpoints of
 *   adjacent levels, each level the mean of the u in its cell (u <= t_1, t_1
 *   < u <= t_2, ...; an empty cell keeps its level), at most `iters` rounds
 *   or until no level moves.  levels_out[4] = the levels clamped to [0, 3]
 *   and rounded to fp16 (as float).  OSCAR_ERR_INVALID_ARG for bad sizes, tau <= 0, iters < 1, no
 *   usable row, or fitted levels that are not strictly increasing in fp16.
 *   Host-only, synchronous.
 */
oscar_status oscar_fit_codebook(const double* x, int64_t n, int32_t d, const double* r, double tau,
                                int32_t iters, float* levels_out);

/*
 * Rotation files: a model's fixed rotations and clip thresholds, computed
 * once offline, stored for serving start-up.  [ZAKER] closing part (the
 * release ships a zoo of precomputed per-layer rotations); [GIST] 2.2 A
 * (R and the thresholds are fixed per layer after calibration).
 *
 *   Layout (little-endian): "OSCARROT", u32 version 1, u32 n_layers, u32
 *   n_kv_heads, u32 d; per layer f32 tau_k, f32 tau_v, R_K [n_kv][d][d] f32,
 *   R_V [n_kv][d][d] f32; then the 64-bit FNV-1a hash of all bytes before it.
 *   r_k / r_v (host) are [n_layers][n_kv][d][d] row-major, tau_k / tau_v
 *   (host) [n_layers].  write creates or replaces the file; info reads the
 *   dimensions; read checks the magic, version, dimensions (the caller's
 *   must equal the file's, else OSCAR_ERR_INVALID_ARG), size and hash before
 *   it writes any output.  OSCAR_ERR_FILE for an unreadable, truncated or
 *   damaged file.  Host-only, synchronous.
 */
oscar_status oscar_rotation_file_write(const char* path, int32_t n_layers, int32_t n_kv_heads, int32_t d,
                                       const float* r_k, const float* r_v, const float* tau_k,
                                       const float* tau_v);
oscar_status oscar_rotation_file_info(const char* path, int32_t* n_layers, int32_t* n_kv_heads, int32_t* d);
oscar_status oscar_rotation_file_read(const char* path, int32_t n_layers, int32_t n_kv_heads, int32_t d,
                                      float* r_k, float* r_v, float* tau_k, float* tau_v);

/*
 * oscar_quantize_append - the fused demotion kernel: rotate, clip, quantise
 * and pack tokens into INT2 history pages.  [ZAKER] pipeline part (the
 * oldest recent token is rotated, clipped, quantised and packed into INT2
 * history; 4 codes per byte; scale/zero point); [GIST] 2.2 B.
 *
 *   For item i < n and every KV head h: x = src row src_index[i] (identity if
 *   src_index is NULL) of k_src / v_src, viewed as [src_rows][row_stride]
 *   bf16 with head h at elements h*d .. h*d+d-1.  A source row outside
 *   [0, src_rows), a request outside the batch or a position beyond the page
 *   table skips the item and sets OSCAR_DEV_LENGTH; a page id outside the
 *   pool skips it and sets OSCAR_DEV_PAGE_BOUNDS.  x~ = x . R[h] (fp32 accumulate),
 *   clamped to [-tau, tau]; per group of g consecutive channels (g =
 *   quant_group_k for K, quant_group_v for V) scale = fp16((max - min) / 3),
 *   zero = fp16(min) over the group; code = clamp(rint((x~ - zero) / scale),
 *   0, 3) (0 if scale is 0).  With desc->codebook == 1 (Lloyd-Max levels;
 *   one group per vector only, else OSCAR_ERR_UNSUPPORTED) the code is
 *   instead the number of thresholds (l_(k-1) + l_k) / 2 of levels_k / levels_v
 *   strictly below u = (x~ - zero) / scale (the nearest level, ties to the
 *   lower), 0 if scale is 0.  The codes and (scale, zero) pairs go to history
 *   position dst_pos[i] of request dst_req[i] through desc->page_table, in the
 *   pool layout above.  K and V are both written.
 *
 *   Any finite bf16 row is accepted at any magnitude: calls of n >= 1024
 *   items (the tensor-core path) multiply the bf16 rows as they are by R
 *   held as three bf16 parts (about 24 significant bits), with exact
 *   products and fp32 sums, like the per-token path's fp32 arithmetic.
 *   Rows holding an infinity or a NaN give unspecified codes.
 *
 *   new_k / new_v (nullable, both or neither): [n][H_kv][d] bf16 rows that
 *   replace the demoted source rows after they have been read - the decode
 *   step's "write the new token into the freed ring slot".  k_src / v_src
 *   are written only then.
 *
 *   src_index, dst_req, dst_pos: device int32 [n].  k_src, v_src, new_k,
 *   new_v: 16-byte aligned; row_stride a multiple of 8 and >= H_kv * d.
 *   The caller owns lengths and page allocation: writing into a page that
 *   another request also references is a caller error.  Items must name
 *   distinct (request, position) pairs.  n = 0 is a no-op.  Async.
 */
oscar_status oscar_quantize_append(const oscar_layer_desc* desc,
                                   uint16_t* k_src, uint16_t* v_src,
                                   int64_t src_rows, int64_t row_stride,
                                   const int32_t* src_index,
                                   const int32_t* dst_req, const int32_t* dst_pos,
                                   int32_t n, const uint16_t* new_k,
                                   const uint16_t* new_v, void* stream);

/*
 * oscar_quantize_append_overlapped - oscar_quantize_append whose reads and
 * arithmetic run while the kernel before it on `stream` is still running.
 * [ZAKER] pipeline part (demote the oldest recent token, write the new one):
 * the same operation, the same arguments, bit for bit the same results.
 *
 *   The per-token kernel reads the rotations, the index arrays, the page
 *   table and the source rows, rotates and quantises, and only then waits
 *   for the previous kernel on the stream to finish; the code stores and
 *   the new-token writes into k_src / v_src (new_k / new_v are read only
 *   then) follow the wait.  This is for a decode loop in which that previous
 *   kernel is the projection that produces new_k / new_v, or the attention
 *   of the layer before (oscar_decode_attention reads, never writes, the
 *   cache).  Precondition (the caller's): no kernel that may still be
 *   running when this one starts writes desc->r_k / r_v, desc->page_table,
 *   src_index, dst_req, dst_pos or the source rows src_index names; new_k /
 *   new_v and anything else may be written.  Those kernels are the one
 *   issued on `stream` just before this call and, if that one lets its
 *   successor start early, the ones still running at that point.  The other
 *   kernels of this library let a successor start only after their own
 *   wait, so after one of them only that kernel counts.  This kernel lets
 *   its successor start at once (the successor's own wait still covers
 *   everything this kernel and its predecessor write), so for a call after
 *   it that reads before its wait, this call's predecessor counts too.
 *   Calls that take the tensor-core path (n >= 1024,
 *   no new rows) wait first, like oscar_quantize_append.  Argument checks
 *   and error codes are those of oscar_quantize_append.  Async.
 */
oscar_status oscar_quantize_append_overlapped(const oscar_layer_desc* desc,
                                              uint16_t* k_src, uint16_t* v_src,
                                              int64_t src_rows, int64_t row_stride,
                                              const int32_t* src_index,
                                              const int32_t* dst_req, const int32_t* dst_pos,
                                              int32_t n, const uint16_t* new_k,
                                              const uint16_t* new_v, void* stream);

/*
 * oscar_decode_attention - one decode step of attention for every request of
 * the batch over BF16 sink | INT2 history | BF16 recent.  [ZAKER] pipeline
 * part (INT2 kernel: unpack, scale/zero dequantisation, float accumulation;
 * BF16 kernel for sink/recent; online-softmax merge); [GIST] 2.2 B (inverse
 * rotation fused into the kernel with no extra memory traffic); [CSDN] the
 * aicoding.csdn.net explainer, section 三.1 (load INT2, rotate back, attend).
 *
 *   q: [B][H_q][d] bf16 (16-byte aligned); out: [B][H_q][d] float32
 *   (16-byte aligned), normalised softmax(q K^T / sqrt(d)) V over the valid
 *   tokens of all three segments; query head j reads KV head j / g.
 *   History keys/values are c * s + z (codebook 0) or l[c] * s + z
 *   (codebook 1) rotated back with R^T; the kernel
 *   computes this as (q . R_K) against c * s + z and one output rotation
 *   . R_V^T per head, which is the same quantity.  A request with no valid
 *   token gets zeros.
 *
 *   Workspace: call with workspace == NULL to receive the required size in
 *   *workspace_bytes (depends on desc dims and the current device) and
 *   return.  Otherwise workspace must be 256-byte aligned device memory of
 *   at least that size, zero-filled before its first use (cudaMemset); each
 *   call leaves it ready for the next one.  It holds per-call merge tickets
 *   and split partials, so two calls in flight at the same time need two
 *   workspaces.  Async.
 */
oscar_status oscar_decode_attention(const oscar_layer_desc* desc, const uint16_t* q,
                                    float* out, void* workspace, size_t* workspace_bytes,
                                    void* stream);

/*
 * oscar_decode_step - one decode step of a layer in one call, for a serving
 * loop that holds the step's inputs in host memory: [ZAKER] pipeline part
 * (demote the oldest recent token, write the new one, attend).
 *
 *   On `stream`, in this order: (1) if in_bytes > 0, bring in_bytes from
 *   host_in (pinned host memory) to dev_in (device), the staging range that
 *   q, new_k / new_v and the index arrays may point into; (2)
 *   oscar_quantize_append with the given arguments (nothing when n = 0);
 *   (3) oscar_decode_attention(desc, q, out, workspace, workspace_bytes);
 *   (4) if host_out is not NULL, copy out ([B][H_q][d] float32) to host_out
 *   (pinned host memory): when host_out is 16-byte aligned the decode kernel
 *   of step (3) writes it with the same stores as `out`, else a copy kernel
 *   follows.  The results are those of the separate calls.
 *   Step (1) is not a copy when it need not be: if q or an argument of (2)
 *   lies inside [dev_in, dev_in + in_bytes), host_in and dev_in are equal
 *   modulo 16 bytes, the per-token demotion kernel runs (new rows given, or
 *   n < 1024) and k_src / v_src lie outside that range, the kernels of (2)
 *   and (3) read those inputs straight from the same offsets of host_in
 *   and dev_in is left unwritten; otherwise a copy kernel fills dev_in.
 *   The copies run in the same launch chain as kernels: the GPU reads
 *   host_in and writes host_out directly (GB300's coherent CPU-GPU link), so
 *   both must be pinned host memory the device addresses at the same pointer
 *   (cudaHostAlloc / cudaMallocHost on a system with unified addressing);
 *   otherwise OSCAR_ERR_INVALID_ARG.  host_in is read anew on every call.
 *   Every argument of (2) and (3) is validated before (1) is issued: a
 *   rejected call copies and launches nothing.  in_bytes > 0 requires
 *   host_in and dev_in (OSCAR_ERR_INVALID_ARG otherwise); workspace must be
 *   given (OSCAR_ERR_WORKSPACE).  Async: host_in must not change until the
 *   stream has passed step (3), and host_out holds the output once the
 *   stream has passed step (4).
 *
 *   flags: 0, or OSCAR_STEP_OVERLAP_PREVIOUS: when no copy kernel of step
 *   (1) runs, step (2) is oscar_quantize_append_overlapped (its reads and
 *   arithmetic overlap the kernel before the call on `stream`), under that
 *   function's precondition on that kernel, which here covers new_k / new_v
 *   too (they are read before the wait as well); in a loop of
 *   oscar_decode_step calls that kernel is the previous call's decode (or
 *   its output copy), which qualifies as long as host_out and out overlap
 *   none of the inputs.
 *   Other bits: OSCAR_ERR_INVALID_ARG.
 */
#define OSCAR_STEP_OVERLAP_PREVIOUS 1u
oscar_status oscar_decode_step(const oscar_layer_desc* desc, const void* host_in, void* dev_in,
                               size_t in_bytes, uint16_t* k_src, uint16_t* v_src, int64_t src_rows,
                               int64_t row_stride, const int32_t* src_index, const int32_t* dst_req,
                               const int32_t* dst_pos, int32_t n, const uint16_t* new_k,
                               const uint16_t* new_v, const uint16_t* q, float* out,
                               void* workspace, size_t workspace_bytes, float* host_out,
                               uint32_t flags, void* stream);

/*
 * oscar_decode_attention_static - oscar_decode_attention for callers that
 * cannot allocate device memory.  The paper has no counterpart: this is a
 * deployment convenience of this library.
 *
 *   Some callers have no way to call cudaMalloc or to hand the library a
 *   workspace: code embedded in a host framework that owns every device
 *   allocation, or a latency-critical serving loop that forbids allocation
 *   after start-up.  This entry point computes exactly what
 *   oscar_decode_attention computes, but its workspace is a fixed array of
 *   OSCAR_STATIC_WORKSPACE_BYTES inside the library, reserved on every GPU
 *   that loads the library until the process exits.  It allocates nothing.
 *
 *   q, out and the cache are the caller's, as for oscar_decode_attention.
 *   Returns OSCAR_ERR_WORKSPACE when the problem needs more workspace than
 *   the fixed array holds (the size oscar_decode_attention reports for a
 *   NULL workspace must not exceed OSCAR_STATIC_WORKSPACE_BYTES; about 0.65
 *   MB for one 100k-token request with 8 KV heads and GQA 4).
 *
 *   The first call on a device looks up the array's device address
 *   (cudaGetSymbolAddress) with that device current, and so does the first
 *   call after the device's context was replaced (cudaDeviceReset); make
 *   those calls before any stream capture.  Each call clears the part of the array that
 *   must start at zero, on `stream`, then launches.  Every call shares the
 *   one array and it keeps the last call's contents: calls whose work
 *   overlaps on the GPU (different streams, or concurrent host threads
 *   without stream ordering) race on it and must not be issued.
 */
#define OSCAR_STATIC_WORKSPACE_BYTES (8u << 20)

oscar_status oscar_decode_attention_static(const oscar_layer_desc* desc, const uint16_t* q,
                                           float* out, void* stream);

/*
 * ---------------------------------------------------------------- 4-bit layers
 *
 * A layer that two bits do not carry (the first and last layers of a model,
 * a model without calibration data) keeps its whole KV cache at 4 bits: no
 * rotation, no BF16 segments; every token goes to its page when it is
 * appended, position-rotated on the way.  Layers of both kinds may share a
 * model: every call takes one layer.
 *
 * Page pool layout of a 4-bit layer: head_dim d is 64 or 128, W = d / 32,
 * 16 tokens per page, quantisation groups of g channels with G_K = d / g_K
 * and G_V = d / g_V groups per vector.  A block of one (page p, KV head h)
 * has 16 d + 64 (G_K + G_V) bytes (oscar_int4_block_bytes) and sits at byte
 * (p * n_kv_heads + h) * block:
 *   [0, 8 d)      K codes: token slot t has d / 2 bytes at t d / 2, 32-bit
 *                 words; channel 32 w + 8 u + n (u < 4, n < 8) is nibble n
 *                 (0 = lowest 4 bits) of word W u + w;
 *   [8 d, 16 d)   V codes, two token slots to a word: channel 32 w + 4 u + n
 *                 (u < 8, n < 4) of slot t is nibble 4 (t % 2) + n of word
 *                 (8 (t / 2) + u) W + w;
 *   [16 d, ...)   slot t: its G_K K (scale, zero) fp16 pairs, then its G_V V
 *                 pairs, at 16 d + 4 (G_K + G_V) t.
 * A value is zero + scale * code, code 0 .. 15.  (So that 4 bytes of K are 8
 * adjacent channels of one token and 2 bytes of V 4 adjacent channels of
 * one token, and one 16-byte load (d = 128) of a warp's lane holds a
 * tensor-core operand's codes.)
 * Logical position x of request b lives in page page_table[b][x / 16], slot
 * x % 16.
 */
typedef struct oscar_int4_desc {
  int32_t batch;              /* B >= 1                                         */
  int32_t n_q_heads;          /* H_q, a multiple of n_kv_heads                  */
  int32_t n_kv_heads;         /* H_kv >= 1                                      */
  int32_t head_dim;           /* 64 or 128                                      */
  int32_t max_pages_per_seq;  /* row length of page_table                       */
  int32_t max_len;            /* host upper bound on every seq_len[b] (decode)  */
  int64_t n_pages;            /* physical pages in the pool                     */
  float tau_k;                /* keys are clamped to [-tau_k, tau_k]; 0 < tau <= 65504 */
  float tau_v;                /* the same for values                            */
  uint8_t* pages;             /* pool, 128-byte aligned (layout above)          */
  const int32_t* page_table;  /* [B][max_pages_per_seq] physical page ids       */
  const int32_t* seq_len;     /* [B] cached tokens of each request (decode)     */
  int32_t* dev_status;        /* optional device word for OSCAR_DEV_* bits      */
  int32_t quant_group_k;      /* g_K: 32, 64 or 128, at most d; 0 = d           */
  int32_t quant_group_v;      /* g_V                                            */
} oscar_int4_desc;

/* Position rotation: pairs of channels of the first rot_dim channels of a
 * head turn by the angle of the token's position. */
typedef struct oscar_rope_desc {
  const float* cos_sin;       /* device [n_positions][rot_dim] fp32, 16-byte aligned: */
                              /* rot_dim / 2 cosines, then rot_dim / 2 sines    */
  int64_t n_positions;        /* rows of cos_sin                                */
  int32_t rot_dim;            /* a multiple of 16, 0 <= rot_dim <= head_dim;    */
                              /* 0: no rotation (cos_sin may be NULL)           */
  int32_t interleaved;        /* 0: pair i is channels (i, i + rot_dim / 2);    */
                              /* 1: pair i is channels (2 i, 2 i + 1)           */
} oscar_rope_desc;

/* What becomes of a score before the softmax.  For query position i and key
 * position j: t = scale (q . k); softcap > 0: t = softcap tanh(t / softcap);
 * slopes: t -= slopes[h] |i - j|; window > 0: keys with i - j >= window are
 * masked.  Scores may be as large as 2^22 in magnitude; a capped one is as exact as
 * an uncapped one, whatever the cap. */
typedef struct oscar_score_desc {
  float scale;                /* > 0 and finite; 0 = 1 / sqrt(head_dim)         */
  float softcap;              /* > 0 and finite; 0 = none                       */
  int32_t window;             /* >= 1; 0 = none                                 */
  int32_t reserved;           /* 0                                              */
  const float* slopes;        /* device [n_q_heads] fp32 or NULL                */
} oscar_score_desc;

/* Bytes of one (page, KV head) block of a 4-bit layer; 0 for an invalid head
 * size or group.  Host-only. */
int64_t oscar_int4_block_bytes(int32_t head_dim, int32_t quant_group_k, int32_t quant_group_v);

/*
 * oscar_rope_append_int4 - rotates the queries and keys of n tokens by their
 * positions and appends their keys and values to a 4-bit layer's pages.  The
 * sources quantise at two bits only; the codec is theirs (scale / zero per
 * group) with sixteen codes.
 *
 *   For item i < n: q row i (q + i * q_stride, H_q heads of d bf16), k row i
 *   and v row i (H_kv heads each).  q' and k' are q and k rotated by row
 *   rope_pos[i] of rope->cos_sin (rope_pos NULL: dst_pos[i]), rounded to
 *   bf16: (a, b) -> (a cos - b sin, a sin + b cos).  q' goes to q_out and k'
 *   to k_out ([n][heads][d], contiguous; each may be NULL, or q / k itself
 *   where that is contiguous).  k' and v, clamped to [-tau, tau], are
 *   quantised per group: scale = fp16((max - min) / 15), zero = fp16(min),
 *   code = clamp(rint((x - zero) / scale), 0, 15) (0 if scale is 0), and
 *   stored at position dst_pos[i] of request dst_req[i].
 *
 *   k' is its exact value rounded to fp32 and that to bf16 (codes do not depend
 *   on how the rotation is computed); q' is within one rounding of fp32 sums.
 *   A NaN is quantised as -tau; other rows are not affected.
 *   dst_req[i] = -1 marks a padding row: nothing of it is written.
 *   Any other request outside the batch, a position beyond the page table
 *   or a rotation row outside cos_sin skips the item and sets
 *   OSCAR_DEV_LENGTH; a page id outside the pool skips it and sets
 *   OSCAR_DEV_PAGE_BOUNDS.  A skipped item writes nothing.
 *
 *   rope may be NULL (no rotation).  q and q_out may be NULL together.
 *   dst_req, dst_pos, rope_pos: device int32 [n].  Rows 16-byte aligned,
 *   strides multiples of 8 elements and at least one row.  seq_len is not
 *   read: the caller advances it.  Items must name distinct (request,
 *   position) pairs.  Outputs may share memory with inputs only as said
 *   above.  n = 0 is a no-op.  Async.
 */
oscar_status oscar_rope_append_int4(const oscar_int4_desc* desc, const oscar_rope_desc* rope,
                                    const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride,
                                    const uint16_t* v, int64_t v_stride, const int32_t* dst_req,
                                    const int32_t* dst_pos, const int32_t* rope_pos, int32_t n,
                                    uint16_t* q_out, uint16_t* k_out, void* stream);

/*
 * oscar_gather_int4 - reads cached rows of a 4-bit layer back as bf16, for
 * instance to go on with a prompt behind a cached prefix.
 *
 *   For item i < n: zero + scale * code, rounded to bf16 by way of fp32, of position
 *   src_pos[i] of request src_req[i], to row i of k_out and v_out
 *   (k_out + i * k_stride, H_kv heads of d).  src_req[i] = -1 and the skips
 *   are those of oscar_rope_append_int4: a skipped row is left as it was.
 *   src_req, src_pos: device int32 [n].  Rows 16-byte aligned, strides
 *   multiples of 8.  seq_len is not read.  n = 0 is a no-op.  Async.
 */
oscar_status oscar_gather_int4(const oscar_int4_desc* desc, const int32_t* src_req, const int32_t* src_pos,
                               int32_t n, uint16_t* k_out, int64_t k_stride, uint16_t* v_out, int64_t v_stride,
                               void* stream);

/*
 * oscar_decode_attention_int4 - one decode step of attention for every
 * request of the batch over a 4-bit layer.
 *
 *   q: row b at q + b * q_stride, H_q heads of d bf16 (16-byte aligned, stride
 *   a multiple of 8); out: [B][H_q][d] bf16 (16-byte aligned).  Request b's
 *   query sits at position seq_len[b] - 1 (its token has been appended) and
 *   attends positions 0 .. seq_len[b] - 1; query head j reads KV head
 *   j / (H_q / H_kv), a group of 1 .. 16.  score may be NULL (all defaults).
 *   Scores, sums and softmax statistics are fp32.  exp(t - max), and its product
 *   with a value's scale, are rounded to fp16 for the tensor cores (2^-11 each of a
 *   key's part in the result; where the scales of one scan lie more than 2^14 apart
 *   they stay fp32), and out to bf16.  A request with no token gets zeros.  Codes,
 *   scales and zeros of slots past seq_len may hold anything.  A length above max_len is
 *   clamped and sets OSCAR_DEV_LENGTH, a negative one counts as 0 and sets
 *   it; a page outside the pool is skipped and sets OSCAR_DEV_PAGE_BOUNDS.
 *   A copy that does not land within 1 s sets OSCAR_DEV_TIMEOUT (the output
 *   must not be used then).  OSCAR_ERR_UNSUPPORTED: groups above 16; max_len
 *   above 2^31 - 513; 2^31 or more of (pages of max_len, or of the window if that
 *   is less, + 64) x B x H_kv x (2 for groups above 8).  out must not overlap q.
 *   The result does not depend on scheduling.
 *
 *   Workspace: NULL asks for the size (it depends on head_dim alone); 256-byte
 *   aligned, zero-filled before its first use; each call leaves it ready for
 *   the next, of whatever sizes; calls that may overlap (other streams, two
 *   graphs replayed at once) need workspaces of their own.  Async.
 */
oscar_status oscar_decode_attention_int4(const oscar_int4_desc* desc, const oscar_score_desc* score,
                                         const uint16_t* q, int64_t q_stride, uint16_t* out, void* workspace,
                                         size_t* workspace_bytes, void* stream);

/* A batch of packed prompts (or documents of one packed sequence). */
typedef struct oscar_prompt_desc {
  int32_t batch;              /* B >= 1 requests                                */
  int32_t n_q_heads;          /* H_q, a multiple of n_kv_heads                  */
  int32_t n_kv_heads;         /* H_kv >= 1                                      */
  int32_t head_dim;           /* 64 or 128                                      */
  int32_t max_q;              /* host upper bound on a request's queries        */
  int32_t max_k;              /* host upper bound on a request's keys           */
  int32_t causal;             /* 1: keys after the query are masked; 0: not     */
  int32_t reserved;           /* 0                                              */
  int64_t total_q;            /* rows of q, out and lse                         */
  int64_t total_k;            /* rows of k and v                                */
  int32_t* dev_status;        /* optional device word for OSCAR_DEV_* bits      */
} oscar_prompt_desc;

/*
 * oscar_prompt_attention - attention of prompt tokens over bf16 rows: the
 * prefill that comes before a cache is decoded from.
 *
 *   Request b has the queries cu_q[b] .. cu_q[b+1] - 1 and the keys cu_k[b] ..
 *   cu_k[b+1] - 1 (device int32 [B + 1], non-decreasing from >= 0): packed
 *   documents do not see one another.  With n_q queries and n_k keys, query
 *   r of the request sits at position i = n_k - n_q + r (the keys' last
 *   n_q positions) and key c at position c.  causal: keys with j > i are
 *   masked; window: keys with i - j >= window; of both, keys j <
 *   prefix_len[b] are excepted (prefix_len NULL: none).  out row =
 *   softmax(t) v over the keys left, t as in oscar_score_desc; a row with no
 *   key left gets zeros and lse -inf.
 *
 *   q, k, v: bf16 rows of H_q / H_kv heads of d, q_stride / k_stride /
 *   v_stride elements apart (multiples of 8), 16-byte aligned; out:
 *   [total_q][H_q][d] bf16 (16-byte aligned); lse: optional [total_q][H_q]
 *   fp32, the natural logarithm of the sum of exp(t).  Scores, statistics and
 *   output sums are fp32; exp(t - max) is rounded to bf16 for its product
 *   with v.  Rows of out and lse outside every request are left as they
 *   were; rows of k and v outside a request never reach it, whatever they
 *   hold.  A query row with a NaN has a NaN result and reaches no other row.  A
 *   request's value rows must be finite where one of its queries sees them (one
 *   with a NaN may reach queries that it is masked for); key and value rows
 *   that the window hides from all of its queries may hold anything.  Lengths above max_q /
 *   max_k or rows outside total_q / total_k are clamped and set
 *   OSCAR_DEV_LENGTH.  A wait within the kernel that runs out (1 s) sets
 *   OSCAR_DEV_TIMEOUT (the output must not be used then).  2^26 or more row
 *   blocks over B x max_q and the head sets (256 rows of (query, head) pairs each):
 *   OSCAR_ERR_UNSUPPORTED.  out must not overlap q, k or v.  The result does not
 *   depend on scheduling.
 *
 *   Workspace: NULL asks for the size (it depends on desc); otherwise 256-byte
 *   aligned device memory, of any content; calls that may overlap need
 *   workspaces of their own.  Async.
 */
oscar_status oscar_prompt_attention(const oscar_prompt_desc* desc, const oscar_score_desc* score,
                                    const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride,
                                    const uint16_t* v, int64_t v_stride, const int32_t* cu_q, const int32_t* cu_k,
                                    const int32_t* prefix_len, uint16_t* out, float* lse, void* workspace,
                                    size_t* workspace_bytes, void* stream);

/*
 * ---------------------------------------------------------------- rotary positions
 *
 * What serves every kind of layer before its cache: the tables that
 * oscar_rope_desc points to, and norm and rotation of query and key rows.  (The
 * pages take keys as given, after both.)
 */

/* How the frequencies theta^(-2 i / rot_dim) of the pairs i are scaled for contexts
 * longer than the trained one. */
enum {
  OSCAR_ROPE_PLAIN = 0,     /* not at all                                         */
  OSCAR_ROPE_LINEAR = 1,    /* all divided by the factor                          */
  OSCAR_ROPE_BASE = 2,      /* theta times factor^(rot_dim / (rot_dim - 2)): the  */
                            /* fastest pair stays, the slowest is divided         */
  OSCAR_ROPE_BY_INDEX = 3,  /* pairs that make turns_high turns or more over the  */
                            /* trained context stay, those of turns_low or fewer  */
                            /* are divided; between, a ramp over the pair's index */
                            /* (its ends rounded outwards to whole indices)       */
  OSCAR_ROPE_BY_TURNS = 4   /* the same with the ramp over the pair's turns       */
};
typedef struct oscar_rope_scaling {
  int32_t kind;               /* OSCAR_ROPE_*                                   */
  int32_t reserved;           /* 0                                              */
  double factor;              /* >= 1 (not read for PLAIN)                      */
  double original_len;        /* positions of the trained context (BY_*)        */
  double turns_low;           /* BY_*: 0 < low < high; both 0: 1 and 32         */
  double turns_high;          /* (BY_INDEX), 1 and 4 (BY_TURNS)                 */
} oscar_rope_scaling;

/*
 * oscar_rope_frequencies - the frequencies of a rotation, in radians per
 * position: freq_out (host, [rot_dim / 2] float64).  scaling may be NULL
 * (PLAIN).  *magnitude_out (nullable): the factor on cosines and sines that goes
 * with the scaling (BY_INDEX: 0.1 ln(factor) + 1; else 1).  rot_dim a multiple of 16,
 * 16 .. 128; theta > 1.  Host-only, synchronous.
 */
oscar_status oscar_rope_frequencies(int32_t rot_dim, double theta, const oscar_rope_scaling* scaling,
                                    double* freq_out, double* magnitude_out);

/*
 * oscar_rope_table - the table of an oscar_rope_desc: cos_sin (device, [n][rot_dim]
 * fp32, 16-byte aligned), row j = the rot_dim / 2 cosines of the angles (first + j) freq[i],
 * then their sines, all times magnitude.
 *
 *   freq: host [rot_dim / 2], 0 <= freq <= 6 radians (of oscar_rope_frequencies, or any
 *   others; read during the call).  An entry is off by 2^-21 of its own size and
 *   (first + j) 2^-65 of a turn at the most (the turn of one position is rounded to 2^-64;
 *   products with it and wraps are exact).  rot_dim a multiple of 16, 16 .. 128;
 *   0 <= first, n <= 2^40.  n = 0 is a no-op.  Async.
 */
oscar_status oscar_rope_table(const double* freq, int32_t rot_dim, double magnitude, int64_t first, int64_t n,
                              float* cos_sin, void* stream);

/* Norm of each head before its rotation: x / sqrt(mean of x^2 + eps), times the weights. */
typedef struct oscar_head_norm {
  const uint16_t* q_weight;   /* device [head_dim] bf16, 16-byte aligned; NULL: */
  const uint16_t* k_weight;   /* query (key) heads have no norm                 */
  float eps;                  /* >= 0 and finite                                */
  int32_t reserved;           /* 0                                              */
} oscar_head_norm;

/*
 * oscar_norm_rope - norm and rotation of the query and key rows of n tokens, for
 * layers whose cache is filled by another call: oscar_quantize_append and
 * oscar_decode_step take keys as they come out of this one, and so does
 * oscar_rope_append_int4, which has no norm of its own, without a rotation (rope NULL).
 *
 *   For item i < n: every head of q row i (q + i * q_stride, n_q_heads heads of
 *   head_dim bf16) and of k row i is normed (norm NULL, or without that weight: not)
 *   and then rotated by row pos[i] of rope->cos_sin as in oscar_rope_append_int4
 *   (rope NULL: not), to row i of q_out and k_out.  fp32 arithmetic, one rounding to
 *   bf16 at the end.  The sum of the squares is fp32: heads with channels above 2^60 in
 *   magnitude are the caller's to scale.  Small ones are normed whatever the eps, and a head
 *   of zeros stays zeros, without an eps too.
 *   pos: device int32 [n]; may be NULL without a rotation.  pos[i] = -1 marks a padding
 *   row: it is left as it was.  With a rotation, any other position outside cos_sin skips
 *   the item and sets OSCAR_DEV_LENGTH in *dev_status (device int32, nullable).
 *   q and q_out may be NULL together, and so may k and k_out.  Rows 16-byte aligned, strides
 *   multiples of 8 elements and at least a row.  q_out may be q where the strides are
 *   equal, and k_out k; no other overlap.  head_dim 64 or 128.  n = 0 is a no-op.  Async.
 */
oscar_status oscar_norm_rope(int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, const oscar_head_norm* norm,
                             const oscar_rope_desc* rope, const uint16_t* q, int64_t q_stride, const uint16_t* k,
                             int64_t k_stride, const int32_t* pos, int32_t n, uint16_t* q_out, int64_t q_out_stride,
                             uint16_t* k_out, int64_t k_out_stride, int32_t* dev_status, void* stream);

/*
 * ---------------------------------------------------------------- 8-bit layers
 *
 * A layer that four bits do not carry keeps its whole KV cache at 8: the paged
 * cache of the 4-bit layers with 256 codes and one (scale, zero) for each vector
 * of a (token, KV head, K|V).
 *
 * Codec: zero = the vector's least channel rounded down to fp16, scale =
 * (greatest - zero) / 255 rounded up to fp16, code = (x - zero) / scale to the nearest
 * integer (ties to even), 0 where scale is 0: no channel lies outside the codes, and
 * every one is within half a scale of zero + scale * code.  Scales and codes are those
 * of exact differences and quotients.
 *
 * Page pool layout: head_dim d is 64 or 128, 16 tokens per page.  A block of one
 * (page p, KV head h) has 32 d + 128 bytes (oscar_int8_block_bytes) and sits at
 * byte (p * n_kv_heads + h) * block:
 *   [0, 16 d)     K codes: channel 16 c + i of token slot t is byte t d +
 *                 16 (c ^ x) + i, x = t % 8 (d = 128) or (t / 2) % 4 (d = 64);
 *   [16 d, 32 d)  V codes the same way;
 *   [32 d, ...)   slot t: K scale, K zero, V scale, V zero (fp16) at 32 d + 8 t.
 * (The order of a slot's 16-byte chunks lets eight slots' chunks of the same
 * channels be read from different shared-memory banks at once.)
 */
typedef struct oscar_int8_desc {
  int32_t batch;              /* B >= 1                                         */
  int32_t n_q_heads;          /* H_q, a multiple of n_kv_heads                  */
  int32_t n_kv_heads;         /* H_kv >= 1                                      */
  int32_t head_dim;           /* 64 or 128                                      */
  int32_t max_pages_per_seq;  /* row length of page_table                       */
  int32_t max_len;            /* host upper bound on every seq_len[b] (decode)  */
  int64_t n_pages;            /* physical pages in the pool                     */
  float tau_k;                /* keys are clamped to [-tau_k, tau_k]; 0 < tau <= 65504 */
  float tau_v;                /* the same for values                            */
  uint8_t* pages;             /* pool, 128-byte aligned (layout above)          */
  const int32_t* page_table;  /* [B][max_pages_per_seq] physical page ids       */
  const int32_t* seq_len;     /* [B] cached tokens of each request (decode)     */
  int32_t* dev_status;        /* optional device word for OSCAR_DEV_* bits      */
} oscar_int8_desc;

/* Bytes of one (page, KV head) block of an 8-bit layer; 0 for an invalid head size.  Host-only. */
int64_t oscar_int8_block_bytes(int32_t head_dim);

/*
 * oscar_rope_append_int8 - norms and rotates the queries and keys of n tokens
 * and appends their keys and values to an 8-bit layer's pages.
 *
 *   For item i < n: q row i and k row i are normed (norm) and rotated by row rope_pos[i]
 *   of rope->cos_sin (rope_pos NULL: dst_pos[i]) as in oscar_norm_rope, rounded to bf16:
 *   q' and k'.  q' goes to q_out and k' to k_out ([n][heads][d], contiguous; each may be
 *   NULL, or q / k itself where that is contiguous).  k' and v row i, clamped to
 *   [-tau, tau], are quantised by the codec above and stored at position dst_pos[i] of
 *   request dst_req[i].  k_held and v_held ([n][H_kv][d] contiguous, each may be NULL, or
 *   k / v itself where that is contiguous) receive what the cache stands for from now on,
 *   the rows that oscar_gather_int8 would read: a prompt's attention over them sees the
 *   values that later decodes see.
 *
 *   A NaN is quantised as -tau; other rows are not affected.
 *   dst_req[i] = -1 marks a padding row: nothing of it is written.  Any other request
 *   outside the batch, a position beyond the page table or a rotation row outside cos_sin
 *   skips the item and sets OSCAR_DEV_LENGTH; a page id outside the pool skips it and
 *   sets OSCAR_DEV_PAGE_BOUNDS.  A skipped item writes nothing.
 *
 *   norm and rope may be NULL.  q and q_out may be NULL together.  dst_req, dst_pos,
 *   rope_pos: device int32 [n].  Rows 16-byte aligned, strides multiples of 8 elements and
 *   at least one row.  seq_len is not read: the caller advances it.  Items must name
 *   distinct (request, position) pairs.  Outputs may share memory with inputs only as said
 *   above, and with one another not at all.  n = 0 is a no-op.  Async.
 */
oscar_status oscar_rope_append_int8(const oscar_int8_desc* desc, const oscar_head_norm* norm,
                                    const oscar_rope_desc* rope, const uint16_t* q, int64_t q_stride,
                                    const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                                    const int32_t* dst_req, const int32_t* dst_pos, const int32_t* rope_pos, int32_t n,
                                    uint16_t* q_out, uint16_t* k_out, uint16_t* k_held, uint16_t* v_held, void* stream);

/*
 * oscar_gather_int8 - reads cached rows of an 8-bit layer back as bf16.
 *
 *   For item i < n: zero + scale * code, rounded to bf16 by way of fp32, of position
 *   src_pos[i] of request src_req[i], to row i of k_out and v_out (k_out + i * k_stride,
 *   H_kv heads of d).  src_req[i] = -1 and the skips are those of
 *   oscar_rope_append_int8: a skipped row is left as it was.  src_req, src_pos: device
 *   int32 [n].  Rows 16-byte aligned, strides multiples of 8; no row of k_out may overlap one
 *   of v_out.  seq_len is not read.  n = 0 is a no-op.  Async.
 */
oscar_status oscar_gather_int8(const oscar_int8_desc* desc, const int32_t* src_req, const int32_t* src_pos, int32_t n,
                               uint16_t* k_out, int64_t k_stride, uint16_t* v_out, int64_t v_stride, void* stream);

/*
 * oscar_decode_attention_int8 - one decode step of attention for every request
 * of the batch over an 8-bit layer.
 *
 *   q: row b at q + b * q_stride, H_q heads of d bf16 (16-byte aligned, stride a multiple
 *   of 8); out: [B][H_q][d] bf16 (16-byte aligned); lse: optional [B][H_q] fp32, the natural
 *   logarithm of the sum of exp(t), by which results over other tokens can be joined.
 *   Request b's query sits at position seq_len[b] - 1 and attends positions 0 ..
 *   seq_len[b] - 1; query head j reads KV head j / (H_q / H_kv), a group of 1 .. 16.  (With
 *   seq_len the length of an encoder's states this is cross attention.)  score may be NULL
 *   (all defaults).
 *   Scores, sums and softmax statistics are fp32; a weight's product with a value's scale
 *   keeps 22 bits (two fp16 parts), as long as the scale is within 2^20 of the largest in
 *   its scan: below that, 2^-32 of the largest scale are lost for each unit of weight and
 *   code.  out is rounded to bf16.  A request with no token gets zeros and lse -inf.
 *   Codes, scales and zeros of slots past seq_len may hold anything.  A query head with a
 *   NaN has a NaN result and reaches no other.  A length above max_len is clamped and
 *   sets OSCAR_DEV_LENGTH, a negative one counts as 0 and sets it; a page outside the pool
 *   is skipped and sets OSCAR_DEV_PAGE_BOUNDS.  A copy that does not land within 1 s sets
 *   OSCAR_DEV_TIMEOUT (the output must not be used then).  OSCAR_ERR_UNSUPPORTED: groups
 *   above 16; max_len above 2^31 - 513; 2^31 or more of (pages of max_len, or of the window
 *   if that is less, + 32) x B x H_kv.  out and lse must not overlap q.  The result does not
 *   depend on scheduling.
 *
 *   Workspace: NULL asks for the size (it depends on head_dim alone); 256-byte aligned,
 *   zero-filled before its first use; each call leaves it ready for the next, of whatever
 *   sizes; calls that may overlap (other streams, two graphs replayed at once) need
 *   workspaces of their own.  Async.
 */
oscar_status oscar_decode_attention_int8(const oscar_int8_desc* desc, const oscar_score_desc* score,
                                         const uint16_t* q, int64_t q_stride, uint16_t* out, float* lse,
                                         void* workspace, size_t* workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* OSCAR_H_ */
