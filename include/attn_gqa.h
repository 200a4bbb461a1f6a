/*
 * attn_gqa.h -- C ABI of libattn_gqa.so: grouped-query scaled-dot-product
 * attention computed in one tiled online-softmax pass on an NVIDIA GB300
 * (sm_103a).  The score matrix is never materialised.
 *
 * The operations are those of three published WGSL compute shaders:
 *   - meganeura 0.2.0, src/shaders/attention.wgsl         -> attn_forward
 *   - meganeura 0.2.0, src/shaders/cached_attention.wgsl  -> attn_decode_cached
 *   - cera, src/backend/shaders/attention_prefill.wgsl    -> attn_prefill
 * Argument lists follow the shaders' parameter lists; shader templating and
 * storage bindings become plain arguments.  Further entry points fill the
 * shaders' open hooks and named future work: sliding windows (*_window),
 * paged caches (*_paged), rotary embedding (*_rope), the backward pass,
 * and an append-and-decode step; each states its reading below.
 *
 * Common rules for every entry point
 *   Notation   H = num_heads, G = num_kv_heads, D = head_dim, gs = H / G.
 *   GQA map    query head h reads kv head g = h / gs (integer division); H
 *              must be a multiple of G (all three shaders divide this way).
 *   Scale      scores are scale * (q . k); forward and decode use
 *              scale = 1 / sqrt(D) (the meganeura shaders' inverseSqrt), prefill
 *              takes scale as an argument (the cera shader's params[5]).
 *   Data       fp32 in, fp32 out (the calls with an attn_dtype_t argument say
 *              otherwise), row-major, all pointers are DEVICE memory
 *              owned by the caller.  The library keeps no pointer after a call
 *              returns.  Some calls need temporary scratch (the 16-bit K/V
 *              operand copies of the tensor-core paths, K turned for RoPE,
 *              the backward's per-row values; sizes from the
 *              attn_*_workspace_bytes queries).  With a workspace bound to the
 *              calling thread (attn_set_workspace) it is carved from that
 *              caller-owned buffer and the library allocates nothing.
 *              Otherwise it is stream-ordered on the call's stream, from a
 *              memory pool the library creates per device and keeps (freed
 *              blocks stay reserved for later calls; attn_release_scratch
 *              returns them).  Besides, every GPU that loads the library holds one
 *              fixed 4 MiB array for attn_decode_cached_noalloc (shared by
 *              all its calls on that device, kept until the process exits).
 *              The backward also runs one of its kernels on a library-owned
 *              stream per device, forked from and joined back into `stream`;
 *              all callers on a device share that stream, so concurrent
 *              backward calls on independent streams serialise there, and a
 *              backward must not be captured into CUDA graphs from two
 *              threads at once.
 *   Streams    every call is asynchronous on `stream` (a cudaStream_t; NULL is
 *              the legacy default stream).  Results are ready when the stream
 *              has reached the call.
 *   Errors     the return value is an attn status code.  Host-side checks run
 *              before anything is launched: on ATTN_ERR_INVALID_ARG or
 *              ATTN_ERR_UNSUPPORTED nothing is written.  ATTN_ERR_CUDA means a
 *              launch failed (the CUDA error is left in place for
 *              cudaGetLastError).  Conditions only the device can see (a
 *              device-resident kv_pos past the cache, a bounded wait that ran
 *              out) are recorded in a per-device status word; read it with
 *              attn_get_status.
 *   Empty      a window of zero keys writes zeros to the output rows and
 *              (-1e30, -1e30) to their LSE pair (attention.wgsl, fn main: the
 *              select() guards on sum_exp == 0).
 *   Precision  ATTN_FP32: fp32 CUDA-core arithmetic throughout.
 *              ATTN_TF32: both products on tcgen05 tensor cores with fp32
 *              accumulation and an fp32 softmax.  QK^T keeps Q to 22
 *              significant bits (two fp16 parts, hi + lo, under a power of
 *              two per query row) and K to 11 (fp16 under a power of two per
 *              128-key tile of a kv head): two products, the tensor time of
 *              one TF32 product.  PV takes TF32 operands (P and V with 11
 *              significant bits).  The scores feed an exponential, so their
 *              operand rounding sets the error: plain TF32 Q and K reach
 *              3.5e-3 of max|V| on scores of standard deviation 9, this
 *              scheme about 1.4e-3.
 *              ATTN_BF16: 16-bit operands at the full 16-bit tensor rate.
 *              QK^T takes fp16 operands (11 significant bits) under powers
 *              of two, one per query row and one per 128-key tile of a kv
 *              head, that keep every value below 2^15 whatever the fp32
 *              magnitudes; PV takes bf16 operands (P <= 2^24 and V; the
 *              fp32 accumulators carry |V| * keys * 2^24 below fp32's range
 *              for any |V| < 2^70).  K and V are converted by a pre-pass, Q
 *              and P on their way into the tensor core.
 *              Tensor-core precisions need D in {64, 128}, else they
 *              return ATTN_ERR_UNSUPPORTED.  Their kernels take
 *              1 <= gs <= 128 (a thread block packs 128/gs queries of gs
 *              heads; when gs does not divide 128 the remaining rows idle),
 *              16-byte aligned pointers, Q/out row strides that are
 *              multiples of 4 floats and K/V row strides that are multiples
 *              of 8 floats (paged caches: page_rows % 32 == 0); a call
 *              outside that runs on the fp32 CUDA-core kernel instead, whose
 *              results lie within every precision's bound.
 *              ATTN_FP32 accepts any 1 <= D <= 128.
 */
#ifndef ATTN_GQA_H
#define ATTN_GQA_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define ATTN_API __attribute__((visibility("default")))
#else
#define ATTN_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t / CUstream; declared here so the header needs no
 * CUDA include. */
typedef struct CUstream_st *attn_stream_t;

typedef enum {
    ATTN_CAUSAL = 0, /* query at position p sees keys 0..p          (kv_seq == q_seq) */
    ATTN_FULL = 1,   /* every query sees keys 0..q_seq-1             (kv_seq == q_seq) */
    ATTN_CROSS = 2   /* every query sees keys 0..kv_seq-1 (any kv_seq, 0 allowed)      */
} attn_mask_t;

typedef enum { ATTN_FP32 = 0, ATTN_TF32 = 1, ATTN_BF16 = 2 } attn_prec_t;

/* Element types of the calls that take more than fp32 (attn_rope_apply,
 * attn_qk_norm_rope, the paged appends, the batched attention). */
typedef enum { ATTN_DT_F32 = 0, ATTN_DT_BF16 = 1, ATTN_DT_F16 = 2 } attn_dtype_t;

/* Which columns of a head make a rotary pair, and how its angles are scaled
 * for contexts longer than the model's own (see attn_rope_table_scaled). */
typedef enum { ATTN_ROPE_HALF = 0, ATTN_ROPE_INTERLEAVED = 1 } attn_rope_layout_t;
typedef enum {
    ATTN_ROPE_NONE = 0,
    ATTN_ROPE_LINEAR = 1,
    ATTN_ROPE_NTK = 2,
    ATTN_ROPE_BY_PARTS = 3
} attn_rope_scaling_t;

enum {
    ATTN_OK = 0,
    ATTN_ERR_INVALID_ARG = 1,
    ATTN_ERR_UNSUPPORTED = 2,
    ATTN_ERR_CUDA = 3,
    ATTN_ERR_TIMEOUT = 4
};

/*
 * Self / cross attention forward with per-row (max, log-sum) output.
 * Source: meganeura attention.wgsl, fn main (variants causal kv_len = pos+1,
 * full kv_len = q_seq, cross kv_len = kv_seq; final store of
 * lse[(pos*H + head)*2 + {0,1}] = (max_score, log(sum_exp))).
 *
 *   q    [q_seq, H*D]     element (pos, h, d) at pos*H*D + h*D + d
 *   k, v [kv_seq, G*D]    element (t, g, d)   at t*G*D + g*D + d
 *   out  [q_seq, H*D]     same layout as q
 *   lse  [q_seq, H, 2]    (m, log l) with m the row's largest scaled score and
 *                         l = sum_t exp(s_t - m), so log-sum-exp = m + log l.
 *                         May be NULL (not written).
 *   mask ATTN_CAUSAL / ATTN_FULL need kv_seq == q_seq.
 *   prec ATTN_FP32, ATTN_TF32 or ATTN_BF16.
 * q_seq == 0 is a no-op (pointers may then be NULL).  Errors: INVALID_ARG for
 * NULL q/k/v/out (or k/v with kv_seq > 0), H % G != 0, G == 0, D == 0 or
 * D > 128, kv_seq != q_seq for causal/full, an unknown mask or precision;
 * UNSUPPORTED as described under Precision.
 */
ATTN_API int attn_forward(const float *q, const float *k, const float *v, float *out, float *lse,
                 uint32_t q_seq, uint32_t kv_seq, uint32_t num_heads, uint32_t num_kv_heads,
                 uint32_t head_dim, attn_mask_t mask, attn_prec_t prec, attn_stream_t stream);

/*
 * Bytes of device workspace attn_decode_cached needs for these sizes on the
 * current device (its SM count sets the number of KV splits).  Returns 0 for
 * sizes attn_decode_cached would reject.
 */
ATTN_API size_t attn_decode_workspace_bytes(uint32_t num_heads, uint32_t num_kv_heads, uint32_t head_dim,
                                   uint32_t max_seq);

/*
 * Cached single-token decode.  Source: meganeura cached_attention.wgsl,
 * fn main (Q = [1, H*D], K/V from a cache, kv_len = kv_pos_buf[0] + 1, so the
 * token attends to positions 0..kv_pos inclusive).
 *
 *   q                  [1, H*D]
 *   k_cache, v_cache   [max_seq, G*D]
 *   kv_pos_dev         one uint32 in DEVICE memory, read by the kernels (so a
 *                      CUDA graph can replay the call as the position grows)
 *   out                [1, H*D]
 *   max_seq            rows of the cache.  The window is cut at max_seq keys
 *                      (the cera prefill shader's defensive clamp); a kv_pos
 *                      >= max_seq also records ATTN_ERR_INVALID_ARG in the
 *                      device status word.
 *   workspace          device buffer of at least
 *                      attn_decode_workspace_bytes(H, G, D, max_seq) bytes,
 *                      16-byte aligned.  Zero it once (cudaMemset) before its
 *                      first use; each completed call leaves it ready for the
 *                      next.  Calls that share a workspace must not overlap on
 *                      the GPU.
 * The work is split over KV ranges; each split keeps its own (max, sum,
 * weighted V) and the last split of each kv head to finish merges them with
 * the log-sum-exp rule.  Errors: INVALID_ARG for NULL pointers, H % G != 0,
 * G == 0, D == 0 or D > 128, max_seq == 0, or a workspace that is too small
 * or misaligned.
 */
ATTN_API int attn_decode_cached(const float *q, const float *k_cache, const float *v_cache,
                       const uint32_t *kv_pos_dev, float *out, uint32_t num_heads,
                       uint32_t num_kv_heads, uint32_t head_dim, uint32_t max_seq,
                       void *workspace, size_t workspace_bytes, attn_stream_t stream);

/*
 * Cached decode of a new token that first appends its own K and V row: the
 * [G*D] rows k_new and v_new are written into row *kv_pos_dev
 * of k_cache and v_cache, then the call is attn_decode_cached over positions
 * 0..kv_pos (the new row included).  The pages leave filling the cache to
 * the host framework; this entry point saves a serving step the separate
 * copies into the cache (the split decode writes the row itself, in the
 * split that ends at kv_pos, before that split reads it).  A kv_pos >=
 * max_seq writes nothing and records ATTN_ERR_INVALID_ARG, as in
 * attn_decode_cached.  Arguments, workspace and errors otherwise as
 * attn_decode_cached, plus NULL k_new / v_new.
 *
 * Step I/O in host memory.  On the shapes the split decode covers (D in
 * {64, 128}, gs = H/G a power of two up to 32; the same holds for
 * attn_decode_cached), q, k_new, v_new, kv_pos_dev and out may also be
 * pinned host memory (cudaHostAlloc / cudaMallocHost, whose addresses are
 * valid on the device under unified addressing): the kernel reads the
 * step's inputs and writes its output across the host link itself, so a
 * serving step needs no staging copies.  The caches and the workspace must
 * be device memory.
 */
ATTN_API int attn_decode_append(const float *q, const float *k_new, const float *v_new, float *k_cache,
                                float *v_cache, const uint32_t *kv_pos_dev, float *out, uint32_t num_heads,
                                uint32_t num_kv_heads, uint32_t head_dim, uint32_t max_seq, void *workspace,
                                size_t workspace_bytes, attn_stream_t stream);

/*
 * Batched causal prefill against a KV cache.  Source: cera
 * attention_prefill.wgsl, fn attention_prefill (params n_heads, n_kv_heads,
 * head_dim, kv_dim, max_seq, scale, start_pos, q_stride, out_stride, q_base;
 * q_global = q_base + i; window min(start_pos + q_global + 1, max_seq)).
 *
 *   q_batch    query i of this call, head h, at (q_base+i)*q_stride + h*D
 *   k_cache,
 *   v_cache    [max_seq, kv_dim]; kv head g at column g*D
 *   out_batch  (q_base+i)*out_stride + h*D; other columns are not written
 *   n_queries  queries in this call (the shader's dispatch height)
 * n_queries == 0 is a no-op.  Errors: INVALID_ARG for NULL pointers,
 * H % G != 0, G == 0, D == 0 or D > 128, kv_dim < G*D, q_stride or
 * out_stride < H*D, start_pos + q_base + n_queries > max_seq (the shader's
 * host-side assertion), a non-finite scale or an unknown precision;
 * UNSUPPORTED as described under Precision.
 */
ATTN_API int attn_prefill(const float *q_batch, const float *k_cache, const float *v_cache,
                 float *out_batch, uint32_t n_queries, uint32_t n_heads, uint32_t n_kv_heads,
                 uint32_t head_dim, uint32_t kv_dim, uint32_t max_seq, float scale,
                 uint32_t start_pos, uint32_t q_stride, uint32_t out_stride, uint32_t q_base,
                 attn_prec_t prec, attn_stream_t stream);

/*
 * Sliding-window (local) attention: the three calls above with one more
 * argument, `window`, placed just before `stream`.  Every other argument,
 * layout, error and result is that of the call without the suffix.
 * Source: meganeura attention.wgsl, fn main -- the key loop of every variant
 * starts at a $KV_START placeholder that the page leaves to the host
 * framework.  This library reads it as a per-row lower bound: a row whose
 * window is keys [0, n) under the rules above attends keys
 *     [max(0, n - window), n)
 * i.e. its last `window` keys (window == 0: no lower bound, the call without
 * the suffix).  A window of 1 returns the V row of the last key; a window at
 * least n changes nothing.  The LSE pair of attn_forward_window describes
 * the kept keys only.  Key tiles that lie wholly before every row's window
 * are neither read nor computed, so the cost follows the window, not the
 * position.  No further errors.
 */
ATTN_API int attn_forward_window(const float *q, const float *k, const float *v, float *out, float *lse,
                                 uint32_t q_seq, uint32_t kv_seq, uint32_t num_heads, uint32_t num_kv_heads,
                                 uint32_t head_dim, attn_mask_t mask, attn_prec_t prec, uint32_t window, attn_stream_t stream);
ATTN_API int attn_decode_cached_window(const float *q, const float *k_cache, const float *v_cache,
                                       const uint32_t *kv_pos_dev, float *out, uint32_t num_heads,
                                       uint32_t num_kv_heads, uint32_t head_dim, uint32_t max_seq,
                                       void *workspace, size_t workspace_bytes, uint32_t window,
                                       attn_stream_t stream);
ATTN_API int attn_prefill_window(const float *q_batch, const float *k_cache, const float *v_cache,
                                 float *out_batch, uint32_t n_queries, uint32_t n_heads, uint32_t n_kv_heads,
                                 uint32_t head_dim, uint32_t kv_dim, uint32_t max_seq, float scale,
                                 uint32_t start_pos, uint32_t q_stride, uint32_t out_stride, uint32_t q_base,
                                 attn_prec_t prec, uint32_t window, attn_stream_t stream);

/*
 * Rotary position embedding (RoPE) fused into the forward.  The forward page
 * has hooks for it ($ROPE_DECL; $ROPE_Q_APPLY on the query value, and the key
 * expression $K_VAL_EXPR) whose bodies it leaves to the host framework.  This
 * library's convention: the pairs (d, d + D/2), d < D/2, of a row at position
 * p turn by the angle p * base^(-2d/D),
 *   x'[d]       = x[d] cos - x[d + D/2] sin
 *   x'[d + D/2] = x[d + D/2] cos + x[d] sin,
 * query row i at position i and key row t at position t; V is not turned.
 *
 * attn_rope_table fills a caller-owned DEVICE table [max_pos, head_dim] of
 * fp32: row p holds the cosines of the D/2 pair angles, then their sines,
 * computed in fp64 (base > 1, head_dim even and <= 128).
 *
 * attn_forward_rope is attn_forward_window with q and k turned first (inside
 * the kernels: the inputs are not modified); rope_table has table_rows >=
 * max(q_seq, kv_seq) rows from attn_rope_table for this head_dim.  Errors as
 * attn_forward_window, plus INVALID_ARG for an odd head_dim, a NULL or short
 * table, and UNSUPPORTED for head_dim % 8 != 0 or a table that is not
 * 16-byte aligned.
 */
ATTN_API int attn_rope_table(float *table, uint32_t max_pos, uint32_t head_dim, double base, attn_stream_t stream);
ATTN_API int attn_forward_rope(const float *q, const float *k, const float *v, float *out, float *lse,
                               uint32_t q_seq, uint32_t kv_seq, uint32_t num_heads, uint32_t num_kv_heads,
                               uint32_t head_dim, attn_mask_t mask, attn_prec_t prec, uint32_t window, const float *rope_table,
                               uint32_t table_rows, attn_stream_t stream);

/*
 * Paged KV cache: decode and prefill against a cache held in pages.  The
 * pages name paged KV only as future work for caches that overflow one buffer
 * (cera attention_prefill.wgsl, header comment); the layout here:
 *   k_pages, v_pages  pools of num_pages pages; page p holds page_rows
 *                     consecutive cache positions as rows
 *                     [p * page_rows, (p + 1) * page_rows) of a
 *                     [num_pages * page_rows, kv_dim] array (decode:
 *                     kv_dim = G*D)
 *   block_table       max_blocks uint32 in DEVICE memory: cache position t
 *                     is in pool page block_table[t / page_rows] at row
 *                     t % page_rows.  Entries may repeat (shared pages).
 * The cache's capacity is max_seq = page_rows * max_blocks; every other
 * argument, the window rule (with `window` as in the *_window calls), the
 * result and the errors are those of attn_decode_cached_window /
 * attn_prefill_window with that max_seq (decode's workspace:
 * attn_decode_workspace_bytes(H, G, D, max_seq)).  Only the block-table
 * entries of pages inside a row's window are read; an entry >= num_pages
 * reads as zeros and records ATTN_ERR_INVALID_ARG in the status word.  The
 * split decode and the tensor-core kernels need page_rows % 32 == 0
 * (otherwise decode, and a tensor-core prefill, run the fp32 CUDA-core
 * kernel).  The TF32 prefill reads named pages in
 * 32-row groups, so rows of such a group past the last attended position
 * must hold finite values.  Further errors: INVALID_ARG for a NULL
 * block_table, page_rows, num_pages or max_blocks of 0, or a capacity or
 * pool of 2^31 rows or more.
 */
ATTN_API int attn_decode_paged(const float *q, const float *k_pages, const float *v_pages,
                               const uint32_t *block_table, const uint32_t *kv_pos_dev, float *out,
                               uint32_t num_heads, uint32_t num_kv_heads, uint32_t head_dim, uint32_t page_rows,
                               uint32_t num_pages, uint32_t max_blocks, void *workspace, size_t workspace_bytes,
                               uint32_t window, attn_stream_t stream);
ATTN_API int attn_prefill_paged(const float *q_batch, const float *k_pages, const float *v_pages,
                                const uint32_t *block_table, float *out_batch, uint32_t n_queries, uint32_t n_heads,
                                uint32_t n_kv_heads, uint32_t head_dim, uint32_t kv_dim, uint32_t page_rows,
                                uint32_t num_pages, uint32_t max_blocks, float scale, uint32_t start_pos,
                                uint32_t q_stride, uint32_t out_stride, uint32_t q_base, attn_prec_t prec, uint32_t window,
                                attn_stream_t stream);

/*
 * Rotary positions as an operator of its own, for fp32, bf16 or fp16 rows:
 *   y = m R(p) x
 * Of every head, the pairs (i, i + R/2) (ATTN_ROPE_HALF) or (2i, 2i + 1)
 * (ATTN_ROPE_INTERLEAVED), i < R/2 with R = rot_dim, turn by the angle
 * p theta_i of the row's position p; columns >= R are copied:
 *   y[a] = m (x[a] cos - x[b] sin),  y[b] = m (x[b] cos + x[a] sin)
 *
 *   x, y        [rows, heads*D]; rows x_stride / y_stride elements apart, so
 *               the Q and K heads of a packed projection are one call.  y may
 *               be x (same stride); otherwise they must not overlap.
 *   dtype       of x and y; the arithmetic is fp32, rounded once
 *   positions   [rows] uint32 in device memory, or NULL: row t is at position t
 *   table       [table_rows, R] fp32: m cos of the R/2 pairs, then m sin
 *               (attn_rope_table_scaled, or attn_rope_table with head_dim = R)
 *   inverse     != 0 turns by -p theta_i and still multiplies by m: the
 *               gradient with respect to x of the call without it, for dy
 * A position >= table_rows writes zeros to the row's turned columns and
 * records ATTN_ERR_INVALID_ARG in the status word.  Sizes, strides or
 * addresses that do not allow 16-byte groups (D, strides % 8; R % 16, or % 8
 * interleaved) run one pair a thread.  rows == 0 is a no-op.  Errors:
 * INVALID_ARG for NULL pointers, addresses not aligned to their element, an
 * unknown type or layout, heads == 0, D == 0 or D > 1024, an odd, zero or too
 * large rot_dim, strides < heads*D, y == x with different strides, or (with
 * positions NULL) table_rows < rows.
 *
 * attn_rope_table_scaled fills such a table, angles in fp64.  theta_i =
 * base^(-2i/R) (base > 1, rot_dim even and <= 1024), changed by `scaling`
 * with factor f > 0:
 *   ATTN_ROPE_NONE      as it is (factor is not read)
 *   ATTN_ROPE_LINEAR    theta_i / f
 *   ATTN_ROPE_NTK       the base becomes base f^(R/(R-2)) (rot_dim >= 4)
 *   ATTN_ROPE_BY_PARTS  theta_i (g + (1 - g)/f) with g = clamp((orig_max_pos
 *                       theta_i / 2 pi - beta_slow) / (beta_fast - beta_slow),
 *                       0, 1): pairs that turn more than beta_fast times over
 *                       the original context keep their angle, those below
 *                       beta_slow are interpolated.  g is linear in the pair's
 *                       turns; weights trained with a ramp over the pair's
 *                       index between two rounded bounds want other angles (a
 *                       table is only data: fill one accordingly)
 * and m = attn_factor on every entry.  Errors: INVALID_ARG for values outside
 * these rules or max_pos * rot_dim >= 2^31; max_pos == 0 is a no-op.
 */
ATTN_API int attn_rope_table_scaled(float *table, uint32_t max_pos, uint32_t rot_dim, double base,
                                    attn_rope_scaling_t scaling, double factor, uint32_t orig_max_pos,
                                    double beta_fast, double beta_slow, double attn_factor, attn_stream_t stream);
ATTN_API int attn_rope_apply(const void *x, void *y, attn_dtype_t dtype, uint32_t rows, uint32_t heads,
                             uint32_t head_dim, uint32_t rot_dim, uint32_t x_stride, uint32_t y_stride,
                             attn_rope_layout_t layout, const uint32_t *positions, const float *table,
                             uint32_t table_rows, int inverse, attn_stream_t stream);

/*
 * Batches of ragged sequences over one paged cache: append, then attention.
 * Both calls take the same description of the batch, in DEVICE memory, so that
 * a captured step replays as the sequences grow:
 *   q_start      [n_seqs + 1]: the new tokens of sequence s are rows
 *                [q_start[s], q_start[s+1]) of the token batch (ascending; a
 *                sequence may have none).  Rows at or past q_start[n_seqs], up
 *                to total_rows, belong to no sequence and are left untouched.
 *   kv_len       [n_seqs]: positions of sequence s after the append, its new
 *                tokens included; they are the last ones, so row i is at
 *                position kv_len[s] - q_start[s+1] + i
 *   block_table  [n_seqs, max_blocks]: position t of sequence s is row
 *                t % page_rows of pool page block_table[s][t / page_rows].
 *                Only entries of positions that are written or attended are
 *                read.  Sequences may share pages they only read.
 *   k_pages,
 *   v_pages      pools of num_pages * page_rows rows of kv_dim elements; kv
 *                head g at column g*D
 * The limits on sizes are those of attn_prefill_paged.
 *
 * attn_append_paged writes the new rows' K, turned by their positions, and V
 * into the pages, and (num_heads > 0) the turned Q into q_out; q and q_out
 * NULL with num_heads == 0 leave Q out.
 *   k_new, v_new, q   [total_rows, ...] of type dtype, rows *_stride elements
 *                     apart; q_out of type cache_dtype
 *   cache_dtype       dtype itself, or any type when dtype is ATTN_DT_F32
 *                     (else ATTN_ERR_UNSUPPORTED); values are rounded once,
 *                     after the turn.  fp32 pools serve attn_decode_paged and
 *                     attn_prefill_paged, 16-bit ones attn_batch_paged.
 *   rot_dim, layout,
 *   table             as attn_rope_apply; rot_dim == 0 (table NULL) turns nothing
 * A row whose position is negative, past the capacity page_rows * max_blocks
 * or past the table, or whose page is >= num_pages, is skipped (nothing of it
 * is written) and ATTN_ERR_INVALID_ARG recorded in the status word.  Two rows
 * must not name the same pool row: its elements would come from either.
 * total_rows == 0 or n_seqs == 0 is a no-op.  q_out may be q when types and
 * strides are the same (else ATTN_ERR_INVALID_ARG); otherwise they must not
 * overlap.
 * Errors: INVALID_ARG for NULL pointers, addresses not
 * aligned to their element, bad heads, sizes, types, layout or strides,
 * total_rows >= 2^31 or n_seqs > 2^30.
 */
ATTN_API int attn_append_paged(const void *q, void *q_out, const void *k_new, const void *v_new, attn_dtype_t dtype,
                               void *k_pages, void *v_pages, attn_dtype_t cache_dtype, const uint32_t *block_table,
                               const uint32_t *q_start, const uint32_t *kv_len, uint32_t total_rows, uint32_t n_seqs,
                               uint32_t num_heads, uint32_t num_kv_heads, uint32_t head_dim, uint32_t kv_dim,
                               uint32_t q_stride, uint32_t q_out_stride, uint32_t k_stride, uint32_t v_stride,
                               uint32_t page_rows, uint32_t num_pages, uint32_t max_blocks, uint32_t rot_dim,
                               attn_rope_layout_t layout, const float *table, uint32_t table_rows,
                               attn_stream_t stream);

/*
 * attn_batch_paged: attention of every new token over its sequence's pages, in
 * bf16 or fp16.  One call takes whole prompts, chunks behind a long cache,
 * single tokens and any mixture.  The row at position p of sequence s, head h,
 * attends the keys [lo, hi) with
 *   lo = max(0, p + 1 - window)                          (window 0: lo = 0)
 *   hi = max(p + 1, min(prefix_len[s], kv_len[s]))       (prefix_len NULL: p + 1)
 * on the scores
 *   s_j = scale (q . k_j)
 *   s_j = softcap tanh(s_j / softcap)                    (softcap > 0)
 *   s_j = s_j - alibi_slopes[h] |p - j|                  (alibi_slopes != NULL)
 * and writes sum_j softmax(s)_j v_j, rounded to dtype; a row without keys
 * writes zeros.
 *
 *   q, out          [total_rows, ...], rows q_stride / out_stride elements
 *                   apart; out must not overlap q or the pools
 *   dtype           of q, the pools and out
 *   alibi_slopes    [n_heads] fp32; prefix_len [n_seqs] uint32 (device), or NULL
 *   workspace       device buffer of attn_batch_paged_workspace_bytes(...)
 *                   bytes, 16-byte aligned.  Zero it once (cudaMemset) before
 *                   its first use; each call leaves it ready for the next, of
 *                   any sizes, also one that recorded ATTN_ERR_TIMEOUT.
 *                   Calls that share it must not overlap on the GPU.
 * Scores, softmax and sums are fp32; P is rounded to dtype for the second
 * product: half a step of each weight, in fp16 at least 2^-32 of the largest
 * so far.  The work is divided over the GPU by each row block's number of key
 * tiles, splitting keys where rows are few; splits are joined in key order,
 * so repeated calls of the same batch give identical bits.  (In another batch a
 * sequence may be cut elsewhere, or run on another of the kernels below, and
 * its results differ in their last bits.)
 * What the pages hold at positions that none of a sequence's rows attends, or
 * past its end, never reaches a result.  K and V at positions that some row of
 * the sequence attends must be finite, |v| below 2^79 (sums are fp32, under
 * weights of up to 2^24; a NaN or infinity may also reach rows of the same
 * sequence that do not attend it).
 * A block-table entry >= num_pages reads as zeros; it, a kv_len[s] past the
 * capacity (the sequence is cut there) or below its number of new rows (rows
 * before position 0 attend no keys of their own), and a q_start that
 * descends or passes total_rows (the sequence is left out, or all of them where
 * they overlap so often that their blocks of rows are too many) record
 * ATTN_ERR_INVALID_ARG in the status word.  total_rows == 0 or n_seqs == 0 is
 * a no-op.  Errors: INVALID_ARG for NULL pointers, bad heads, sizes or
 * strides, a scale that is not finite or beyond 2e38, a softcap that is
 * negative, above 2e38 or so small that scale / softcap is not finite, or a
 * workspace that is too small or misaligned; UNSUPPORTED for ATTN_DT_F32
 * (attn_decode_paged and attn_prefill_paged serve fp32 pools), head_dim % 8 !=
 * 0, kv_dim or strides % 8 != 0, addresses of q, out or the pools that are not
 * 16-byte aligned, more than 16384 sequences, a capacity of more than 2^24
 * positions, a pool of more than 2^31 - 257 rows, or total_rows * n_heads >
 * 2^30.
 * Kernels: pages of whole 8-row groups (page_rows % 8 == 0) run on the tensor
 * cores (tcgen05) or, for about one row a sequence (total_rows <= n_seqs) with
 * H/G <= 16, on a kernel that streams K and V; other pages on warp-level
 * products.  Results lie within the same bounds.
 */
ATTN_API size_t attn_batch_paged_workspace_bytes(uint32_t n_heads, uint32_t n_kv_heads, uint32_t head_dim);
ATTN_API int attn_batch_paged(const void *q, const void *k_pages, const void *v_pages, void *out, attn_dtype_t dtype,
                              const uint32_t *block_table, const uint32_t *q_start, const uint32_t *kv_len,
                              uint32_t total_rows, uint32_t n_seqs, uint32_t n_heads, uint32_t n_kv_heads,
                              uint32_t head_dim, uint32_t kv_dim, uint32_t q_stride, uint32_t out_stride,
                              uint32_t page_rows, uint32_t num_pages, uint32_t max_blocks, float scale,
                              uint32_t window, float softcap, const float *alibi_slopes, const uint32_t *prefix_len,
                              void *workspace, size_t workspace_bytes, attn_stream_t stream);

/*
 * attn_batch_paged_sinks: attn_batch_paged with one more argument, `sinks`,
 * placed just before `stream`: the sequence's first positions stay visible
 * behind the window.  The row at position p attends the keys
 *   [0, min(sinks, lo)) and [lo, hi)
 * with lo and hi as above (sinks == 0, or a window that reaches the first
 * positions: attn_batch_paged; bias and cap are those of each key's own
 * position).  Key tiles between the two ranges are neither read nor computed.
 * No further errors.
 */
ATTN_API int attn_batch_paged_sinks(const void *q, const void *k_pages, const void *v_pages, void *out,
                                    attn_dtype_t dtype, const uint32_t *block_table, const uint32_t *q_start,
                                    const uint32_t *kv_len, uint32_t total_rows, uint32_t n_seqs, uint32_t n_heads,
                                    uint32_t n_kv_heads, uint32_t head_dim, uint32_t kv_dim, uint32_t q_stride,
                                    uint32_t out_stride, uint32_t page_rows, uint32_t num_pages, uint32_t max_blocks,
                                    float scale, uint32_t window, float softcap, const float *alibi_slopes,
                                    const uint32_t *prefix_len, void *workspace, size_t workspace_bytes,
                                    uint32_t sinks, attn_stream_t stream);

/*
 * Norms of query and key heads with their rotary turn in the same pass, and
 * the gradients, for fp32, bf16 or fp16 rows.  Of every head x of Q and of K
 *   z = w x r,  r = 1 / sqrt(mean(x^2) + eps)      (over its head_dim columns)
 *   y = m R(p) z                                   (as attn_rope_apply)
 * with one weight vector for the heads of Q and one for those of K.
 *
 *   q, k            [rows, heads*D], rows *_stride elements apart, so both are
 *                   read where a packed projection left them; num_heads or
 *                   num_kv_heads 0 leaves one of them out
 *   q_out, k_out    as q and k; each may be its input (same stride), otherwise
 *                   they must not overlap any input
 *   q_weight,
 *   k_weight        [D] of type weight_dtype, or NULL: ones
 *   dtype           of the rows; the arithmetic is fp32, rounded once
 *   rot_dim, layout, positions, table, table_rows
 *                   as attn_rope_apply; rot_dim == 0 (table NULL): no turn
 * A position >= table_rows writes zeros to the row's turned columns (the
 * backward takes their upstream gradient as zero) and records
 * ATTN_ERR_INVALID_ARG in the status word.  The sum of squares is fp32: |x|
 * below 1e18.  rows == 0 is a no-op.  Errors: INVALID_ARG for NULL or
 * misaligned pointers, unknown types or layouts, both head counts 0, D == 0 or
 * D > 256, an odd or too large rot_dim, strides < heads*D, an output in place
 * with another stride, an eps that is not finite or below 1e-30, or (with
 * positions NULL) table_rows < rows.
 *
 * The backward takes the forward's inputs and the upstream gradients dq, dk
 * of q_out and k_out:
 *   dz = m R(p)^T dy,  dw = sum over rows and heads of dz x r,
 *   dx = r (w dz - x r mean(w dz x r))
 * dq_out and dk_out are written as q_out and k_out are (each may be dq or q,
 * dk or k); dq_weight and dk_weight ([D] of weight_dtype, either may be NULL:
 * not wanted) are written in full, also for rows == 0 and for a tensor that is
 * left out (zeros).  Sums are fp32, in a fixed order: repeated calls give
 * identical bits.  workspace (16-byte aligned; not needed when both are NULL)
 * holds attn_qk_norm_rope_backward_workspace_bytes bytes and keeps nothing
 * between calls; calls that share it must not overlap on the GPU.
 */
ATTN_API int attn_qk_norm_rope(const void *q, const void *k, void *q_out, void *k_out, const void *q_weight,
                               const void *k_weight, attn_dtype_t dtype, attn_dtype_t weight_dtype, uint32_t rows,
                               uint32_t num_heads, uint32_t num_kv_heads, uint32_t head_dim, uint32_t q_stride,
                               uint32_t k_stride, uint32_t q_out_stride, uint32_t k_out_stride, float eps,
                               uint32_t rot_dim, attn_rope_layout_t layout, const uint32_t *positions,
                               const float *table, uint32_t table_rows, attn_stream_t stream);
ATTN_API size_t attn_qk_norm_rope_backward_workspace_bytes(uint32_t head_dim);
ATTN_API int attn_qk_norm_rope_backward(const void *dq, const void *dk, const void *q, const void *k, void *dq_out,
                                        void *dk_out, const void *q_weight, const void *k_weight, void *dq_weight,
                                        void *dk_weight, attn_dtype_t dtype, attn_dtype_t weight_dtype, uint32_t rows,
                                        uint32_t num_heads, uint32_t num_kv_heads, uint32_t head_dim,
                                        uint32_t dq_stride, uint32_t dk_stride, uint32_t q_stride, uint32_t k_stride,
                                        uint32_t dq_out_stride, uint32_t dk_out_stride, float eps, uint32_t rot_dim,
                                        attn_rope_layout_t layout, const uint32_t *positions, const float *table,
                                        uint32_t table_rows, void *workspace, size_t workspace_bytes,
                                        attn_stream_t stream);

/*
 * The paged cache in 8 bits.  The batch is described as for attn_append_paged;
 * the pools hold e4m3 codes and two arrays their scales:
 *   k_pages, v_pages    [num_pages * page_rows, kv_dim] bytes; kv head g at
 *                       column g*D
 *   k_scales, v_scales  [num_pages * page_rows / scale_rows, num_kv_heads]
 *                       bytes: pool rows [b * scale_rows, (b + 1) * scale_rows)
 *                       of head g share the scale 2^(k_scales[b][g] - 127)
 *   scale_rows          divides page_rows (1: a scale for every position and
 *                       head; page_rows: one a page)
 * A value is code times scale.  Scales run from 2^-14 to 2^7 (bytes outside
 * read as the nearest of these), so every value is exactly a bf16 and an fp16
 * number, from steps of 2^-23 up to 57344.
 *
 * attn_append_paged8 writes the new rows' K and V: K normed (k_weight, [D] of
 * weight_dtype, not NULL; as attn_qk_norm_rope) and turned by its position
 * (rot_dim > 0), both then rounded to codes of the smallest scale 2^e with
 * max|x| <= 448 * 2^e over all rows of the scale's block written so far; and
 * Q, normed (q_weight) and turned, into q_out.
 *   - A block whose first position is among the new rows starts anew,
 *     whatever its page held.  In a block that held earlier positions of the
 *     sequence, these keep their codes, or, where the scale grows, are
 *     multiplied by the scales' quotient and rounded again (exact but for
 *     codes that become subnormal).
 *   - Magnitudes above 57344, and infinities, become 57344; a NaN stays one
 *     and counts for no scale.  The arithmetic is fp32 up to the rounding.
 *   - q_out_dtype is ATTN_DT_BF16 or ATTN_DT_F16: dtype itself unless that is
 *     ATTN_DT_F32 (else ATTN_ERR_UNSUPPORTED).  q, q_out NULL with num_heads == 0
 *     leave Q out.
 * Rows that attn_append_paged skips are skipped here (their q_out, too), with
 * the same status.  No two rows may belong to the same scale of the pools
 * unless they are of one sequence; a page that sequences share is written by
 * none of them, so they share whole blocks of scale_rows positions (what is
 * written into a block may move all of its codes).  total_rows == 0 or n_seqs == 0 is a no-op.
 * Errors: INVALID_ARG as attn_append_paged, and for a scale_rows that does not
 * divide page_rows, NULL scales, a weight for Q without Q, or (with a weight)
 * an eps as attn_qk_norm_rope; UNSUPPORTED for head_dim % 16 != 0, kv_dim %
 * 16 != 0, pools that are not 16-byte aligned, or total_rows * 2 *
 * num_kv_heads beyond 2^31 - 256.
 *
 * attn_read_paged8 writes the values of a range of each sequence's positions,
 * rounded to dtype (bf16 and fp16 hold them exactly):
 *   starts       [n_seqs + 1]: rows [starts[s], starts[s+1]) of k_out and
 *                v_out are sequence s's positions first[s], first[s] + 1, ...
 *                Rows of no sequence are left untouched.
 *   first        [n_seqs], or NULL: from position 0
 *   kv_len       [n_seqs]: a position past it (or past the capacity, or in a
 *                page outside the pool) reads as zeros and records
 *                ATTN_ERR_INVALID_ARG in the status word
 *   k_out, v_out [total_rows, ...] of type dtype, rows k_stride / v_stride
 *                elements apart
 * Errors as attn_append_paged8's.
 *
 * attn_batch_paged8 is attn_batch_paged_sinks over such a cache: dtype
 * (ATTN_DT_BF16 or ATTN_DT_F16) is that of q and out.  The products run on
 * fp16 operands: K and V exactly, Q of bf16 times a power of two of its row
 * (entries below 2^-28 of the row's largest lose bits), P with half a step of
 * fp16 of each weight and at least 2^-32 of the largest so far (single tokens:
 * of each weight times its key's V scale, and of the largest of these).
 * Neither K nor V may hold a NaN code at positions that some row of the
 * sequence attends; at others, and in pages of other sequences, codes and
 * scales are free.  The workspace is attn_batch_paged's, also the same one by
 * turns, and the kernels are chosen as there.  Errors as attn_batch_paged;
 * INVALID_ARG for a scale_rows that does not divide page_rows or NULL scales,
 * UNSUPPORTED for head_dim % 16 != 0 and kv_dim % 16 != 0.
 */
ATTN_API int attn_append_paged8(const void *q, void *q_out, const void *k_new, const void *v_new, attn_dtype_t dtype,
                                attn_dtype_t q_out_dtype, void *k_pages, void *v_pages, uint8_t *k_scales,
                                uint8_t *v_scales, const uint32_t *block_table, const uint32_t *q_start,
                                const uint32_t *kv_len, uint32_t total_rows, uint32_t n_seqs, uint32_t num_heads,
                                uint32_t num_kv_heads, uint32_t head_dim, uint32_t kv_dim, uint32_t q_stride,
                                uint32_t q_out_stride, uint32_t k_stride, uint32_t v_stride, uint32_t page_rows,
                                uint32_t num_pages, uint32_t max_blocks, uint32_t scale_rows, const void *q_weight,
                                const void *k_weight, attn_dtype_t weight_dtype, float eps, uint32_t rot_dim,
                                attn_rope_layout_t layout, const float *table, uint32_t table_rows,
                                attn_stream_t stream);
ATTN_API int attn_read_paged8(const void *k_pages, const void *v_pages, const uint8_t *k_scales,
                              const uint8_t *v_scales, void *k_out, void *v_out, attn_dtype_t dtype,
                              const uint32_t *block_table, const uint32_t *starts, const uint32_t *first,
                              const uint32_t *kv_len, uint32_t total_rows, uint32_t n_seqs, uint32_t num_kv_heads,
                              uint32_t head_dim, uint32_t kv_dim, uint32_t k_stride, uint32_t v_stride,
                              uint32_t page_rows, uint32_t num_pages, uint32_t max_blocks, uint32_t scale_rows,
                              attn_stream_t stream);
ATTN_API int attn_batch_paged8(const void *q, const void *k_pages, const void *v_pages, const uint8_t *k_scales,
                               const uint8_t *v_scales, void *out, attn_dtype_t dtype, const uint32_t *block_table,
                               const uint32_t *q_start, const uint32_t *kv_len, uint32_t total_rows, uint32_t n_seqs,
                               uint32_t n_heads, uint32_t n_kv_heads, uint32_t head_dim, uint32_t kv_dim,
                               uint32_t q_stride, uint32_t out_stride, uint32_t page_rows, uint32_t num_pages,
                               uint32_t max_blocks, uint32_t scale_rows, float scale, uint32_t window, uint32_t sinks,
                               float softcap, const float *alibi_slopes, const uint32_t *prefix_len, void *workspace,
                               size_t workspace_bytes, attn_stream_t stream);

/*
 * Backward of attn_forward / attn_forward_window: the gradients of `out` with
 * respect to q, k and v for an upstream gradient dout.  The pages emit the
 * per-row (max, log-sum) pair for a backward pass (meganeura attention.wgsl:
 * header comment and the final LSE store) but print none; this is the plain
 * gradient of the forward definition, rebuilt from that pair:
 *   p_t  = exp(scale q.k_t - lse0 - lse1)      over the row's kept keys
 *   ds_t = p_t (dout.v_t - dout.out)
 *   dq   = scale sum_t ds_t k_t
 *   dk_t = scale sum over rows of ds_t q      (every query head of the kv head)
 *   dv_t = sum over rows of p_t dout
 * The LSE output is not differentiated (its gradient is taken as zero).
 *
 *   q, out, dout, dq   [q_seq, H*D]  (out and lse exactly as the forward wrote
 *   k, v, dk, dv       [kv_seq, G*D]  them for these q, k, v, mask, window)
 *   lse                [q_seq, H, 2]
 *   mask, window       as attn_forward_window (window 0 = none)
 *   prec               ATTN_FP32: CUDA cores, fp32 arithmetic.
 *                      ATTN_BF16: tensor cores; q, k, v, dout and the
 *                      P and dS tiles rounded to bf16, fp32 accumulation
 *                      (D in {64, 128}, else ATTN_ERR_UNSUPPORTED; a group
 *                      H/G that is not a power of two up to 128 runs the
 *                      fp32 backward instead).
 *                      ATTN_TF32 returns ATTN_ERR_UNSUPPORTED.
 * dq, dk and dv are written in full (keys no row attends get zero).  Each
 * element is computed by one thread block, without atomics, so repeated
 * calls give identical bits.  Needs D % 4 == 0 and 16-byte-aligned pointers,
 * else ATTN_ERR_UNSUPPORTED.  Scratch (8 bytes per (row, head); with
 * ATTN_BF16 also bf16 copies of q, dout, k and v) comes from the bound
 * workspace or the library pool (see the Data rule above).  q_seq == 0 is a
 * no-op; kv_seq == 0 zeroes
 * dq.  Errors otherwise as attn_forward, plus NULL out, dout, lse or
 * gradient pointers.
 */
ATTN_API int attn_backward(const float *q, const float *k, const float *v, const float *out, const float *dout,
                           const float *lse, float *dq, float *dk, float *dv, uint32_t q_seq, uint32_t kv_seq,
                           uint32_t num_heads, uint32_t num_kv_heads, uint32_t head_dim, attn_mask_t mask, attn_prec_t prec,
                           uint32_t window, attn_stream_t stream);

/*
 * Backward of attn_forward_rope: attn_backward's arguments plus the RoPE
 * table of that forward (rope_table, table_rows as there).  The gradients
 * are with respect to the unturned q and k: the plain gradient at the turned
 * q, k (turned into library scratch) is turned back.  out and lse are those
 * attn_forward_rope wrote.  Errors as attn_backward plus those of
 * attn_forward_rope's table checks.
 */
ATTN_API int attn_backward_rope(const float *q, const float *k, const float *v, const float *out, const float *dout,
                                const float *lse, float *dq, float *dk, float *dv, uint32_t q_seq, uint32_t kv_seq,
                                uint32_t num_heads, uint32_t num_kv_heads, uint32_t head_dim, attn_mask_t mask, attn_prec_t prec,
                                uint32_t window, const float *rope_table, uint32_t table_rows,
                                attn_stream_t stream);

/*
 * Cached single-token decode that allocates nothing and takes no workspace.
 * The shader pages have no counterpart to this entry point; it exists for
 * callers that cannot provide device scratch memory -- a plugin inside a
 * framework that owns every device allocation, or a serving loop that must
 * never call cudaMalloc (an allocation may synchronise the device and has no
 * latency bound).
 *
 * Arguments, layouts, the window rule and the result are those of
 * attn_decode_cached, minus the workspace.  In its place the library uses a
 * fixed 4 MiB array of device memory that is part of the library image: every
 * GPU that loads libattn_gqa.so holds it until the process exits.
 *   - Sizes whose split decode would need more than 4 MiB of scratch (about
 *     H * 2 * SMs / G * D * 4 bytes), shapes the split kernels do not cover
 *     (they take D in {64, 128} with gs = H/G a power of two up to 32) and
 *     pointers that are not 16-byte aligned return ATTN_ERR_UNSUPPORTED;
 *     nothing is launched.
 *   - All calls on a device share the one array, and it keeps what the last
 *     call left there; each call first clears the counters that must start
 *     at zero, on `stream`.  Calls that can overlap on the GPU (different
 *     streams without ordering between them) race on the array and give
 *     wrong results: order them on one stream.
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture begins.
 * Errors: as attn_decode_cached (INVALID_ARG for bad sizes or NULL pointers),
 * plus the UNSUPPORTED cases above.
 */
ATTN_API int attn_decode_cached_noalloc(const float *q, const float *k_cache, const float *v_cache,
                                        const uint32_t *kv_pos_dev, float *out, uint32_t num_heads,
                                        uint32_t num_kv_heads, uint32_t head_dim, uint32_t max_seq,
                                        attn_stream_t stream);

/*
 * Caller-owned scratch.  attn_set_workspace binds a DEVICE buffer of
 * workspace_bytes bytes (256-byte aligned) to the calling thread: from then
 * on every call this thread makes takes its temporary scratch from it, from
 * offset 0 each call, and allocates nothing; a call whose scratch does not
 * fit returns ATTN_ERR_INVALID_ARG before launching anything.
 * attn_set_workspace(NULL, 0) returns to the library pool.  The buffer is
 * read and written on the calls' streams: calls that share it must be
 * ordered on one stream (or synchronised), and it must stay allocated until
 * the last of them has run.  Errors: INVALID_ARG for a misaligned buffer.
 *
 * The queries give the bytes one call needs (0: none, or arguments the call
 * would reject); a bound workspace must hold the largest of the calls it
 * serves.
 *   attn_forward_workspace_bytes   attn_forward, attn_forward_window and, with
 *                                  rope != 0, attn_forward_rope
 *   attn_prefill_workspace_bytes   attn_prefill, attn_prefill_window and
 *                                  attn_prefill_paged (max_seq = page_rows *
 *                                  max_blocks)
 *   attn_backward_workspace_bytes  attn_backward and, with rope != 0,
 *                                  attn_backward_rope
 * Decode takes its workspace as an argument (attn_decode_workspace_bytes).
 */
ATTN_API int attn_set_workspace(void *workspace, size_t workspace_bytes);
ATTN_API size_t attn_forward_workspace_bytes(uint32_t q_seq, uint32_t kv_seq, uint32_t num_heads,
                                             uint32_t num_kv_heads, uint32_t head_dim, attn_mask_t mask,
                                             attn_prec_t prec, uint32_t window, int rope);
ATTN_API size_t attn_prefill_workspace_bytes(uint32_t n_queries, uint32_t n_heads, uint32_t n_kv_heads,
                                             uint32_t head_dim, uint32_t kv_dim, uint32_t max_seq,
                                             uint32_t start_pos, uint32_t q_base, attn_prec_t prec,
                                             uint32_t window);
ATTN_API size_t attn_backward_workspace_bytes(uint32_t q_seq, uint32_t kv_seq, uint32_t num_heads,
                                              uint32_t num_kv_heads, uint32_t head_dim, attn_prec_t prec, int rope);

/*
 * The library pool on the current device (the scratch of calls made without
 * a bound workspace): attn_scratch_reserved_bytes is the memory it holds;
 * attn_scratch_peak_bytes the most it has had in use at once since the last
 * reset (reset != 0 resets it to 0 after reading); attn_release_scratch
 * returns the reserved memory not in use (call it after synchronising the
 * streams that used the pool).  Errors: ATTN_ERR_CUDA if the pool is not
 * available.
 */
ATTN_API size_t attn_scratch_reserved_bytes(void);
ATTN_API size_t attn_scratch_peak_bytes(int reset);
ATTN_API int attn_release_scratch(void);

/*
 * Waits for `stream`, then returns and clears the current device's status
 * word: ATTN_OK, or the largest code a kernel recorded since the last read
 * (ATTN_ERR_INVALID_ARG for a decode kv_pos past the cache, ATTN_ERR_TIMEOUT
 * for a bounded device wait that gave up; its kernel returned early and its
 * output is not valid).  Returns ATTN_ERR_CUDA if the stream or the read
 * failed.
 */
ATTN_API int attn_get_status(attn_stream_t stream);

/*
 * Failure-path self test.  Launches one CTA that waits, with the bounded wait
 * every kernel of this library uses, on a barrier that nothing completes, but
 * with a limit of timeout_us microseconds (1 .. 1000000) instead of the usual
 * one second.  The wait gives up, the kernel records ATTN_ERR_TIMEOUT in the
 * device status word and returns normally: no fault, no hang, and the CUDA
 * context stays usable.  Read the outcome with attn_get_status.  Errors:
 * INVALID_ARG for a timeout outside the range.
 */
ATTN_API int attn_selftest_wait_timeout(uint32_t timeout_us, attn_stream_t stream);

/*
 * The same for the warp-wide wait of the batched kernels: one warp's wait gives
 * up, seven others wait for a barrier that completes just then.  lanes
 * [8] uint32 (device): the lanes of each warp whose wait succeeded, all or
 * none.  Errors: INVALID_ARG for a timeout outside the range or NULL lanes.
 * attn_selftest_short_wait is this for the wait of the tcgen05 kernels with a
 * cap, a bias, first positions or an 8-bit cache, which has its own code.
 *
 * attn_selftest_batch_wait sets the limit of the waits inside the kernels of
 * attn_batch_paged, attn_batch_paged_sinks and attn_batch_paged8 for this
 * process's later calls in bf16 on pages of whole 8-row groups (other calls
 * keep the usual limit): limit_ns nanoseconds, at most one second, 0 for the
 * usual one.  With limits of a microsecond waits of an
 * ordinary call run out: it records ATTN_ERR_TIMEOUT, drains what it has in
 * flight and returns; its output is not valid.
 */
ATTN_API int attn_selftest_batch_wait(uint32_t limit_ns);
ATTN_API int attn_selftest_warp_wait(uint32_t timeout_us, uint32_t *lanes, attn_stream_t stream);
ATTN_API int attn_selftest_short_wait(uint32_t timeout_us, uint32_t *lanes, attn_stream_t stream);

/* Static, human-readable name of a status code. */
ATTN_API const char *attn_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_GQA_H */
