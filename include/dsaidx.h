/*
 * libdsaidx -- the DeepSeek Sparse Attention (DSA) indexer hot path on one
 * GB300 GPU: the index-key store and the score + top-k selection; and the
 * attention it serves: rotary positions, the K/V cache, attention of drafted
 * tokens over it and over the selection.
 *
 * Sources (web pages on the bf16 index-K fix in the DSA indexer):
 *  [VAL] "The Moment of Validation: Diagnosing an OOM Crash in the bf16 Index-K
 *        Fix for DeepSeek V4 Sparse Attention", section "Input Knowledge
 *        Required to Understand This Message": fp8 index keys take 128 bytes of
 *        data plus a 4-byte scale (132 B/token), bf16 keys 128 x 2 = 256
 *        B/token; the fused store normalises, applies RoPE and stores in one
 *        kernel call.
 *  [DEC] "The Fused Kernel Decision: Precision Archaeology in the CUDA Sparse
 *        Attention Indexer", section "The Message": the indexer buffer is
 *        paged, page_size = 64, [npages, 64*128] bf16; each token maps to a
 *        page and an offset and its 128 values are written there.
 *  [CRA] "The Crash That Changed Direction", sections "The Experiment: Why
 *        fp32?" and "Assumptions Made and Broken": scores come from a batched
 *        matrix product of queries and index keys followed by a ReLU; the
 *        pages up-convert fp8 keys exactly before the product (this library
 *        gives them to the tensor cores as stored, see dsa_index_topk); the
 *        top-512 (or 1024) key positions are kept.
 *  [WFK] "When the Fused Kernel Isn't Enough", section "The Message:
 *        Validation and Discovery": materialising the logits over the whole
 *        context ran out of memory at about 22K tokens. This library never
 *        materialises the [q_len x ctx] logits: key tiles stream through a
 *        running per-query top-k.
 *
 * Conventions for every call:
 *  - Pointers marked (device) are CUDA device pointers owned by the caller;
 *    pointers marked (host) are host memory. The library keeps no pointer
 *    after a call returns.
 *  - Work is enqueued on `stream` and is asynchronous; argument errors are
 *    returned before anything is enqueued. Calls that enqueue work must be
 *    made with the context's device current (the one current at
 *    dsa_ctx_create); otherwise they return DSA_ERR_INVALID_ARG and enqueue
 *    nothing. A launch failure returns
 *    DSA_ERR_CUDA. Errors found on the device (a page id out of range, a
 *    bounded wait that ran out) do not trap: the kernel skips the access,
 *    records the error in a status word of the context and carries on;
 *    dsa_get_device_status() reads and clears it.
 *  - Sizes are int32 element counts; the byte layouts are stated per call.
 *  - Index heads H = 64 and head_dim D = 128 are fixed. Page size is 64.
 */
#ifndef DSAIDX_H
#define DSAIDX_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* dsa_stream_t; /* a cudaStream_t; NULL = legacy default stream */

typedef enum {
  DSA_OK = 0,
  DSA_ERR_INVALID_ARG = 1,   /* null pointer, negative size, misaligned pointer ... */
  DSA_ERR_UNSUPPORTED = 2,   /* k not in 1..2048, unknown format, no sm_103 device */
  DSA_ERR_CUDA = 3,          /* a CUDA runtime/driver call failed */
  DSA_ERR_DEVICE_BOUNDS = 4, /* device saw a page id / position / sequence out of range (or a
                                top-k candidate buffer would have overflowed: the keys are
                                dropped, never written past the buffer) */
  DSA_ERR_TIMEOUT = 5,       /* a bounded device-side wait ran out */
  DSA_ERR_WORKSPACE = 6      /* workspace too small */
} dsa_status;

typedef enum {
  DSA_FMT_BF16 = 0, /* 128 bf16 per token = 256 B; page = [64][128] bf16 = 16384 B      [DEC] */
  DSA_FMT_FP8 = 1,  /* 128 e4m3 + 1 fp32 scale = 132 B per token; page = [64][128] e4m3
                       followed by [64] fp32 scales = 8448 B                            [VAL] */
  DSA_FMT_FP4 = 2   /* 128 e2m1 (OCP MX FP4: 1 sign, 2 exponent bits with bias 1, 1
                       mantissa bit; magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6) packed two
                       per byte, the even dimension in the low nibble, + 1 fp32 scale
                       = 68 B per token; page = [64][64] code bytes followed by [64]
                       fp32 scales = 4352 B. [DEC], section "The Message: A Blueprint
                       for Kernel Modification", names an fp4 variant of the indexer
                       kernel for more aggressive compression without a layout; this
                       one is the fp8 key with its element type narrowed to e2m1. */
} dsa_fmt;

enum { DSA_HEADS = 64, DSA_HEAD_DIM = 128, DSA_PAGE_SIZE = 64 };

typedef struct dsa_ctx dsa_ctx; /* opaque; one per device */

/* Create a context on the current CUDA device.
 *  rope_theta  RoPE base theta (> 0); frequency of pair i is theta^(-2i/128).
 *  rms_eps     RMSNorm epsilon (>= 0).
 *  max_pos     positions the store accepts are 0 .. max_pos-1 (> 0). The
 *              context holds a cos/sin table of max_pos x 64 x 8 bytes built
 *              on the host in double precision and rounded to fp32.
 *  gamma_bf16  (host) 128 bf16 RMSNorm weights, or NULL for all ones.
 * Allocates device memory (the table, gamma, a status word). Returns
 * DSA_ERR_UNSUPPORTED if the device is not compute capability 10.3. */
dsa_status dsa_ctx_create(dsa_ctx** out, float rope_theta, float rms_eps, int32_t max_pos,
                          const uint16_t* gamma_bf16);

/* Free the context's device memory. Synchronises the device first. */
dsa_status dsa_ctx_destroy(dsa_ctx* ctx);

/* Bytes per cache page for a format (16384, 8448 or 4352); 0 for an unknown format. */
size_t dsa_cache_page_bytes(dsa_fmt fmt);

/* Index-key store ([VAL], [DEC]): for each token t,
 *   y  = RMSNorm(k_raw[t]) * gamma            (fp32, eps = rms_eps)
 *   y' = RoPE(y, rope_pos[t])                 (dims i and i+64 rotated together)
 *   written to page page_table[seq_id[t]][rope_pos[t] / 64], slot rope_pos[t] % 64:
 *   bf16: round-to-nearest-even of y'; fp8: scale = max(max|y'|, 1e-4) / 448,
 *   e4m3 (round to nearest even, saturating) of y' * (1/scale), and the scale;
 *   fp4: the same with 6 for 448 and e2m1 for e4m3.
 * The fp32 operations follow one fixed order, so the stored bytes are
 * reproducible bit for bit (sum of squares: 16 sequential partials over 8
 * consecutive dims, then a pairwise tree; every product and sum of the
 * rotation rounded separately).
 *  k_raw       (device) [T][128] bf16, 16-byte aligned rows.
 *  rope_pos    (device) [T] int32: the token's position in its sequence; also
 *              its cache position. Must be in [0, min(max_pos, 64*max_pages)).
 *  seq_id      (device) [T] int32 in [0, B).
 *  page_table  (device) [B][max_pages] int32 page ids in [0, num_pages).
 *  cache       (device) num_pages * dsa_cache_page_bytes(fmt) bytes, 256-byte aligned.
 * Tokens must not share a slot within one call. Out-of-range seq/pos/page on
 * the device: the token is skipped and DSA_ERR_DEVICE_BOUNDS is recorded. */
dsa_status dsa_index_store(dsa_ctx* ctx, const void* k_raw, const int32_t* rope_pos,
                           const int32_t* seq_id, const int32_t* page_table, int32_t T,
                           int32_t B, int32_t max_pages, void* cache, int32_t num_pages,
                           dsa_fmt fmt, dsa_stream_t stream);

/* Hadamard rotation ("The Moment of Validation", section "Input Knowledge
 * Required to Understand This Message": the fused store applies a Hadamard
 * transform between RoPE and quantisation; "The Fused Kernel Decision",
 * section "Assumptions and Their Validity": queries and keys must use the
 * same order). When on, dsa_index_store writes H y' instead of y', H the
 * unnormalised 128-point Walsh-Hadamard transform in natural (Sylvester)
 * order (entries +-1, fp32 butterflies h = 1, 2, ..., 64, each pair
 * (i, i+h) -> (a + b, a - b)), and dsa_index_topk rotates every query head by
 * the same H and divides the dot products by 128, so scores keep their
 * meaning: (H q) . (H k) / 128 = q . k. The query is rotated exactly, as far
 * as the scores can tell: the fp32 rotation is carried as two bf16 terms
 * (hi + lo, 16 significant bits) for bf16 caches and three e4m3 terms (12
 * bits) for fp8 and fp4 caches, each term its own pass of the tensor cores,
 * and the queries run in tiles of two queries of one sequence (one for a
 * decode batch, one query per sequence) instead of four.
 * A cache must be written and read with the same setting. Off by default;
 * applies to the calls made after it, and changes the size
 * dsa_index_topk_workspace_size reports. */
dsa_status dsa_ctx_set_hadamard(dsa_ctx* ctx, int32_t on);

/* Slot output: when on, dsa_index_topk writes into out_idx the cache slot of
 * each selected key, page_table[b][pos / 64] * 64 + pos % 64 (the row the
 * sparse attention gathers), instead of its position pos; padding stays -1.
 * The pages feed the selected tokens to the attention ("The Crash That
 * Changed Direction", section "The Experiment: Why fp32?"); the slot is what
 * a paged gather needs. dsa_sparse_attn reads its selection by the same
 * setting: a top-k and the attention over its answer are called under one
 * setting, and a caller that changes it in between changes how the other's
 * selection is read. Off by default; applies to the calls made after it. */
dsa_status dsa_ctx_set_slot_output(dsa_ctx* ctx, int32_t on);

/* Upper bound of the workspace bytes dsa_index_topk needs for these sizes.
 * It does not grow with the context length: it holds the schedule
 * (O(Tq + B)), split-context partial lists (O(#SMs * k)) and one shared
 * threshold per query (8 bytes). The same for both cache formats: the
 * queries are turned into their tensor-core terms inside the scorer, in
 * shared memory. */
size_t dsa_index_topk_workspace_size(const dsa_ctx* ctx, int32_t Tq, int32_t B, int32_t k,
                                     dsa_fmt fmt);

/* Score + top-k ([CRA]): for each query row r of sequence b (rows
 * cu_q[b] .. cu_q[b+1]-1, position p = seq_lens[b] - n_q(b) + j for the j-th),
 *   s[r, key] = sum_h head_w[r][h] * max(0, sum_d q[r][h][d] * k[key][d])
 * over the visible keys of sequence b: positions 0..p when causal, else
 * 0..seq_lens[b]-1; k is the stored key (fp8 / fp4: e4m3 / e2m1 value times
 * its scale).
 * Output row r holds the positions (within the sequence) and fp32 scores of
 * the min(k, visible) best keys, ordered by (score desc, position asc);
 * unused slots are -1 / -inf. Products accumulate in fp32. For fp8 caches
 * the stored e4m3 keys enter the tensor cores as they are and each query row
 * (one head) as two e4m3 terms under a power-of-two scale: exact for every
 * query value of at least 2^-10 of its row's largest magnitude, smaller
 * values off by at most 2^-17 of that magnitude. fp4 caches take the same
 * path: the scorer widens each tile's e2m1 codes to e4m3 in shared memory
 * (exact: every e2m1 value is an e4m3 value), so only the bytes read from
 * memory shrink.
 *  q           (device) [Tq][64][128] bf16, 16-byte aligned.
 *  head_w      (device) [Tq][64] fp32, 16-byte aligned.
 *  cache       (device) as written by dsa_index_store, num_pages pages of fmt.
 *  page_table  (device) [B][max_pages] int32; entries past a sequence's last
 *              page are not read.
 *  seq_lens    (device) [B] int32, n_q(b) <= seq_lens[b] <= 64*max_pages.
 *  cu_q        (device) [B+1] int32, cu_q[0] = 0, non-decreasing, cu_q[B] = Tq.
 *  k           1 .. 2048 (the pages use 512 and 1024, and a downstream
 *              gather may take 2048; other k run the top-512, top-1024 or
 *              top-2048 selection and keep the first k of each sorted row;
 *              k > 1024 runs in one-query tiles, the decode kernel, whatever
 *              the batch: a 2048-key candidate buffer only fits there).
 *              B <= 16384 and Tq < 2^25, else DSA_ERR_UNSUPPORTED.
 *  out_idx     (device) [Tq][k] int32;  out_score (device) [Tq][k] fp32.
 *  workspace   (device) >= dsa_index_topk_workspace_size(...) bytes, 256-byte
 *              aligned; contents need not be initialised and are scratch.
 * Scratch memory is O(#SMs * tile) + O(Tq * k): the logits are never stored. */
dsa_status dsa_index_topk(dsa_ctx* ctx, const void* q, const float* head_w, const void* cache,
                          int32_t num_pages, dsa_fmt fmt, const int32_t* page_table,
                          int32_t max_pages, const int32_t* seq_lens, const int32_t* cu_q,
                          int32_t B, int32_t Tq, int32_t causal, int32_t k, int32_t* out_idx,
                          float* out_score, void* workspace, size_t ws_bytes,
                          dsa_stream_t stream);

/* Allocation-free top-k, for callers that cannot allocate device memory
 * (an engine whose memory is already carved into its own pools, or a
 * latency-critical path that must not call cudaMalloc). The pages have no
 * counterpart; it is an addition of this library.
 * Same arguments and results as dsa_index_topk, without the workspace: the
 * scratch is a fixed array of DSA_STATIC_WORKSPACE_BYTES in the library's
 * device image, held by every GPU that loads the library until exit. The
 * call allocates nothing. Its first call on a device looks up the array's
 * device address (cudaGetSymbolAddress); make that first call before any
 * stream capture. A device reset (cudaDeviceReset) invalidates that address:
 * the next call notices the new CUDA context and looks it up again, so make
 * it, too, outside a capture. All calls share the array: calls that overlap on the GPU
 * race. Nothing in it needs clearing; each call rewrites what must start at
 * zero. Returns DSA_ERR_WORKSPACE, without launching anything, when
 * dsa_index_topk_workspace_size(ctx, Tq, B, k, fmt) exceeds
 * DSA_STATIC_WORKSPACE_BYTES (on a 152-SM GB300 with one sequence: batches
 * up to about 1.29M queries with k <= 512 and 1.07M with 512 < k <= 1024,
 * any cache format; with the Hadamard rotation on, about 970K and 892K;
 * with k > 1024, about 549K, rotation on or off). */
#define DSA_STATIC_WORKSPACE_BYTES (32u << 20)
dsa_status dsa_index_topk_static(dsa_ctx* ctx, const void* q, const float* head_w,
                                 const void* cache, int32_t num_pages, dsa_fmt fmt,
                                 const int32_t* page_table, int32_t max_pages,
                                 const int32_t* seq_lens, const int32_t* cu_q, int32_t B,
                                 int32_t Tq, int32_t causal, int32_t k, int32_t* out_idx,
                                 float* out_score, dsa_stream_t stream);

/* ---------------------------------------------------------------- attention
 * What follows the indexer in a serving step: rotating the queries, the main
 * K/V cache, and attention over it, for all keys or for the selected ones.
 * These calls keep the conventions above; element strides are in elements,
 * the innermost dimension is contiguous. */

/* A rotary plan: the cos/sin table of one set of rotary parameters. The
 * rotated part of a head has rot_dim dimensions; pair i of it is (i, i +
 * rot_dim/2) in the half layout, (2i, 2i+1) in the interleaved one, and turns
 * by position * f_i, f_i = theta^(-2i/rot_dim), scaled for long contexts:
 *  DSA_ROPE_LINEAR    f_i / factor
 *  DSA_ROPE_BY_PARTS  with turns r_i = orig_max_pos f_i / (2 pi) and
 *                     g = clamp((r_i - beta_slow) / (beta_fast - beta_slow), 0, 1):
 *                     f_i / factor * (1 - g) + f_i * g
 * Every cos and sin is multiplied by mscale (1 leaves lengths as they are).
 * Angles are computed in double, cos and sin rounded once to fp32. */
typedef enum { DSA_ROPE_HALF = 0, DSA_ROPE_INTERLEAVED = 1 } dsa_rope_layout;
typedef enum { DSA_ROPE_PLAIN = 0, DSA_ROPE_LINEAR = 1, DSA_ROPE_BY_PARTS = 2 } dsa_rope_scaling;
typedef enum { DSA_BF16 = 0, DSA_F16 = 1, DSA_F32 = 2 } dsa_dtype;
typedef struct {
  double theta;         /* > 0 */
  int32_t rot_dim;      /* even, 2 .. 1024 */
  int32_t max_pos;      /* positions 0 .. max_pos-1; the table takes max_pos * rot_dim * 4 bytes */
  int32_t layout;       /* dsa_rope_layout */
  int32_t scaling;      /* dsa_rope_scaling */
  double factor;        /* LINEAR, BY_PARTS: > 0 */
  double orig_max_pos;  /* BY_PARTS: > 0 */
  double beta_slow;     /* BY_PARTS: < beta_fast */
  double beta_fast;
  double mscale;        /* > 0 */
} dsa_rope_desc;
typedef struct dsa_rope dsa_rope;

/* Allocates the table on the context's device and fills it; synchronises, so
 * not during a stream capture. dsa_rope_destroy synchronises the device. */
dsa_status dsa_rope_create(dsa_ctx* ctx, dsa_rope** out, const dsa_rope_desc* desc);
dsa_status dsa_rope_destroy(dsa_rope* rope);

/* y[t][h] = x[t][h] with dimensions rot_start .. rot_start + rot_dim - 1
 * rotated to position pos[t] and the others copied; `inverse` turns the other
 * way, which is also the gradient with respect to x of a forward rotation.
 * fp32 arithmetic, every product and sum rounded separately, one rounding to
 * the type.
 *  x, y   (device) [T][H][D] of dtype, any strides of tokens and heads. y == x
 *         with the same strides rotates in place; otherwise they must not overlap.
 *         Rows of y that share elements are refused (those of x may, unless in
 *         place).
 *  pos    (device) [T] int32. A token whose position is out of range is not
 *         written and DSA_ERR_DEVICE_BOUNDS is recorded.
 * Any D, H and alignment of the type's own size; 16-byte aligned rows and
 * parts run 16 bytes at a time. */
dsa_status dsa_rope_apply(dsa_ctx* ctx, const dsa_rope* rope, const void* x, void* y, dsa_dtype dtype,
                          const int32_t* pos, int32_t T, int32_t H, int32_t D, int32_t rot_start,
                          int64_t x_stride_t, int64_t x_stride_h, int64_t y_stride_t,
                          int64_t y_stride_h, int32_t inverse, dsa_stream_t stream);

/* The K/V cache: pages of 64 tokens like the index cache (a page table can
 * serve both), for kv_heads heads of head_dim 64 or 128. A page is kv_heads
 * blocks of
 *   K codes [64][CB], V codes [64][CB], K scales [64][SB], V scales [64][SB]
 *   DSA_FMT_BF16  CB = 2 head_dim, SB = 0
 *   DSA_FMT_FP8   CB = head_dim (e4m3), SB = head_dim / 32
 *   DSA_FMT_FP4   CB = head_dim / 2 (e2m1, the even dimension in the low
 *                 nibble), SB = head_dim / 32
 * In fp8 and fp4, 32 dimensions share the power of two 2^e, stored as the
 * byte e + 127: e is the smallest integer with max|y| <= 448 * 2^e (fp8) or
 * 6 * 2^e (fp4), within -117 .. 119 or -125 .. 125, so a stored value is a
 * bf16 number exactly and a code saturates only beyond 448 * 2^119 (2.98e38)
 * or 6 * 2^125 (2.55e38) (OCP microscaling layouts with the exponent rounded
 * up). 32 dimensions of which one is not finite get the
 * byte 255 and read as NaN. Not the index cache's scales: those are one fp32
 * per token. Returns 0 for unsupported arguments. */
size_t dsa_kv_page_bytes(int32_t kv_heads, int32_t head_dim, dsa_fmt fmt);

/* Write tokens: k (rotated first, when rope is given) and v to slot
 * cache_pos % 64 of page page_table[seq_id][cache_pos / 64], rounded to
 * nearest even once, from fp32.
 *  k, v        (device) [T][kv_heads][head_dim] bf16, 16-byte aligned, strides
 *              multiples of 8 elements.
 *  cache_pos   (device) [T] int32: the token's place in its sequence's pages.
 *  rope_pos    (device) [T] int32 rotary positions, or NULL for cache_pos
 *              (drafted tokens of a tree lie one after another in the cache
 *              but their positions follow their depth).
 *  rope        rotates dimensions rot_start .. of k; NULL for none.
 *  cache       (device) num_pages * dsa_kv_page_bytes bytes, 256-byte aligned.
 * Tokens must not share a slot within one call. A token whose sequence,
 * place, page or rotary position is out of range is skipped and
 * DSA_ERR_DEVICE_BOUNDS recorded. */
dsa_status dsa_kv_store(dsa_ctx* ctx, const void* k, const void* v, int64_t k_stride_t, int64_t k_stride_h,
                        int64_t v_stride_t, int64_t v_stride_h, const int32_t* cache_pos,
                        const int32_t* seq_id, const int32_t* page_table, int32_t T, int32_t B,
                        int32_t max_pages, int32_t kv_heads, int32_t head_dim, void* cache,
                        int32_t num_pages, dsa_fmt fmt, const dsa_rope* rope, const int32_t* rope_pos,
                        int32_t rot_start, dsa_stream_t stream);

/* Read tokens back as bf16 (exact: the values the cache stands for) into k
 * and v, laid out and aligned as dsa_kv_store's; rows that share elements are
 * refused, and k and v must not overlap. A token whose sequence,
 * place or page is out of range reads as zeros, and DSA_ERR_DEVICE_BOUNDS is
 * recorded. */
dsa_status dsa_kv_load(dsa_ctx* ctx, const void* cache, int32_t num_pages, dsa_fmt fmt, int32_t kv_heads,
                       int32_t head_dim, const int32_t* cache_pos, const int32_t* seq_id,
                       const int32_t* page_table, int32_t T, int32_t B, int32_t max_pages, void* k,
                       void* v, int64_t k_stride_t, int64_t k_stride_h, int64_t v_stride_t,
                       int64_t v_stride_h, dsa_stream_t stream);

/* Arguments of the attention calls. Rows cu_q[b] .. cu_q[b+1]-1 of q are the
 * n_b query tokens of sequence b, whose own keys and values are the last n_b
 * of its seq_lens[b] cache places (written before the call); the others are
 * its committed context. Query head h reads kv head h / (heads / kv_heads). */
typedef struct {
  const void* q;            /* (device) [Tq][heads][head_dim] bf16, 16-byte aligned */
  int64_t q_stride_t, q_stride_h;      /* multiples of 8 */
  void* out;                /* (device) [Tq][heads][head_dim] bf16, 16-byte aligned */
  int64_t out_stride_t, out_stride_h;  /* multiples of 8; no two rows may share elements */
  float* lse;               /* (device) [Tq][heads] log of the sum of exp(score), or NULL */
  const void* cache;        /* (device) as written by dsa_kv_store, 256-byte aligned */
  int32_t num_pages;
  dsa_fmt fmt;
  int32_t heads, kv_heads, head_dim;
  const int32_t* page_table;  /* (device) [B][max_pages] */
  int32_t max_pages;
  const int32_t* seq_lens;    /* (device) [B], n_b <= seq_lens[b] <= 64 * max_pages */
  const int32_t* cu_q;        /* (device) [B+1], cu_q[0] = 0, non-decreasing, cu_q[B] = Tq */
  int32_t B, Tq;
  const uint32_t* mask;       /* (device) [Tq][mask_words] bits, or NULL */
  int32_t mask_words;
  double scale;               /* of q.k, > 0 */
  void* workspace;            /* (device) >= dsa_attn_workspace_size bytes, 256-byte aligned, scratch */
  size_t ws_bytes;
} dsa_attn_args;

/* Workspace of both calls: two partial results of up to 256 rows per SM,
 * whatever the sizes of the call (40 MB for head_dim 128 on 152 SMs). 0 for an unsupported head_dim. */
size_t dsa_attn_workspace_size(const dsa_ctx* ctx, int32_t head_dim);

/* Attention of drafted tokens over the cache: query i of sequence b sees the
 * whole committed context and the drafted token j of its own sequence where
 * bit j of its mask row is set (usually its ancestors in the tree and
 * itself; bits past mask_words count as clear), or where j <= i without a
 * mask (a chain: a chunk of a prefill; one token: a decode step). out = softmax(scale q.k) v; a row that sees no key
 * gives zeros and lse -inf. What the cache holds in places a row does not see
 * does not reach it, infinities and NaN included. Keys of a page out of range
 * are left out and DSA_ERR_DEVICE_BOUNDS recorded; so are whole sequences
 * whose lengths are inconsistent (their rows are not written).
 * A row all of whose visible scores are -inf counts as one that sees no key.
 * Sums over the keys are fp32, taken before the division by the weights' sum
 * with weights of up to 2^8: they stay finite where the visible |v| add up to
 * less than 2^119.
 * Tq * heads < 2^31, kv_heads <= 65536, 64 * num_pages < 2^31 and, in bf16,
 * 128 * num_pages * kv_heads < 2^31, else DSA_ERR_UNSUPPORTED. Results do not
 * depend on timing. */
dsa_status dsa_tree_attn(dsa_ctx* ctx, const dsa_attn_args* args, dsa_stream_t stream);

/* Attention over a selection: query row t sees the keys sel[t][0 .. k-1] of
 * its sequence (as dsa_index_topk writes them: positions, or cache slots when
 * slot output is on; negative entries are skipped), and, with a mask, the
 * drafted tokens whose bits are set. An entry out of range (a position at or
 * past seq_lens[b], a slot past the cache) is left out and
 * DSA_ERR_DEVICE_BOUNDS recorded; a key listed twice counts twice. Otherwise
 * as dsa_tree_attn (a query of an inconsistent sequence gives zeros).
 *  sel  (device) [Tq][k] int32, 1 <= k <= 65536.  heads / kv_heads <= 128. */
dsa_status dsa_sparse_attn(dsa_ctx* ctx, const dsa_attn_args* args, const int32_t* sel, int32_t k,
                           dsa_stream_t stream);

/* Kernel timing, for benchmarks and profiling. While enabled, the library
 * records a CUDA event pair on the launch stream around each kernel it
 * launches (at most 8192 pairs between reads; later launches are counted but
 * not timed). Reading synchronises the device, writes per-kind total
 * milliseconds and launch counts since the previous read (launches are
 * counted whether or not timing is on), and resets both, those of kinds that
 * are not asked for too. dsa_profile_read_kinds writes `kinds` (>= 1) entries,
 * zeros past the last kind there is. dsa_profile_read writes the indexer's
 * DSA_K_COUNT, a number that stays: programs have arrays of that length. */
typedef enum {
  DSA_K_STORE = 0,      /* dsa_index_store */
  DSA_K_PLAN = 1,       /* dsa_index_topk: schedule */
  DSA_K_SCORE_BF16 = 2, /* dsa_index_topk: tensor-core scorer + running top-k, bf16 cache */
  DSA_K_SCORE_FP8 = 3,  /* the same, fp8 cache */
  DSA_K_SCORE_FP4 = 4,  /* the same, fp4 cache */
  DSA_K_COUNT = 5,      /* kinds that dsa_profile_read reports */
  DSA_K_ROPE = 5,       /* dsa_rope_apply */
  DSA_K_KV_STORE = 6,   /* dsa_kv_store */
  DSA_K_KV_LOAD = 7,    /* dsa_kv_load */
  DSA_K_ATTN = 8,       /* dsa_tree_attn, dsa_sparse_attn: the attention */
  DSA_K_ATTN_JOIN = 9,  /* the same: joining units that were divided */
  DSA_K_ALL = 10        /* kinds there are */
} dsa_kernel_kind;
dsa_status dsa_profile_enable(dsa_ctx* ctx, int on);
dsa_status dsa_profile_read(dsa_ctx* ctx, float* ms /* [DSA_K_COUNT] */,
                            int32_t* launches /* [DSA_K_COUNT] */);
dsa_status dsa_profile_read_kinds(dsa_ctx* ctx, float* ms /* [kinds] */, int32_t* launches /* [kinds] */,
                                  int32_t kinds);

/* Synchronise `stream`, then read and clear the context's device status
 * word. Returns DSA_OK or the first device-side error recorded. */
dsa_status dsa_get_device_status(dsa_ctx* ctx, dsa_stream_t stream);

/* Failure-detection self-test: enqueues a one-CTA kernel that waits, with
 * the scorer's bounded mbarrier wait, on a barrier nothing ever signals;
 * after about a millisecond the wait gives up, DSA_ERR_TIMEOUT is recorded
 * in the status word (read it with dsa_get_device_status) and the kernel
 * returns, leaving the context usable. Exercises the error path of a stalled
 * pipeline without faulting or hanging the GPU. */
dsa_status dsa_selftest_bounded_wait(dsa_ctx* ctx, dsa_stream_t stream);

/* Static string for a status code. */
const char* dsa_status_str(dsa_status s);

#ifdef __cplusplus
}
#endif
#endif /* DSAIDX_H */
