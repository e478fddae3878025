/*
 * ua.h -- C ABI of libua.so: unified paged, variable-length GQA attention for
 * NVIDIA GB300 (sm_103a).
 *
 * One call computes attention for a batch of sequences whose keys and values sit
 * in a paged cache indexed by a block table ("RocKE unified_attention parity &
 * benchmark harness", gfx950 README, "Running" step 1: paged KV cache, block
 * tables, cumulative query lengths, optional sliding window, softcap, sinks, ALiBi
 * slopes, QQ-bias).  The library chooses between two execution paths ("2D": one
 * CTA per q-block x kv-head walks every key; "split": the key range is cut into
 * partitions whose max / sum / partial output are merged, as in the aiter PR #3962
 * "split-K long-context decode for shuffled fp8 SWA", "Changes" -- inside the
 * thread-block cluster of a decode slot's partitions, or by a second kernel).
 *
 * Semantics, for sequence b with q_len = cu_seqlens_q[b+1] - cu_seqlens_q[b],
 * kv_len = seq_lens_k[b] and ctx = kv_len - q_len, query row i (0 <= i < q_len)
 * of head h at position p = ctx + i, kv-head g = h / (num_q_heads / num_kv_heads):
 *   allowed keys   0 <= j < kv_len, j <= p, and p - j <= window_left if window_left >= 0
 *   s_j  = scale * q . K_j                 (fp8 cache: K_j = e4m3 * k_scale)
 *   s_j  = softcap * tanh(s_j / softcap)   if softcap > 0
 *   s_j += alibi_slopes[h] * (j - ctx)     if alibi_slopes != NULL
 *   s_j += qq_bias[i * qq_bias_stride + (j - ctx)]  if qq_bias != NULL and j >= ctx
 *   out  = sum_j e^{s_j} V_j / (e^{sinks[h]} (if sinks != NULL) + sum_j e^{s_j})
 *                                      (fp8 cache: V_j = e4m3 * v_scale; per-token
 *                                       scales, when given, replace k_scale / v_scale
 *                                       key by key, and per-block scales block by block,
 *                                       of e4m3 or int8 codes: see ua_shape_t)
 * A row with no allowed key (possible only when kv_len < q_len, e.g. a decode slot
 * with kv_len 0) is written as 0.
 *
 * Layouts (all contiguous, row-major, device memory owned by the caller):
 *   q            [total_q, num_q_heads, head_dim]               q_dtype (F16 or BF16)
 *   k_cache      [num_blocks, block_size, num_kv_heads, head_dim] kv_dtype
 *   v_cache      same shape and type as k_cache
 *   out          [total_q, num_q_heads, head_dim]               out_dtype (F16, BF16, F32)
 *   cu_seqlens_q [num_seqs + 1] int32, non-decreasing, cu_seqlens_q[0] = 0
 *   seq_lens_k   [num_seqs] int32
 *   block_table  [num_seqs, max_blocks_per_seq] int32 physical block ids
 *   alibi_slopes [num_q_heads] float32, sinks [num_q_heads] float32
 *   qq_bias      float32 rows of qq_bias_stride elements, at least max_seqlen_q rows;
 *                qq_bias_stride >= max_seqlen_q
 *   kv_scale     float32[2] = {k_scale, v_scale}; required for the fp8 cache only
 *
 * Conventions: every call is asynchronous on `stream` (a cudaStream_t; NULL is the
 * legacy default stream) and never synchronises; the library keeps no pointer to
 * caller memory after the call returns.  Errors are returned as ua_status_t and no
 * C++ exception crosses the ABI.  Per device, the library keeps what it looks up once
 * (the SM count, the device address of its status word, recently encoded tensor maps of
 * the caller's buffers, keyed by address and layout); none of it survives cudaDeviceReset,
 * after which the library must not be called on that device again.
 * Block ids outside [0, num_blocks) are not read:
 * the kernel treats the key as zero and raises UA_ERR_DEVICE_CHECK in the device
 * status word (see ua_device_status).
 */
#ifndef UA_H_
#define UA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define UA_VERSION 100

/* Size of the fixed device scratch array used by ua_unified_attention_noalloc. */
#define UA_NOALLOC_SCRATCH_BYTES (16u << 20)

typedef enum {
  UA_OK = 0,
  UA_ERR_INVALID_ARG = 1,  /* a size, pointer, alignment or enum value is not accepted */
  UA_ERR_UNSUPPORTED = 2,  /* a valid combination this build has no kernel for */
  UA_ERR_CUDA = 3,         /* a CUDA runtime call failed (launch, allocation, query) */
  UA_ERR_WORKSPACE = 4,    /* the caller's workspace is smaller than ua_plan() asks */
  UA_ERR_DEVICE_CHECK = 5, /* a kernel saw a block id outside [0, num_blocks), or ua_append_kv a
                              position outside the rotation table */
  UA_ERR_TIMEOUT = 6,      /* a kernel gave up waiting on its own copy pipeline */
  UA_ERR_SCRATCH_LIMIT = 7 /* ua_unified_attention_noalloc: the call needs more scratch than
                              its fixed UA_NOALLOC_SCRATCH_BYTES */
} ua_status_t;

typedef enum {
  UA_DT_F16 = 0,
  UA_DT_BF16 = 1,
  UA_DT_F8E4M3 = 2,
  UA_DT_F32 = 3,
  UA_DT_I8 = 4 /* caches only: signed codes -127 .. 127 with a scale per block and kv-head */
} ua_dtype_t;

typedef enum {
  UA_BACKEND_AUTO = 0,  /* dispatcher picks from grid fill and key-walk length */
  UA_BACKEND_2D = 1,    /* force one pass per q-block x kv-head */
  UA_BACKEND_SPLIT = 2  /* force the split-KV partition + merge path */
} ua_backend_t;

typedef enum { UA_PATH_2D = 1, UA_PATH_SPLIT = 2 } ua_path_t;

/* Host-side sizes of one call (host ints, so the library never reads device data
 * to size its grids), plus optional caller workspace and profiling events. */
typedef struct {
  int32_t num_seqs;
  int32_t total_q;            /* = cu_seqlens_q[num_seqs] */
  int32_t max_seqlen_q;       /* >= every q_len */
  int32_t max_seqlen_k;       /* >= every kv_len */
  int32_t max_blocks_per_seq; /* row length of block_table */
  int32_t num_blocks;         /* physical blocks in each cache */
  int32_t qq_bias_stride;     /* elements per qq_bias row (ignored without qq_bias) */
  int32_t q_dtype;            /* ua_dtype_t: F16 or BF16 */
  int32_t out_dtype;          /* ua_dtype_t: F16, BF16 or F32 */
  int32_t num_splits;         /* 0: the dispatcher decides; > 0: partitions for the split path */
  void* workspace;            /* device scratch for the split path, or NULL: the library keeps
                                 a grow-only buffer per (device, stream), and one for each
                                 capture on a stream, and never frees them (nor a replaced one)
                                 while the process lives */
  size_t workspace_bytes;     /* bytes at `workspace` */
  void* events;               /* NULL, or cudaEvent_t[3] recorded on `stream` before the
                                 attention kernel, after it, and after the merge kernel */
  /* fp8 caches: per-token scales (aiter PR #3962 "split-K long-context decode for shuffled
   * fp8 SWA", test matrix: per-token scales, K and V scales with different strides), or
   * NULL for the per-tensor kv_scale.  Device float32 arrays over (block, slot, kv-head):
   * the scale of key slot s of physical block b, kv-head g, is
   * k_scale_tok[b * k_scale_stride[0] + s * k_scale_stride[1] + g * k_scale_stride[2]]
   * (strides in elements, each >= 0); V likewise with its own strides.  Both or neither;
   * ignored for fp16 / bf16 caches.  Read by the decode tile (at most 8 rows per kv-head,
   * head_dim <= 128, 16 | block_size); other calls with them return UA_ERR_UNSUPPORTED.
   * Every scale a call reads must be finite, and V scales below 256 (a key's P times its V
   * scale is an f16 MMA operand). */
  const float* k_scale_tok;
  const float* v_scale_tok;
  int64_t k_scale_stride[3];
  int64_t v_scale_stride[3];
  /* e4m3 or int8 caches: a scale for each block and kv-head, as ua_append_kv writes them, or
   * NULL.  Device float32 arrays over (block, kv-head): the scale of physical block b, kv-head
   * g, is k_scale_blk[b * k_scale_blk_stride[0] + g * k_scale_blk_stride[1]] (strides in
   * elements, each >= 0); V likewise.  Both or neither, and not together with the per-token
   * scales; an int8 cache needs them.  Every kernel reads them (any head_dim, block_size and
   * batch shape).  Values are taken within [2^-40, 2^40]. */
  const float* k_scale_blk;
  const float* v_scale_blk;
  int64_t k_scale_blk_stride[2];
  int64_t v_scale_blk_stride[2];
} ua_shape_t;

/* What the dispatcher chose for a call (see ua_plan). */
typedef struct {
  int32_t path;        /* ua_path_t */
  int32_t kernel;      /* 1: warp-MMA tile kernel, 16 rows per CTA (decode-shaped q-blocks);
                          2: key-major decode tile, 8 rows per CTA (decode with at most 8
                          rows per kv-head, head_dim <= 128, 16 | block_size);
                          4: warp-MMA tile kernel, 64 rows per CTA (fp8 caches at head_dim
                          256, block sizes not a multiple of 16); 8: tensor-memory
                          (tcgen05) kernel with 128-row q-blocks of floor(128 / G) tokens x
                          G heads (16-bit caches, or fp8 at head_dim <= 128: codes dequantised
                          to f16 in shared memory as in RocKE "fp8 KV cache", a bf16 q
                          taken as f16); 16: the same
                          kernel with two such tiles of consecutive tokens per CTA; 32: the
                          key-major decode tile of code 2 with eight consumer warps (128-key
                          stages, one CTA per SM), for decode grids of at most one CTA per SM;
                          64: the decode tile of code 2 with two kv-heads per CTA (fp8 caches
                          with per-tensor scales, or caches with per-block ones, at most 4
                          rows per kv-head, an even num_kv_heads): one page box carries both
                          heads' rows; 128: the decode tile of code 2 or 64 for caches with
                          per-block scales, a CTA walking an even share of all sequences'
                          keys: grid_x ranges, and n_part the most partitions of one row */
  int32_t block_m;     /* (query token x head) rows per q-block */
  int32_t n_part;      /* key-range partitions (1 on the 2D path) */
  int32_t grid_x;      /* q-block slots: num_seqs when slot_per_seq, else
                          floor(total_q * G / block_m) + num_seqs */
  int32_t grid_y;      /* num_kv_heads (num_kv_heads / 2 for kernel 64) */
  int32_t grid_z;      /* n_part */
  int32_t num_sms;     /* SM count the plan was made for */
  int32_t cluster_y;   /* CTAs of one q-block slot (different kv-heads) launched as a cluster */
  int32_t cluster_z;   /* > 1: the n_part partitions of a slot are one cluster too (cluster
                          cluster_y x cluster_z, at most 16 CTAs) and merge through
                          distributed shared memory, with no merge kernel and no workspace */
  int32_t slot_per_seq; /* 1: every sequence fits one q-block and grid slot x is sequence x */
  size_t workspace_bytes; /* scratch the split path needs (0 on the 2D path) */
} ua_plan_t;

/*
 * ua_unified_attention -- the attention call described at the top of this file.
 *
 * scale         multiplies q . k (usually 1 / sqrt(head_dim))
 * softcap       > 0 enables s -> softcap * tanh(s / softcap); <= 0 disables it
 * window_left   >= 0: a query at position p sees keys p - window_left .. p
 *               (a window of W keys including the query itself is W - 1); < 0: off
 * alibi_slopes, qq_bias, sinks: device float32 arrays, or NULL to disable
 * kv_dtype      ua_dtype_t of both caches: F16, BF16 (q_dtype must match), F8E4M3
 *               (OCP e4m3fn) or I8 (both: q may be F16 or BF16, |q| < 65504)
 * kv_scale      device float32[2] {k_scale, v_scale}, required with F8E4M3 unless the shape
 *               gives per-token or per-block scales
 * backend       ua_backend_t
 * stream        cudaStream_t to launch on
 * shape         host-side sizes (must not be NULL)
 *
 * Returns UA_OK after the kernels are enqueued.  UA_ERR_INVALID_ARG for: a NULL
 * required pointer or shape; a tensor pointer not 16-byte aligned; num_q_heads not
 * a positive multiple of num_kv_heads; head_dim not 64, 128 or 256; block_size < 1;
 * negative sizes; qq_bias with qq_bias_stride < max_seqlen_q; an unknown enum.
 * UA_ERR_UNSUPPORTED for q_dtype != kv_dtype with a 16-bit cache.  UA_ERR_WORKSPACE
 * when `shape->workspace` is given but smaller than the plan needs.  UA_ERR_CUDA
 * when a launch or allocation fails.
 */
int ua_unified_attention(const void* q, const void* k_cache, const void* v_cache, void* out,
                         const int32_t* cu_seqlens_q, const int32_t* seq_lens_k,
                         const int32_t* block_table, int block_size, int num_q_heads,
                         int num_kv_heads, int head_dim, float scale, float softcap,
                         int window_left, const float* alibi_slopes, const float* qq_bias,
                         const float* sinks, int kv_dtype, const float* kv_scale, int backend,
                         void* stream, const ua_shape_t* shape);

/*
 * ua_unified_attention_call -- the same call with its arguments in one struct, for bindings that
 * pay for every argument and make one call again and again (Python's ctypes takes 2.0 us for the
 * 22 arguments above and 0.4 us for two).  NULL: UA_ERR_INVALID_ARG.
 */
typedef struct {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  void* out;
  const int32_t* cu_seqlens_q;
  const int32_t* seq_lens_k;
  const int32_t* block_table;
  const float* alibi_slopes;
  const float* qq_bias;
  const float* sinks;
  const float* kv_scale;
  const ua_shape_t* shape;
  int32_t block_size;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  float scale;
  float softcap;
  int32_t window_left;
  int32_t kv_dtype;
  int32_t backend;
} ua_attention_t;
int ua_unified_attention_call(const ua_attention_t* call, void* stream);

/*
 * ua_unified_attention_noalloc -- ua_unified_attention for callers that may not
 * allocate device memory (the pages have no counterpart: this is a library service).
 *
 * Some callers cannot call cudaMalloc: a serving runtime that gives all free device
 * memory to its own cache pool at start-up, a process held to a fixed memory budget,
 * or a latency-critical loop where an allocation (which can block and synchronise the
 * device) is not allowed.  ua_unified_attention allocates only when the split-KV path
 * runs without a caller workspace; this entry point runs the same kernels but keeps the
 * split path's scratch in one fixed device array of UA_NOALLOC_SCRATCH_BYTES that the
 * library holds on every GPU that loads it, until the process exits.  It never calls
 * cudaMalloc or cudaFree.
 *
 * Arguments and results are those of ua_unified_attention, except that
 * shape->workspace is ignored.  Extra behaviour:
 *   - UA_ERR_SCRATCH_LIMIT, before anything is launched, when the plan needs more than
 *     UA_NOALLOC_SCRATCH_BYTES of scratch (ua_plan reports workspace_bytes).
 *   - The first call on a device looks up the array's device address (with that device
 *     current); make that first call before any stream capture on the device.  The
 *     address is kept until the process exits and does not survive cudaDeviceReset:
 *     after a reset of the device, do not call this entry point again.
 *   - Every call on a device shares the one array: calls whose kernels overlap on the
 *     GPU (different streams, or several host threads) race on it and give wrong
 *     results.  Calls on one stream are ordered and safe.  The array keeps the last
 *     call's contents; nothing in it needs to start at zero.
 */
int ua_unified_attention_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                 void* out, const int32_t* cu_seqlens_q,
                                 const int32_t* seq_lens_k, const int32_t* block_table,
                                 int block_size, int num_q_heads, int num_kv_heads, int head_dim,
                                 float scale, float softcap, int window_left,
                                 const float* alibi_slopes, const float* qq_bias,
                                 const float* sinks, int kv_dtype, const float* kv_scale,
                                 int backend, void* stream, const ua_shape_t* shape);

/*
 * One ua_append_kv call: what to write, where, and how it is rotated.  Sizes are host ints;
 * tensors are device memory.  Strides are in elements.
 */
typedef struct {
  const void* k;       /* [total_q, num_kv_heads, head_dim] of `dtype`, strides k_stride */
  const void* v;       /* likewise, v_stride */
  const void* q;       /* [total_q, num_q_heads, head_dim] to rotate, or NULL */
  void* q_out;         /* the rotated queries, q_out_stride: q itself, or memory that overlaps
                          none of q, k and v */
  void* k_cache;       /* [num_blocks, block_size, num_kv_heads, head_dim] kv_dtype, contiguous */
  void* v_cache;
  const int32_t* cu_seqlens_q;  /* [num_seqs + 1] */
  const int32_t* seq_lens_k;    /* [num_seqs]: lengths with the new tokens */
  const int32_t* block_table;   /* [num_seqs, max_blocks_per_seq] */
  const float* cos_sin;         /* [max_position, rot_dim]: a row's rot_dim / 2 cosines, then its
                                   sines; 16-byte aligned; NULL: no rotation (rot_dim 0) */
  const int32_t* positions;     /* [n_axes][total_q], or NULL: a token's place in the cache */
  const float* kv_scale;        /* e4m3 cache, per tensor: {k_scale, v_scale} */
  float* k_scale_tok;           /* e4m3 cache, per token: written at (block, slot, kv-head) */
  float* v_scale_tok;
  float* k_scale_blk;           /* e4m3 or int8 cache, per block: updated at (block, kv-head) */
  float* v_scale_blk;
  int64_t q_stride[2];          /* token, head: multiples of 8; the head dim has stride 1 */
  int64_t k_stride[2];
  int64_t v_stride[2];
  int64_t q_out_stride[2];
  int64_t k_scale_tok_stride[3];
  int64_t v_scale_tok_stride[3];
  int64_t k_scale_blk_stride[2];
  int64_t v_scale_blk_stride[2];
  int64_t positions_stride;     /* from one axis' positions to the next's */
  int32_t num_seqs;
  int32_t total_q;
  int32_t max_seqlen_q;         /* >= every q_len */
  int32_t max_blocks_per_seq;
  int32_t num_blocks;
  int32_t block_size;
  int32_t num_q_heads;          /* 0 without q */
  int32_t num_kv_heads;
  int32_t head_dim;             /* 64, 128 or 256 */
  int32_t dtype;                /* of q, k, v and q_out: F16 or BF16 */
  int32_t kv_dtype;             /* of the caches: `dtype`, F8E4M3 or I8 */
  int32_t rot_dim;              /* rotated elements at a head's front: a multiple of 16, 0 .. head_dim */
  int32_t max_position;         /* rows of cos_sin */
  int32_t interleaved;          /* pairs: 0: (f, f + rot_dim / 2); 1: (2 f, 2 f + 1) */
  int32_t n_axes;               /* 1 .. 4 (1 without positions) */
  const uint8_t* axis_of;       /* n_axes > 1: host array [rot_dim / 2], the axis of each frequency */
} ua_append_t;

/*
 * ua_append_kv -- appends the batch's new keys and values to the paged cache, the keys rotated
 * by their position on the way, and rotates the queries beside them, in one launch.  (The
 * pages describe the cache that ua_unified_attention reads; this call writes it.)
 *
 * Token i of sequence b goes to cache position seq_lens_k[b] - q_len + i; its slot follows
 * from the block table, as ua_unified_attention reads it.  With cos_sin, pair f = 0 ..
 * rot_dim / 2 - 1 of each q and k head turns by the angle in row positions[axis_of[f]][token]
 * (or, without positions, the cache position):
 *   a' = a cos - b sin,  b' = b cos + a sin      fp32, every product and sum rounded on its own
 * and elements from rot_dim on pass through.  What is stored, with x the fp32 value:
 *   16-bit cache        x rounded once
 *   e4m3, kv_scale      rne(x * (1 / scale)), saturating at 448
 *   e4m3, *_scale_tok   scale = amax * (1 / 448) of the token's head, within [2^-40, 2^40];
 *                       written beside the codes
 *   *_scale_blk         one scale for each block and kv-head, qmax 448 (e4m3) or 127 (int8):
 *                       s = amax over the block's new tokens * (1 / qmax), within [2^-40,
 *                       2^40], or the block's present scale if it holds tokens of the sequence
 *                       already and that is larger.  New codes are rne(x * (1 / s)); codes
 *                       held already become rne(code * (present / s)) when s grew.
 * Slots past the new tokens, and blocks that no new token reaches, keep what they hold (a
 * block's slots past kv_len too).  Values must be finite where a scale is computed.  A block
 * reached by two sequences of one call, or twice by one, is the caller's error.
 *
 * A token whose cache position is negative (kv_len < q_len) is skipped, as are rows of k, v
 * and q past cu_seqlens_q[num_seqs], and a sequence's tokens from total_q on.  A block id
 * outside [0, num_blocks) or past the table's row is not written; a position outside [0,
 * max_position) skips its token, queries included; both raise UA_ERR_DEVICE_CHECK in the
 * device status word.
 *
 * Asynchronous on `stream`, capturable, no workspace, no allocation.  Returns UA_OK or
 * UA_ERR_INVALID_ARG (a missing or misaligned pointer, a size, stride or enum value that is
 * not accepted, strides by which q_out or a scale array overlaps itself, scales that do not fit
 * the cache's type), UA_ERR_UNSUPPORTED (a 16-bit cache
 * of another type than k and v), UA_ERR_CUDA.
 */
int ua_append_kv(const ua_append_t* call, void* stream);

/*
 * Latent caches: one vector a token, shared by all heads, instead of keys and values a kv-head
 * (the pages have no counterpart).  Row t of a cache [num_blocks, block_size, latent_dim +
 * rope_dim] is [c_t | r_t]: c_t, the normalised latent, is a key and a value at once; r_t, the
 * rotated rope key, is a part of the key only.  latent_dim is 128, 256 or 512, rope_dim a multiple
 * of 16 up to 64, elements are F16 or BF16.  Caches, block tables, lengths and the device status
 * word are used as by ua_unified_attention; every call below is asynchronous on `stream`,
 * capturable, and returns a ua_status_t.
 */

/* One ua_append_latent call.  Strides are in elements; the last dim of each tensor has stride 1. */
typedef struct {
  const void* latent;           /* [total_q, latent_dim] of `dtype`, row stride latent_stride */
  const void* k_rope;           /* [total_q, rope_dim], k_rope_stride */
  const void* q_rope;           /* [total_q, num_heads, rope_dim] to rotate, or NULL */
  void* q_rope_out;             /* the rotated queries: q_rope itself (with its strides), or memory
                                   that overlaps none of the inputs */
  void* cache;                  /* [num_blocks, block_size, latent_dim + rope_dim], contiguous */
  const int32_t* cu_seqlens_q;  /* [num_seqs + 1] */
  const int32_t* seq_lens_k;    /* [num_seqs]: lengths with the new tokens */
  const int32_t* block_table;   /* [num_seqs, max_blocks_per_seq] */
  const void* norm_weight;      /* [latent_dim] of norm_dtype, 16-byte aligned (as latent, k_rope,
                                   q_rope, q_rope_out and cache), or NULL: latents are stored as
                                   they are */
  const float* cos_sin;         /* [max_position, rope_dim]: a row's rope_dim / 2 cosines, then its
                                   sines; 16-byte aligned; NULL: no rotation */
  const int32_t* positions;     /* [total_q], or NULL: a token's place in the cache */
  int64_t latent_stride;        /* token strides and q_rope's head strides: multiples of 8 (any
                                   where there is one token, or one head) */
  int64_t k_rope_stride;
  int64_t q_rope_stride[2];     /* token, head */
  int64_t q_rope_out_stride[2];
  int32_t num_seqs;
  int32_t total_q;
  int32_t max_blocks_per_seq;
  int32_t num_blocks;
  int32_t block_size;
  int32_t num_heads;            /* of q_rope; 0 without it */
  int32_t latent_dim;
  int32_t rope_dim;
  int32_t dtype;                /* of every tensor but norm_weight: F16 or BF16 */
  int32_t norm_dtype;           /* `dtype` or F32 */
  int32_t max_position;         /* rows of cos_sin */
  int32_t interleaved;          /* pairs: 0: (f, f + rope_dim / 2); 1: (2 f, 2 f + 1) */
  float norm_eps;
} ua_append_latent_t;

/*
 * ua_append_latent -- appends the batch's new tokens to a latent cache, in one launch:
 *   c_j = x_j * (mean_j(x_j^2) + norm_eps)^(-1/2) * norm_weight_j     (fp32, rounded once)
 *   r   = k_rope rotated as ua_append_kv rotates keys, over its whole rope_dim
 * and rotates q_rope beside it.  Token i of sequence b goes to cache position seq_lens_k[b] - q_len
 * + i.  What ua_append_kv skips (tokens at negative positions, rows past cu_seqlens_q[num_seqs])
 * and refuses on the device (block ids outside the cache: not written; positions outside the table:
 * the token is skipped, its queries included) holds here too.
 */
int ua_append_latent(const ua_append_latent_t* call, void* stream);

/* One ua_tree_mask call. */
typedef struct {
  const int32_t* parents;       /* [total_q]: the parent's index among its sequence's new tokens, below
                                   the token's own; -1: none */
  const int32_t* cu_seqlens_q;
  const int32_t* seq_lens_k;    /* lengths with the new tokens */
  int32_t* mask;                /* [total_q, mask_words] out, or NULL */
  int32_t* positions;           /* [total_q] out, or NULL */
  int64_t mask_stride;          /* words from one row of mask to the next, >= mask_words */
  int32_t num_seqs;
  int32_t total_q;
  int32_t max_seqlen_q;         /* >= every q_len; at most 4096 */
  int32_t mask_words;           /* 32 mask_words >= max_seqlen_q */
} ua_tree_t;

/*
 * ua_tree_mask -- what the tokens of drafted trees see, from their parents: bit j of token i's mask
 * (word j / 32) says that new token j of the sequence is i itself or an ancestor of i.  positions
 * receives kv_len - q_len + the token's depth (its rotary position: siblings share one).  A parent
 * that is not below its token (or below -1) counts as none, and raises UA_ERR_DEVICE_CHECK in the
 * device status word, as does a q_len above max_seqlen_q, whose tokens from there on are left out.
 * Rows past cu_seqlens_q[num_seqs] stay as they are.
 */
int ua_tree_mask(const ua_tree_t* call, void* stream);

/*
 * One ua_latent_attention call.  Tensors are contiguous; q, cache, out and workspace are 16-byte
 * aligned; out and lse overlap none of the others.
 */
typedef struct {
  const void* q;                /* [total_q, num_heads, latent_dim + rope_dim] of `dtype` */
  const void* cache;            /* [num_blocks, block_size, latent_dim + rope_dim] of `dtype` */
  void* out;                    /* [total_q, num_heads, latent_dim] of out_dtype */
  float* lse;                   /* [total_q, num_heads] or NULL: ln of each row's sum (-inf: no key) */
  const int32_t* cu_seqlens_q;
  const int32_t* seq_lens_k;
  const int32_t* block_table;
  const int32_t* tree_mask;     /* [total_q, tree_words] bits, or NULL: causal */
  void* workspace;              /* device scratch, or NULL: the library's own (see ua_shape_t) */
  size_t workspace_bytes;
  int64_t tree_mask_stride;     /* words from one row of tree_mask to the next */
  int32_t num_seqs;
  int32_t total_q;
  int32_t max_seqlen_q;         /* >= every q_len and kv_len: the grid's size follows from them */
  int32_t max_seqlen_k;
  int32_t max_blocks_per_seq;
  int32_t num_blocks;
  int32_t block_size;
  int32_t num_heads;
  int32_t latent_dim;
  int32_t rope_dim;
  int32_t dtype;
  int32_t out_dtype;            /* F16, BF16 or F32 */
  int32_t tree_words;           /* 32 tree_words >= max_seqlen_q */
  float scale;                  /* > 0 */
} ua_latent_t;

/*
 * ua_latent_attention -- attention over a latent cache with absorbed projections: q is in the
 * latent space (the key up-projection applied to it), and so is out.  For row i of head h at
 * position p = kv_len - q_len + i:
 *   s_j = scale * q . [c_j | r_j],   out = sum_j e^{s_j} c_j / sum_j e^{s_j}
 * over 0 <= j < kv_len with j <= p, or with tree_mask over j < kv_len - q_len and those new tokens
 * j of the sequence whose bit j - (kv_len - q_len) is set in the row's mask (no other rule: a
 * token sees itself only if its own bit is set).  A row that sees no key is written as 0.  Every
 * slot below kv_len must hold finite values (their weight may be 0, but they are multiplied); slots
 * past it may hold anything.  Every block size works; a copy takes as many rows at a time as the
 * largest power of two that divides it (up to 64).
 * Returns UA_ERR_UNSUPPORTED where total_q * num_heads or num_blocks * block_size passes 31 bits,
 * UA_ERR_WORKSPACE where `workspace` is smaller than ua_latent_workspace_bytes().
 */
int ua_latent_attention(const ua_latent_t* call, void* stream);

/* Bytes of scratch that the call needs on the current device (0: none, or an invalid argument). */
size_t ua_latent_workspace_bytes(const ua_latent_t* call);

/*
 * One ua_latent_prefill call.  Strides are in elements: multiples of 8, not 0 (the last dim has stride
 * 1; a dim of one element may have any).  q, k_nope, k_rope, v and out are 16-byte aligned; out and lse
 * overlap none of the others.
 */
typedef struct {
  const void* q;                /* [total_q, num_heads, nope_dim + rope_dim] of `dtype` */
  const void* k_nope;           /* [total_k, num_heads, nope_dim] */
  const void* k_rope;           /* [total_k, rope_dim], shared by the heads */
  const void* v;                /* [total_k, num_heads, value_dim] */
  void* out;                    /* [total_q, num_heads, value_dim] of out_dtype, contiguous */
  float* lse;                   /* [total_q, num_heads] or NULL: ln of each row's sum (-inf: no key) */
  const int32_t* cu_seqlens_q;  /* [num_seqs + 1] */
  const int32_t* cu_seqlens_k;  /* [num_seqs + 1] */
  int64_t q_stride[2];          /* token, head */
  int64_t k_nope_stride[2];
  int64_t v_stride[2];
  int64_t k_rope_stride;
  int32_t num_seqs;
  int32_t total_q;
  int32_t total_k;
  int32_t max_seqlen_q;         /* >= every q_len and k_len: the grid's order follows from them */
  int32_t max_seqlen_k;
  int32_t num_heads;
  int32_t nope_dim;             /* 64 or 128 */
  int32_t rope_dim;             /* a multiple of 16 up to 64 */
  int32_t value_dim;            /* 64 or 128 */
  int32_t dtype;
  int32_t out_dtype;            /* F16, BF16 or F32 */
  float scale;                  /* > 0 */
} ua_latent_prefill_t;

/*
 * ua_latent_prefill -- the expanded form, for prompts: keys and values of every head, as the
 * up-projection of the latents gives them (k_nope and v may be slices of one tensor), and the rope
 * keys.  For row i of a sequence of q_len queries and k_len keys, at position p = k_len - q_len + i:
 *   s_j = scale * (q_nope . k_nope_j + q_rope . k_rope_j),  j <= p,   out = softmax(s) v
 * A row that sees no key is written as 0.  Rows past cu_seqlens_q[num_seqs] stay as they are.
 * Returns UA_ERR_UNSUPPORTED where total_q / 256 + num_seqs passes 65535.
 */
int ua_latent_prefill(const ua_latent_prefill_t* call, void* stream);

/*
 * ua_plan -- the dispatcher's decision for a call with these sizes, without touching
 * the GPU: path, kernel, partitions, grid and workspace bytes.  The split path is
 * taken (UA_BACKEND_AUTO) when the 2D grid fills less than one wave of SMs and the
 * longest key walk of a q-block spans at least two minimum partitions (grid fill and
 * walk length, as in the aiter PR #3962 gating and the RocKE harness "Why three
 * tables").  num_sms <= 0 asks the current CUDA device.  Returns UA_OK or
 * UA_ERR_INVALID_ARG / UA_ERR_CUDA (device query).
 */
int ua_plan(const ua_shape_t* shape, int block_size, int num_q_heads, int num_kv_heads,
            int head_dim, int window_left, int kv_dtype, int backend, int num_sms,
            ua_plan_t* plan);

/*
 * ua_workspace_bytes -- bytes of split-path scratch a call with these sizes needs on the
 * current device (0 when it takes the 2D path or merges its partitions inside a
 * thread-block cluster): fp32 max and sum per (query token, head, partition), then the
 * unnormalised partial output rows, each piece 256-byte aligned.  The scratch rules follow
 * the author's follow-up on the review of aiter PR #3962 ("split-K long-context decode for
 * shuffled fp8 SWA"): the partition count is capped, the scratch belongs to one stream at a
 * time (a caller workspace, or the library's own buffer per device and stream or per
 * capture), and every entry the merge reads is written by the same call, so the scratch needs
 * no clearing.
 * Returns 0 on an invalid argument too.
 */
size_t ua_workspace_bytes(const ua_shape_t* shape, int block_size, int num_q_heads,
                          int num_kv_heads, int head_dim, int window_left, int kv_dtype,
                          int backend);

/*
 * ua_device_status -- synchronises `stream`, then stores in *status the device
 * check word the kernels of this library raised since the last reset, mapped to
 * UA_OK, UA_ERR_DEVICE_CHECK (a block id outside the cache, a position outside the
 * rotation table, or a q_len above max_seqlen_q in a decode-shaped call) or
 * UA_ERR_TIMEOUT (a bounded wait expired).  Returns UA_OK or UA_ERR_CUDA / UA_ERR_INVALID_ARG.
 * The word reports what the kernels refuse to read rather than faulting: a bad block id
 * is never dereferenced (its keys count as zero).  Slots of a sequence's last page at or
 * past kv_len are never an input either: whatever they hold (NaN included) gets weight
 * exactly 0 and its V values are zeroed before P.V, after the NaN-in-unused-V-slots
 * finding of the follow-up on aiter PR #3962's review.
 */
int ua_device_status(void* stream, int* status);

/* Clears the device check word (enqueued on `stream`). */
int ua_device_status_reset(void* stream);

/*
 * sizeof(ua_shape_t) in the loaded library.  The struct grows as calls learn new options (its
 * per-block scales are such), and a call reads all of it: a caller built against another header
 * compares this with its own sizeof(ua_shape_t) before its first call, and makes none when they
 * differ.  UA_VERSION stays as long as every older member keeps its place and meaning.
 */
size_t ua_shape_bytes(void);

/* Static text for a ua_status_t code. */
const char* ua_status_string(int status);

/* UA_VERSION of the loaded library. */
int ua_version(void);

#ifdef __cplusplus
}
#endif

#endif /* UA_H_ */
