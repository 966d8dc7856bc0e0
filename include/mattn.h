/*
 * mattn.h - C ABI of the masked-attention library (libmattn.so) for one
 * NVIDIA GB300 GPU (sm_103a).
 *
 * The library computes fused scaled-dot-product attention with an element-wise
 * score modification and a mask, in one pass over key/value tiles with an
 * online softmax, so the Sq x Skv score matrix never reaches device memory:
 *
 *   s[b,h,i,j] = scale * <q[b,h,i,:], k[b,hk,j,:]>            hk = h / (Hq/Hkv)
 *   s'         = score_mod(s, b, h, i, j)                       (before softmax)
 *   O[b,h,i,:] = sum over kept j of softmax_j(s') * v[b,hk,j,:]
 *   LSE[b,h,i] = ln sum over kept j of exp(s'[b,h,i,j])
 *
 * Sources: the FlexAttention page (section "FlexAttention": a user function
 * score_mod(score, b, h, q_idx, kv_idx) modifies every score before the
 * softmax; the variant list: causal, relative position, ALiBi, sliding window,
 * PrefixLM, document masking; the item on exploiting mask sparsity; section
 * "Performance": a deterministic backward that recomputes intermediates) and
 * the Online-Softmax/FlashAttention page (abstract: 3-pass safe softmax,
 * 2-pass online softmax, 1-pass FlashAttention).
 *
 * Conventions for every entry point:
 *  - Buffers are caller-owned. Tensor arguments are DEVICE pointers; structs
 *    (attn_params, attn_block_mask) live in HOST memory. The library allocates
 *    no device memory on any call.
 *  - Layout: contiguous [B, H, S, D], D innermost. Base pointers of q, k, v,
 *    o, dO, dq, dk, dv must be 16-byte aligned.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *    stream). Argument errors are returned before anything is launched. A
 *    failed launch returns ATTN_ERR_CUDA. Device-side failures (a bounded wait
 *    that ran out) are written to the status word and read back with
 *    attn_check_status().
 *  - No C++ exception crosses this boundary. The functions are thread-safe.
 */
#ifndef MATTN_H_
#define MATTN_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st; /* cudaStream_t is `struct CUstream_st*` */

typedef enum attn_status {
  ATTN_OK = 0,
  ATTN_ERR_INVALID_ARG = 1,        /* NULL pointer, bad size, inconsistent shapes */
  ATTN_ERR_UNSUPPORTED = 2,        /* valid but not built: D, dtype, tails, variant */
  ATTN_ERR_MISALIGNED = 3,         /* a tensor base pointer is not 16-byte aligned */
  ATTN_ERR_WORKSPACE_TOO_SMALL = 4,/* the caller's buffer is smaller than required */
  ATTN_ERR_CUDA = 5,               /* a CUDA runtime call or a launch failed */
  ATTN_ERR_TIMEOUT = 6             /* a device-side bounded wait ran out */
} attn_status;

/* Variant: OR of the bits below; 0 = full (bidirectional) attention with the
 * identity score_mod. Mask terms combine as
 *   keep(b,i,j) = (CAUSAL: j <= i) AND (WINDOW: i - j < window)
 *                 AND (DOCUMENT: doc_id[b][i] == doc_id[b][j])
 *                 OR  (PREFIX: j < prefix_len[b])
 * with absent AND-terms true and an absent PREFIX false. i and j are absolute
 * positions: i = q_offset + query row, j = kv_offset + key column (both
 * offsets 0 unless the call is one shard of a longer sequence, see
 * attn_params and attn_combine).
 * Score terms apply in this order: s <- scale * q.k; ALIBI: s <- s - slope_h
 * * (i - j); RELBIAS: s <- s + rel_bias[h][i - j + Skv - 1]; SOFTCAP:
 * s <- softcap * tanh(s / softcap). */
enum {
  ATTN_MASK_CAUSAL = 1u << 0,   /* FlexAttention page, "Causal Mask" */
  ATTN_MASK_WINDOW = 1u << 1,   /* "Sliding Window + Causal" (1024 tokens there) */
  ATTN_MASK_DOCUMENT = 1u << 2, /* variant list: document masking */
  ATTN_MASK_PREFIX = 1u << 3,   /* variant list: PrefixLM (prefix is bidirectional) */
  ATTN_SCORE_ALIBI = 1u << 8,   /* variant list: ALiBi; slope_h = 2^(-8(h+1)/Hq) */
  ATTN_SCORE_SOFTCAP = 1u << 9, /* "Soft-capping" section (Gemma 2, Grok-1) */
  ATTN_SCORE_RELBIAS = 1u << 10 /* relative position encoding: the score is adjusted by
                                   the query-key distance, from a per-head table the
                                   call captures (no S x S tensor); forward only */
};
#define ATTN_MASK_BITS 0x0Fu
#define ATTN_SCORE_BITS 0x700u

enum { ATTN_BF16 = 0, ATTN_F32 = 1 };

/* Tile size of the block mask and of the kernels (query rows x key columns). */
#define ATTN_TILE 128

/* Block mask: per (batch, 128-row query tile) the ascending lists of
 * 128-column key tiles that are FULL (every pair kept: no mask evaluated) or
 * PARTIAL (some pairs kept: the mask is evaluated per element); EMPTY tiles
 * are skipped (FlexAttention page: exploiting the sparsity of the mask). The
 * mask does not depend on the head, so one list serves every head. All
 * pointers below point into the caller's device buffer given to
 * build_block_mask(); this host struct only describes it.
 *   full_cnt, part_cnt  int32 [B][nq]
 *   full_idx, part_idx  int32 [B][nq][nkv]  (first *_cnt entries valid)
 *   order               int32 [B*nq]: b*nq+qt by descending full+part count
 *                       (ties by ascending index): longest work first
 * The t_* members hold the transposed lists (per key tile, its query tiles,
 * [B][nkv] and [B][nkv][nq]) when built with transposed = 1, else NULL;
 * t_order lists their rows batch element by batch element (ascending b),
 * within one by descending full+part count (ties by ascending index). */
typedef struct attn_block_mask {
  int B, Sq, Skv;
  int nq, nkv;
  unsigned variant;      /* mask bits it was built for */
  int window;            /* parameters it was built for */
  const int* doc_id;
  const int* prefix_len;
  const int* full_cnt;
  const int* part_cnt;
  const int* full_idx;
  const int* part_idx;
  const int* order;
  const int* t_full_cnt;
  const int* t_part_cnt;
  const int* t_full_idx;
  const int* t_part_idx;
  const int* t_order;
  int q_offset, kv_offset;  /* position offsets it was built for */
  int doc_len;              /* row length of doc_id it was built for */
} attn_block_mask;

/* Parameters of a call (host struct). */
typedef struct attn_params {
  int dtype;                   /* ATTN_BF16 or ATTN_F32: type of q, k, v, o, do, dq, dk, dv */
  float scale;                 /* multiplies q.k, > 0; 0 selects 1/sqrt(D) */
  int window;                  /* ATTN_MASK_WINDOW: keys with i - j < window; >= 1 */
  float softcap;               /* ATTN_SCORE_SOFTCAP: cap c > 0 */
  const float* alibi_slopes;   /* ATTN_SCORE_ALIBI: device fp32 [Hq], or NULL for 2^(-8(h+1)/Hq) */
  const int* doc_id;           /* ATTN_MASK_DOCUMENT: device int32 [B][doc_len], indexed
                                  by absolute position */
  const int* prefix_len;       /* ATTN_MASK_PREFIX: device int32 [B] */
  const attn_block_mask* block_mask; /* from build_block_mask() for the same mask, or NULL:
                                        then every key tile allowed by the causal bound is
                                        visited with the mask evaluated per element */
  int* status;                 /* device int32 status word, or NULL for the library's own */
  unsigned long long timeout_ns; /* limit of each device-side wait; 0 = 4 s */
  const float* rel_bias;       /* ATTN_SCORE_RELBIAS: device fp32 [Hq][Sq + Skv - 1]; entry
                                  d + Skv - 1 is added to the score of a query-key pair at
                                  distance d = i - j (4-byte aligned). Not differentiated:
                                  attn_bwd returns ATTN_ERR_UNSUPPORTED with this bit */
  unsigned fault_inject;       /* 0 in normal use. ATTN_FAULT_NO_LOADS: the tensor-core
                                  kernels' load warp issues no copy, so every wait for data
                                  runs out after timeout_ns and the call reports
                                  ATTN_ERR_TIMEOUT (tests the bounded-wait path; no GPU
                                  fault is involved) */
  /* Paged K/V cache (variant list: PagedAttention), bf16 forward only. NULL
   * page_table: k and v are contiguous [B,Hkv,Skv,D]. Otherwise k and v are
   * page pools [num_pages][Hkv][page_size][D] and key j of batch b is row
   * j % page_size of page page_table[b * pages_per_seq + j / page_size].
   * page_size is 16, 32, 64 or 128; pages_per_seq * page_size >= Skv. Rows
   * of the last page past Skv are read (and masked): they must hold finite
   * values. A page index outside [0, num_pages) reads zeros. Not combined
   * with ATTN_SCORE_RELBIAS (ATTN_ERR_UNSUPPORTED). */
  const int* page_table;       /* device int32 [B][pages_per_seq], or NULL */
  int page_size;
  int pages_per_seq;
  int num_pages;
  /* Shards of a longer sequence (FlexAttention page, variant list: sliding
   * window + document masking + causal + context parallel): query row r and
   * key column c of this call sit at absolute positions q_offset + r and
   * kv_offset + c, which every mask term, the ALiBi bias and the document ids
   * use. Results over disjoint key shards merge with attn_combine(). >= 0.
   * Forward, backward and block mask; not combined with ATTN_SCORE_RELBIAS. */
  int q_offset;
  int kv_offset;
  /* Row length of doc_id: 0 selects L = max(q_offset + Sq, kv_offset + Skv);
   * otherwise >= L (e.g. the whole sequence's length when the call is one
   * shard of it). */
  int doc_len;
} attn_params;

#define ATTN_FAULT_NO_LOADS 1u

/* Forward: O = softmax(score_mod(scale*QK^T) under the mask) V and LSE.
 *   q [B,Hq,Sq,D], k and v [B,Hkv,Skv,D], o [B,Hq,Sq,D] (dtype p->dtype),
 *   lse fp32 [B,Hq,Sq] (natural log; -inf for a row with no kept key, whose
 *   O row is 0).
 * Supported: D in {64, 128}; Hq % Hkv == 0 (GQA: query head h reads key/value
 * head h / (Hq/Hkv)); any Sq, Skv >= 1 for both ATTN_BF16 (tcgen05
 * tensor-core kernel: a last tile that runs past Sq or Skv reads zero-filled
 * rows, its extra keys are masked and its extra query rows are not stored)
 * and ATTN_F32 (fp32 FFMA kernel). Returns ATTN_ERR_UNSUPPORTED for anything
 * else. */
attn_status attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                     int B, int Hq, int Hkv, int Sq, int Skv, int D,
                     unsigned variant, const attn_params* p, struct CUstream_st* stream);

/* Decode: a few new query rows per sequence against a long key/value cache
 * (FlexAttention page, variant list: PagedAttention, alone and with a
 * sliding window). Same arguments, layouts and results as attn_fwd for
 * ATTN_BF16, D = 64 or 128, with (Hq / Hkv) * Sq <= 16: the query rows of all
 * query heads that share a key/value head are computed together, so each
 * key and value row is read from memory once. K and V are contiguous or a
 * paged cache (attn_params page_table etc., page_size 16, 32, 64 or 128); a
 * page index outside [0, num_pages) reads as zeros. Every mask and score term
 * is supported; for a new token at absolute position P, pass q_offset = P
 * so the causal and window terms see it. p->block_mask is not used.
 * The keys are split across CTAs when that gives more parallelism: the
 * splits' partial results (fp32) go to `workspace` (device, 256-byte aligned,
 * attn_decode_workspace_bytes() bytes for the full split count) and are
 * merged into o and lse by the online-softmax merge. A smaller workspace (or
 * NULL) means fewer splits (none with NULL). Asynchronous on `stream`;
 * argument errors before any launch; ATTN_ERR_UNSUPPORTED for other dtypes,
 * D or row counts, or B * Hkv > 65535. */
attn_status attn_decode(const void* q, const void* k, const void* v, void* o, float* lse,
                        int B, int Hq, int Hkv, int Sq, int Skv, int D,
                        unsigned variant, const attn_params* p,
                        void* workspace, size_t workspace_bytes, struct CUstream_st* stream);

/* Bytes of workspace attn_decode() uses for its full split count on the
 * current device (0 when it does not split the keys). */
size_t attn_decode_workspace_bytes(int B, int Hq, int Hkv, int Sq, int Skv, int D);

/* Merge of partial results over disjoint key sets, e.g. the key/value shards
 * of context-parallel attention (FlexAttention page, variant list: ... +
 * context parallel). It is the merge step of the online softmax
 * (Online-Softmax/FlashAttention page, 2-pass online softmax: partial maxima
 * and sums combine as m = max(m1, m2), l = l1 e^(m1-m) + l2 e^(m2-m)) applied
 * to whole results, each normalised by its own sum:
 *   LSE = ln sum_k exp(LSE_k),   O = sum_k exp(LSE_k - LSE) O_k
 * and a row with no kept key in any part (every LSE_k = -inf) gets O = 0 and
 * LSE = -inf. A part whose LSE_k is -inf is not read.
 *   o_parts   device [n_parts][rows][D] of `dtype` (ATTN_BF16 or ATTN_F32),
 *             part k = the forward output of the same queries against key
 *             set k (rows = B * H * S in [B, H, S, D] order)
 *   lse_parts device fp32 [n_parts][rows]
 *   o, lse    device [rows][D] of `dtype` and fp32 [rows]; they must not
 *             overlap the parts.
 * D is 64 or 128; n_parts >= 1; 16-byte aligned tensors. Asynchronous on
 * `stream`. ATTN_ERR_INVALID_ARG / ATTN_ERR_UNSUPPORTED / ATTN_ERR_MISALIGNED
 * before any launch. */
attn_status attn_combine(const void* o_parts, const float* lse_parts, int n_parts,
                         long long rows, int D, int dtype, void* o, float* lse,
                         struct CUstream_st* stream);

/* Jagged batches (FlexAttention page, variant list: irregular tensors): n
 * sequences packed back to back with no padding, cu_seqlens (device int32
 * [n + 1]: 0 = cu[0] <= cu[1] <= ... <= cu[n] = total) their cumulative
 * lengths. Writes doc_id (device int32 [total]) = the index of the sequence
 * each packed position belongs to. With B = 1, S = total and
 * ATTN_MASK_DOCUMENT (plus ATTN_MASK_CAUSAL etc.) the forward, backward and
 * block mask then attend within each sequence only. Asynchronous on
 * `stream`; ATTN_ERR_INVALID_ARG for n < 1, total < 0 or null pointers. The
 * lengths are not validated on the device: non-monotone input gives
 * undefined ids. */
attn_status attn_doc_ids_from_seqlens(const int* cu_seqlens, int n, int total, int* doc_id,
                                      struct CUstream_st* stream);

/* A [B, H, S, D] tensor of any strides (in elements), D contiguous. `data`
 * is 16-byte aligned and every stride of a dimension longer than 1 is a
 * multiple of 16 bytes, >= 0, and in a tensor that is written > 0. */
typedef struct attn_view {
  void* data;
  long long stride_b, stride_h, stride_s;
} attn_view;

/* Page tables and slot maps of a serving step, from the requests' lengths.
 * Request b (of B) holds cached_lens[b] tokens in the first
 * ceil(cached / page_size) entries of page_table[b] and gets new_lens[b] more
 * (0 for an empty place of the batch; a negative length counts as 0). Pages it
 * then needs beyond those are taken from free_pages in order, request by
 * request, and written to its next entries; other entries stay as they are.
 *   seq_lens   int32 [B]          cached + new
 *   cu_new     int32 [B + 1]      cumulative new lengths (cu_new[0] = 0)
 *   slots      int64 [max_tokens] page * page_size + position % page_size of
 *                                 each new token, packed request by request
 *   positions  int32 [max_tokens] its position in its sequence
 *   seq_ids    int32 [max_tokens] its request
 *   info       int32 [4]          new tokens, pages taken, pages lacking,
 *                                 requests longer than their table
 * Entries past the last new token are -1 (attn_qk_norm_rope and the cache
 * calls skip them, so a captured graph may keep max_tokens fixed); new tokens
 * past max_tokens are dropped. A page that free_pages cannot give is entered
 * as -1, and tokens without a page (that one, or past pages_per_seq) get slot
 * -1: info tells. free_pages itself is not changed: the caller moves its front
 * past the info[1] pages taken before the next call, between replays of a graph
 * too. page_size 16, 32, 64 or 128; B <= 16384 (else
 * ATTN_ERR_UNSUPPORTED). What is written (page_table and the outputs) may
 * overlap no other argument (ATTN_ERR_INVALID_ARG): seq_lens is not
 * cached_lens. Asynchronous on `stream`, one launch. */
attn_status attn_page_plan(const int* cached_lens, const int* new_lens, int B, int* page_table,
                           int pages_per_seq, int page_size, const int* free_pages, int num_free,
                           int* seq_lens, int* cu_new, long long* slots, int* positions,
                           int* seq_ids, int max_tokens, int* info, struct CUstream_st* stream);

/* Parameters of the norm and rotation of queries and keys (host struct). */
typedef struct attn_rope_params {
  int dtype;              /* ATTN_BF16 or ATTN_F32: type of the tensors */
  float eps;              /* >= 0, added to the mean of squares */
  const float* q_weight;  /* device fp32 [D], or NULL: no norm of the queries */
  const float* k_weight;  /* device fp32 [D], or NULL: no norm of the keys */
  const float* cos_sin;   /* device fp32 [max_pos][rot_dim], 16-byte aligned: rot_dim / 2
                             cosines, then as many sines; NULL: no rotation */
  int max_pos;
  int rot_dim;            /* leading channels that are rotated: a multiple of 16, <= D */
  int interleaved;        /* pairs (2i, 2i + 1) if nonzero, else (i, i + rot_dim / 2) */
  const int* positions;   /* device int32 [B][S], or NULL: position s */
} attn_rope_params;

/* Per-head RMS norm and position rotation of queries and keys, one pass:
 *   y = x / sqrt(mean(x^2) + eps) * weight,
 *   out[c] = y[c] cos_i - y[c'] sin_i,  out[c'] = y[c'] cos_i + y[c] sin_i
 * for the i-th channel pair (c, c') and row `position` of cos_sin; channels
 * from rot_dim on are y. q and q_out are [B, Hq, S, D], k and k_out
 * [B, Hkv, S, D], each with strides of its own: the inputs may be slices of a
 * projection's output, the outputs what attn_fwd takes. Hq or Hkv may be 0
 * (its tensors are then not used). q_out may be q itself with the same strides
 * (k likewise); no other overlap. With cos_sin, a row whose position lies
 * outside [0, max_pos) is not written (places of a padded batch). D is 64 or
 * 128. Sums are fp32, squares among them (they stay finite up to |x| = 2^60);
 * each output is rounded once. Infinities and NaN act as the formulas say: what
 * is not rotated does not see its neighbours'. Asynchronous on `stream`. */
attn_status attn_qk_norm_rope(const attn_view* q, const attn_view* k, const attn_view* q_out,
                              const attn_view* k_out, int B, int Hq, int Hkv, int S, int D,
                              const attn_rope_params* p, struct CUstream_st* stream);

/* Bytes of workspace attn_qk_norm_rope_bwd() needs (the weights' partial sums). */
size_t attn_qk_norm_rope_bwd_workspace_bytes(int D);

/* Gradient of attn_qk_norm_rope: from its inputs q, k and the gradients
 * dq_out, dk_out of its outputs computes dq, dk and dq_weight, dk_weight (device
 * fp32 [D], summed over every row, 0 without rows; NULL: not wanted, and invalid
 * for a weight that is NULL). Rows that the forward did not write are not
 * written either and add nothing: where dq and dk are parts of a gradient that
 * goes on (a projection's), zero it before its first use, as what stands in
 * those rows is what the next product reads. q (k) is not read and may be NULL when its weight is NULL. dq may
 * be dq_out itself with the same strides. No atomics: results are bitwise
 * reproducible. The workspace is 256-byte aligned device memory whose contents
 * need not be kept between calls; calls that may run at the same time need
 * one each. */
attn_status attn_qk_norm_rope_bwd(const attn_view* q, const attn_view* k, const attn_view* dq_out,
                                  const attn_view* dk_out, const attn_view* dq,
                                  const attn_view* dk, float* dq_weight, float* dk_weight,
                                  void* workspace, size_t workspace_bytes, int B, int Hq, int Hkv,
                                  int S, int D, const attn_rope_params* p,
                                  struct CUstream_st* stream);

/* attn_qk_norm_rope with positions on several axes (tokens of images and video: time, height,
 * width): channel pair i (of rot_dim / 2) turns by the angle of the token's position on axis
 * pair_axis[i], row `position` and column i of cos_sin. `axes` is 1 to 4 and pair_axis a host
 * array of rot_dim / 2 entries below it, read before the call returns; p->positions is then
 * device int32 [axes][B][S], and neither it nor p->cos_sin may be NULL. A row is not written
 * where a position on any axis lies outside [0, max_pos). Everything else is as for
 * attn_qk_norm_rope, which gives the same bits for equal positions on every axis. */
attn_status attn_qk_norm_rope_axes(const attn_view* q, const attn_view* k, const attn_view* q_out,
                                   const attn_view* k_out, int B, int Hq, int Hkv, int S, int D,
                                   const attn_rope_params* p, int axes,
                                   const unsigned char* pair_axis, struct CUstream_st* stream);

/* Gradient of attn_qk_norm_rope_axes, as attn_qk_norm_rope_bwd is of attn_qk_norm_rope (the
 * workspace is attn_qk_norm_rope_bwd_workspace_bytes() too). */
attn_status attn_qk_norm_rope_axes_bwd(const attn_view* q, const attn_view* k,
                                       const attn_view* dq_out, const attn_view* dk_out,
                                       const attn_view* dq, const attn_view* dk, float* dq_weight,
                                       float* dk_weight, void* workspace, size_t workspace_bytes,
                                       int B, int Hq, int Hkv, int S, int D,
                                       const attn_rope_params* p, int axes,
                                       const unsigned char* pair_axis, struct CUstream_st* stream);

/* The 4-bit paged key/value cache. A pool is num_pages * Hkv records, record
 * (page, head) being
 *   K codes  [page_size][D / 2]   bytes: channel 2b in the low nibble of byte
 *   V codes  [page_size][D / 2]   b, channel 2b + 1 in the high one
 *   K scales [page_size][D / 32]  bf16, one per 32 consecutive channels
 *   V scales [page_size][D / 32]  bf16
 * and a code n stands for (n - 8) * scale (4.5 bits an element). Scales are
 * not negative. D is 64 or 128, page_size 16, 32, 64 or 128. The pool is 16-byte aligned. */
size_t attn_cache_q4_bytes(int num_pages, int Hkv, int page_size, int D);

/* Writes K and V rows (bf16 [B, Hkv, S, D], strides of their own) to slots
 * (device int64 [B][S]; page = slot / page_size). Per 32 channels
 * scale = bf16(max|x| / 7) and code = clamp(rint(x / scale), -8, 7) + 8, ties
 * to even; a zero scale stores code 8, and a group with an infinity or NaN
 * gets scale NaN (it reads back as NaN). A slot outside
 * [0, num_pages * page_size) is skipped. The slots of one call must differ:
 * what two tokens write to the same slot is unspecified. Asynchronous on
 * `stream`. */
attn_status attn_cache_store_q4(const attn_view* k, const attn_view* v, const long long* slots,
                                void* pool, int num_pages, int page_size, int B, int Hkv, int S,
                                int D, struct CUstream_st* stream);

/* Reads the rows at `slots` back as bf16 (one rounding), e.g. a cached
 * prefix that attn_fwd attends to as a packed batch. A slot outside the pool
 * reads as zeros; slots may repeat. */
attn_status attn_cache_load_q4(const void* pool, int num_pages, int page_size,
                               const long long* slots, const attn_view* k, const attn_view* v,
                               int B, int Hkv, int S, int D, struct CUstream_st* stream);

/* attn_decode over a 4-bit paged cache and sequences of their own lengths.
 * q, o [B, Hq, Sq, D] bf16 and lse fp32 [B, Hq, Sq] as for attn_decode, with
 * (Hq / Hkv) * Sq <= 16. seq_lens (device int32 [B]) counts each sequence's
 * keys, its Sq query rows' own tokens included: row r sits at absolute
 * position i = seq_lens[b] - Sq + r and key j at j. max_len bounds seq_lens
 * on the host (a length outside [0, max_len] counts as the nearest bound) and
 * p->pages_per_seq * page_size must hold it. p gives dtype (ATTN_BF16), scale,
 * window, softcap, alibi_slopes, page_table, page_size, pages_per_seq and
 * num_pages; its other fields are not used, except that offsets must be 0.
 * Variant: ATTN_MASK_CAUSAL, ATTN_MASK_WINDOW, ATTN_SCORE_ALIBI and
 * ATTN_SCORE_SOFTCAP (a finite softcap >= 1e-38) in any combination (others:
 * ATTN_ERR_UNSUPPORTED), and with a window the first `sink` keys stay visible:
 *   keep(i, j) = j < seq_len AND i >= 0 AND (CAUSAL: j <= i)
 *                AND (WINDOW: i - j < window OR j < sink)
 * Keys that no row sees are not read, and what a masked key's record holds,
 * NaN included, changes nothing. Products run on the codes, exact in fp16, and
 * sums are fp32. A query row is scaled by a power of two and rounded to fp16:
 * exact but for channels 2^28 and more below its largest, whose bits below 2^-38 of
 * that are lost. A probability times its V scale is rounded to 11 bits, and sums of
 * a group of 32 channels drop what lies 2^-25 below its largest such product; the
 * groups may differ in size by up to 2^100. A row without a key (an empty place of
 * the batch) gets O = 0, LSE = -inf. A page index outside [0, num_pages) reads as
 * zeros. With a workspace the keys of all sequences are shared out evenly over the
 * SMs, and results of sequences that several CTAs share are joined from it: 256-byte
 * aligned device memory, attn_decode_q4_workspace_bytes() for the full spread, less
 * or NULL means fewer CTAs (one per sequence and key/value head with NULL); its
 * contents need not be kept between calls, and calls that may run at the same time
 * need one each. ATTN_ERR_UNSUPPORTED for B * Hkv > 65535 or max_len > INT_MAX -
 * 255. */
attn_status attn_decode_q4(const void* q, const void* pool, void* o, float* lse, int B, int Hq,
                           int Hkv, int Sq, int max_len, int D, unsigned variant,
                           const attn_params* p, const int* seq_lens, int sink, void* workspace,
                           size_t workspace_bytes, struct CUstream_st* stream);

/* Bytes of workspace attn_decode_q4() uses for its full spread on the current
 * device (0 when a sequence's keys are too few to share out). */
size_t attn_decode_q4_workspace_bytes(int B, int Hq, int Hkv, int Sq, int max_len, int D);

/* Decode over a bf16 paged cache for sequences of their own lengths, groups of which share
 * their first keys (a prompt behind many requests): O and LSE of every sequence over its own
 * keys and those that its group shares, which (512 of them or more) are read once for up to 128
 * query rows of a key/value head. Arguments as for attn_decode_q4 (no sinks), with k and v bf16
 * page pools [num_pages][Hkv][page_size][D] (p: page_table, page_size, pages_per_seq, num_pages)
 * and
 *   group_starts  device int32 [G + 1], ascending: group g is sequences group_starts[g] to
 *                 group_starts[g + 1] - 1 (entries are cut to [0, B], and one below an earlier
 *                 one counts as that); sequences in no group share nothing
 *   shared_lens   device int32 [G]: the first shared_lens[g] keys of the group's sequences are
 *                 the same, in the same pages; the first sequence's table row may stand for all
 *                 there, so each row of page_table must hold them
 * G may be 0 (then both may be NULL): a decode of ragged lengths. A shared key past a
 * sequence's own length is not seen by it. Row r of sequence b sits at absolute position
 * i = seq_lens[b] - Sq + r and sees key j where
 *   keep(i, j) = j < seq_len AND i >= 0 AND (CAUSAL: j <= i) AND (WINDOW: i - j < window).
 * A row without a key gets O = 0, LSE = -inf. Products are of bf16 pairs and sums fp32;
 * a probability is rounded to bf16 before it multiplies its value row. What a key that no row of
 * its sequence (a shared one: of its group) sees holds, NaN included, changes nothing; of the
 * seen ones, values must be finite for the rows that do not see them. A page index outside
 * [0, num_pages) reads as zeros. `workspace`: device memory, 256-byte aligned, of
 * attn_decode_shared_workspace_bytes() bytes (less: ATTN_ERR_WORKSPACE_TOO_SMALL); its contents
 * need not be kept between calls, and calls that may run at the same time need one each.
 * Results are bitwise reproducible. Asynchronous on `stream`, three launches.
 * ATTN_ERR_UNSUPPORTED for (Hq / Hkv) * Sq > 16, B or G > 4096, B * Hkv > 65535. */
attn_status attn_decode_shared(const void* q, const void* k, const void* v, void* o, float* lse,
                               int B, int Hq, int Hkv, int Sq, int max_len, int D,
                               unsigned variant, const attn_params* p, const int* seq_lens,
                               const int* group_starts, const int* shared_lens, int G,
                               void* workspace, size_t workspace_bytes,
                               struct CUstream_st* stream);

/* Bytes of workspace that attn_decode_shared() needs on the current device. */
size_t attn_decode_shared_workspace_bytes(int B, int Hq, int Hkv, int Sq, int G, int max_len,
                                          int D);

/* The attention weight that each cached key received, e.g. to decide which keys a cache
 * gives up (attn_cache_evict):
 *   weights[b][hk][j] = decay * previous[b][hk][j]
 *                       + sum over the query rows (h, r) of key/value head hk that see key j
 *                         of exp(s'[b,h,r,j] - lse[b,h,r])
 * for j < seq_lens[b]; entries from there on are left as they were. q [B, Hq, Sq, D] bf16 and
 * lse fp32 [B, Hq, Sq] are those of an attention call over the same keys (Sq >= 1: the token of
 * a decode step, or the last tokens of a prompt), k its bf16 keys: page pools and
 * p->page_table, or NULL and contiguous [B, Hkv, max_len, D]. Row r sits at absolute position
 * i = seq_lens[b] - Sq + r and key j at j; seq_lens (device int32 [B]) counts each sequence's
 * keys, the rows' own tokens included, NULL: max_len each. max_len bounds seq_lens on the host
 * (a length outside [0, max_len] counts as the nearest bound). Variant and p as for
 * attn_decode_q4 (no sinks). weights and previous are device fp32 [B][Hkv][weights_stride],
 * weights_stride >= max_len; previous may be weights itself (weights added up step by step),
 * or NULL (0), and is not read where decay is 0; no other overlap. A row whose LSE is -inf adds
 * nothing, and what a key that no row sees holds, NaN included, changes nothing. A page index
 * outside [0, num_pages) reads as zeros. Sums are fp32 in a fixed order: bitwise reproducible.
 * Asynchronous on `stream`; ATTN_ERR_UNSUPPORTED for B * Hkv > 65535. */
attn_status attn_key_weights(const void* q, const void* k, const float* lse, const float* previous,
                             float decay, float* weights, int B, int Hq, int Hkv, int Sq,
                             int max_len, int D, int weights_stride, unsigned variant,
                             const attn_params* p, const int* seq_lens, struct CUstream_st* stream);

/* Eviction from the bf16 paged cache by accumulated attention weight (attn_key_weights), per
 * sequence and key/value head. With first = starts[b], or sink where starts is NULL (both cut to
 * seq_lens[b]), the first `first` keys stay; of the n = seq_lens[b] - first others, where they
 * are more than `keep`, the last `recent` (<= keep) stay and the keep - recent of the largest
 * weights (equal ones: the lowest index; NaN counts as the largest), else all. The held keys move
 * together in their order: held key m behind the first ones to position first + m. Each head
 * keeps keys of its own, as many as the others, so positions count places of the cache from then
 * on, not tokens: rotations that the rows hold stay true, positions of new tokens
 * (attn_qk_norm_rope) are the caller's to count, and window and ALiBi terms see places.
 *   weights      fp32 [B][Hkv][weights_stride]
 *   weights_out  the same, the held keys' weights at their new positions and 0 from there to
 *                seq_lens[b]; entries past seq_lens[b] stay. May be weights itself
 *   k, v         bf16 page pools [num_pages][Hkv][page_size][D], D 64 or 128
 *   page_table   int32 [B][pages_per_seq]
 *   new_table    int32 [B][new_pages_per_seq], or NULL: the rows move in place. Otherwise held
 *                rows are copied to the pages that it names, from position first rounded down
 *                to whole pages on (pages before that, e.g. a shared prefix, stay in both tables,
 *                and a row whose place is the same in both is left alone), and the old pages
 *                keep what they hold. Rows past its end are not written
 *   kept         int32 [B][Hkv][keep]  old positions of the held keys behind the first ones,
 *                ascending, then -1
 *   new_lens     int32 [B]   first + min(n, keep)
 *   freed        int32 [max_freed]  the pages that the sequences no longer use, one sequence
 *                after the other (a page that several gave up, once for each): entries of
 *                page_table from ceil(new_lens / page_size) on in place, from first / page_size
 *                on with new_table, up to ceil(seq_lens / page_size). An entry that new_table has
 *                in the same place, below ceil(new_lens / page_size), is in use and not listed.
 *                Those past max_freed are dropped; other entries stay
 *   info         int32 [2]   pages freed, sequences that gave up keys
 * A page outside the pool reads as zeros and is not written. In place, a page that several
 * sequences hold must lie among their first keys (whole pages before `first`); with new_table,
 * its pages must hold no row that the call reads, other than in its own place. Lengths outside
 * [0, max_len] count as the nearest bound. What is written overlaps nothing else
 * (ATTN_ERR_INVALID_ARG). page_size 16, 32, 64 or 128; B <= 16384, B * Hkv <= 65535 and
 * num_pages * Hkv * page_size < 2^32 (ATTN_ERR_UNSUPPORTED). Asynchronous on `stream`, two
 * launches. */
attn_status attn_cache_evict(const float* weights, float* weights_out, int weights_stride,
                             const int* seq_lens, const int* starts, int sink, int keep,
                             int recent, void* k, void* v, int num_pages, int page_size,
                             const int* page_table, int pages_per_seq, const int* new_table,
                             int new_pages_per_seq, int B, int Hkv, int max_len, int D, int* kept,
                             int* new_lens, int* freed, int max_freed, int* info,
                             struct CUstream_st* stream);

/* Bytes of device buffer build_block_mask() needs (256-byte aligned pieces). */
size_t attn_block_mask_bytes(int B, int Sq, int Skv, int transposed);

/* Classifies every (query tile, key tile) pair as full, partial or empty
 * under the mask bits of `variant` (score bits are ignored) and writes the
 * lists into `buf` (device, `bytes` long, 256-byte aligned). Fills `*out`
 * (host) with pointers into `buf`. The result is exact: a tile is full iff
 * every pair in it is kept and empty iff none is. */
attn_status build_block_mask(unsigned variant, const attn_params* p, int B, int Sq, int Skv,
                             void* buf, size_t bytes, int transposed, attn_block_mask* out,
                             struct CUstream_st* stream);

/* Bytes of fp32 workspace attn_bwd() needs: B*Hq*Sq*4 (the row terms
 * Delta_i = <dO_i, O_i>). */
size_t attn_bwd_workspace_bytes(int B, int Hq, int Sq);

/* Bytes of workspace for attn_bwd()'s fp16 path: the row terms, then fp16
 * copies of q, k, v and dO (about 2 (B Hq Sq + B Hkv Skv) D * 2 bytes more).
 * A call given at least this much, with Sq and Skv multiples of 128, no
 * position offsets and no relative-position bias, converts its inputs to fp16
 * (recording their largest |x|) and, where every |x| <= 60000 and
 * 2 D max|dO| max|V| <= 60000, computes the gradients from fp16 operands: each
 * product of a probability or dS term with an input is then one tensor-core
 * product instead of the bf16 path's two (the bf16 value and its rounding
 * remainder). Otherwise, and with a smaller workspace, the bf16 path runs.
 * Both meet the same bound. */
size_t attn_bwd_workspace_bytes_f16(int B, int Hq, int Hkv, int Sq, int Skv, int D);

/* Backward of the forward above (FlexAttention page, "Performance": a
 * deterministic backward that recomputes intermediates instead of storing
 * them): from q, k, v, o, lse and dO computes
 *   dq [B,Hq,Sq,D], dk and dv [B,Hkv,Skv,D] (dtype p->dtype; with GQA, dk and
 *   dv sum over the query heads of their group).
 * `workspace` is device memory of attn_bwd_workspace_bytes() bytes, or of
 * attn_bwd_workspace_bytes_f16() bytes for the fp16 path (see there). No
 * atomics: results are bitwise reproducible. Supported: ATTN_BF16, D = 128 and
 * 64, any Sq, Skv >= 1 (a last tile that runs past Sq or Skv reads zero rows,
 * its padding keys are masked and its padding rows are not stored); a block
 * mask built with transposed = 1 (or NULL); position offsets (attn_params
 * q_offset, kv_offset), with a block mask built for the same offsets: the
 * gradients of this call's own attention (its o and lse over its keys); the
 * relative-position bias (a constant of the call: no gradient flows to the
 * table), not together with offsets. Not supported (ATTN_ERR_UNSUPPORTED):
 * paged K/V. */
attn_status attn_bwd(const void* q, const void* k, const void* v, const void* o,
                     const float* lse, const void* dO, void* dq, void* dk, void* dv,
                     void* workspace, size_t workspace_bytes,
                     int B, int Hq, int Hkv, int Sq, int Skv, int D,
                     unsigned variant, const attn_params* p, struct CUstream_st* stream);

/* attn_bwd for callers that cannot allocate device memory. The page this
 * library follows has no counterpart: it exists for code that is handed its
 * tensors but has no way to obtain a workspace (a framework that owns every
 * device allocation and forbids raw cudaMalloc, a plug-in without an
 * allocator). Same arguments and results as attn_bwd without `workspace`:
 * the Delta row terms live in a fixed array inside the library (8 MiB per
 * GPU that loads it, held until the process exits), so B*Hq*Sq may be at most
 * 2,097,152; larger problems return ATTN_ERR_WORKSPACE_TOO_SMALL before
 * anything runs (every other argument is checked first, with no CUDA call).
 * No cudaMalloc, cudaFree or other allocating call is made. The first call
 * on a device looks up the array's device address and keeps it (make that
 * call before any stream capture); the address belongs to the device's
 * primary context, so after cudaDeviceReset the entry point must not be
 * called again in the same process. Every call shares the array, which keeps the
 * last call's contents (none needs to start at zero); calls that overlap on
 * the GPU race on it. */
attn_status attn_bwd_noalloc(const void* q, const void* k, const void* v, const void* o,
                             const float* lse, const void* dO, void* dq, void* dk, void* dv,
                             int B, int Hq, int Hkv, int Sq, int Skv, int D,
                             unsigned variant, const attn_params* p, struct CUstream_st* stream);

/* Synchronises `stream`, reads the device status word (`status_dev`, or the
 * library's own when NULL), resets it to 0 and returns it as an attn_status. */
attn_status attn_check_status(int* status_dev, struct CUstream_st* stream);

/* Static string naming a status code. */
const char* attn_status_str(attn_status s);

/* Name of the CUDA runtime error behind the calling thread's most recent
 * ATTN_ERR_CUDA (e.g. "cudaErrorLaunchOutOfResources"), or "cudaSuccess"
 * if none occurred on this thread. Static string; makes no CUDA call that
 * can fail. */
const char* attn_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MATTN_H_ */
