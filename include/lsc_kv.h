/*
 * lsc_kv.h -- C ABI of liblsc's attention K/V block pool: page-strided K and V
 * views of every attention layer; copy_prefix, the device copy that moves a
 * reused prefix's K/V rows into another sequence's blocks; and the calls of a
 * step over one layer's blocks: append (write the new tokens' K/V rows,
 * quantised when the pool holds e4m3), gather (read rows back dense) and
 * attend (softmax attention of the new tokens over the cached ones).
 *
 * Sources, cited by page title and section:
 *   [VA] "非连续 KV Cache" (vLLM-Ascend design document) §3 (block stride =
 *        physical page size / element size; padding skipped by stride), §3.2
 *        (K and V are separate views), §3.4 (the 48-element block example; the
 *        merged two-lane view (2, blocks, block_tokens, kv_heads, head_dim)
 *        whose lane and block strides come from the physical allocation)
 *   [KP] "Kapitsa 源码拆解 05：前缀缓存与模型状态恢复", figure 2 (reusing a prefix
 *        in another slot copies its KV with copy_prefix)
 *
 * Layout: attention layer l owns one region of two lanes, [K lane][V lane];
 * each lane holds num_blocks physical pages; a block's logical payload is
 * block_tokens rows of kv_heads x head_dim elements (token-major, the §3.4
 * order), followed by padding to page_bytes that no call reads or writes.
 * Regions follow one another in layer order.
 *
 * E4M3 pools hold one 8-bit code per element and one scale byte per (token row,
 * kv head): the payload is block_tokens rows of kv_heads x head_dim codes, then,
 * at byte round_up(codes, 16) of the page, [block_tokens, kv_heads] scale bytes.
 * Element x of a row is code * 2^(byte - 127); byte 255 marks a row that held a
 * NaN or an infinity and reads back as NaN.  A written row takes the smallest
 * power of two, at least 2^-127 (byte 0; a row of zeros too), that brings its
 * largest magnitude to 448 or less, the largest e4m3 value, and each element is
 * rounded once, to nearest even.  A power of two keeps the product exact, so the
 * only error is that one rounding (half a step: 2^-4 of the element, or 2^-10
 * times the scale below 2^-6 times it).
 *
 * Conventions are those of lsc.h (return codes, host/device pointers, streams,
 * no host sync except create/destroy).
 */
#ifndef LSC_KV_H
#define LSC_KV_H

#include "lsc.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int32_t num_layers;   /* attention layers holding K/V (> 0) */
  int32_t num_blocks;   /* physical blocks per lane (> 0) */
  int32_t block_tokens; /* token rows per block (> 0) */
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t dtype;        /* lsc_dtype */
  int64_t page_bytes;   /* physical page per block: >= payload, multiple of 16 and of the element size */
} lsc_kv_pool_desc;

typedef struct lsc_kv_pool lsc_kv_pool;

/* Typed strided views of one attention layer ([VA] §3.2, §3.4); strides and
 * offsets in elements of dtype. */
typedef struct {
  void *region;            /* device: the layer's [K lane][V lane] */
  int64_t region_bytes;
  void *k;                 /* device: block 0 of the K lane */
  void *v;                 /* device: block 0 of the V lane */
  int64_t shape[4];        /* num_blocks, block_tokens, kv_heads, head_dim */
  int64_t strides[4];      /* page_bytes / es, kv_heads * head_dim, head_dim, 1 */
  int64_t lane_stride;     /* v - k: num_blocks * page_bytes / es (dim 0 of the merged view) */
  int64_t page_bytes, payload_bytes, row_bytes;
  int32_t dtype;
  int32_t scale_offset;    /* E4M3: byte of a page where its scale bytes begin; 0 for other types */
} lsc_kv_layer_view;

/* One block of a prefix copy: token rows [0, n_tokens) of src_block go to
 * dst_block, in both lanes of every attention layer. */
typedef struct {
  int32_t src_block;
  int32_t dst_block;
  int32_t n_tokens;  /* 0 .. block_tokens; 0 copies nothing */
  int32_t reserved;  /* must be 0 */
} lsc_kv_copy_op;

/* Bytes a pool with this description needs: num_layers * 2 * num_blocks *
 * page_bytes.  Errors: INVALID_ARG, LAYOUT (page smaller than the payload or
 * not a multiple of the element size, or an E4M3 block of 2 GiB or more), MISALIGNED (page not a multiple of 16). */
int lsc_kv_pool_required_bytes(const lsc_kv_pool_desc *desc, size_t *total_bytes);

/* Create a K/V pool; device_base == NULL allocates (cudaMalloc, owned),
 * otherwise the 256-byte-aligned buffer is borrowed.  Without a GPU a borrowed
 * base gives a host-only pool (views work, copies return CUDA).  On a GPU the
 * library also allocates a device status word.  A pool may be created, and one on a
 * borrowed base destroyed, while the thread captures a stream into a graph.
 * Errors: as lsc_kv_pool_required_bytes, plus MISALIGNED (base), NO_MEMORY, CUDA. */
int lsc_kv_pool_create(const lsc_kv_pool_desc *desc, void *device_base, size_t base_bytes, lsc_kv_pool **out);
int lsc_kv_pool_destroy(lsc_kv_pool *pool);
/* Errors: OUT_OF_RANGE (layer). */
int lsc_kv_pool_layer_view(const lsc_kv_pool *pool, int32_t layer, lsc_kv_layer_view *out);
/* As lsc_pool_status, for the K/V pool's status word: waits for `stream` (host
 * sync), stores LSC_OK or the first device-side error (OUT_OF_RANGE,
 * INVALID_ARG, DEV_TIMEOUT) and clears the word. */
int lsc_kv_pool_status(lsc_kv_pool *pool, void *stream, int32_t *host_status);

/*
 * copy_prefix ([KP] figure 2): for every op with n_tokens > 0, token rows
 * [0, n_tokens) of src_block are copied to dst_block in the K and V lanes of
 * every attention layer (with their scale bytes in an E4M3 pool); nothing else
 * changes (rows past n_tokens, padding, source blocks, other blocks).  A prefix of T tokens is passed block by block:
 * its full blocks with n_tokens = block_tokens, then the partial last one.
 * One persistent launch per 2560 ops, 16-byte vector copies, on `stream`;
 * `done_event` (may be NULL) is recorded after the last launch.  ops is a host
 * array, read during the call.  bytes_copied (may be NULL) receives the bytes
 * written.  Errors (nothing enqueued): INVALID_ARG (n_tokens outside
 * [0, block_tokens], reserved != 0, NULL ops with n_ops > 0), OUT_OF_RANGE
 * (a block id), DUP_DST (two copying ops share a destination), SRC_IS_DST (a
 * source is a destination of the same call), CUDA.
 */
int lsc_copy_prefix(lsc_kv_pool *pool, const lsc_kv_copy_op *ops, int32_t n_ops, void *stream,
                    void *done_event, int64_t *bytes_copied);

/* ---- one step over a layer's blocks ----------------------------------------- */

/*
 * The sequences of a step.  Sequence i brings n_i = cu_seqlens[i+1] -
 * cu_seqlens[i] new tokens, rows [cu_seqlens[i], cu_seqlens[i+1]) of the dense
 * arrays, and has kv_lens[i] tokens in the cache, the new ones included: new
 * token j sits at position kv_lens[i] - n_i + j.  Position p is row
 * p % block_tokens of block block_table[i][p / block_tokens].  Everything that
 * varies from step to step is on the device, so a captured graph can be replayed
 * with new lengths and tables.
 *
 * Rows of the dense arrays at and behind cu_seqlens[n_seq] belong to no sequence
 * and are left as they were.  A token of a negative position (n_i > kv_lens[i])
 * has no row in the cache: append does not write it, gather gives zeros, and
 * attend, when causal, gives it an empty row.
 *
 * Found on the device, recorded in the pool's status word, never faulting:
 *  - INVALID_ARG: cu_seqlens that does not begin with 0, decreases or exceeds
 *    total_tokens.  No call reads or writes outside its arrays then; the batch's
 *    dense rows (append: its blocks' rows) are unspecified.
 *  - INVALID_ARG: kv_lens[i] < 0, > max_blocks * block_tokens or >
 *    LSC_KV_MAX_TOKENS.  The sequence is taken to have no cached tokens.
 *  - OUT_OF_RANGE: a block id outside [0, num_blocks) where a position needs it.
 *    append skips the row, gather gives zeros; what attend gives for that
 *    sequence is unspecified.
 */
#define LSC_KV_MAX_TOKENS (0x7fffffff - 1024)

typedef struct {
  int32_t n_seq;
  int32_t total_tokens;       /* rows of the dense arrays, >= cu_seqlens[n_seq] */
  int32_t max_blocks;         /* row length of block_table */
  int32_t reserved;           /* must be 0 */
  const int32_t *block_table; /* device [n_seq, max_blocks]; entries past a sequence's last block are not read */
  const int32_t *cu_seqlens;  /* device [n_seq + 1], cu_seqlens[0] == 0, non-decreasing */
  const int32_t *kv_lens;     /* device [n_seq] */
} lsc_kv_batch;

typedef struct {
  lsc_kv_batch batch;
  const void *k;    /* device [total_tokens, kv_heads, head_dim] at dtype */
  const void *v;    /* the same */
  int32_t dtype;    /* F32, BF16 or F16 */
  int32_t reserved; /* must be 0 */
  int64_t k_stride; /* elements from a token to the next (a slice of a wider projection); 0 = kv_heads * head_dim */
  int64_t v_stride;
} lsc_kv_append_args;

/*
 * Write the new tokens' K and V rows into layer `layer`'s blocks, in one launch.
 * The pool's type is the dense type (bit-exact), another float type (each
 * element rounded to nearest even, beyond the largest value to infinity) or E4M3
 * (quantised as described at the top; the row's scale byte is written with it).
 * Nothing else of the pool changes.  When two tokens of a call share a row of a
 * block, what it holds then is unspecified: heads, elements and (E4M3) scale bytes
 * of either, in any mixture.  Errors: INVALID_ARG (NULL, negative
 * or zero sizes, reserved != 0, dtype, a stride below kv_heads * head_dim),
 * OUT_OF_RANGE (layer), MISALIGNED (an array not aligned to its element),
 * CUDA, WRONG_DEVICE.
 */
int lsc_kv_append(lsc_kv_pool *pool, int32_t layer, const lsc_kv_append_args *args, void *stream);

typedef struct {
  lsc_kv_batch batch;
  void *k;          /* device [total_tokens, kv_heads, head_dim] at dtype */
  void *v;
  int32_t dtype;    /* F32, BF16 or F16 */
  int32_t reserved; /* must be 0 */
  int64_t k_stride;
  int64_t v_stride;
} lsc_kv_gather_args;

/*
 * The inverse: the rows that the batch's tokens sit in, dense, in one launch.
 * With n_i = kv_lens[i] it reads back whole sequences.  Elements are the pool's
 * values (E4M3: code times scale) rounded once to dtype.  Errors as lsc_kv_append.
 */
int lsc_kv_gather(lsc_kv_pool *pool, int32_t layer, const lsc_kv_gather_args *args, void *stream);

typedef struct {
  lsc_kv_batch batch;
  int32_t num_q_heads;    /* a multiple of kv_heads: q head h reads kv head h / (num_q_heads / kv_heads) */
  int32_t dtype;          /* of q and out: F32, BF16 or F16 */
  const void *q;          /* device [total_tokens, num_q_heads, head_dim] */
  void *out;              /* device, same shape; overlaps no input */
  float *lse;             /* device [total_tokens, num_q_heads] or NULL */
  float scale;            /* of the scores, > 0 */
  int32_t causal;         /* 1: a token sees positions up to its own; 0: all kv_lens[i] positions */
  int64_t q_stride;       /* elements from a token to the next; 0 = num_q_heads * head_dim */
  int64_t out_stride;
  int32_t max_seq_tokens; /* bound of every n_i that the host knows; 0 = total_tokens.  It picks the kernel: give a
                             decode step its 1 (or its few speculated tokens), or a prefill kernel serves it */
  int32_t max_kv_tokens;  /* bound of every kv_lens[i] that the host knows; 0 = max_blocks * block_tokens.  It says
                             how far work is cut and how large the workspace is */
  void *workspace;        /* device scratch of workspace_bytes, what
                             lsc_kv_attend_workspace_bytes says or more, 16-byte aligned, untouched by
                             others until the call's work on the stream completes; NULL = the
                             library takes it from the device's stream-ordered pool */
  size_t workspace_bytes;
} lsc_kv_attend_args;

/*
 * Attention of the new tokens over layer `layer`'s cached tokens (the new ones
 * included: append first):
 *   s_j = scale q . k_j,  out = sum_j exp(s_j) v_j / sum_j exp(s_j),
 *   lse = log sum_j exp(s_j)   (natural logarithm)
 * over the positions j that the token sees.  A token that sees none gets zeros
 * and lse = -infinity.  A score of NaN or +infinity makes the row NaN, and so do
 * scores of -infinity alone; a row of q that holds one of the three gives such
 * scores.  Its lse is not finite.  Positions it does not see, and rows behind a sequence's
 * last token, do not enter, whatever they hold.  Sums and softmax statistics
 * are 32-bit; with 16-bit q the weights exp(s_j - max) are rounded before they
 * meet v: to bf16 in bf16 pools; to f16 in f16 and E4M3 pools, in full down to
 * 2^-21 of a row's largest weight and to a multiple of 2^-31 of it below (E4M3
 * pools, more than 64 rows of q a kv head: to nine significant bits or more down
 * to 2^-17 of it, to a multiple of 2^-25 of it below, and elements of q below 2^-9
 * of their row's largest are off by up to 2^-18 of it; in E4M3 pools a weight is
 * one times the scale of its row of v).  E4M3 rows of v with a scale below 2^-76 add an
 * absolute error of up to 2^-93 a position; beside rows with a scale of 2^e above
 * 2^100, positions lighter than 2^(e - 133) of the heaviest drop out of the sums,
 * and rows of k with such a scale may overflow their scores.
 * Two calls with the same inputs give the same bits.
 * A sequence that exceeds max_kv_tokens is recorded as INVALID_ARG in the status
 * word and taken to have no cached tokens; one that exceeds max_seq_tokens is
 * recorded too, and its rows of out and lse stay as they are.  If a bounded device
 * wait expires (DEV_TIMEOUT in the status word), out and lse are
 * unspecified.
 * Supported: head_dim <= 512.  Pools of q's 16-bit type, and E4M3 pools with
 * 16-bit q, at head_dim 64, 128 and 256, with q and out 16-byte aligned in base
 * and stride, run on the tensor cores (E4M3 pools with F16 q: up to 64 rows of q
 * a kv head, max_seq_tokens times the group); every other combination (F32, q of
 * another type than the pool's, other head sizes) on the CUDA cores.
 * Errors: INVALID_ARG (as lsc_kv_append; num_q_heads no multiple of kv_heads;
 * scale not positive and finite; causal not 0 or 1; negative bounds; a
 * workspace that is too small), OUT_OF_RANGE (layer), UNSUPPORTED, MISALIGNED
 * (an array, or the workspace), NO_MEMORY (no workspace to be had), CUDA,
 * WRONG_DEVICE.
 */
int lsc_kv_attend(lsc_kv_pool *pool, int32_t layer, const lsc_kv_attend_args *args, void *stream);

/* Bytes of workspace that lsc_kv_attend asks for with these arguments, and that
 * serve every call over this pool of the same types and heads whose n_seq,
 * total_tokens, max_seq_tokens and max_kv_tokens (0 meaning total_tokens and
 * max_blocks * block_tokens) are no larger: asked once with the largest sizes, one
 * workspace serves every layer and step of a stream, prefill and decode alike.
 * 0: none.  The pointers are checked and do not matter otherwise.  Errors: as
 * lsc_kv_attend's argument checks; CUDA (a host-only pool). */
int lsc_kv_attend_workspace_bytes(const lsc_kv_pool *pool, const lsc_kv_attend_args *args, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* LSC_KV_H */
