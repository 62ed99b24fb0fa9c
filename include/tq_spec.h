/*
 * tq_spec.h -- the operators around the packed cache of a speculative-decoding
 * round (same library and conventions as tq.h: ownership, streams, errors,
 * block and cache layout):
 *
 *   tq_qk_norm_rope          rows of a q/k/v projection -> the rows that
 *                            tq_encode_kv, tq_decode_step and the decode
 *                            entry points take (norm, rotation, layout)
 *   tq_decode_attention_tree attention of a tree of drafted tokens
 *   tq_cache_compact         keep chosen rows of every sequence, in place
 *   tq_cache_copy            copy row ranges between cache slots (fork a prompt)
 *
 * A round: tq_qk_norm_rope on the drafted tokens (position = context + depth),
 * tq_encode_kv of their k and v behind the context, tq_decode_attention_tree,
 * then tq_cache_compact with the accepted path.
 */
#ifndef TQ_SPEC_H_
#define TQ_SPEC_H_

#include "tq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TQ_BF16 2              /* a third element type, of these entry points only */
#define TQ_MAX_TREE_NODES 64   /* drafted tokens of one sequence */
#define TQ_MAX_ROT_DIM 512

typedef enum { TQ_ROPE_NONE = 0, TQ_ROPE_LINEAR = 1, TQ_ROPE_NTK = 2, TQ_ROPE_YARN = 3 } tq_rope_scaling;

/* A position rotation.  Pair i turns by turns[i] * 2^-64 of a full turn per
 * position: the phase of a position is an integer product modulo 2^64, so
 * angles of far positions lose nothing. */
typedef struct {
  int32_t rot_dim;      /* rotated leading elements of a row, even; 0: none   */
  int32_t interleaved;  /* pairs (2i, 2i+1) if nonzero, else (i, i + rot/2)   */
  float gain;           /* factor on the rotated elements                     */
  int32_t reserved;
  uint64_t turns[TQ_MAX_ROT_DIM / 2];
} tq_rope;

/*
 * tq_make_rope -- fill `out` (host, synchronous).  Pair i of r = rot_dim / 2
 * turns by f_i = base^(-2i / rot_dim) radians per position, changed by
 * `scaling` for contexts longer than the trained one:
 *   NONE    f_i;
 *   LINEAR  f_i / factor;
 *   NTK     base replaced by base * factor^(rot_dim / (rot_dim - 2));
 *   YARN    (Peng, Quesnelle, Fan, Shippole 2023) f_i (1 - w_i) + f_i / factor w_i,
 *           w_i a ramp over i from 0 at floor(d(beta_fast)) to 1 at
 *           ceil(d(beta_slow)), d(n) = rot_dim ln(orig_ctx / (2 pi n)) / (2 ln base),
 *           the ends clamped to [0, rot_dim - 1]; gain 0.1 ln(factor) + 1.
 * gain is 1 otherwise.  TQ_ERR_INVALID_ARG for a null `out`, an odd or
 * negative rot_dim, a base not above 1, a factor below 1, and (YARN) an
 * orig_ctx, beta_fast or beta_slow not above 0 or beta_fast < beta_slow;
 * TQ_ERR_UNSUPPORTED for rot_dim above TQ_MAX_ROT_DIM or an unknown scaling.
 */
int tq_make_rope(int rot_dim, int interleaved, double base, int scaling, double factor,
                 double orig_ctx, double beta_fast, double beta_slow, tq_rope* out);

/* Rows of one side of a projection.  Element d of head h of token t of batch
 * entry b is in[b * batch_stride + t * token_stride + h * head_stride + d]
 * (strides in elements, so a slice of a joint projection needs no copy). */
typedef struct {
  const void* in;
  void* out;
  const void* weight;  /* norm weight [head_dim] or NULL (all ones); not read for v */
  int32_t heads;
  int64_t batch_stride, token_stride, head_stride;
} tq_rows;

/*
 * tq_qk_norm_rope -- for every row x of q and k:
 *   norm != 0:  x <- x / sqrt(mean(x^2) + eps) * (weight + weight_bias);
 *   rotation of the first rot_dim elements by the row's position:
 *   (a, b) <- gain * (a cos - b sin, b cos + a sin);
 * v rows are only converted and laid out.  All arithmetic is fp32 with one
 * rounding at the end.
 *   - q, k, v: any may be NULL (not all).  q->out is [batch, seq_new, heads,
 *     head_dim] (what the decode entry points take), k->out and v->out
 *     [batch, heads, seq_new, head_dim] (what tq_encode_kv takes), contiguous,
 *     16-byte aligned, overlapping no input.
 *   - in_dtype: of q, k and v; w_dtype: of the weights; out_dtype: of the
 *     outputs; each TQ_F32, TQ_F16 or TQ_BF16.  Every row must start 16-byte
 *     aligned.
 *   - head_dim: a multiple of 128 up to 512, at least rope->rot_dim.
 *   - rope: host pointer, may be NULL (no rotation).  positions: device int32
 *     [batch, seq_new], any value (required when something is rotated).
 *   - n_tok: device int32 [batch] or NULL; outputs of the tokens
 *     t >= n_tok[b] are left as they were.
 *   - eps: finite and >= 0; weight_bias: finite.
 * seq_new == 0 is a no-op.  TQ_ERR_INVALID_ARG / TQ_ERR_UNSUPPORTED on bad
 * arguments (nothing launched), TQ_ERR_CUDA if the launch fails.
 */
int tq_qk_norm_rope(const tq_rope* rope, int batch, int seq_new, int head_dim, const tq_rows* q,
                    const tq_rows* k, const tq_rows* v, int in_dtype, int w_dtype, int out_dtype,
                    int norm, float eps, float weight_bias, const int32_t* positions,
                    const int32_t* n_tok, void* stream);

/*
 * tq_tree_masks -- ancestor masks and depths of a drafted tree (host,
 * synchronous).  parents[j] is the node that node j continues, or -1 for a
 * child of the context; every parent comes before its children.  masks[j]
 * gets bit j and the bits of j's ancestors; depths[j] (may be NULL) the number
 * of ancestors: node j's position is the context length + depths[j].
 * TQ_ERR_INVALID_ARG for null pointers, n outside 1..TQ_MAX_TREE_NODES or a
 * parent outside [-1, j).
 */
int tq_tree_masks(const int32_t* parents, int n, uint64_t* masks, int32_t* depths);

/*
 * tq_tree_workspace_size -- bytes of device workspace of
 * tq_decode_attention_tree; 0 for invalid arguments.
 */
size_t tq_tree_workspace_size(const tq_kv_desc* desc, int q_heads, int n_q);

/*
 * tq_decode_attention_tree -- attention of a tree of drafted tokens over the
 * packed cache.  The last n_nodes[b] of sequence b's seq_lens[b] cached
 * positions are its drafted nodes; C = seq_lens[b] - n_nodes[b] positions are
 * its context.  Query row j (j < n_nodes[b]) sees every context position, and
 * node i (position C + i) if and only if bit i of tree[b][j] is set (i below
 * n_nodes[b]; a node sees itself only if its own bit is set).  The scores and
 * the V sum are those of tq_decode_attention, plain V format, no sparse-V.
 *   - n_q: query rows per sequence, 1..TQ_MAX_TREE_NODES; n_nodes: device
 *     int32 [batch] or NULL (= n_q), clamped to [0, n_q] (TQ_DEV_LEN_RANGE).
 *   - tree: device uint64 [batch, n_q], 8-byte aligned.
 *   - q: device [batch, n_q, q_heads, head_dim], q_dtype TQ_F32, TQ_F16 or
 *     TQ_BF16; out: the same shape, out_dtype TQ_F16 or TQ_BF16 (the products
 *     run on 16-bit operands; a 32-bit output would claim more than they hold).
 *   - Rows j >= n_nodes[b] of out are left as they were.  A row that sees no
 *     position is zero.  When seq_lens[b] < n_nodes[b] the nodes before the
 *     cache's start do not exist: no row sees them.
 *   - Values in positions that a row does not see (infinite or NaN norms
 *     included) do not reach it.
 *   - Range: the rows of a kv-head are worked on in groups of up to 128, whose
 *     queries share one power-of-two scale; a row whose largest finite |q| is
 *     below 2^-20 of its group's keeps less of q than fp16 would.  V norms share
 *     a scale along the sequence: one below 2^-21 of the largest (of any cached
 *     position, seen or not) is rounded coarser than fp16 at a weight of 1.
 *   - workspace: tq_tree_workspace_size() bytes, 256-byte aligned, any
 *     content; calls that share one must not overlap in time.  Three launches
 *     (queries, attention, join), the last two as programmatic dependents.
 *   - Every wait inside the kernel is bounded, at 2^20 tries of about a
 *     microsecond (fewer if the environment sets TQ_TREE_WAIT_TRIES before the
 *     process's first call).  One that runs out sets TQ_DEV_INTERNAL: out is
 *     invalid, nothing of the call is left in flight, the context stays usable.
 * seq_lens, limits and errors otherwise as tq_decode_attention (head_dim 128
 * or 256, even seq_cap, batch <= 2048, any q_heads / kv_heads ratio).
 */
int tq_decode_attention_tree(const tq_kv_desc* desc, const tq_codebook* k_cb, const tq_codebook* v_cb,
                             int q_heads, int n_q, const void* q, int q_dtype,
                             const uint8_t* k_codes, const uint16_t* k_norms, const uint8_t* v_codes,
                             const uint16_t* v_norms, const int32_t* seq_lens,
                             const int32_t* n_nodes, const uint64_t* tree, float scale, void* out,
                             int out_dtype, void* workspace, size_t workspace_bytes,
                             uint32_t* dev_status, void* stream);

/* The buffers of one cache (tq.h layout).  values: the v3 outlier values, or
 * NULL with outliers = 0. */
typedef struct {
  uint8_t* k_codes;
  uint16_t* k_norms;
  uint8_t* v_codes;
  uint16_t* v_norms;
  uint16_t* values;
  int32_t outliers;  /* v3 outlier channels per kv-head (0: none) */
} tq_cache_bufs;

/*
 * tq_cache_compact -- in place, for every sequence b, kv-head and
 * i < n_keep[b]: row keep[b][i] becomes row start[b] + i.  It is as if all
 * rows were read before any is written.  Rows elsewhere stay as they are.
 * Works on every V format (rows are moved as bytes; the v3 values with them).
 *   - keep: device int32 [batch, max_keep] positions; each needs
 *     start[b] + i <= keep[b][i] < seq_cap (a list that ascends from start[b]
 *     on always has the first).  An entry outside that is skipped (its row is
 *     left as it was) and sets TQ_DEV_POS_RANGE.  Repeats are allowed.
 *   - n_keep: device int32 [batch], clamped to [0, max_keep]
 *     (TQ_DEV_LEN_RANGE); start: device int32 [batch] or NULL (= 0); a
 *     negative start skips the sequence (TQ_DEV_POS_RANGE).
 *   - new_lens: device int32 [batch] or NULL; gets start[b] + n_keep[b]
 *     (clamped to [0, seq_cap]).  May be the seq_lens array of the decode
 *     calls that follow on the stream, but none of the arrays above
 *     (TQ_ERR_INVALID_ARG where they overlap).
 * max_keep == 0 is a no-op apart from new_lens.  head_dim up to 512.
 */
int tq_cache_compact(const tq_kv_desc* desc, const tq_cache_bufs* cache, const int32_t* keep,
                     int max_keep, const int32_t* n_keep, const int32_t* start, int32_t* new_lens,
                     uint32_t* dev_status, void* stream);

/*
 * tq_cache_copy -- for every copy c: rows [src_pos[c], src_pos[c] + n_rows[c])
 * of slot (batch entry) src_slot[c] of cache `src` to rows from dst_pos[c] of
 * slot dst_slot[c] of cache `dst`, all kv-heads.  The caches may be the same
 * one, or differ in batch and seq_cap; every other field of the two
 * descriptors and the outlier counts must be equal.  Rows that are written
 * must be neither read nor written by another part of the same call (they
 * would hold one of the values).  Consecutive copies of the same source
 * range read it once.
 *   - src_slot, dst_slot, n_rows: device int32 [n_copies]; src_pos, dst_pos:
 *     the same or NULL (= 0).  max_rows: host bound of n_rows.
 *   - A copy with a slot or position outside its cache is skipped
 *     (TQ_DEV_POS_RANGE); n_rows is clamped to [0, max_rows]
 *     (TQ_DEV_LEN_RANGE) and to both caches' ends (TQ_DEV_POS_RANGE).
 */
int tq_cache_copy(const tq_kv_desc* src_desc, const tq_cache_bufs* src, const tq_kv_desc* dst_desc,
                  const tq_cache_bufs* dst, int n_copies, const int32_t* src_slot,
                  const int32_t* dst_slot, const int32_t* src_pos, const int32_t* dst_pos,
                  const int32_t* n_rows, int max_rows, uint32_t* dev_status, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* TQ_SPEC_H_ */
