// Host layer of the speculative-decoding operators (include/tq_spec.h):
// argument validation and dispatch.  Validation never touches the GPU.

#include <cmath>
#include <cstring>

#include "../../include/tq_spec.h"
#include "tq_spec_internal.h"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlap(const void* a, size_t n, const void* b, size_t m) {  // of two given ranges
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + m && y < x + n;
}

bool valid_dtype(int t) { return t == TQ_F32 || t == TQ_F16 || t == TQ_BF16; }
size_t dtype_size(int t) { return t == TQ_F32 ? 4 : 2; }

// Units (16 bytes) of one row of K codes, V codes and v3 values, and the
// checks of a cache's buffers.
int check_cache(const tq_kv_desc* d, const tq_cache_bufs* c, int units[3]) {
  int st = tq::validate_desc(d);
  if (st != TQ_OK) return st;
  if (!c || !c->k_codes || !c->k_norms || !c->v_codes || !c->v_norms) return TQ_ERR_INVALID_ARG;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_norms, 4) || !aligned(c->v_norms, 4))
    return TQ_ERR_INVALID_ARG;
  if (c->outliers < 0 || c->outliers > TQ_MAX_OUTLIERS) return TQ_ERR_INVALID_ARG;
  if ((c->outliers > 0) != (c->values != nullptr) || !aligned(c->values, 16)) return TQ_ERR_INVALID_ARG;
  const int nb = d->head_dim / tq::kBlock;
  units[0] = nb * d->k_bits;
  units[1] = nb * d->v_bits;
  units[2] = c->outliers == 0 ? 0 : c->outliers <= 8 ? 1 : 2;
  return TQ_OK;
}

tq::CacheView view(const tq_kv_desc* d, const tq_cache_bufs* c) {
  return tq::CacheView{{c->k_codes, c->v_codes, reinterpret_cast<uint8_t*>(c->values)},
                       {c->k_norms, c->v_norms},
                       d->batch,
                       d->seq_cap};
}

int check_rows(const tq_rows* r, int dtype, int w_dtype, bool weighted, tq::RowSide* out) {
  *out = tq::RowSide{};
  if (!r) return TQ_OK;
  if (r->heads < 1 || !r->in || !r->out || !aligned(r->in, 16) || !aligned(r->out, 16)) return TQ_ERR_INVALID_ARG;
  const long long size = (long long)dtype_size(dtype);
  const long long strides[3] = {r->batch_stride, r->token_stride, r->head_stride};
  for (long long s : strides)
    if (s < 0 || (s % (16 / size)) != 0) return TQ_ERR_INVALID_ARG;
  out->in = r->in;
  out->out = r->out;
  out->weight = weighted ? r->weight : nullptr;
  if (out->weight && !aligned(out->weight, dtype_size(w_dtype))) return TQ_ERR_INVALID_ARG;
  out->heads = r->heads;
  out->batch_stride = r->batch_stride;
  out->token_stride = r->token_stride;
  out->head_stride = r->head_stride;
  return TQ_OK;
}

}  // namespace

extern "C" {

int tq_make_rope(int rot_dim, int interleaved, double base, int scaling, double factor,
                 double orig_ctx, double beta_fast, double beta_slow, tq_rope* out) {
  if (!out || rot_dim < 0 || rot_dim % 2 != 0) return TQ_ERR_INVALID_ARG;
  if (rot_dim > TQ_MAX_ROT_DIM) return TQ_ERR_UNSUPPORTED;
  if (scaling < TQ_ROPE_NONE || scaling > TQ_ROPE_YARN) return TQ_ERR_UNSUPPORTED;
  if (!std::isfinite(base) || !(base > 1.0) || !std::isfinite(factor) || !(factor >= 1.0)) return TQ_ERR_INVALID_ARG;
  if (scaling == TQ_ROPE_YARN) {
    if (!std::isfinite(orig_ctx) || !(orig_ctx > 0.0) || !std::isfinite(beta_fast) || !(beta_slow > 0.0) ||
        !(beta_fast >= beta_slow))
      return TQ_ERR_INVALID_ARG;
  }
  std::memset(out, 0, sizeof(*out));
  out->rot_dim = rot_dim;
  out->interleaved = interleaved ? 1 : 0;
  out->gain = scaling == TQ_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  long double b = base;
  if (scaling == TQ_ROPE_NTK && rot_dim > 2)
    b = b * powl((long double)factor, (long double)rot_dim / (rot_dim - 2));
  double lo = 0.0, hi = 0.0;
  if (scaling == TQ_ROPE_YARN && rot_dim > 0) {
    const double two_pi = 6.283185307179586;
    auto at = [&](double turns) { return rot_dim * std::log(orig_ctx / (turns * two_pi)) / (2.0 * std::log(base)); };
    lo = std::fmin(std::fmax(std::floor(at(beta_fast)), 0.0), rot_dim - 1.0);
    hi = std::fmax(std::fmin(std::ceil(at(beta_slow)), rot_dim - 1.0), 0.0);
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    long double f = powl(b, -2.0L * i / rot_dim);
    if (scaling == TQ_ROPE_LINEAR) f /= factor;
    if (scaling == TQ_ROPE_YARN) {
      const double w = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
      f = f * (1.0L - w) + f / factor * w;
    }
    // turns per position in units of 2^-64: f <= 1 radian, below 2^62
    out->turns[i] = (uint64_t)(f / 6.283185307179586476925286766559005768L * 18446744073709551616.0L + 0.5L);
  }
  return TQ_OK;
}

int tq_qk_norm_rope(const tq_rope* rope, int batch, int seq_new, int head_dim, const tq_rows* q,
                    const tq_rows* k, const tq_rows* v, int in_dtype, int w_dtype, int out_dtype,
                    int norm, float eps, float weight_bias, const int32_t* positions,
                    const int32_t* n_tok, void* stream) {
  if (batch < 1 || seq_new < 0 || head_dim < 1 || (!q && !k && !v)) return TQ_ERR_INVALID_ARG;
  if (!valid_dtype(in_dtype) || !valid_dtype(w_dtype) || !valid_dtype(out_dtype)) return TQ_ERR_INVALID_ARG;
  if (head_dim % tq::kBlock != 0 || head_dim > tq::kMaxHeadDim) return TQ_ERR_UNSUPPORTED;
  if (rope) {
    if (rope->rot_dim < 0 || rope->rot_dim % 2 != 0 || rope->rot_dim > head_dim || !std::isfinite(rope->gain))
      return TQ_ERR_INVALID_ARG;
  }
  if (norm && (!std::isfinite(eps) || !(eps >= 0.0f) || !std::isfinite(weight_bias))) return TQ_ERR_INVALID_ARG;
  if (seq_new == 0) return TQ_OK;  // empty tensors need not have addresses
  const bool rotates = rope && rope->rot_dim > 0 && (q || k);
  if (rotates && !positions) return TQ_ERR_INVALID_ARG;
  if (!aligned(positions, 4) || !aligned(n_tok, 4)) return TQ_ERR_INVALID_ARG;
  tq::RopeParams p{};
  const tq_rows* sides[3] = {q, k, v};
  for (int s = 0; s < 3; ++s) {
    const int st = check_rows(sides[s], in_dtype, w_dtype, norm && s < 2, &p.side[s]);
    if (st != TQ_OK) return st;
  }
  const long long rows = (long long)p.side[0].heads + p.side[1].heads + p.side[2].heads;
  if (rows > (1 << 20) || (long long)batch * seq_new >= (1LL << 31)) return TQ_ERR_UNSUPPORTED;
  p.batch = batch;
  p.seq_new = seq_new;
  p.head_dim = head_dim;
  p.rows = (int)rows;
  p.rot_dim = rotates ? rope->rot_dim : 0;
  p.interleaved = rotates ? rope->interleaved : 0;
  p.gain = rotates ? rope->gain : 1.0f;
  if (rotates) std::memcpy(p.turns, rope->turns, sizeof(uint64_t) * (size_t)(rope->rot_dim / 2));
  p.in_dtype = in_dtype;
  p.w_dtype = w_dtype;
  p.out_dtype = out_dtype;
  p.norm = norm ? 1 : 0;
  p.eps = eps;
  p.weight_bias = weight_bias;
  p.positions = positions;
  p.n_tok = n_tok;
  return tq::launch_qk_norm_rope(p, static_cast<cudaStream_t>(stream));
}

int tq_tree_masks(const int32_t* parents, int n, uint64_t* masks, int32_t* depths) {
  if (!parents || !masks || n < 1 || n > TQ_MAX_TREE_NODES) return TQ_ERR_INVALID_ARG;
  for (int j = 0; j < n; ++j)
    if (parents[j] < -1 || parents[j] >= j) return TQ_ERR_INVALID_ARG;
  for (int j = 0; j < n; ++j) {
    const int u = parents[j];
    masks[j] = (1ull << j) | (u >= 0 ? masks[u] : 0ull);
    if (depths) depths[j] = u >= 0 ? depths[u] + 1 : 0;
  }
  return TQ_OK;
}

size_t tq_tree_workspace_size(const tq_kv_desc* desc, int q_heads, int n_q) {
  if (tq::validate_desc(desc) != TQ_OK) return 0;
  if (desc->head_dim > tq::kMaxDecodeHeadDim || desc->batch > tq::kMaxBatch) return 0;
  if (q_heads < desc->kv_heads || q_heads % desc->kv_heads != 0) return 0;
  if (n_q < 1 || n_q > TQ_MAX_TREE_NODES) return 0;
  if ((long long)desc->batch * q_heads * n_q >= (1LL << 31)) return 0;
  return tq::tree_workspace_bytes(desc->batch, desc->kv_heads, q_heads, desc->head_dim, n_q);
}

int tq_decode_attention_tree(const tq_kv_desc* desc, const tq_codebook* k_cb, const tq_codebook* v_cb,
                             int q_heads, int n_q, const void* q, int q_dtype,
                             const uint8_t* k_codes, const uint16_t* k_norms, const uint8_t* v_codes,
                             const uint16_t* v_norms, const int32_t* seq_lens,
                             const int32_t* n_nodes, const uint64_t* tree, float scale, void* out,
                             int out_dtype, void* workspace, size_t workspace_bytes,
                             uint32_t* dev_status, void* stream) {
  if (!valid_dtype(q_dtype) || (out_dtype != TQ_F16 && out_dtype != TQ_BF16)) return TQ_ERR_INVALID_ARG;
  if (n_q < 1 || n_q > TQ_MAX_TREE_NODES) return TQ_ERR_INVALID_ARG;
  int st = tq::validate_decode(desc, k_cb, v_cb, q_heads, 1, q, TQ_F16, k_codes, k_norms, v_codes, v_norms,
                               seq_lens, scale, 0.0f, static_cast<const float*>(out), dev_status);
  if (st != TQ_OK) return st;
  if (!tree || !aligned(tree, 8) || !aligned(n_nodes, 4)) return TQ_ERR_INVALID_ARG;
  if ((long long)desc->batch * q_heads * n_q >= (1LL << 31)) return TQ_ERR_UNSUPPORTED;
  const size_t need = tq_tree_workspace_size(desc, q_heads, n_q);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return TQ_ERR_WORKSPACE;
  tq::TreeParams p{};
  p.q = q;
  p.out = out;
  p.k_codes = k_codes;
  p.k_norms = k_norms;
  p.v_codes = v_codes;
  p.v_norms = v_norms;
  p.seq_lens = seq_lens;
  p.n_nodes = n_nodes;
  p.tree = tree;
  p.status = dev_status;
  for (int j = 0; j < 16; ++j) {
    p.kcent[j] = j < (1 << desc->k_bits) ? k_cb->centroids[j] : 0.0f;
    p.vcent[j] = j < (1 << desc->v_bits) ? v_cb->centroids[j] : 0.0f;
  }
  tq::sign_bits(desc->sign_seed, p.sign_mask);
  p.q_dtype = q_dtype;
  p.out_dtype = out_dtype;
  p.k_bits = desc->k_bits;
  p.v_bits = desc->v_bits;
  p.batch = desc->batch;
  p.kv_heads = desc->kv_heads;
  p.q_heads = q_heads;
  p.head_dim = desc->head_dim;
  p.seq_cap = desc->seq_cap;
  p.n_q = n_q;
  p.score_mult = (float)((double)scale * 1.4426950408889634 / tq::kBlock);
  p.workspace = workspace;
  return tq::launch_tree(p, static_cast<cudaStream_t>(stream));
}

int tq_cache_compact(const tq_kv_desc* desc, const tq_cache_bufs* cache, const int32_t* keep,
                     int max_keep, const int32_t* n_keep, const int32_t* start, int32_t* new_lens,
                     uint32_t* dev_status, void* stream) {
  tq::CompactParams p{};
  const int st = check_cache(desc, cache, p.units);
  if (st != TQ_OK) return st;
  if (max_keep < 0 || !n_keep || (max_keep > 0 && !keep)) return TQ_ERR_INVALID_ARG;
  if (!aligned(keep, 4) || !aligned(n_keep, 4) || !aligned(start, 4) || !aligned(new_lens, 4) ||
      !aligned(dev_status, 4))
    return TQ_ERR_INVALID_ARG;
  // new_lens is written while other CTAs still read the lists
  const size_t per_seq = sizeof(int32_t) * (size_t)desc->batch;
  if (overlap(new_lens, per_seq, start, per_seq) || overlap(new_lens, per_seq, n_keep, per_seq) ||
      overlap(new_lens, per_seq, keep, per_seq * (size_t)max_keep))
    return TQ_ERR_INVALID_ARG;
  if ((long long)desc->batch * desc->kv_heads >= (1LL << 27)) return TQ_ERR_UNSUPPORTED;
  if (max_keep == 0 && !new_lens) return TQ_OK;
  p.c = view(desc, cache);
  p.kv_heads = desc->kv_heads;
  p.nb = desc->head_dim / tq::kBlock;
  p.max_keep = max_keep;
  p.keep = keep;
  p.n_keep = n_keep;
  p.start = start;
  p.new_lens = new_lens;
  p.status = dev_status;
  return tq::launch_cache_compact(p, static_cast<cudaStream_t>(stream));
}

int tq_cache_copy(const tq_kv_desc* src_desc, const tq_cache_bufs* src, const tq_kv_desc* dst_desc,
                  const tq_cache_bufs* dst, int n_copies, const int32_t* src_slot,
                  const int32_t* dst_slot, const int32_t* src_pos, const int32_t* dst_pos,
                  const int32_t* n_rows, int max_rows, uint32_t* dev_status, void* stream) {
  tq::CopyParams p{};
  int units[3];
  int st = check_cache(src_desc, src, p.units);
  if (st != TQ_OK) return st;
  if ((st = check_cache(dst_desc, dst, units)) != TQ_OK) return st;
  if (src_desc->kv_heads != dst_desc->kv_heads || src_desc->head_dim != dst_desc->head_dim ||
      src_desc->sign_seed != dst_desc->sign_seed || src_desc->k_bits != dst_desc->k_bits ||
      src_desc->v_bits != dst_desc->v_bits || src->outliers != dst->outliers)
    return TQ_ERR_INVALID_ARG;
  if (n_copies < 0 || max_rows < 0) return TQ_ERR_INVALID_ARG;
  if (n_copies > 0 && (!src_slot || !dst_slot || !n_rows)) return TQ_ERR_INVALID_ARG;
  if (!aligned(src_slot, 4) || !aligned(dst_slot, 4) || !aligned(src_pos, 4) || !aligned(dst_pos, 4) ||
      !aligned(n_rows, 4) || !aligned(dev_status, 4))
    return TQ_ERR_INVALID_ARG;
  if (n_copies == 0 || max_rows == 0) return TQ_OK;
  p.src = view(src_desc, src);
  p.dst = view(dst_desc, dst);
  p.kv_heads = src_desc->kv_heads;
  p.nb = src_desc->head_dim / tq::kBlock;
  p.n_copies = n_copies;
  p.max_rows = max_rows;
  p.src_slot = src_slot;
  p.dst_slot = dst_slot;
  p.src_pos = src_pos;
  p.dst_pos = dst_pos;
  p.n_rows = n_rows;
  p.status = dev_status;
  return tq::launch_cache_copy(p, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
