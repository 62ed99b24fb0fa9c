// Internal interface between the host layer of the speculative-decoding
// operators (tq_spec_host.cpp) and their sm_100a kernels.
#pragma once

#include "../../include/tq_spec.h"
#include "tq_internal.h"

namespace tq {

struct RowSide {
  const void* in;
  void* out;
  const void* weight;
  long long batch_stride, token_stride, head_stride;  // elements
  int heads;
};

struct RopeParams {
  RowSide side[3];  // q, k, v (heads = 0: absent)
  int batch, seq_new, head_dim, rows;  // rows: heads of the three sides together
  int rot_dim, interleaved;
  int in_dtype, w_dtype, out_dtype;
  int norm;
  float eps, weight_bias, gain;
  const int32_t* positions;
  const int32_t* n_tok;
  uint64_t turns[TQ_MAX_ROT_DIM / 2];
};
int launch_qk_norm_rope(const RopeParams& p, cudaStream_t stream);

// The row parts of a cache as 16-byte units: K codes, V codes, v3 values.
struct CacheView {
  uint8_t* codes[3];   // K codes, V codes, v3 values (null: none)
  uint16_t* norms[2];
  int batch, seq_cap;
};
struct CompactParams {
  CacheView c;
  int units[3];        // 16-byte units per row of each part
  int kv_heads, nb, max_keep;
  const int32_t* keep;
  const int32_t* n_keep;
  const int32_t* start;
  int32_t* new_lens;
  uint32_t* status;
};
int launch_cache_compact(const CompactParams& p, cudaStream_t stream);

struct CopyParams {
  CacheView src, dst;
  int units[3];
  int kv_heads, nb, n_copies, max_rows;
  const int32_t* src_slot;
  const int32_t* dst_slot;
  const int32_t* src_pos;
  const int32_t* dst_pos;
  const int32_t* n_rows;
  uint32_t* status;
};
int launch_cache_copy(const CopyParams& p, cudaStream_t stream);

struct TreeParams {
  const void* q;
  void* out;
  const uint8_t* k_codes;
  const uint16_t* k_norms;
  const uint8_t* v_codes;
  const uint16_t* v_norms;
  const int32_t* seq_lens;
  const int32_t* n_nodes;
  const uint64_t* tree;
  uint32_t* status;
  float kcent[16], vcent[16];
  uint32_t sign_mask[4];
  int q_dtype, out_dtype;
  int k_bits, v_bits;
  int batch, kv_heads, q_heads, head_dim, seq_cap, n_q;
  float score_mult;  // scale * log2(e) / 128
  int wait_tries;    // limit of a wait inside the kernel, set by launch_tree
  void* workspace;
};
size_t tree_workspace_bytes(int batch, int kv_heads, int q_heads, int head_dim, int n_q);
int launch_tree(const TreeParams& p, cudaStream_t stream);

// of tq_host.cpp
void sign_bits(uint64_t seed, uint32_t mask[4]);
int validate_desc(const tq_kv_desc* d);

}  // namespace tq
