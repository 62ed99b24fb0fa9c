// Attention of a tree of drafted tokens over the packed cache.
//
// For query row (node j, head h) of sequence b, with q^ = H (s o q) per block:
//   x_t = scale / 128 * sum_blk nK_t q^ . cK[idx_t],  t visible to j,
//   w = softmax(x), o = s o H (sum_t w_t nV_t / 128 cV[idx_t]).
//
// One CTA per row: a tile of 128 positions is scored by 128 threads, then
// each thread adds the tile to its dimension of the output.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tq_spec_internal.h"

namespace tq {
namespace {

constexpr int kTreeTile = 128;

__device__ __forceinline__ float load_q(const TreeParams& p, size_t i) {
  if (p.q_dtype == TQ_F32) return static_cast<const float*>(p.q)[i];
  if (p.q_dtype == TQ_F16) return __half2float(static_cast<const __half*>(p.q)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[i]);
}

__device__ __forceinline__ uint32_t code_at(const uint8_t* row, int bits, int i) {
  const int bit = bits * i;
  uint32_t w = row[bit >> 3];
  if ((bit & 7) + bits > 8) w |= (uint32_t)row[(bit >> 3) + 1] << 8;
  return (w >> (bit & 7)) & ((1u << bits) - 1u);
}

__device__ void block_wht(float* x, int D, int tid) {  // 128 threads
  for (int m = 1; m < kBlock; m <<= 1) {
    __syncthreads();
    float r[2];
    for (int k = 0; k * kBlock < D; ++k) {
      const float a = x[k * kBlock + tid], b = x[k * kBlock + (tid ^ m)];
      r[k] = (tid & m) ? b - a : a + b;
    }
    __syncthreads();
    for (int k = 0; k * kBlock < D; ++k) x[k * kBlock + tid] = r[k];
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kTreeTile) tree_rows_kernel(const __grid_constant__ TreeParams p) {
  __shared__ float qs[kMaxDecodeHeadDim], os[kMaxDecodeHeadDim], ps[kTreeTile], red[4];
  __shared__ float kc[16], vc[16];
  const int tid = threadIdx.x, D = p.head_dim, nb = D / kBlock;
  const int h = (int)(blockIdx.x % (unsigned)p.q_heads);
  const int j = (int)(blockIdx.x / (unsigned)p.q_heads % (unsigned)p.n_q);
  const int b = (int)(blockIdx.x / (unsigned)p.q_heads / (unsigned)p.n_q);
  const int raw_len = p.seq_lens[b], raw_n = p.n_nodes ? p.n_nodes[b] : p.n_q;
  const int len = min(max(raw_len, 0), p.seq_cap), n = min(max(raw_n, 0), p.n_q);
  if ((len != raw_len || n != raw_n) && tid == 0 && p.status) atomicOr(p.status, TQ_DEV_LEN_RANGE);
  if (j >= n) return;
  const int ctx = len - n;
  const uint64_t seen = p.tree[(size_t)b * p.n_q + j];
  const size_t row = ((size_t)b * p.n_q + j) * p.q_heads + h;
  const int kvh = h / (p.q_heads / p.kv_heads);
  const size_t base = ((size_t)b * p.kv_heads + kvh) * p.seq_cap;
  if (tid < 16) {
    kc[tid] = p.kcent[tid];
    vc[tid] = p.vcent[tid];
  }
  const bool neg = (p.sign_mask[tid >> 5] >> (tid & 31)) & 1u;
  for (int k = 0; k < nb; ++k) {
    const float x = load_q(p, row * D + k * kBlock + tid);
    qs[k * kBlock + tid] = neg ? -x : x;
  }
  block_wht(qs, D, tid);
  float m = -INFINITY, l = 0.0f, acc[2] = {0.0f, 0.0f};
  for (int t0 = 0; t0 < len; t0 += kTreeTile) {
    const int t = t0 + tid, node = t - ctx;
    float x = -INFINITY;
    const bool sees = t < len && (node < 0 || ((seen >> node) & 1u));
    if (sees) {
      x = 0.0f;
      for (int k = 0; k < nb; ++k) {
        const uint8_t* codes = p.k_codes + ((base + t) * nb + k) * 16 * p.k_bits;
        float s = 0.0f;
        for (int i = 0; i < kBlock; ++i) s = fmaf(qs[k * kBlock + i], kc[code_at(codes, p.k_bits, i)], s);
        x = fmaf(s, __half2float(__ushort_as_half(p.k_norms[(base + t) * nb + k])), x);
      }
      x *= p.score_mult;
    }
    float mx = x;
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    mx = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float alpha = mx == -INFINITY ? 1.0f : exp2f(m - mx);
    ps[tid] = !sees ? -1.0f : x == -INFINITY ? 0.0f : exp2f(x - mx);  // -1: not seen
    m = mx;
    __syncthreads();
    l *= alpha;
    for (int k = 0; k < nb; ++k) acc[k] *= alpha;
    for (int i = 0; i < kTreeTile && t0 + i < len; ++i) {
      const float w = ps[i];
      if (w == -1.0f) continue;
      l += w;
      for (int k = 0; k < nb; ++k) {
        const size_t r = (base + t0 + i) * nb + k;
        const float nv = __half2float(__ushort_as_half(p.v_norms[r]));
        acc[k] = fmaf(w * nv, vc[code_at(p.v_codes + r * 16 * p.v_bits, p.v_bits, tid)], acc[k]);
      }
    }
    __syncthreads();
  }
  for (int k = 0; k < nb; ++k) os[k * kBlock + tid] = acc[k];
  block_wht(os, D, tid);
  const float inv = l > 0.0f || l != l ? 1.0f / (l * kBlock) : 0.0f;
  for (int k = 0; k < nb; ++k) {
    const float x = os[k * kBlock + tid] * (neg ? -inv : inv);
    if (p.out_dtype == TQ_F16) static_cast<__half*>(p.out)[row * D + k * kBlock + tid] = __float2half_rn(x);
    else static_cast<__nv_bfloat16*>(p.out)[row * D + k * kBlock + tid] = __float2bfloat16_rn(x);
  }
}

}  // namespace

size_t tree_workspace_bytes(int, int, int, int, int) { return 256; }

int launch_tree(const TreeParams& p, cudaStream_t stream) {
  const long long rows = (long long)p.batch * p.n_q * p.q_heads;
  if (rows >= (1LL << 31)) return TQ_ERR_UNSUPPORTED;
  tree_rows_kernel<<<(unsigned)rows, kTreeTile, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // namespace tq
