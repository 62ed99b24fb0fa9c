// Per-head RMS norm of q and k rows, position rotation, and the layouts that
// the cache and the decode kernels take, in one pass over a projection.
//
//   y = x / sqrt(mean(x^2) + eps) * w,   (a, b) -> g (a cos - b sin, b cos + a sin)
//
// Bound by HBM: every row is read once and written once and nothing else
// moves.  A group of LPR lanes (8, 16 or 32 for rows of up to 128, 256, 512)
// holds a row as two 8-element chunks per lane.  In the half layout (pairs
// (i, i + rot/2)) with rot/2 a multiple of 8 the two chunks are the two halves
// of the same pairs, and in the interleaved layout a chunk holds whole pairs,
// so the rotation stays in the lane; other half-layout widths fetch each
// element's partner from a shared copy of the row.
//
// The phase of (position, pair) is position * turns modulo 2^64, an exact
// integer product; its top 32 bits, reduced to the nearest quarter turn, leave
// at most 1/8 turn for sincospi, so far positions cost no accuracy.  A CTA
// takes TT tokens and computes each token's cosines once for all its heads.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tq_spec_internal.h"

namespace tq {
namespace {

constexpr int kRopeThreads = 256;

template <int DT>
struct Elem;
template <>
struct Elem<TQ_F32> {
  static constexpr int kVec = 2;  // uint4 words of an 8-element chunk
};
template <>
struct Elem<TQ_F16> {
  static constexpr int kVec = 1;
};
template <>
struct Elem<TQ_BF16> {
  static constexpr int kVec = 1;
};

template <int DT>
__device__ __forceinline__ void unpack8(const uint4 (&r)[Elem<DT>::kVec], float (&x)[8]) {
  if constexpr (DT == TQ_F32) {
    const uint32_t w[8] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  } else {
    const uint32_t w[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f;
      if constexpr (DT == TQ_F16) f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      else f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <int DT>
__device__ __forceinline__ void pack8(const float (&x)[8], uint4 (&r)[Elem<DT>::kVec]) {
  if constexpr (DT == TQ_F32) {
    r[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    r[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == TQ_F16) {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    r[0] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__device__ __forceinline__ float load_weight(const void* w, int dt, int i) {
  if (dt == TQ_F32) return static_cast<const float*>(w)[i];
  if (dt == TQ_F16) return __half2float(static_cast<const __half*>(w)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
}

// cos and sin of 2 pi * phase / 2^64
__device__ __forceinline__ float2 phase_cs(uint64_t phase) {
  const uint32_t top = (uint32_t)(phase >> 32);
  const uint32_t quarter = (top + 0x20000000u) >> 30;     // nearest quarter turn
  const int32_t rest = (int32_t)(top - (quarter << 30));  // in [-2^29, 2^29): 1/8 turn
  float s, c;
  sincospif((float)rest * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
  const float c1 = (quarter & 1u) ? -s : c, s1 = (quarter & 1u) ? c : s;
  return (quarter & 2u) ? make_float2(-c1, -s1) : make_float2(c1, s1);
}

// Shared memory: cos and sin [TT][D / 2], weights [2][D], then (GEN) one row
// of floats per group.
template <int IN, int OUT, int LPR, bool GEN>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p, int TT, FastDiv by_rows,
                                                            FastDiv by_seq) {
  constexpr int kGroups = kRopeThreads / LPR;
  constexpr int VI = Elem<IN>::kVec, VO = Elem<OUT>::kVec;
  extern __shared__ __align__(16) float sm[];
  const int D = p.head_dim, hp = p.rot_dim / 2, half_d = D / 2;
  float* cos_t = sm;
  float* sin_t = sm + TT * half_d;
  float* wts = sm + 2 * TT * half_d;
  float* scratch = wts + 2 * D;
  const int tid = threadIdx.x, sub = tid % LPR, group = tid / LPR;
  const uint32_t n_tokens = (uint32_t)p.batch * (uint32_t)p.seq_new;
  const uint32_t tok0 = blockIdx.x * (uint32_t)TT;
  const int toks = (int)min((uint32_t)TT, n_tokens - tok0);
  const int items = toks * p.rows;

  // chunk indices of this lane (see the file comment)
  const int hc = hp / 8;
  int ca, cb;
  if (!GEN && !p.interleaved && sub < hc) {
    ca = sub;
    cb = sub + hc;
  } else if (!GEN && !p.interleaved) {
    ca = 2 * hc + 2 * (sub - hc);
    cb = ca + 1;
  } else {
    ca = 2 * sub;
    cb = ca + 1;
  }
  const bool has = 16 * sub < D;  // rows of 384 leave the last lanes idle

  struct Where {
    const void* src;
    int b, t, side, head;
    bool live;
  };
  auto locate = [&](int item) {
    Where w{};
    const uint32_t tk = by_rows.div((uint32_t)item);
    int r = item - (int)tk * p.rows;
    const uint32_t token = tok0 + tk;
    w.b = (int)by_seq.div(token);
    w.t = (int)(token - (uint32_t)w.b * (uint32_t)p.seq_new);
    w.side = 0;
    if (r >= p.side[0].heads) {
      r -= p.side[0].heads;
      w.side = 1;
      if (r >= p.side[1].heads) {
        r -= p.side[1].heads;
        w.side = 2;
      }
    }
    w.head = r;
    const RowSide& s = p.side[w.side];
    const long long off = w.b * s.batch_stride + w.t * s.token_stride + r * s.head_stride;
    w.src = static_cast<const char*>(s.in) + off * (IN == TQ_F32 ? 4 : 2);
    w.live = !p.n_tok || w.t < __ldg(p.n_tok + w.b);
    return w;
  };
  auto load = [&](const Where& w, uint4 (&a)[VI], uint4 (&b)[VI]) {
    if (!has || !w.live) return;
    const uint4* src = static_cast<const uint4*>(w.src);
#pragma unroll
    for (int i = 0; i < VI; ++i) {
      a[i] = __ldcs(src + ca * VI + i);
      b[i] = __ldcs(src + cb * VI + i);
    }
  };

  // the first rows' loads are in flight while the tables are filled
  uint4 ra[VI] = {}, rb[VI] = {};
  Where cur{};
  if (group < items) {
    cur = locate(group);
    load(cur, ra, rb);
  }
  for (int i = tid; i < toks * hp; i += kRopeThreads) {
    const int tk = i / hp, m = i - tk * hp;
    const long long pos = __ldg(p.positions + tok0 + tk);
    const float2 cs = phase_cs((uint64_t)pos * p.turns[m]);
    cos_t[tk * half_d + m] = p.gain * cs.x;
    sin_t[tk * half_d + m] = p.gain * cs.y;
  }
  if (p.norm)
    for (int i = tid; i < 2 * D; i += kRopeThreads) {
      const void* w = p.side[i / D].weight;
      wts[i] = (w ? load_weight(w, p.w_dtype, i % D) : 1.0f) + p.weight_bias;
    }
  __syncthreads();

  for (int item = group; item - group < items; item += kGroups) {
    const bool mine = item < items;
    Where w = cur;
    float xa[8], xb[8];
    unpack8<IN>(ra, xa);
    unpack8<IN>(rb, xb);
    if (item + kGroups < items) {
      cur = locate(item + kGroups);
      load(cur, ra, rb);
    }
    const bool rotated = w.side < 2;
    if (p.norm) {  // every lane takes part in the shuffles
      float ss = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(xa[k], xa[k], fmaf(xb[k], xb[k], ss));
      if (!has || !mine) ss = 0.0f;
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (rotated && has) {
        const float inv = 1.0f / sqrtf(ss / (float)D + p.eps);
        const float* wt = wts + w.side * D;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          xa[k] *= inv * wt[8 * ca + k];
          xb[k] *= inv * wt[8 * cb + k];
        }
      }
    }
    const int tk = (int)by_rows.div((uint32_t)min(item, items - 1));
    if (hp > 0) {
      const float* ct = cos_t + tk * half_d;
      const float* st = sin_t + tk * half_d;
      if constexpr (GEN) {
        float* row = scratch + group * (D + 4);
        if (has) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            row[8 * ca + k] = xa[k];
            row[8 * cb + k] = xb[k];
          }
        }
        __syncwarp();
        if (rotated && has) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int e = 16 * sub + k;
            float& x = k < 8 ? xa[k & 7] : xb[k & 7];
            if (e < hp) x = x * ct[e] - row[e + hp] * st[e];
            else if (e < 2 * hp) x = x * ct[e - hp] + row[e - hp] * st[e - hp];
          }
        }
        __syncwarp();
      } else if (rotated && has) {
        if (p.interleaved) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {  // pairs 8 sub + k: four in each chunk
            const int m = 8 * sub + k;
            float& a = k < 4 ? xa[(2 * k) & 7] : xb[(2 * k) & 7];
            float& b = k < 4 ? xa[(2 * k + 1) & 7] : xb[(2 * k + 1) & 7];
            if (m < hp) {
              const float c = ct[m], s = st[m], a0 = a;
              a = a0 * c - b * s;
              b = b * c + a0 * s;
            }
          }
        } else if (sub < hc) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float c = ct[8 * sub + k], s = st[8 * sub + k], a0 = xa[k];
            xa[k] = a0 * c - xb[k] * s;
            xb[k] = xb[k] * c + a0 * s;
          }
        }
      }
    }
    if (mine && has && w.live) {
      const RowSide& s = p.side[w.side];
      const size_t row = w.side == 0 ? ((size_t)w.b * p.seq_new + w.t) * s.heads + w.head
                                     : ((size_t)w.b * s.heads + w.head) * p.seq_new + w.t;
      uint4* dst = static_cast<uint4*>(s.out) + row * (size_t)(D / 8 * VO);
      uint4 oa[VO], ob[VO];
      pack8<OUT>(xa, oa);
      pack8<OUT>(xb, ob);
#pragma unroll
      for (int i = 0; i < VO; ++i) {
        dst[ca * VO + i] = oa[i];
        dst[cb * VO + i] = ob[i];
      }
    }
  }
}

template <int IN, int OUT, int LPR, bool GEN>
int run_rope(const RopeParams& p, cudaStream_t stream) {
  // One token per CTA while the GPU is not full, then four: the table of
  // cosines is filled by all threads at once.
  const long long tokens = (long long)p.batch * p.seq_new;
  const int TT = tokens > 4 * 148 * 4 ? 4 : 1;
  const size_t smem = sizeof(float) * ((size_t)TT * p.head_dim + 2 * p.head_dim +
                                       (GEN ? (size_t)(kRopeThreads / LPR) * (p.head_dim + 4) : 0));
  rope_kernel<IN, OUT, LPR, GEN><<<(unsigned)((tokens + TT - 1) / TT), kRopeThreads, smem, stream>>>(
      p, TT, FastDiv::make((uint32_t)p.rows), FastDiv::make((uint32_t)p.seq_new));
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

template <int IN, int OUT>
int dispatch_lpr(const RopeParams& p, cudaStream_t stream) {
  const bool gen = p.rot_dim > 0 && !p.interleaved && (p.rot_dim / 2) % 8 != 0;
  if (p.head_dim <= 128) return gen ? run_rope<IN, OUT, 8, true>(p, stream) : run_rope<IN, OUT, 8, false>(p, stream);
  if (p.head_dim <= 256) return gen ? run_rope<IN, OUT, 16, true>(p, stream) : run_rope<IN, OUT, 16, false>(p, stream);
  return gen ? run_rope<IN, OUT, 32, true>(p, stream) : run_rope<IN, OUT, 32, false>(p, stream);
}

template <int IN>
int dispatch_out(const RopeParams& p, cudaStream_t stream) {
  switch (p.out_dtype) {
    case TQ_F32: return dispatch_lpr<IN, TQ_F32>(p, stream);
    case TQ_F16: return dispatch_lpr<IN, TQ_F16>(p, stream);
  }
  return dispatch_lpr<IN, TQ_BF16>(p, stream);
}

}  // namespace

int launch_qk_norm_rope(const RopeParams& p, cudaStream_t stream) {
  switch (p.in_dtype) {
    case TQ_F32: return dispatch_out<TQ_F32>(p, stream);
    case TQ_F16: return dispatch_out<TQ_F16>(p, stream);
  }
  return dispatch_out<TQ_BF16>(p, stream);
}

}  // namespace tq
