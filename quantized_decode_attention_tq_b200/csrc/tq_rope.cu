// Per-head RMS norm of q and k rows, position rotation, and the layouts that
// the cache and the decode kernels take, in one pass over a projection.
//
//   y = x / sqrt(mean(x^2) + eps) * w,   (a, b) -> g (a cos - b sin, b cos + a sin)
//
// Bound by HBM: every row is read once and written once and nothing else
// moves.  A group of LPR lanes (8, 16 or 32 for rows of up to 128, 256, 512)
// holds a row as two 8-element chunks per lane and loads the next row while it
// works on one.  In the half layout (pairs (i, i + rot/2)) with rot/2 a
// multiple of 8 the two chunks are the two halves of the same pairs, and in
// the interleaved layout a chunk holds whole pairs, so the rotation stays in
// the lane; other half-layout widths fetch each element's partner from a
// shared copy of the row, whose padding keeps the lanes on different banks.
// Measured on 8 x 4096 tokens of 48 rows of 128 in bf16 to fp16: 148 us in
// both layouts, 83 % of a copy's rate; 253 us at a half-layout width of 100
// (308 us when lanes held 16 consecutive elements, padded per 16).
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
constexpr int kMaxTT = 8;

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

// two fp32 operations in one instruction
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{ .reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z; }"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{ .reg .b64 x, y, z, w; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7};\n"
      "fma.rn.f32x2 w, x, y, z; mov.b64 {%0, %1}, w; }"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
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

// Where element e of a row or table lies in shared memory when lanes hold 8
// consecutive ones (kAnyHalves): a word of padding per 8, so that lanes 8
// elements apart use different banks; rows of a warp's groups are spaced so
// that all 32 do (lane s of group g at bank 9 (s + LPR g)).
__device__ __forceinline__ int padded(int e) { return e + (e >> 3); }
__host__ __device__ constexpr int row_pitch(int d, int lpr) { return d + d / 8 + (lpr == 8 ? 24 : lpr == 16 ? 16 : 0); }

enum Layout { kHalves = 0, kNeighbours = 1, kAnyHalves = 2 };  // kAnyHalves: rot/2 not a multiple of 8

// Shared memory: cos and sin [TT][pitch], weights [2][D], then (kAnyHalves) one
// row of floats per group.
template <int IN, int OUT, int LPR, int MODE>
__global__ void __launch_bounds__(kRopeThreads, IN == TQ_F32 || MODE == kAnyHalves ? 3 : 4)
rope_kernel(const __grid_constant__ RopeParams p, int TT, FastDiv by_rows, FastDiv by_seq) {
  constexpr bool GEN = MODE == kAnyHalves, split = MODE == kHalves;
  constexpr int kGroups = kRopeThreads / LPR;
  constexpr int VI = Elem<IN>::kVec, VO = Elem<OUT>::kVec, kIn = IN == TQ_F32 ? 4 : 2, kOut = OUT == TQ_F32 ? 4 : 2;
  struct Base {
    const char* in;  // null: a token that is left alone
    char* out;
  };
  struct Step {
    long long in, out;  // bytes from one head to the next
  };
  __shared__ Base base[kMaxTT][4];
  __shared__ Step step[4];
  extern __shared__ __align__(16) float sm[];
  const int D = p.head_dim, hp = p.rot_dim / 2, half_d = D / 2;
  const int pitch = GEN ? half_d + half_d / 8 : half_d;  // of a token's table
  float* cos_t = sm;
  float* sin_t = sm + TT * pitch;
  float* wts = sm + 2 * TT * pitch;
  float* scratch = wts + 2 * D;
  const int tid = threadIdx.x, sub = tid % LPR, group = tid / LPR;
  const uint32_t n_tokens = (uint32_t)p.batch * (uint32_t)p.seq_new;
  const uint32_t tok0 = blockIdx.x * (uint32_t)TT;
  const int toks = (int)min((uint32_t)TT, n_tokens - tok0);
  const int items = toks * p.rows;
  const float inv_d = 1.0f / (float)D;
  const int end_q = p.side[0].heads, end_k = end_q + p.side[1].heads;

  // chunk indices of this lane (see the file comment)
  const int hc = hp / 8;
  // (otherwise chunks sub and sub + D / 16, so that lanes read side by side)
  const int ca = split ? (sub < hc ? sub : 2 * hc + 2 * (sub - hc)) : sub;
  const int cb = split ? (sub < hc ? sub + hc : ca + 1) : sub + D / 16;
  const bool has = 16 * sub < D;  // rows of 384 leave the last lanes idle
  // this lane's pairs: ma .. ma + 3 and mb .. mb + 3; whether all or some of them turn
  const int ma = split ? 8 * sub : 4 * ca, mb = split ? ma + 4 : 4 * cb;
  const bool all = !GEN && has && mb + 4 <= hp, some = !GEN && has && ma < hp;

  // where each token's rows of each side begin
  if (tid < 3 * toks) {
    const int tk = tid / 3, s = tid - 3 * tk;
    const RowSide& side = p.side[s];
    const uint32_t token = tok0 + (uint32_t)tk;
    const int b = (int)by_seq.div(token), t = (int)(token - (uint32_t)b * (uint32_t)p.seq_new);
    Base x{nullptr, nullptr};
    if (!p.n_tok || t < __ldg(p.n_tok + b)) {
      const long long row = s == 0 ? ((long long)b * p.seq_new + t) * side.heads : (long long)b * side.heads * p.seq_new + t;
      x.in = static_cast<const char*>(side.in) + (b * side.batch_stride + t * side.token_stride) * kIn;
      x.out = static_cast<char*>(side.out) + row * (D * kOut);
    }
    base[tk][s] = x;
    if (tk == 0) step[s] = Step{side.head_stride * kIn, (s == 0 ? 1LL : (long long)p.seq_new) * (D * kOut)};
  }
  __syncthreads();

  struct Row {
    uint4 a[VI], b[VI];
    char* out;  // null: nothing to write
    int token, side;
  } cur;
  auto load = [&](int item) {
    const int tk = (int)by_rows.div((uint32_t)min(item, items - 1)), r = min(item, items - 1) - tk * p.rows;
    const int s = r < end_q ? 0 : r < end_k ? 1 : 2, h = r - (s == 0 ? 0 : s == 1 ? end_q : end_k);
    const Base x = base[tk][s];
    const Step d = step[s];
    cur.token = tk;
    cur.side = s;
    cur.out = item < items && has && x.in ? x.out + h * d.out : nullptr;
    if (cur.out) {
      const uint4* src = reinterpret_cast<const uint4*>(x.in + h * d.in);
#pragma unroll
      for (int i = 0; i < VI; ++i) {
        cur.a[i] = __ldcs(src + ca * VI + i);
        cur.b[i] = __ldcs(src + cb * VI + i);
      }
    }
  };

  load(group);  // in flight while the tables are filled
  for (int i = tid; i < toks * hp; i += kRopeThreads) {
    const int tk = i / hp, m = i - tk * hp;
    const long long pos = __ldg(p.positions + tok0 + tk);
    const float2 c = phase_cs((uint64_t)pos * p.turns[m]);
    const int at = tk * pitch + (GEN ? padded(m) : m);
    cos_t[at] = p.gain * c.x;
    sin_t[at] = p.gain * c.y;
  }
  if (p.norm)
    for (int i = tid; i < 2 * D; i += kRopeThreads) {
      const int s = i >= D ? 1 : 0;
      const void* w = p.side[s].weight;
      wts[i] = (w ? load_weight(w, p.w_dtype, i - s * D) : 1.0f) + p.weight_bias;
    }
  __syncthreads();

  for (int item = group; item - group < items; item += kGroups) {
    const int s = cur.side;
    char* const out = cur.out;
    const float* ct = cos_t + cur.token * pitch;
    const float* st = sin_t + cur.token * pitch;
    float xa[8], xb[8];  // the lane's two chunks
    unpack8<IN>(cur.a, xa);
    unpack8<IN>(cur.b, xb);
    load(item + kGroups);
    if (p.norm) {  // every lane takes part in the shuffles
      float2 q = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        q = fma2(make_float2(xa[k], xa[k + 1]), make_float2(xa[k], xa[k + 1]), q);
        q = fma2(make_float2(xb[k], xb[k + 1]), make_float2(xb[k], xb[k + 1]), q);
      }
      float ss = out ? q.x + q.y : 0.0f;
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (s < 2 && has) {
        const float inv = rsqrtf(fmaf(ss, inv_d, p.eps));
        const float2 i2 = make_float2(inv, inv);
        const float4* wa = reinterpret_cast<const float4*>(wts + s * D + 8 * ca);
        const float4* wb = reinterpret_cast<const float4*>(wts + s * D + 8 * cb);
        const float4 a0 = wa[0], a1 = wa[1], b0 = wb[0], b1 = wb[1];
        const float2 ea[4] = {{a0.x, a0.y}, {a0.z, a0.w}, {a1.x, a1.y}, {a1.z, a1.w}};
        const float2 eb[4] = {{b0.x, b0.y}, {b0.z, b0.w}, {b1.x, b1.y}, {b1.z, b1.w}};
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const float2 x = mul2(make_float2(xa[k], xa[k + 1]), mul2(ea[k / 2], i2));
          const float2 y = mul2(make_float2(xb[k], xb[k + 1]), mul2(eb[k / 2], i2));
          xa[k] = x.x, xa[k + 1] = x.y;
          xb[k] = y.x, xb[k + 1] = y.y;
        }
      }
    }
    if (s < 2 && some) {
      const float4 c0 = *reinterpret_cast<const float4*>(ct + ma), c1 = *reinterpret_cast<const float4*>(ct + mb);
      const float4 n0 = *reinterpret_cast<const float4*>(st + ma), n1 = *reinterpret_cast<const float4*>(st + mb);
      if constexpr (split) {  // pairs (xa[k], xb[k]), two at a time
        const float2 cs[4] = {{c0.x, c0.y}, {c0.z, c0.w}, {c1.x, c1.y}, {c1.z, c1.w}};
        const float2 sn[4] = {{n0.x, n0.y}, {n0.z, n0.w}, {n1.x, n1.y}, {n1.z, n1.w}};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 c = cs[k], n = sn[k];
          const float2 x = make_float2(xa[2 * k], xa[2 * k + 1]), y = make_float2(xb[2 * k], xb[2 * k + 1]);
          const float2 z = mul2(y, n), o = fma2(x, c, make_float2(-z.x, -z.y)), q = fma2(y, c, mul2(x, n));
          xa[2 * k] = o.x, xa[2 * k + 1] = o.y;
          xb[2 * k] = q.x, xb[2 * k + 1] = q.y;
        }
      } else {  // pairs of neighbours, perhaps not all turning
        const float cs[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        const float sn[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float& x = k < 4 ? xa[(2 * k) & 7] : xb[(2 * k) & 7];
          float& y = k < 4 ? xa[(2 * k + 1) & 7] : xb[(2 * k + 1) & 7];
          if (all || (k < 4 ? ma + k : mb + k - 4) < hp) {
            const float o = x * cs[k] - y * sn[k];
            y = y * cs[k] + x * sn[k];
            x = o;
          }
        }
      }
    }
    if constexpr (GEN) {
      float* copy = scratch + group * row_pitch(D, LPR);
      if (has) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          copy[9 * ca + k] = xa[k];
          copy[9 * cb + k] = xb[k];
        }
      }
      __syncwarp();
      if (s < 2 && has) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int e = k < 8 ? 8 * ca + k : 8 * cb + k - 8;
          float& x = k < 8 ? xa[k & 7] : xb[k & 7];
          if (e < 2 * hp) {
            const int m = e < hp ? e : e - hp;
            const float n = st[padded(m)];
            x = fmaf(copy[padded(e < hp ? e + hp : m)], e < hp ? -n : n, x * ct[padded(m)]);
          }
        }
      }
      __syncwarp();
    }
    if (out) {
      uint4* dst = reinterpret_cast<uint4*>(out);
      uint4 oa[VO], ob[VO];
      pack8<OUT>(xa, oa);
      pack8<OUT>(xb, ob);
#pragma unroll
      for (int k = 0; k < VO; ++k) {
        dst[ca * VO + k] = oa[k];
        dst[cb * VO + k] = ob[k];
      }
    }
  }
}

template <int IN, int OUT, int LPR, int MODE>
int run_rope(const RopeParams& p, cudaStream_t stream) {
  // One token per CTA, and more while that leaves every SM sixteen CTAs: the
  // tables are filled by all threads at once, but a last wave of few CTAs
  // costs more (4004 tokens of 24 rows: 31 us at eight tokens a CTA, 24.7 at two).
  constexpr int kGroups = kRopeThreads / LPR;
  const int D = p.head_dim, pitch = MODE == kAnyHalves ? D / 2 + D / 16 : D / 2;
  const long long tokens = (long long)p.batch * p.seq_new;
  int TT = 1;
  while (TT < kMaxTT && tokens > (long long)TT * 16 * 148) TT *= 2;
  const size_t smem = sizeof(float) * ((size_t)2 * TT * pitch + 2 * D + (MODE == kAnyHalves ? kGroups * row_pitch(D, LPR) : 0));
  rope_kernel<IN, OUT, LPR, MODE><<<(unsigned)((tokens + TT - 1) / TT), kRopeThreads, smem, stream>>>(
      p, TT, FastDiv::make((uint32_t)p.rows), FastDiv::make((uint32_t)p.seq_new));
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

template <int IN, int OUT, int LPR>
int dispatch_mode(const RopeParams& p, cudaStream_t stream) {
  if (p.interleaved) return run_rope<IN, OUT, LPR, kNeighbours>(p, stream);
  if ((p.rot_dim / 2) % 8 != 0) return run_rope<IN, OUT, LPR, kAnyHalves>(p, stream);
  return run_rope<IN, OUT, LPR, kHalves>(p, stream);
}

template <int IN, int OUT>
int dispatch_lpr(const RopeParams& p, cudaStream_t stream) {
  if (p.head_dim <= 128) return dispatch_mode<IN, OUT, 8>(p, stream);
  if (p.head_dim <= 256) return dispatch_mode<IN, OUT, 16>(p, stream);
  return dispatch_mode<IN, OUT, 32>(p, stream);
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
