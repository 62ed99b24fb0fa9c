// Attention of a tree of drafted tokens over the packed cache.
//
// For query row (node j, head h) of sequence b, with q^ = H (s o q) per block:
//   x_t = scale / 128 * sum_blk nK_t q^ . cK[idx_t],  t visible to j,
//   w = softmax(x), o = s o H (sum_t w_t nV_t / 128 cV[idx_t]).
//
// Mapping.  A unit is a (sequence, kv-head, group of up to N query rows); the
// rows of a kv-head (nodes x heads of the group) share its K and V.  All
// 128-position tiles of all units are laid end to end and cut evenly over one
// persistent CTA per SM (tq_tree_cut.h).  Per tile, codes become fp16 once for all N rows:
//   S^T [128 positions x N rows] = K^ [128 x D] . Q^T     (tcgen05, M = 128)
//   O^T [128 dims x N rows]     += V^T [128 x 128] . P    per 128-block
// Positions are the MMA's rows, so N adapts to the tree (16 to 128 columns), a
// thread owns one position (its two norms are registers), and both operands
// made from codes are written in the cache's own order: K^ as rows of tensor
// memory, V^ as M-major and P as N-major rows of shared memory, 128-byte
// swizzled.  Shared-memory bandwidth ran out first (table lookups, V^ and P in
// and out: 96% taken with K^ there too), so K^ does not pass through it.
//
// Softmax in the log2 domain with a lazy reference maximum per row: a tile is
// scored against it, and only when some score exceeds it by 2^kTau do the
// warps reduce the tile's maxima and rescale O in tensor memory.  The norm of
// V multiplies the weight, scaled by a power of two so that fp16 holds it.
//
// Roundings to fp16, all others are fp32: the query is split in two fp16 terms
// (two MMAs), the centroids are scaled by a factor that makes their rounding
// small (centroid_scale), and weight * norm is rounded once.  A row group's
// queries share one power-of-two scale (a scale per row would cost the softmax a
// product per score), and a part's V norms another.
//
// What it measured (on the device, one B200; a pass through the binding takes
// some 6 us more): trees of 16 nodes on 8 x 32768 positions of 3 + 3 bits
// 166 us, 64 nodes on 131072 of 4 + 2 bits 269 us.  A tile of 64 columns takes
// about 2500 cycles and 6500 warp instructions (1300 for K, 930 for V, 3600 in
// the softmax) with 57% of the issue slots, 60% of the shared-memory bandwidth
// and 24% of the tensor pipe taken: no unit is full, the latencies of its 28
// warps bind.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <type_traits>

#include "tq_spec_internal.h"
#include "tq_tree_cut.h"

namespace tq {
namespace tree {
namespace {

constexpr int kTok = 128;  // positions per tile

// Roles by warpgroup (four warps): softmax groups of 128 threads, each with its
// share of the row group's columns; one group that turns K codes into fp16 and
// one for V; one whose warps issue the score MMAs, the V MMAs and the copies.
// Four softmax groups from 64 columns on: with two, 64 columns took 198 us
// where four take 188 (8 x 32768 positions).  Registers per thread at launch,
// then by role; the shares must fit the launch's total.  Other splits were 3 to
// 25% slower.  With this one a thread spills up to 8 bytes in heads of one block
// at 16 to 64 columns, 52 at 128, and 72 to 216 in heads of two.
template <int N>
struct Roles {
  static constexpr int kGroups = N >= 64 ? 4 : 2;
  static constexpr int kSoftWarps = 4 * kGroups, kCodeWarp = kSoftWarps, kMmaWarp = kSoftWarps + 8;
  static constexpr int kWarps = kMmaWarp + 4, kThreads = 32 * kWarps;
  static constexpr int kLaunch = kGroups == 4 ? 72 : 96;
  static constexpr int kSoft = kGroups == 4 ? 80 : 136, kCodes = kGroups == 4 ? 64 : 72, kMma = kGroups == 4 ? 56 : 64;
  static_assert(kGroups * kSoft + 2 * kCodes + kMma <= (kWarps / 4) * kLaunch, "register split");
};

constexpr int kMaxGrid = 256;       // CTAs at most (slots of the workspace)
constexpr uint32_t kBase = 1024;    // shared-window address of dynamic shared memory
constexpr uint32_t kMaxDyn = 227 * 1024;
constexpr float kTau = 6.0f;        // log2: how far a score may exceed the reference maximum
constexpr float kUnset = -1e30f;    // reference of a row that has seen no position
// V norms are scaled by a power of two that puts the largest one seen when it
// is chosen at 2^7: norms down to 2^-21 of it keep full fp16 precision at weight
// 1, and the scale is chosen anew when one exceeds 2^9 (2^(6 + 9) fits fp16).
constexpr int kNormTop = 7;
constexpr float kNormRoom = 512.0f;
// The scale before one is chosen: the smallest norm that is not zero exceeds it,
// so the first tile that holds one chooses (until then the sum over V is zero).
constexpr float kNoScale = 0x1p100f;
constexpr uint32_t kPanel = 128 * 128;  // bytes of a 64-element x 128-row panel

struct Plan {
  uint32_t bytes;
  uint32_t q, vt, pt;           // Q^ (hi, lo), V^ stages, P stages
  uint32_t lut_k, lut_v;
  uint32_t ring_k, ring_v;      // code rings, a tile per slot
  uint32_t bar, misc, prefix;
  int v_stages, p_stages, depth;
};

// fp16 levels of a codebook by bytes: low bytes of levels 0-3 and 4-7, high bytes of the same
struct Levels {
  uint32_t lo0, lo1, hi0, hi1;
};

// What the join kernel needs of the unit that a CTA's range starts inside of:
// parts first - 1 .. last (of the split) hold it.
struct Join {
  int b, kvh, hg, first, last, nodes;  // first = 0: the CTA's range starts with a unit, or the cut was not its first
};

struct Params {
  TreeParams t;
  Plan pl;
  float kscale, vscale;         // centroid scales
  Levels klev;                  // K levels of 2- and 3-bit codes
  int n_hg;                     // row groups per kv-head
  FastDiv group;                // q_heads / kv_heads
  // workspace
  float* ws_mul;                // [units] factor of a unit's scores
  uint8_t* ws_q;                // [units] Q^ as it lies in shared memory
  Join* ws_join;                // [grid]
  float* ws_ml;                 // [2 * grid][N][2]
  float* ws_acc;                // [2 * grid][N][D]
};

// ------------------------------------------------------------- primitives --

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t x;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(a));
  return x;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a));
  return x;
}
__device__ __forceinline__ float4 lds128f(uint32_t a) {
  float4 x;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(a));
  return x;
}
// a code table never changes after the prologue: the compiler may move these
__device__ __forceinline__ uint32_t lds_table(uint32_t a) {
  uint32_t x;
  asm("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(a));
  return x;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t a, unsigned short x) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(a), "h"(x) : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ void bar_init(uint32_t a, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(a), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t a) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(a) : "memory");
}
// Copy `bytes` (a multiple of 16) and let the barrier expect them.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t a, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.b32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(a), "r"(parity), "n"(1000)
      : "memory");
  return ok != 0;
}
// Wait for a phase, for at most as many tries of about a microsecond as the
// limit word says.  One that runs out sets the word to zero (aborted) and
// reports it.  From then on every wait returns at once, no copy is issued, the
// loops run to their end on whatever the buffers hold (all accesses stay in
// bounds), and what is in flight is drained (bar_drain).
__device__ __forceinline__ void bar_wait(uint32_t a, uint32_t parity, uint32_t limit_word, uint32_t* status) {
#pragma unroll 1
  for (uint32_t i = 1; !bar_try(a, parity); ++i) {
    const uint32_t limit = lds32(limit_word);
    if (i < limit) continue;
    if (limit != 0) {
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(limit_word), "r"(0) : "memory");
      if (status) atomicOr(status, TQ_DEV_INTERNAL);
    }
    return;
  }
}
// Wait for a copy or a product that was issued, whether or not the kernel was
// aborted: neither shared nor tensor memory may go while one is in flight.
// Both end by themselves; the limit is a second here too.
__device__ __forceinline__ void bar_drain(uint32_t a, uint32_t parity, uint32_t* status) {
#pragma unroll 1
  for (int i = 0; i < (1 << 20); ++i)
    if (bar_try(a, parity)) return;
  if (status) atomicOr(status, TQ_DEV_INTERNAL);
}

__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool named_or(int id, int threads, bool v) {
  uint32_t r;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.b32 p, %3, 0; bar.red.or.pred q, %1, %2, p; selp.b32 %0, 1, 0, q; }"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// the same with A in tensor memory (lane: row, a column: two consecutive k)
__device__ __forceinline__ void tc_mma_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.b32 %0, 1, 0, p; }" : "=r"(r));
  return r != 0;
}
template <typename T>
__device__ __forceinline__ T uniform(T x) {  // the same value in every lane, and known to be
  return __shfl_sync(0xffffffffu, x, 0);
}

// Shared-memory matrix descriptor, 128-byte swizzle: K-major operands step
// 1024 bytes per 8 rows (sbo); MN-major ones 1024 bytes per 8 k (sbo) and one
// panel per 64 rows or columns (lbo).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}
// kind::f16, fp16 operands, fp32 accumulator, M = 128
__host__ __device__ constexpr uint32_t mma_desc(int n, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(128 >> 4) << 24);
}

template <int R>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R, int Launch>
__device__ __forceinline__ void regs_dec_to() {
  if constexpr (R < Launch) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

__device__ __forceinline__ float warp_max(float x) {  // NaN counts only where all are
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// two fp32 operations in one instruction
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{ .reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z; }"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{ .reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; add.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z; }"
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

template <int C>
__device__ __forceinline__ void tm_load(uint32_t addr, float (&r)[C]) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  if constexpr (C == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                 : "r"(addr));
  } else if constexpr (C == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(addr));
  } else {
    static_assert(C == 32, "column chunk");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
          "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
          "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(addr));
  }
}
template <int C>
__device__ __forceinline__ void tm_store(uint32_t addr, const float (&r)[C]) {
  const uint32_t* u = reinterpret_cast<const uint32_t*>(r);
  if constexpr (C == 8) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(u[0]),
                 "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
  } else if constexpr (C == 16) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            addr),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
        "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
        : "memory");
  } else {
    static_assert(C == 32, "column chunk");
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
        "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
        "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]),
        "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]),
        "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
        : "memory");
  }
}

// Unnormalised Walsh-Hadamard transform of the 128-blocks of one row held by a
// warp (lane l: elements 4l..4l+3 of every block).
template <int NB>
__device__ __forceinline__ void wht(float (&v)[NB][4], int lane) {
#pragma unroll
  for (int blk = 0; blk < NB; ++blk) {
    const float t0 = v[blk][0] + v[blk][1], t1 = v[blk][0] - v[blk][1];
    const float t2 = v[blk][2] + v[blk][3], t3 = v[blk][2] - v[blk][3];
    v[blk][0] = t0 + t2;
    v[blk][2] = t0 - t2;
    v[blk][1] = t1 + t3;
    v[blk][3] = t1 - t3;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float o = __shfl_xor_sync(0xffffffffu, v[blk][k], m);
        v[blk][k] = (lane & m) ? o - v[blk][k] : v[blk][k] + o;
      }
  }
}

// ------------------------------------------------------------ codes -> fp16 --

// Address of pair q (codes 2q, 2q + 1) of a B-bit stream in the lane's table:
// entry f of lane l at table + f * 128 + 4 l, the table aligned to its size.
template <int B>
__device__ __forceinline__ uint32_t pair_addr(const uint32_t* w, int q, uint32_t lane_base) {
  const int pos = 2 * B * q, wi = pos >> 5, sh = pos & 31;
  uint32_t x;
  if (sh + 2 * B > 32) x = __funnelshift_r(w[wi], w[wi + 1], sh - 7);
  else x = sh >= 7 ? w[wi] >> (sh - 7) : w[wi] << (7 - sh);
  return (x & (((1u << (2 * B)) - 1u) << 7)) | lane_base;
}

// Whether K codes go through a table in shared memory.  Byte permutes take no
// shared-memory bandwidth but a third more instructions: for heads of one
// block they win where that bandwidth binds (rows of 16 to 64 columns: 130,
// 137, 166 us against 136, 143, 171 on 8 x 32768 positions of 3 + 3 bits), for
// heads of two the K warps bind (291 against 249 us, 256-wide heads, 3 + 2 bits).
__host__ __device__ constexpr bool k_table(int nb, int bits) { return bits == 4 || nb == 2; }

// Codes of 2 or 3 bits without a table: eight codes are spread
// to one per nibble (x + (x & high) * (2^s - 1) moves the high half up by s), a
// byte permute picks the low bytes of four levels and another the high bytes,
// and two more interleave them to fp16 pairs.
template <int B>
__device__ __forceinline__ uint32_t spread8(const uint32_t* w, int g) {  // codes 8g .. 8g + 7 of the stream
  if constexpr (B == 2) {
    uint32_t x = (g & 1) ? w[g >> 1] >> 16 : w[g >> 1] & 0xFFFFu;
    x += (x & 0xFF00u) * 255u;
    x += (x & 0x00F000F0u) * 15u;
    return x + (x & 0x0C0C0C0Cu) * 3u;
  } else {
    static_assert(B == 3, "spread codes");
    const int pos = 24 * g, wi = pos >> 5, sh = pos & 31;
    uint32_t x = sh == 8 ? w[wi] >> 8 : (sh == 0 ? w[wi] : __funnelshift_r(w[wi], w[wi + 1], sh)) & 0xFFFFFFu;
    x += (x & 0xFFF000u) * 15u;
    x += (x & 0x0FC00FC0u) * 3u;
    return x + (x & 0x38383838u);
  }
}
__device__ __forceinline__ void pick4(const Levels& t, uint32_t z, uint32_t& a, uint32_t& b) {
  const uint32_t lo = __byte_perm(t.lo0, t.lo1, z), hi = __byte_perm(t.hi0, t.hi1, z);
  a = __byte_perm(lo, hi, 0x5140);
  b = __byte_perm(lo, hi, 0x7362);
}

// The codes of one position and block.
template <int B>
__device__ __forceinline__ void read_codes(uint32_t slot_row, uint32_t (&w)[4 * B]) {
#pragma unroll
  for (int i = 0; i < B; ++i) {
    const uint4 x = lds128(slot_row + 16u * i);
    w[4 * i] = x.x;
    w[4 * i + 1] = x.y;
    w[4 * i + 2] = x.z;
    w[4 * i + 3] = x.w;
  }
}
// Their values as 16 chunks of 8 fp16, into the row of a swizzled tile whose
// chunk 0 is at dst_row.
template <int B>
__device__ __forceinline__ void expand_to_smem(const uint32_t (&w)[4 * B], uint32_t dst_row, uint32_t lane_base) {
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = lds_table(pair_addr<B>(w, 4 * c + i, lane_base));
    sts128((dst_row ^ (uint32_t)((c & 7) << 4)) + (uint32_t)(c >> 3) * kPanel, v[0], v[1], v[2], v[3]);
  }
}
// Their values as 64 columns of this lane's row of tensor memory.
template <int B, bool TABLE>
__device__ __forceinline__ void expand_to_tmem(const uint32_t (&w)[4 * B], uint32_t addr, uint32_t lane_base, const Levels& lv) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t v[16];
    if constexpr (TABLE) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = lds_table(pair_addr<B>(w, 16 * c + i, lane_base));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t z = spread8<B>(w, 4 * c + i);
        pick4(lv, z, v[4 * i], v[4 * i + 1]);
        pick4(lv, z >> 16, v[4 * i + 2], v[4 * i + 3]);
      }
    }
    tm_store<16>(addr + 16 * c, reinterpret_cast<const float(&)[16]>(v));
  }
  tc_wait_st();
}

// ------------------------------------------------------------------ output --

// One row of the output: acc / (128 l), rotated back.  v holds acc / 128.
template <int NB>
__device__ __forceinline__ void emit_row(const TreeParams& p, float (&v)[NB][4], float l, int lane, size_t row) {
  wht<NB>(v, lane);
  const uint32_t sgn = p.sign_mask[lane >> 3] >> (4 * (lane & 7));
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;  // l = 0: no position seen
#pragma unroll
  for (int blk = 0; blk < NB; ++blk) {
    float o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = l != 0.0f ? (((sgn >> k) & 1u) ? -v[blk][k] : v[blk][k]) * inv : 0.0f;
    uint2 w;
    if (p.out_dtype == TQ_F16) {
      const __half2 a = __floats2half2_rn(o[0], o[1]), b = __floats2half2_rn(o[2], o[3]);
      w = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
      const __nv_bfloat162 a = __floats2bfloat162_rn(o[0], o[1]), b = __floats2bfloat162_rn(o[2], o[3]);
      w = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
    *reinterpret_cast<uint2*>(static_cast<char*>(p.out) + (row * NB * kBlock + blk * kBlock + 4 * lane) * 2) = w;
  }
}

__device__ __forceinline__ int clamp_nodes(const TreeParams& p, int b) {
  return p.n_nodes ? min(max(__ldg(p.n_nodes + b), 0), p.n_q) : p.n_q;
}
// The output row of column n of a row group, or -1.
__device__ __forceinline__ long long out_row(const Params& P, int b, int kvh, int vl, int nodes) {
  const TreeParams& p = P.t;
  const int G = (int)P.group.d;
  const int j = (int)P.group.div((uint32_t)vl);
  if (j >= nodes) return -1;
  return ((long long)b * p.n_q + j) * p.q_heads + kvh * G + (vl - j * G);
}

// --------------------------------------------------------------- the kernel --

// barriers, two stages each but the last
enum Bar { kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kSFull = 8, kSEmpty = 10, kPFull = 12, kPFree = 14, kQFull = 16,
           kQFree = 17, kRingFull = 18, kRingFree = 24, kDrain = 30, kBars = 32 };  // rings: three slots for K, three for V

// word offsets in the misc area
template <int NB, int N>
struct Misc {
  static constexpr int kLimit = 0, kTmem = 1, kRing = 2, kUnits = 3, kBegin = 4, kVmax = 8;  // [16]
  static constexpr int kMoff = kVmax + 16;                                   // [N]
  static constexpr int kAlpha = kMoff + N;                                   // [N]
  static constexpr int kRed = kAlpha + N;                                    // [4][N]
  static constexpr int kMask = kRed + 4 * N;                                 // [N] 64-bit
  static constexpr int kScan = kMask + 2 * N;                                // [2][16]
  static constexpr int kNorm = kScan + 32;                                   // [4 tiles][block][K, V][128]
  static constexpr int kWords = kNorm + 4 * NB * 2 * kTok;
};

template <int NB, int N>
__global__ void __launch_bounds__(Roles<N>::kThreads, 1) tree_kernel(const __grid_constant__ Params P) {
  constexpr int D = NB * kBlock;
  using Ro = Roles<N>;
  constexpr int kGroups = Ro::kGroups, kSoftWarps = Ro::kSoftWarps, kThreads = Ro::kThreads;
  constexpr int HC = N / kGroups;           // rows (columns of S) of a softmax group
  constexpr int CH = HC < 16 ? HC : 16;     // columns per tensor-memory load
  // tensor memory: two stages of S, O, two stages of K^ (64 columns each)
  constexpr uint32_t kColsO = 2 * NB * N, kColsK = 3 * NB * N, kColsUsed = 3 * NB * N + 128;
  constexpr uint32_t kCols = kColsUsed <= 256 ? 256 : 512;
  static_assert(kColsUsed <= 512, "tensor memory");
  constexpr uint32_t kQPanel = N * 128;     // bytes of a 64-dim panel of Q^
  constexpr uint32_t kPBlock = (uint32_t)((N + 63) / 64) * kPanel, kPStage = NB * kPBlock;
  using M = Misc<NB, N>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const TreeParams& p = P.t;
  const Plan& pl = P.pl;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  {
    uint32_t dyn;
    asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(dyn));
    if (smem_u32(smem) != kBase || dyn < pl.bytes) {  // another layout of the shared window: reported, never used
      if (tid == 0) {
        if (p.status) atomicOr(p.status, TQ_DEV_INTERNAL);
        P.ws_join[blockIdx.x] = Join{};
      }
      return;
    }
  }
  auto gen = [&](uint32_t a) { return smem + (a - kBase); };
  uint32_t* misc = reinterpret_cast<uint32_t*>(gen(pl.misc));
  float* miscf = reinterpret_cast<float*>(misc);
  int* prefix = reinterpret_cast<int*>(gen(pl.prefix));
  const uint32_t limit_word = pl.misc + 4 * M::kLimit;
  auto bar = [&](int i) { return pl.bar + 8u * (uint32_t)i; };
  auto wait = [&](int i, uint32_t parity) { bar_wait(bar(i), parity, limit_word, p.status); };
  auto aborted = [&]() { return lds32(limit_word) == 0; };

  // ---- set-up: barriers, tensor memory, code tables, lengths ----------------
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      bar_init(bar(kKFull + s), 4);
      bar_init(bar(kKEmpty + s), 1);
      bar_init(bar(kVFull + s), 4);
      bar_init(bar(kVEmpty + s), 1);
      bar_init(bar(kSFull + s), 1);
      bar_init(bar(kSEmpty + s), kSoftWarps);
      bar_init(bar(kPFull + s), kSoftWarps);
      bar_init(bar(kPFree + s), 1);
      bar_init(bar(kDrain + s), 1);
    }
    bar_init(bar(kQFull), 1);
    bar_init(bar(kQFree), 1);
    for (int r = 0; r < 6; ++r) {
      bar_init(bar(kRingFull + r), 1);
      bar_init(bar(kRingFree + r), 4);
    }
    misc[M::kLimit] = (uint32_t)p.wait_tries;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == Ro::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(pl.misc + 4 * M::kTmem),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  int lens_r[4], local = 0, local_live = 0;  // kMaxBatch / 512; tiles, entries that have some
  const int per = (p.batch + 511) / 512;
  if (tid < 512) {
#pragma unroll
    for (int i = 0; i < 4; ++i) lens_r[i] = (i < per && tid * per + i < p.batch) ? __ldg(p.seq_lens + tid * per + i) : 0;
  }
  auto fill = [&](int bits, const float* cent, float scale, uint32_t base) {
    const int n = 32 << (2 * bits), m = (1 << bits) - 1;
    for (int e = tid; e < n; e += kThreads) {
      const int f = e >> 5;
      const __half2 h = __floats2half2_rn(cent[f & m] * scale, cent[f >> bits] * scale);
      *reinterpret_cast<__half2*>(gen(base + 4u * (uint32_t)e)) = h;
    }
  };
  if (k_table(NB, p.k_bits) && pl.lut_k != pl.lut_v) fill(p.k_bits, p.kcent, P.kscale, pl.lut_k);
  fill(p.v_bits, p.vcent, P.vscale, pl.lut_v);
  if (tid < 512) {
    int live = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool there = i < per && tid * per + i < p.batch;
      const int len = min(max(lens_r[i], 0), p.seq_cap);
      if (there && blockIdx.x == 0 && p.status) {
        const int nn = p.n_nodes ? __ldg(p.n_nodes + tid * per + i) : 0;
        if (len != lens_r[i] || nn < 0 || nn > p.n_q) atomicOr(p.status, TQ_DEV_LEN_RANGE);
      }
      lens_r[i] = (len + kTok - 1) / kTok;
      local += lens_r[i];
      if (i < per) {
        const uint32_t have = __ballot_sync(0xffffffffu, len > 0);
        local_live += __popc(have & ((1u << lane) - 1u));
        live += __popc(have);
      }
    }
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) {
      misc[M::kScan + warp] = (uint32_t)incl;
      misc[M::kScan + 16 + warp] = (uint32_t)live;
    }
    local = incl - local;  // before this thread, inside the warp
  }
  tc_before();
  __syncthreads();
  tc_after();
  const int ub = p.kv_heads * P.n_hg;
  const uint32_t warp_tiles = lane < 16 ? misc[M::kScan + lane] : 0;
  const int sw = switch_length((long long)__reduce_add_sync(0xffffffffu, warp_tiles) * ub, (int)gridDim.x);
  if (tid < 512) {
    int run = local + (int)__reduce_add_sync(0xffffffffu, lane < warp ? warp_tiles : 0u) +
              sw * (local_live + (int)__reduce_add_sync(0xffffffffu, lane < warp ? misc[M::kScan + 16 + lane] : 0u));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= per || tid * per + i >= p.batch) break;
      prefix[tid * per + i] = run;
      run += unit_length(lens_r[i], sw);
      if (tid * per + i == p.batch - 1) prefix[p.batch] = run;
    }
  }
  __syncthreads();
  const uint32_t tmem = misc[M::kTmem];
  const Cut cut(prefix, p.batch, ub, sw, (int)gridDim.x);
  // This CTA's part of the line; its beginning is kept in shared memory, not in
  // two registers of every role.
  int span;
  {
    const long long begin = cut.start(blockIdx.x);
    span = blockIdx.x < cut.parts ? (int)(cut.start(blockIdx.x + 1) - begin) : 0;
    *reinterpret_cast<volatile long long*>(misc + M::kBegin) = begin;  // every thread: the same value
  }
  auto segment = [&](int x) {  // the unit at x from the beginning
    const long long begin = *reinterpret_cast<volatile long long*>(misc + M::kBegin);
    return cut.find(begin + x, begin + span, P.n_hg);
  };
  const uint32_t tm_o = tmem + kColsO;
  // P: tile n uses stage n mod p_stages (1 or 2)
  const uint32_t p_shift = (uint32_t)pl.p_stages - 1;
  auto p_stage = [&](uint32_t n) { return n & p_shift; };
  auto p_phase = [&](uint32_t n) { return (n >> p_shift) & 1u; };

  if (warp < kSoftWarps) {
    // ================================================================ softmax
    regs_inc<Ro::kSoft>();
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the query kernel's factors
    const int quad = warp & 3, grp = warp >> 2, tk = 32 * quad + lane;
    const int c0 = grp * HC;  // first column of this group
    const uint32_t tm_lane = (uint32_t)(32 * quad) << 16;
    const uint32_t tk_row = (uint32_t)tk * 128u + (uint32_t)((tk & 7) << 4);  // P row, chunk 0
    const uint32_t moff_a = pl.misc + 4u * (M::kMoff + c0), alpha_a = pl.misc + 4u * (M::kAlpha + c0);
    const uint32_t mask_a = pl.misc + 4u * (M::kMask + 2 * c0);
    float* red = miscf + M::kRed;  // [quad][N]
    const int gid = 2 + grp;       // named barrier of the group
    uint32_t tile_no = 0, seg_no = 0;  // across segments
    const int rows = (int)P.group.d * p.n_q;  // of a kv-head
    for (int x = 0; x < span; ++seg_no) {
      const Seg sg = segment(x);
      const int len = min(max(__ldg(p.seq_lens + sg.b), 0), p.seq_cap);
      const int nodes = clamp_nodes(p, sg.b), ctx = len - nodes;
      named_sync(1, 32 * kSoftWarps);  // every group is done with the unit before
      if (tid < N) {  // which nodes each row sees
        const int vl = sg.hg * N + tid, j = (int)P.group.div((uint32_t)vl);
        uint64_t w = 0;
        if (vl < rows && j < nodes)
          w = __ldg(reinterpret_cast<const unsigned long long*>(p.tree) + (size_t)sg.b * p.n_q + j);
        *reinterpret_cast<uint64_t*>(misc + M::kMask + 2 * tid) = w;
      }
      const float mul = *(volatile const float*)(P.ws_mul + (size_t)sg.b * ub + sg.r);
      if (tk < HC) miscf[M::kMoff + c0 + tk] = -kUnset;  // the references are kept negated
      named_sync(1, 32 * kSoftWarps);
      float2 l[HC / 2];
#pragma unroll
      for (int c = 0; c < HC / 2; ++c) l[c] = make_float2(0.0f, 0.0f);
      float vpow = kNoScale;  // 2^-e of the V norms, e the segment's scale
      for (int tile = sg.lo; tile < sg.hi; ++tile, ++tile_no) {
        const uint32_t st = tile_no & 1, ph = (tile_no >> 1) & 1;
        const int t = tile * kTok + tk, node = t - ctx;
        const bool masked = (tile + 1) * kTok > ctx;  // the tile holds drafted nodes or the end
        const uint32_t tm_s = tmem + tm_lane + st * (NB * N) + c0;
        const uint32_t pt = pl.pt + p_stage(tile_no) * kPStage;
        bool grown = false;  // the V scale changed in this tile
        float beta = 1.0f;
        wait(kSFull + st, ph);
        tc_after();
        // this position's norms, left there with its codes
        float f[NB], vs[NB], vbig = 0.0f, vbig_all = 0.0f;
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
          const float* nrm = miscf + M::kNorm + ((tile_no & 3) * NB + blk) * 2 * kTok + tk;
          f[blk] = nrm[0] * mul;
          vs[blk] = nrm[kTok];
          const float size = fabsf(vs[blk]);
          vbig = fmaxf(vbig, size < INFINITY ? size : 0.0f);
          vbig_all = size < INFINITY ? vbig_all : INFINITY;
        }
#pragma unroll
        for (int ch = 0; ch < HC / CH; ++ch) {
          float x[CH];  // scores, then scores against the references
          auto sees = [&](int c) {  // whether column c's row sees this position
            uint64_t w;
            asm volatile("ld.shared.b64 %0, [%1];" : "=l"(w) : "r"(mask_a + 8u * (ch * CH + c)));
            return t < len && (node < 0 || ((w >> node) & 1ull));
          };
          auto load_scores = [&]() {
            tm_load<CH>(tm_s + ch * CH, x);
            if constexpr (NB == 2) {
              float y[CH];
              tm_load<CH>(tm_s + N + ch * CH, y);
              tc_wait_ld();
#pragma unroll
              for (int c = 0; c < CH; c += 2) {
                const float2 r = fma2(make_float2(y[c], y[c + 1]), make_float2(f[NB - 1], f[NB - 1]),
                                      mul2(make_float2(x[c], x[c + 1]), make_float2(f[0], f[0])));
                x[c] = r.x;
                x[c + 1] = r.y;
              }
            } else {
              tc_wait_ld();
#pragma unroll
              for (int c = 0; c < CH; c += 2) {
                const float2 r = mul2(make_float2(x[c], x[c + 1]), make_float2(f[0], f[0]));
                x[c] = r.x;
                x[c + 1] = r.y;
              }
            }
            if (masked) {
#pragma unroll
              for (int c = 0; c < CH; ++c)
                if (!sees(c)) x[c] = -INFINITY;
            }
          };
          // rounded product first, then the difference: the maximum itself gives exactly 0
          auto against = [&]() {
            float top = -INFINITY;
#pragma unroll
            for (int c = 0; c < CH; c += 4) {
              const float4 m = lds128f(moff_a + 4u * (ch * CH + c));
              const float2 u = add2(make_float2(x[c], x[c + 1]), make_float2(m.x, m.y));
              const float2 w = add2(make_float2(x[c + 2], x[c + 3]), make_float2(m.z, m.w));
              x[c] = u.x; x[c + 1] = u.y; x[c + 2] = w.x; x[c + 3] = w.y;
              top = max3(max3(top, u.x, u.y), w.x, w.y);
            }
            return top;
          };
          load_scores();
          const float top = against();
          const bool wide = ch == 0 ? vbig * vpow > kNormRoom : grown;
          if (named_or(gid, 128, top > kTau || wide)) {
            // ---- new references (and V scale): the tile's maximum of each row
            load_scores();
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              const float y = warp_max(x[c]);
              if (lane == 0) red[quad * N + c0 + ch * CH + c] = y;
            }
            if (ch == 0) {
              const float y = warp_max(vbig);
              if (lane == 0) miscf[M::kVmax + warp] = y;
            }
            named_sync(gid, 128);
            if (tk < CH) {
              const int c = c0 + ch * CH + tk;
              const float y = fmaxf(fmaxf(red[c], red[N + c]), fmaxf(red[2 * N + c], red[3 * N + c]));
              const float old = -miscf[M::kMoff + c];
              float a = 1.0f;
              if (y > old + kTau) {
                a = old == kUnset ? 0.0f : ex2(old - y);
                miscf[M::kMoff + c] = -y;
              }
              miscf[M::kAlpha + c] = a;
            }
            if (ch == 0) {
              float vm = 0.0f;
#pragma unroll
              for (int w = 0; w < 4; ++w) vm = fmaxf(vm, miscf[M::kVmax + 4 * grp + w]);
              if (vm * vpow > kNormRoom) {
                const float np = ldexpf(1.0f, kNormTop - ilogbf(vm));
                beta = np / vpow;
                vpow = np;
                grown = true;
              }
            }
            named_sync(gid, 128);
            if (tile > sg.lo) {
              wait(kPFree + p_stage(tile_no - 1), p_phase(tile_no - 1));  // the sum so far
              tc_after();
            }
            float a[CH];
#pragma unroll
            for (int c = 0; c < CH; c += 4) {
              const float4 m = lds128f(alpha_a + 4u * (ch * CH + c));
              a[c] = m.x; a[c + 1] = m.y; a[c + 2] = m.z; a[c + 3] = m.w;
            }
#pragma unroll
            for (int c = 0; c < CH; c += 2) {
              float2& y = l[(ch * CH + c) / 2];
              y = mul2(y, make_float2(a[c], a[c + 1]));
            }
            if (tile > sg.lo) {
#pragma unroll
              for (int blk = 0; blk < NB; ++blk) {
                float o[CH];
                tm_load<CH>(tm_o + tm_lane + blk * N + c0 + ch * CH, o);
                tc_wait_ld();
#pragma unroll
                for (int c = 0; c < CH; ++c) o[c] *= a[c] * beta;
                tm_store<CH>(tm_o + tm_lane + blk * N + c0 + ch * CH, o);
              }
              tc_wait_st();
            }
            load_scores();
            against();
          }
          // ---- weights, their sums, and weight * norm as the MMA's operand
          if (ch == 0) {
#pragma unroll
            for (int blk = 0; blk < NB; ++blk) vs[blk] *= vpow;
            wait(kPFree + p_stage(tile_no), p_phase(tile_no) ^ 1);
          }
          if (ch == HC / CH - 1) {  // the scores are in registers
            tc_before();
            __syncwarp();
            if (lane == 0) bar_arrive(bar(kSEmpty + st));
          }
#pragma unroll
          for (int c = 0; c < CH; c += 8) {
            float2 w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              w[k] = make_float2(ex2(x[c + 2 * k]), ex2(x[c + 2 * k + 1]));
              float2& y = l[(ch * CH + c) / 2 + k];
              y = add2(y, w[k]);
            }
            const int col = c0 + ch * CH + c;
#pragma unroll
            for (int blk = 0; blk < NB; ++blk) {
              uint32_t h[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float2 y = mul2(w[k], make_float2(vs[blk], vs[blk]));
                const __half2 hh = __floats2half2_rn(y.x, y.y);
                h[k] = *reinterpret_cast<const uint32_t*>(&hh);
              }
              // column col's chunk of this position's row, swizzled
              sts128(pt + (uint32_t)blk * kPBlock + (uint32_t)(col >> 6) * kPanel + (tk_row ^ (uint32_t)((col & 63) << 1)),
                     h[0], h[1], h[2], h[3]);
            }
          }
          if (masked && !(vbig_all < INFINITY)) {
            // an infinite or NaN norm times a weight of zero: rows that do not
            // see the position get a plain zero
#pragma unroll 1
            for (int c = 0; c < CH; ++c) {
              if (sees(c)) continue;
              const int col = c0 + ch * CH + c;
              for (int blk = 0; blk < NB; ++blk)
                sts16(pt + (uint32_t)blk * kPBlock + (uint32_t)(col >> 6) * kPanel + (tk_row ^ (uint32_t)((col & 56) << 1)) +
                          2u * (col & 7),
                      0);
            }
          }
        }
        tc_before();
        fence_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(bar(kPFull + p_stage(tile_no)));
      }
      // ---- the segment's partial: l over the positions, O, reference maxima
      wait(kPFree + p_stage(tile_no - 1), p_phase(tile_no - 1));
      tc_after();
#pragma unroll
      for (int c = 0; c < HC; ++c) {
        float y = c & 1 ? l[c / 2].y : l[c / 2].x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (lane == 0) red[quad * N + c0 + c] = y;
      }
      named_sync(gid, 128);
      const long long slot = 2 * (long long)blockIdx.x + (sg.lo == 0 ? 1 : 0);
      float* ml = P.ws_ml + slot * N * 2;
      float* acc = P.ws_acc + slot * N * D;
      if (tk < HC) {
        const int c = c0 + tk;
        const float m = -miscf[M::kMoff + c], sum = red[c] + red[N + c] + red[2 * N + c] + red[3 * N + c];
        // a row with a NaN score keeps it through the join: its maximum is made infinite
        *reinterpret_cast<float2*>(ml + 2 * c) = make_float2(sum != sum ? INFINITY : m == kUnset ? -INFINITY : m, sum);
      }
      const float osc = 1.0f / (vpow * P.vscale * kBlock);
#pragma unroll
      for (int blk = 0; blk < NB; ++blk)
#pragma unroll
        for (int ch = 0; ch < HC / CH; ++ch) {
          float o[CH];
          tm_load<CH>(tm_o + tm_lane + blk * N + c0 + ch * CH, o);
          tc_wait_ld();
#pragma unroll
          for (int c = 0; c < CH; ++c) acc[(size_t)(c0 + ch * CH + c) * D + blk * kBlock + tk] = o[c] * osc;
        }
      tc_before();
      if (sg.lo == 0 && sg.hi == sg.nt) {  // the whole unit: emit its rows
        named_sync(1, 32 * kSoftWarps);
        for (int n = warp; n < N; n += kSoftWarps) {
          const int vl = sg.hg * N + n;
          const long long row = vl < rows ? out_row(P, sg.b, sg.kvh, vl, nodes) : -1;
          if (row < 0) continue;
          float v[NB][4];
#pragma unroll
          for (int blk = 0; blk < NB; ++blk) {
            const float4 a = __ldcg(reinterpret_cast<const float4*>(acc + (size_t)n * D + blk * kBlock + 4 * lane));
            v[blk][0] = a.x; v[blk][1] = a.y; v[blk][2] = a.z; v[blk][3] = a.w;
          }
          emit_row<NB>(p, v, __ldcg(ml + 2 * n + 1), lane, (size_t)row);
        }
      }
      x += sg.nt - sg.lo + sw;
    }
  } else if (warp < Ro::kMmaWarp) {
    // ============================================================ dequantise
    // A warp takes 32 positions of every tile from the code ring; the K warps'
    // lanes also fetch their position's norms, a tile ahead.
    regs_dec_to<Ro::kCodes, Ro::kLaunch>();
    const int cw = warp - Ro::kCodeWarp, side = cw >> 2, quarter = cw & 3, tok = 32 * quarter + lane;
    auto work = [&](auto bits_tag, auto side_tag) {
      constexpr int B = decltype(bits_tag)::value;
      constexpr bool V = decltype(side_tag)::value;
      constexpr uint32_t kRow = NB * 16 * B;  // bytes of a position
      const uint32_t ring = (V ? pl.ring_v : pl.ring_k) + (uint32_t)tok * kRow, depth = (uint32_t)pl.depth;
      const uint32_t lane_base = (V ? pl.lut_v : pl.lut_k) + 4u * lane;
      const uint32_t tm_k = tmem + ((uint32_t)(32 * quarter) << 16) + kColsK;
      const uint32_t v_row = pl.vt + (uint32_t)tok * 128u + (uint32_t)((tok & 7) << 4);
      const uint32_t shift = V ? (uint32_t)pl.v_stages - 1 : 1u;
      uint32_t slot = 0, slot_ph = 0, stage = 0, stage_ph = 1, tile_no = 0;
      for (int x = 0; x < span;) {
        const Seg sg = segment(x);
        const int len = min(max(__ldg(p.seq_lens + sg.b), 0), p.seq_cap);
        const size_t row0 = ((size_t)sg.b * p.kv_heads + sg.kvh) * p.seq_cap;
        const int tiles = sg.hi - sg.lo;
        const int t_first = sg.lo * kTok + tok;  // this lane's position in the first tile
        uint16_t kn[NB], vn[NB];
        auto fetch_norms = [&](int i) {
          const int t = t_first + i * kTok;
#pragma unroll
          for (int blk = 0; blk < NB; ++blk) {
            kn[blk] = vn[blk] = 0;
            if (t < len) {
              kn[blk] = __ldg(p.k_norms + (row0 + t) * NB + blk);
              vn[blk] = __ldg(p.v_norms + (row0 + t) * NB + blk);
            }
          }
        };
        if (!V) fetch_norms(0);
        for (int i = 0; i < tiles; ++i, ++tile_no) {
          wait(kRingFull + (V ? 3 : 0) + (int)slot, slot_ph);
#pragma unroll
          for (int blk = 0; blk < NB; ++blk) {
            uint32_t w[4 * B];
            read_codes<B>(ring + slot * (kTok * kRow) + (uint32_t)(blk * 16 * B), w);
            if (blk == NB - 1) {  // this warp has read the slot
              __syncwarp();
              if (lane == 0) bar_arrive(bar(kRingFree + (V ? 3 : 0) + (int)slot));
            }
            wait((V ? kVEmpty : kKEmpty) + stage, stage_ph);
            if constexpr (V) {
              expand_to_smem<B>(w, v_row + stage * 2 * kPanel, lane_base);
              fence_async_smem();
            } else {
              tc_after();
              if (blk == 0) {
                // The softmax warps read the norms of tile n - 4 before they
                // free its S stage, which the product of tile n - 2 waited
                // for, as this stage did for that product.
                float* dst = miscf + M::kNorm + (tile_no & 3u) * NB * 2 * kTok + tok;
#pragma unroll
                for (int k = 0; k < NB; ++k) {
                  dst[k * 2 * kTok] = __half2float(__ushort_as_half(kn[k]));
                  dst[k * 2 * kTok + kTok] = __half2float(__ushort_as_half(vn[k]));
                }
                if (i + 1 < tiles) fetch_norms(i + 1);
              }
              expand_to_tmem<B, k_table(NB, B)>(w, tm_k + stage * 64, lane_base, P.klev);
              tc_before();
            }
            __syncwarp();
            if (lane == 0) bar_arrive(bar((V ? kVFull : kKFull) + stage));
            stage = (stage + 1) & shift;
            stage_ph ^= stage == 0 ? 1u : 0u;
          }
          if (++slot == depth) {
            slot = 0;
            slot_ph ^= 1;
          }
        }
        x += sg.nt - sg.lo + sw;
      }
    };
    auto by_bits = [&](int bits, auto side_tag) {
      if (bits == 2) work(std::integral_constant<int, 2>{}, side_tag);
      else if (bits == 3) work(std::integral_constant<int, 3>{}, side_tag);
      else work(std::integral_constant<int, 4>{}, side_tag);
    };
    if (side) by_bits(p.v_bits, std::true_type{});
    else by_bits(p.k_bits, std::false_type{});
  } else {
    // ================================================================= MMAs
    // The first warp issues the score products, the second the V sums, the
    // third the copies of the codes, the fourth those of Q^.  Descriptors and
    // loop bounds are warp-uniform, so that they stay in uniform registers: an
    // MMA of these shapes takes 32 to 64 cycles, and moving its descriptors
    // into place must not take longer.
    regs_dec<Ro::kMma>();
    if (warp == Ro::kMmaWarp) {
      constexpr uint32_t id_s = mma_desc(N, false, false);
      uint32_t ks = 0, kph = 0, tile_no = 0, seg_no = 0;
      const uint64_t dq = smem_desc(pl.q, 16, 1024);
      const uint32_t tm = uniform(tmem);
      for (int x = 0; x < span; ++seg_no) {
        const Seg sg = segment(x);
        const int tiles = uniform(sg.hi - sg.lo);
        wait(kQFull, seg_no & 1);
        for (int i = 0; i < tiles; ++i, ++tile_no) {
          const uint32_t st = tile_no & 1, ph = (tile_no >> 1) & 1;
          wait(kSEmpty + st, ph ^ 1);
#pragma unroll
          for (int blk = 0; blk < NB; ++blk) {
            wait(kKFull + ks, kph);
            tc_after();
            if (elect_one()) {
              const uint32_t a = tm + kColsK + ks * 64;
              const uint64_t b = dq + (2 * blk * kQPanel >> 4);
              const uint32_t d = tm + st * (NB * N) + blk * N;
#pragma unroll
              for (int half = 0; half < 2; ++half)  // the two terms of the query
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  tc_mma_ta(d, a + 8 * k,
                         b + (((half * 2 * NB + (k >> 2)) * kQPanel + 32u * (k & 3)) >> 4), id_s,
                         half == 0 && k == 0 ? 0u : 1u);
              tc_commit(bar(kKEmpty + ks));
              if (blk == NB - 1) tc_commit(bar(kSFull + st));
            }
            __syncwarp();
            ks ^= 1;
            kph ^= ks ^ 1;
          }
        }
        if (elect_one()) tc_commit(bar(kQFree));
        __syncwarp();
        x += sg.nt - sg.lo + sw;
      }
    } else if (warp == Ro::kMmaWarp + 1) {
      constexpr uint32_t id_o = mma_desc(N, true, true);
      uint32_t vs = 0, vph = 0, tile_no = 0;
      const uint64_t dv = smem_desc(pl.vt, kPanel, 1024), dp = smem_desc(pl.pt, kPanel, 1024);
      const uint32_t to = uniform(tm_o);
      for (int x = 0; x < span;) {
        const Seg sg = segment(x);
        const int tiles = uniform(sg.hi - sg.lo);
        for (int i = 0; i < tiles; ++i, ++tile_no) {
          wait(kPFull + p_stage(tile_no), p_phase(tile_no));
#pragma unroll
          for (int blk = 0; blk < NB; ++blk) {
            wait(kVFull + vs, vph);
            tc_after();
            if (elect_one()) {
              const uint64_t a = dv + (vs * 2 * kPanel >> 4);
              const uint64_t b = dp + ((p_stage(tile_no) * kPStage + blk * kPBlock) >> 4);
              const uint32_t d = to + blk * N;
#pragma unroll
              for (int k = 0; k < 8; ++k)
                tc_mma(d, a + (2048u * k >> 4), b + (2048u * k >> 4), id_o, k == 0 ? (i > 0 ? 1u : 0u) : 1u);
              tc_commit(bar(kVEmpty + vs));
              if (blk == NB - 1) tc_commit(bar(kPFree + p_stage(tile_no)));
            }
            __syncwarp();
            if (++vs == (uint32_t)pl.v_stages) {
              vs = 0;
              vph ^= 1;
            }
          }
        }
        x += sg.nt - sg.lo + sw;
      }
      // no product is in flight when tensor memory is freed (the softmax warps
      // waited for every score product)
      if (tile_no > 0) wait(kPFree + p_stage(tile_no - 1), p_phase(tile_no - 1));
    } else if (warp == Ro::kMmaWarp + 2 && lane == 0) {
      // Codes into the rings: a tile's positions are contiguous in the cache.
      // Positions past the end keep what the slot held: any code is a level,
      // and their weights are zero.
      const uint32_t depth = (uint32_t)pl.depth;
      uint32_t slot = 0, free_ph = 1;
      bool stop = false, half = false;  // half: K's copy of this slot was issued, V's not
      for (int x = 0; x < span && !stop;) {
        const Seg sg = segment(x);
        const int len = min(max(__ldg(p.seq_lens + sg.b), 0), p.seq_cap);
        const size_t row0 = ((size_t)sg.b * p.kv_heads + sg.kvh) * p.seq_cap;
        for (int tile = sg.lo; tile < sg.hi; ++tile) {
          const uint32_t rows = (uint32_t)min(len - tile * kTok, kTok);
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            const uint32_t row_bytes = NB * 16u * (uint32_t)(side ? p.v_bits : p.k_bits);
            const uint8_t* src = (side ? p.v_codes : p.k_codes) + (row0 + (size_t)tile * kTok) * row_bytes;
            // Aborted, the slot's last copy may still be in flight: a second
            // one would arrive on a barrier that expects no arrival.  Heads of
            // one block look once for both sides (132 and 137 us against 134 and
            // 138 at 16 and 32 columns); in heads of two K would wait for V
            // (258 against 251 us).
            if (NB == 2 || side == 0) {
              if (NB == 1) wait(kRingFree + 3 + (int)slot, free_ph);
              wait(kRingFree + 3 * side + (int)slot, free_ph);
              if ((stop = aborted())) break;
            }
            fence_async_smem();  // the slot's reads before the copy
            bulk_copy((side ? pl.ring_v : pl.ring_k) + slot * (kTok * row_bytes), src, rows * row_bytes,
                      bar(kRingFull + 3 * side + (int)slot));
            half = side == 0;
          }
          if (stop) break;
          if (++slot == depth) {
            slot = 0;
            free_ph ^= 1;
          }
        }
        x += sg.nt - sg.lo + sw;
      }
      misc[M::kRing] = 4 * slot + 2 * free_ph + (half ? 1 : 0);
    } else if (warp == Ro::kMmaWarp + 3 && lane == 0) {
      // Q^ of each unit, as the query kernel left it; and the join's record
      Join j{};
      if (span > 0) {
        const Seg sg = segment(0);
        if (sg.lo > 0 && cut.part_of(sg.b, sg.r, 0) == (long long)blockIdx.x - 1)
          j = Join{sg.b, sg.kvh, sg.hg, (int)blockIdx.x, (int)cut.part_of(sg.b, sg.r, sg.nt - 1), clamp_nodes(p, sg.b)};
      }
      P.ws_join[blockIdx.x] = j;
      asm volatile("griddepcontrol.wait;" ::: "memory");
      asm volatile("fence.proxy.async;" ::: "memory");
      uint32_t seg_no = 0;
      for (int x = 0; x < span; ++seg_no) {
        const Seg sg = segment(x);
        wait(kQFree, (seg_no & 1) ^ 1);
        if (aborted()) break;  // as for the codes
        bulk_copy(pl.q, P.ws_q + ((size_t)sg.b * ub + sg.r) * (4 * NB * kQPanel), 4 * NB * kQPanel, bar(kQFull));
        x += sg.nt - sg.lo + sw;
      }
      misc[M::kUnits] = seg_no;
    }
  }

  tc_before();
  __syncthreads();
  tc_after();
  if (misc[M::kLimit] == 0) {  // waits were cut short: wait for what is in flight
    if (warp == Ro::kMmaWarp || warp == Ro::kMmaWarp + 1) {  // the products that this warp issued
      const uint32_t b = bar(kDrain + warp - Ro::kMmaWarp);
      if (elect_one()) tc_commit(b);
      __syncwarp();
      bar_drain(b, 0, p.status);
    } else if (warp == Ro::kMmaWarp + 2) {
      // Slots below the next one were last filled in this pass over the ring,
      // the others in the pass before (at first none was, and parity 1 is over).
      const uint32_t slot = misc[M::kRing] >> 2, before = (misc[M::kRing] >> 1) & 1u, half = misc[M::kRing] & 1u;
#pragma unroll 1
      for (uint32_t i = 0; i < 2 * (uint32_t)pl.depth; ++i) {
        const uint32_t k = i & 1u, n = i >> 1;
        bar_drain(bar(kRingFull + 3 * (int)k + (int)n), n < slot + (k == 0 ? half : 0u) ? before ^ 1u : before, p.status);
      }
    } else if (warp == Ro::kMmaWarp + 3 && misc[M::kUnits] > 0) {
      bar_drain(bar(kQFull), (misc[M::kUnits] - 1) & 1u, p.status);
    }
    __syncthreads();
  }
  if (warp == Ro::kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
}

// The rows of every unit, ready for the score products: q^ = H (s o q) under
// one power-of-two scale (|q^| <= 128 max |q|, scaled to below 2^15), split into
// two fp16 terms, in the layout of the kernel's Q^ buffer.  One CTA per unit.
// The units of an empty sequence have no tiles: their rows see no position, and
// this kernel writes their zeros.
template <int NB, int N>
__global__ void __launch_bounds__(512) query_kernel(const __grid_constant__ Params P) {
  constexpr int D = NB * kBlock, kWarpsQ = 16;
  constexpr uint32_t kQPanel = N * 128;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float wmax[kWarpsQ];
  const TreeParams& p = P.t;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ub = p.kv_heads * P.n_hg, b = (int)(blockIdx.x / (unsigned)ub), r = (int)(blockIdx.x % (unsigned)ub);
  const int kvh = r / P.n_hg, hg = r % P.n_hg, nodes = clamp_nodes(p, b), rows = (int)P.group.d * p.n_q;
  constexpr int RW = (N + kWarpsQ - 1) / kWarpsQ;  // rows of a warp
  if (__ldg(p.seq_lens + b) <= 0) {
    for (int n = warp; n < N; n += kWarpsQ) {
      const int vl = hg * N + n;
      const long long row = vl < rows ? out_row(P, b, kvh, vl, nodes) : -1;
      if (row < 0) continue;
#pragma unroll
      for (int blk = 0; blk < NB; ++blk)
        *reinterpret_cast<uint2*>(static_cast<char*>(p.out) + ((size_t)row * D + blk * kBlock + 4 * lane) * 2) = make_uint2(0, 0);
    }
    return;
  }
  float v[RW][NB][4];
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const int n = warp + kWarpsQ * i, vl = hg * N + n;
    const long long row = n < N && vl < rows ? out_row(P, b, kvh, vl, nodes) : -1;
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      v[i][blk][0] = v[i][blk][1] = v[i][blk][2] = v[i][blk][3] = 0.0f;
      if (row < 0) continue;
      const size_t e = (size_t)row * D + blk * kBlock + 4 * lane;
      if (p.q_dtype == TQ_F32) {
        const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + e);
        v[i][blk][0] = a.x; v[i][blk][1] = a.y; v[i][blk][2] = a.z; v[i][blk][3] = a.w;
      } else {
        const uint2 h = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.q) + e);
        float2 a, c;
        if (p.q_dtype == TQ_F16) {
          a = __half22float2(*reinterpret_cast<const __half2*>(&h.x));
          c = __half22float2(*reinterpret_cast<const __half2*>(&h.y));
        } else {
          a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&h.x));
          c = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&h.y));
        }
        v[i][blk][0] = a.x; v[i][blk][1] = a.y; v[i][blk][2] = c.x; v[i][blk][3] = c.y;
      }
    }
  }
  float mx = 0.0f;
#pragma unroll
  for (int i = 0; i < RW; ++i)
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = fabsf(v[i][blk][k]);
        mx = fmaxf(mx, a < INFINITY ? a : 0.0f);  // elements that are not finite have no say
      }
  mx = warp_max(mx);
  if (lane == 0) wmax[warp] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarpsQ; ++w) mx = fmaxf(mx, wmax[w]);
  const int qe = mx > 0.0f ? max(ilogbf(mx) - 7, -110) : 0;
  const float sc = ldexpf(1.0f, -qe);
  if (threadIdx.x == 0) P.ws_mul[blockIdx.x] = p.score_mult * ldexpf(1.0f, qe) / P.kscale;
  const uint32_t sgn = p.sign_mask[lane >> 3] >> (4 * (lane & 7));
  uint8_t* image = P.ws_q + (size_t)blockIdx.x * (4 * NB * kQPanel);
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const int n = warp + kWarpsQ * i;
    if (n >= N) break;
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i][blk][k] *= ((sgn >> k) & 1u) ? -sc : sc;
    wht<NB>(v[i], lane);
    // lane l holds dims 4l..4l+3: chunk l / 2 of the block, half l & 1
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      uint8_t* a = image + (uint32_t)(2 * blk + (lane >> 4)) * kQPanel + (uint32_t)n * 128u +
                   (uint32_t)((((lane >> 1) & 7) ^ (n & 7)) << 4) + 8u * (lane & 1);
      const float(&y)[4] = v[i][blk];
      __half2 h[2], t[2];
      h[0] = __floats2half2_rn(y[0], y[1]);
      h[1] = __floats2half2_rn(y[2], y[3]);
      const float2 b0 = __half22float2(h[0]), b1 = __half22float2(h[1]);
      t[0] = __floats2half2_rn(y[0] - b0.x, y[1] - b0.y);
      t[1] = __floats2half2_rn(y[2] - b1.x, y[3] - b1.y);
      *reinterpret_cast<uint2*>(a) = make_uint2(*reinterpret_cast<uint32_t*>(&h[0]), *reinterpret_cast<uint32_t*>(&h[1]));
      *reinterpret_cast<uint2*>(a + 2 * NB * kQPanel) =
          make_uint2(*reinterpret_cast<uint32_t*>(&t[0]), *reinterpret_cast<uint32_t*>(&t[1]));
    }
  }
}

// Join of the units that a cut went through.  Block (c, g): the unit that CTA
// c + 1 starts inside of (its first cut), rows 8 g .. 8 g + 7.
template <int NB, int N>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Params P) {
  constexpr int D = NB * kBlock;
  const TreeParams& p = P.t;
  const int lane = threadIdx.x & 31, n = blockIdx.y * 8 + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Join jn = P.ws_join[blockIdx.x + 1];
  if (jn.first == 0) return;
  const int vl = jn.hg * N + n;
  if (vl >= (int)P.group.d * p.n_q) return;
  const long long row = out_row(P, jn.b, jn.kvh, vl, jn.nodes);
  if (row < 0) return;
  // part c - 1 holds the unit's first tiles (its last segment: slot 2 (c-1) + 1),
  // parts c, c + 1, ... the rest (their first segments: slots 2 c', ...)
  const long long c = jn.first;
  const int parts = jn.last - jn.first + 2;
  auto slot = [&](int i) { return i == 0 ? 2 * (c - 1) + 1 : 2 * (c - 1 + i); };
  float top = -INFINITY, l = 0.0f;
  float v[NB][4] = {};
  for (int i0 = 0; i0 < parts; i0 += 32) {
    const int i = i0 + lane;
    float2 ml = make_float2(-INFINITY, 0.0f);
    if (i < parts) ml = *reinterpret_cast<const float2*>(P.ws_ml + (slot(i) * N + n) * 2);
    float m = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = fmaxf(m, top);
    const float down = top == -INFINITY ? 0.0f : ex2(top - m);
    top = m;
    const float w = ml.x == -INFINITY ? 0.0f : ex2(ml.x - m);
    float s = w != 0.0f ? ml.y * w : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    l = l * down + s;
#pragma unroll
    for (int blk = 0; blk < NB; ++blk)
#pragma unroll
      for (int k = 0; k < 4; ++k) v[blk][k] *= down;
    const int m_parts = min(32, parts - i0);
#pragma unroll 8
    for (int j = 0; j < m_parts; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const float* acc = P.ws_acc + (slot(i0 + j) * N + n) * D + 4 * lane;
#pragma unroll
      for (int blk = 0; blk < NB; ++blk) {
        const float4 a = *reinterpret_cast<const float4*>(acc + blk * kBlock);
        if (wj != 0.0f) {
          v[blk][0] = fmaf(a.x, wj, v[blk][0]);
          v[blk][1] = fmaf(a.y, wj, v[blk][1]);
          v[blk][2] = fmaf(a.z, wj, v[blk][2]);
          v[blk][3] = fmaf(a.w, wj, v[blk][3]);
        }
      }
    }
  }
  emit_row<NB>(p, v, l, lane, (size_t)row);
}

// --------------------------------------------------------------- host side --

// A factor for a codebook's levels that makes their rounding to fp16 small:
// the best of 8192 in [1, 2), by the mean squared error over N(0,1) (levels of
// 2, 3, 4 bits: 0.7e-5, 1.6e-5, 4.9e-5 of their size, against 2e-4 unscaled).
// The kernel divides it out in fp32.
float find_scale(const float* cent, int levels) {
  float weight[16], best = 1.0f, least = INFINITY;
  for (int j = 0; j < levels; ++j) {  // density at the level times the width of its cell
    const float lo = j > 0 ? cent[j - 1] : 2.0f * cent[j] - cent[j + 1];
    const float hi = j + 1 < levels ? cent[j + 1] : 2.0f * cent[j] - cent[j - 1];
    weight[j] = std::exp(-0.5f * cent[j] * cent[j]) * std::fabs(hi - lo) + 1e-6f;
  }
  for (int k = 0; k < 8192; ++k) {
    const float a = 1.0f + k * (1.0f / 8192.0f), stop = least * a * a;
    float err = 0.0f;
    for (int j = levels - 1; j >= 0 && err < stop; --j) {
      const float x = cent[j] * a;
      uint32_t u;
      memcpy(&u, &x, 4);
      u = (u + 0xFFFu + ((u >> 13) & 1u)) & ~0x1FFFu;  // 10 mantissa bits, to nearest even
      float r;
      memcpy(&r, &u, 4);
      err += weight[j] * (r - x) * (r - x);
    }
    if (err < stop) {
      least = err / (a * a);
      best = a;
    }
  }
  return best;
}

// The search takes some 0.1 ms, so a thread keeps the last factors it found,
// by the levels' values.
float centroid_scale(const float* cent, int bits) {
  struct Known {
    float cent[16], scale;
    int bits;
  };
  static thread_local Known known[4] = {};
  static thread_local int next = 0;
  const size_t size = sizeof(float) << bits;
  for (const Known& k : known)
    if (k.bits == bits && memcmp(k.cent, cent, size) == 0) return k.scale;
  Known& k = known[next];
  next = (next + 1) & 3;
  memcpy(k.cent, cent, size);
  k.scale = find_scale(cent, 1 << bits);
  k.bits = bits;
  return k.scale;
}

Levels level_bytes(const float* cent, float scale, int bits) {
  uint32_t w[4] = {0, 0, 0, 0};
  for (int j = 0; j < (1 << bits) && j < 8; ++j) {
    const uint16_t h = __half_as_ushort(__float2half_rn(cent[j] * scale));
    w[j >> 2] |= (uint32_t)(h & 255u) << (8 * (j & 3));
    w[2 + (j >> 2)] |= (uint32_t)(h >> 8) << (8 * (j & 3));
  }
  return Levels{w[0], w[1], w[2], w[3]};
}

// First-fit placement in the shared window.
struct Place {
  uint32_t lo[16], hi[16];
  int n = 1;
  Place() { lo[0] = kBase, hi[0] = kBase + kMaxDyn; }
  uint32_t take(uint32_t size, uint32_t align) {
    for (int i = 0; i < n; ++i) {
      const uint32_t a = (lo[i] + align - 1) / align * align;
      if (a + size > hi[i]) continue;
      const uint32_t l0 = lo[i];
      lo[i] = a + size;
      if (a > l0 && n < 16) {
        for (int j = n; j > i; --j) lo[j] = lo[j - 1], hi[j] = hi[j - 1];
        lo[i] = l0;
        hi[i] = a;
        ++n;
      }
      return a;
    }
    return 0;
  }
};

template <int NB, int N>
bool plan(const TreeParams& p, Plan& pl) {
  // in order of preference: stages of V^ and P, slots of a code ring
  static const int tries[7][3] = {{2, 2, 3}, {2, 2, 2}, {2, 1, 3}, {2, 1, 2}, {1, 1, 3}, {1, 1, 2}, {1, 1, 1}};
  for (const auto& t : tries) {
    pl = Plan{};
    Place at;
    uint32_t end = 0;
    bool ok = true;
    auto take = [&](uint32_t size, uint32_t align) {
      const uint32_t a = at.take(size, align);
      ok = ok && a != 0;
      if (a + size > end) end = a + size;
      return a;
    };
    pl.v_stages = t[0];
    pl.p_stages = t[1];
    pl.depth = t[2];
    // tables: V's, and K's where it has one, one for both where the levels are
    pl.lut_v = take(128u << (2 * p.v_bits), 128u << (2 * p.v_bits));
    if (k_table(NB, p.k_bits)) {
      const bool same = p.v_bits == p.k_bits && memcmp(p.kcent, p.vcent, sizeof(p.kcent)) == 0;
      pl.lut_k = same ? pl.lut_v : take(128u << (2 * p.k_bits), 128u << (2 * p.k_bits));
    }
    pl.vt = take(2 * kPanel * t[0], 1024);
    pl.q = take((uint32_t)(4 * NB * N * 128), 1024);
    pl.pt = take((uint32_t)(t[1] * NB * ((N + 63) / 64)) * kPanel, 1024);
    pl.ring_k = take(kTok * NB * 16u * (uint32_t)(p.k_bits * t[2]), 128);
    pl.ring_v = take(kTok * NB * 16u * (uint32_t)(p.v_bits * t[2]), 128);
    pl.bar = take(8 * kBars, 128);
    pl.misc = take(4 * Misc<NB, N>::kWords, 128);
    pl.prefix = take(4u * (uint32_t)(p.batch + 1), 128);
    pl.bytes = end - kBase;
    if (ok) return true;
  }
  return false;
}

template <int NB, int N>
int run(Params& P, cudaStream_t stream) {
  const TreeParams& p = P.t;
  const int rows = p.q_heads / p.kv_heads * p.n_q;
  P.n_hg = (rows + N - 1) / N;
  P.group = FastDiv::make((uint32_t)(p.q_heads / p.kv_heads));
  const long long tiles =
      (long long)p.batch * p.kv_heads * P.n_hg * ((p.seq_cap + kTok - 1) / kTok);
  // set up once per device
  auto kern = tree_kernel<NB, N>;
  static int sm_counts[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return TQ_ERR_CUDA;
  if (sm_counts[dev] == 0) {
    int sms = 0;
    cudaFuncAttributes attrs;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxDyn) != cudaSuccess ||
        cudaFuncGetAttributes(&attrs, kern) != cudaSuccess)
      return TQ_ERR_CUDA;
    if (attrs.numRegs < Roles<N>::kLaunch) return TQ_ERR_UNSUPPORTED;  // the register split would never be granted
    sm_counts[dev] = sms;
  }
  const int grid = (int)min(min((long long)sm_counts[dev], (long long)kMaxGrid), tiles);
  char* ws = static_cast<char*>(p.workspace);
  const size_t units = (size_t)p.batch * p.kv_heads * P.n_hg;
  P.ws_mul = reinterpret_cast<float*>(ws);
  ws += (units * 4 + 255) / 256 * 256;
  P.ws_join = reinterpret_cast<Join*>(ws);
  ws += kMaxGrid * 32;
  P.ws_ml = reinterpret_cast<float*>(ws);
  ws += (size_t)2 * kMaxGrid * N * 2 * 4;
  P.ws_acc = reinterpret_cast<float*>(ws);
  ws += (size_t)2 * kMaxGrid * N * NB * kBlock * 4;
  P.ws_q = reinterpret_cast<uint8_t*>(ws);
  // The kernel's set-up runs beside the query kernel, the join kernel's launch
  // beside the kernel's end (programmatic dependent launches).
  query_kernel<NB, N><<<(unsigned)units, 512, 0, stream>>>(P);
  if (cudaGetLastError() != cudaSuccess) return TQ_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(Roles<N>::kThreads);
  cfg.dynamicSmemBytes = P.pl.bytes;
  if (cudaLaunchKernelEx(&cfg, kern, P) != cudaSuccess) return TQ_ERR_CUDA;
  if (grid == 1) return TQ_OK;  // no cut
  cfg.gridDim = dim3((unsigned)(grid - 1), N / 8);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  if (cudaLaunchKernelEx(&cfg, join_kernel<NB, N>, P) != cudaSuccess) return TQ_ERR_CUDA;
  return TQ_OK;
}

// The narrowest N that holds a kv-head's rows, or else the widest that fits.
template <int NB, int N>
int pick(Params& P, cudaStream_t stream) {
  const int rows = P.t.q_heads / P.t.kv_heads * P.t.n_q;
  if constexpr (N < (NB == 1 ? 128 : 64)) {
    if (rows > N) {
      const int st = pick<NB, 2 * N>(P, stream);
      if (st != TQ_ERR_UNSUPPORTED) return st;
    }
  }
  if (plan<NB, N>(P.t, P.pl)) return run<NB, N>(P, stream);
  return TQ_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace tree

size_t tree_workspace_bytes(int batch, int kv_heads, int q_heads, int head_dim, int n_q) {
  // slots of the widest row group, and Q^ of every unit (two fp16 terms); the
  // rows of a kv-head fill whole row groups
  const size_t rows = (size_t)(q_heads / kv_heads) * n_q, wide = head_dim == kBlock ? 128 : 64;
  size_t n = 16;
  while (n < rows && n < wide) n *= 2;
  const size_t padded = (rows + n - 1) / n * n, units16 = (size_t)batch * kv_heads * ((rows + 15) / 16);
  return (units16 * 4 + 255) / 256 * 256 + tree::kMaxGrid * 32 + (size_t)2 * tree::kMaxGrid * n * (head_dim + 2) * 4 +
         (size_t)batch * kv_heads * padded * head_dim * 4;
}

int launch_tree(const TreeParams& t, cudaStream_t stream) {
  // tries of a wait (see bar_wait), read once a process
  static const int tries = [] {
    const char* s = std::getenv("TQ_TREE_WAIT_TRIES");
    const long n = s ? std::strtol(s, nullptr, 10) : 1L << 20;
    return (int)std::min(std::max(n, 1L), 1L << 20);
  }();
  tree::Params P{};
  P.t = t;
  P.t.wait_tries = tries;
  P.kscale = tree::centroid_scale(t.kcent, t.k_bits);
  P.vscale = tree::centroid_scale(t.vcent, t.v_bits);
  P.klev = tree::level_bytes(t.kcent, P.kscale, t.k_bits);
  return t.head_dim == kBlock ? tree::pick<1, 16>(P, stream) : tree::pick<2, 16>(P, stream);
}

}  // namespace tq
