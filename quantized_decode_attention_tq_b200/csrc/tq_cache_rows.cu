// Moving rows of the packed cache: in-place compaction and slot copies.  A row
// of one (slot, kv-head) is its K codes, V codes and v3 values (16-byte units)
// and its fp16 norms.  Nothing is computed: both are bound by HBM, at one read
// and one write of each moved row.

#include <type_traits>

#include "tq_spec_internal.h"

namespace tq {
namespace {

constexpr int kRowThreads = 256;

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ------------------------------------------------------------- compaction --
//
// A cluster of C CTAs owns one (sequence, kv-head) and walks its list in
// blocks of C * R entries, R per CTA.  A block's rows are read into shared
// memory by every CTA before any CTA of the cluster writes one (one cluster
// barrier per block).  Reads of the next block start before this block's
// writes: entry i reads a row >= start + i, and the rows written so far lie
// below start + (first entry of the next block), so no read meets a write
// that comes before it in the list.
template <int NB>
__global__ void __launch_bounds__(kRowThreads) compact_kernel(const __grid_constant__ CompactParams p, int R, int C,
                                                              FastDiv by_units) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x;
  const uint32_t unit = blockIdx.x / (unsigned)C;  // (sequence, kv-head)
  const int rank = (int)(blockIdx.x % (unsigned)C);
  const int b = (int)(unit / (unsigned)p.kv_heads), h = (int)(unit % (unsigned)p.kv_heads);
  const int per_row = p.units[0] + p.units[1] + p.units[2];
  const int n_raw = __ldg(p.n_keep + b), start = p.start ? __ldg(p.start + b) : 0;
  int n = min(max(n_raw, 0), p.max_keep);
  if (rank == 0 && h == 0 && tid == 0) {
    if (n != n_raw && p.status) atomicOr(p.status, TQ_DEV_LEN_RANGE);
    if (start < 0 && p.status) atomicOr(p.status, TQ_DEV_POS_RANGE);
    if (p.new_lens) p.new_lens[b] = (int)min(max((long long)start + n, 0LL), (long long)p.c.seq_cap);
  }
  if (start < 0) n = 0;
  uint8_t* rows_sm[2] = {smem, smem + (size_t)R * per_row * 16};
  int* idx_sm[2] = {reinterpret_cast<int*>(smem + (size_t)2 * R * per_row * 16),
                    reinterpret_cast<int*>(smem + (size_t)2 * R * per_row * 16) + R};
  uint16_t* norm_sm = reinterpret_cast<uint16_t*>(idx_sm[1] + R) + (size_t)tid * 2 * NB;  // this thread's entry
  const size_t base = (size_t)unit * p.c.seq_cap;  // first row of this (sequence, kv-head)
  const int32_t* keep = p.keep + (size_t)b * p.max_keep;
  const int block = C * R, blocks = (n + block - 1) / block;

  // entry of this thread in block n (thread t < R handles entry rank * R + t)
  auto entry = [&](int blk) {
    const long long i = (long long)blk * block + (long long)rank * R + tid;
    if (tid >= R || i >= n) return -1;
    const int s = __ldg(keep + i);
    if (s < start + i || s >= p.c.seq_cap) {
      if (h == 0 && p.status) atomicOr(p.status, TQ_DEV_POS_RANGE);
      return -1;
    }
    return s;
  };
  // the part and the unit inside it of row unit u
  auto part_of = [&](int u, int& part) {
    part = 0;
    if (u >= p.units[0]) {
      u -= p.units[0];
      part = 1;
      if (u >= p.units[1]) {
        u -= p.units[1];
        part = 2;
      }
    }
    return u;
  };
  uint16_t norm_r[2][2][NB] = {};  // [buffer][K, V][block]: norms of this thread's entry
  auto issue = [&](int buf, int idx) {
    int* ids = idx_sm[buf];
    if (tid < R) ids[tid] = idx;
    __syncthreads();
    for (int j = tid; j < R * per_row; j += kRowThreads) {
      const int r = (int)by_units.div((uint32_t)j);
      const int s = ids[r];
      if (s < 0) continue;
      int part;
      const int u = part_of(j - r * per_row, part);
      copy16_async(smem_u32(rows_sm[buf]) + 16u * (uint32_t)j,
                   p.c.codes[part] + ((base + s) * p.units[part] + u) * 16);
    }
    async_commit();
    if (idx >= 0) {
#pragma unroll
      for (int sd = 0; sd < 2; ++sd)
#pragma unroll
        for (int k = 0; k < NB; ++k) norm_r[buf][sd][k] = p.c.norms[sd][(base + idx) * NB + k];
    }
  };
  auto store = [&](int buf, int blk) {
    const int* ids = idx_sm[buf];
    const size_t row0 = base + start + (size_t)blk * block + (size_t)rank * R;
    for (int j = tid; j < R * per_row; j += kRowThreads) {
      const int r = (int)by_units.div((uint32_t)j);
      if (ids[r] < 0) continue;
      int part;
      const int u = part_of(j - r * per_row, part);
      *reinterpret_cast<uint4*>(p.c.codes[part] + ((row0 + r) * p.units[part] + u) * 16) =
          *reinterpret_cast<const uint4*>(rows_sm[buf] + (size_t)16 * j);
    }
    if (tid < R && ids[tid] >= 0) {
#pragma unroll
      for (int sd = 0; sd < 2; ++sd)
#pragma unroll
        for (int k = 0; k < NB; ++k) p.c.norms[sd][(row0 + tid) * NB + k] = norm_sm[sd * NB + k];
    }
  };

  if (blocks == 0) return;  // uniform over the cluster
  int next = entry(0);
  issue(0, next);
  if (blocks > 1) next = entry(1);
  // two blocks per round, so that the register buffers have fixed indices
  auto turn = [&](int blk, auto cur_tag) {
    constexpr int cur = decltype(cur_tag)::value;
    if (blk + 1 < blocks) {
      issue(cur ^ 1, next);
      if (blk + 2 < blocks) next = entry(blk + 2);
      async_wait<1>();
    } else {
      async_wait<0>();
    }
    // putting this block's norms into shared memory completes their loads,
    // which must be before another CTA of the cluster may write
    if (tid < R) {
#pragma unroll
      for (int sd = 0; sd < 2; ++sd)
#pragma unroll
        for (int k = 0; k < NB; ++k) norm_sm[sd * NB + k] = norm_r[cur][sd][k];
    }
    __syncthreads();
    if (C > 1) {
      // Every load of the block has returned (the wait above, the norms in
      // shared memory), so the cluster needs to meet but no fence (with one,
      // half of the rows of 8 x 32768 took 56 us instead of 51).
      asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
      asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    }
    store(cur, blk);
    __syncthreads();  // the buffer is free for block blk + 2
  };
  for (int blk = 0; blk < blocks; blk += 2) {
    turn(blk, std::integral_constant<int, 0>{});
    if (blk + 1 < blocks) turn(blk + 1, std::integral_constant<int, 1>{});
  }
}

// ------------------------------------------------------------------ copies --
//
// One CTA takes RC rows of one kv-head through `per` copies in order and keeps
// them in registers, so consecutive copies of the same source rows (a fork)
// read them once.  (Loading the next copy's rows ahead of the stores needs
// twice the registers: 43 -> 53 us on a fork of 32768 rows to 7 slots.)
constexpr int kUnitsPerThread = 8;

__global__ void __launch_bounds__(kRowThreads) copy_kernel(const __grid_constant__ CopyParams p, int RC, int per) {
  const int tid = threadIdx.x;
  const int h = (int)(blockIdx.x % (unsigned)p.kv_heads);
  const long long t0 = (long long)(blockIdx.x / (unsigned)p.kv_heads) * RC;
  uint4 reg[kUnitsPerThread];
  uint16_t nreg[2][2];
  int have_slot = -1, have_rows = 0;
  long long have_pos = -1;
  const int c_end = min((int)(blockIdx.y + 1) * per, p.n_copies);
  for (int c = (int)blockIdx.y * per; c < c_end; ++c) {
    const int ss = __ldg(p.src_slot + c), ds = __ldg(p.dst_slot + c);
    const long long sp = p.src_pos ? __ldg(p.src_pos + c) : 0, dp = p.dst_pos ? __ldg(p.dst_pos + c) : 0;
    const int want = __ldg(p.n_rows + c);
    long long n = min(max(want, 0), p.max_rows);
    uint32_t bad = n != want ? TQ_DEV_LEN_RANGE : 0u;
    if (ss < 0 || ss >= p.src.batch || ds < 0 || ds >= p.dst.batch || sp < 0 || dp < 0) {
      bad |= TQ_DEV_POS_RANGE;
      n = 0;
    } else if (n > min(p.src.seq_cap - sp, p.dst.seq_cap - dp)) {
      bad |= TQ_DEV_POS_RANGE;
      n = max(0LL, min(p.src.seq_cap - sp, p.dst.seq_cap - dp));
    }
    if (bad && blockIdx.x == 0 && tid == 0 && p.status) atomicOr(p.status, bad);
    const int m = (int)min((long long)RC, n - t0);  // rows of this CTA in copy c
    if (m <= 0) continue;
    const bool load = !(ss == have_slot && sp == have_pos && m <= have_rows);
    const size_t srow = ((size_t)ss * p.kv_heads + h) * p.src.seq_cap + sp + t0;
    const size_t drow = ((size_t)ds * p.kv_heads + h) * p.dst.seq_cap + dp + t0;
    // Unit j of the CTA's rows, counted part by part at RC rows each, sits in
    // register j / threads; the parts are contiguous in both caches.
#pragma unroll
    for (int i = 0; i < kUnitsPerThread; ++i) {
      int j = tid + i * kRowThreads, part = 0;
      if (j >= RC * p.units[0]) {
        j -= RC * p.units[0];
        part = 1;
        if (j >= RC * p.units[1]) {
          j -= RC * p.units[1];
          part = 2;
        }
      }
      if (j < m * p.units[part]) {
        if (load) reg[i] = *reinterpret_cast<const uint4*>(p.src.codes[part] + (srow * p.units[part] + j) * 16);
      }
    }
    const int nn = m * p.nb;  // norms per side, at most 2 per thread
#pragma unroll
    for (int sd = 0; sd < 2; ++sd)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (load && tid + i * kRowThreads < nn) nreg[sd][i] = p.src.norms[sd][srow * p.nb + tid + i * kRowThreads];
#pragma unroll
    for (int i = 0; i < kUnitsPerThread; ++i) {
      int j = tid + i * kRowThreads, part = 0;
      if (j >= RC * p.units[0]) {
        j -= RC * p.units[0];
        part = 1;
        if (j >= RC * p.units[1]) {
          j -= RC * p.units[1];
          part = 2;
        }
      }
      if (j < m * p.units[part])
        *reinterpret_cast<uint4*>(p.dst.codes[part] + (drow * p.units[part] + j) * 16) = reg[i];
    }
#pragma unroll
    for (int sd = 0; sd < 2; ++sd)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (tid + i * kRowThreads < nn) p.dst.norms[sd][drow * p.nb + tid + i * kRowThreads] = nreg[sd][i];
    if (load) {
      have_slot = ss;
      have_pos = sp;
      have_rows = m;
    }
  }
}

template <int NB>
int run_compact(const CompactParams& p, cudaStream_t stream) {
  const int per_row = p.units[0] + p.units[1] + p.units[2];
  // rows per CTA and block: as many as two buffers of 96 KiB together hold
  int R = kRowThreads;
  while (R > 32 && (size_t)2 * R * per_row * 16 > 96 * 1024) R /= 2;
  while (R > 32 && R / 2 >= p.max_keep) R /= 2;  // a short list needs no more
  int C = 1;
  while (C < 8 && (long long)C * R < p.max_keep) C *= 2;
  const size_t smem = (size_t)2 * R * per_row * 16 + (size_t)2 * R * 4 + (size_t)2 * R * NB * 2;
  auto kern = compact_kernel<NB>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return TQ_ERR_CUDA;
  static bool ready[64] = {false};
  if (!ready[dev]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 104 * 1024) != cudaSuccess)
      return TQ_ERR_CUDA;
    ready[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.c.batch * p.kv_heads) * (unsigned)C);
  cfg.blockDim = dim3(kRowThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p, R, C, FastDiv::make((uint32_t)per_row)) != cudaSuccess) return TQ_ERR_CUDA;
  return TQ_OK;
}

}  // namespace

int launch_cache_compact(const CompactParams& p, cudaStream_t stream) {
  switch (p.nb) {
    case 1: return run_compact<1>(p, stream);
    case 2: return run_compact<2>(p, stream);
    case 3: return run_compact<3>(p, stream);
  }
  return run_compact<4>(p, stream);
}

int launch_cache_copy(const CopyParams& p, cudaStream_t stream) {
  const int per_row = p.units[0] + p.units[1] + p.units[2];
  // rows per CTA: what 8 units and 2 norms a side per thread hold, fewer
  // while that leaves SMs without work
  int RC = kRowThreads * kUnitsPerThread / per_row;
  if (RC > 2 * kRowThreads / p.nb) RC = 2 * kRowThreads / p.nb;
  while (RC > 16 && ((long long)p.max_rows + RC - 1) / RC * p.kv_heads < 4 * 148) RC /= 2;
  const long long ctas = ((long long)p.max_rows + RC - 1) / RC * p.kv_heads;
  if (ctas >= (1LL << 31)) return TQ_ERR_UNSUPPORTED;
  // all copies in one CTA where that gives every SM eight, else split
  const long long want = min((8LL * 148 + ctas - 1) / ctas, (long long)min(p.n_copies, 1 << 15));
  const int per = (int)((p.n_copies + want - 1) / want);
  copy_kernel<<<dim3((unsigned)ctas, (unsigned)((p.n_copies + per - 1) / per)), kRowThreads, 0, stream>>>(p, RC, per);
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // namespace tq
