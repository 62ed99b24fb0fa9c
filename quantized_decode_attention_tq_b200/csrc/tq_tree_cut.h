// How the tiles of the tree kernel are cut over its CTAs (device code; host
// code too, so that it can be checked on its own).
#pragma once

#ifdef __CUDACC__
#define TQ_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define TQ_HOST_DEVICE inline
#endif

namespace tq {
namespace tree {

// a / b for 0 <= a, 0 < b: 32-bit where both fit (a 64-bit division is a long
// subroutine, and several stand in a launch's critical path)
TQ_HOST_DEVICE long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (long long)((unsigned)a / (unsigned)b);
  return a / b;
}

// All units are laid end to end on one line: a tile takes a length of 1, and
// the end of a unit that has tiles kSwitch more (the partial, the next unit's
// query and the references of its first tile).  The line is cut into parts of
// equal length.  A tree of 64 nodes on 131072 positions: 277 us with no such
// length, 272 with 3, 5 or 8; other cases within 1%.  With few tiles per part
// the ends count nothing.  No part is without a tile: those with ends are at
// least 4 kSwitch long, and unit ends have a tile between them.
constexpr int kSwitch = 3;
TQ_HOST_DEVICE int switch_length(long long tiles, int grid) { return tiles >= 4LL * kSwitch * grid ? kSwitch : 0; }
TQ_HOST_DEVICE int unit_length(int tiles, int sw) { return tiles > 0 ? tiles + sw : 0; }  // empty slots take none

struct Seg {
  int b, r, kvh, hg;  // batch entry, unit of it: kv-head and row group
  int nt, lo, hi;     // tiles of the unit; lo .. hi - 1: those of the part (the next unit: nt - lo + sw on)
};

struct Cut {
  const int* prefix;  // [batch + 1]: unit_length of every entry before b, added up
  int batch, ub, sw;  // units per batch entry; length of a unit's end
  long long length, parts;
  TQ_HOST_DEVICE Cut(const int* pre, int b, int units, int end, int grid) : prefix(pre), batch(b), ub(units), sw(end) {
    length = (long long)pre[b] * units;
    parts = length < grid ? length : (long long)grid;  // (with ends, it is longer than the grid)
  }
  TQ_HOST_DEVICE int entry(long long x) const {  // the last entry that starts at or before x
    int lo = 0, hi = batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((long long)prefix[mid] * ub <= x) lo = mid;
      else hi = mid;
    }
    return lo;
  }
  // where part c begins: at a tile, or at the line's end
  TQ_HOST_DEVICE long long start(long long c) const {
    if (c >= parts) return length;
    const long long y = quotient(c * length, parts);
    if (sw == 0) return y;
    const int b = entry(y);
    const long long first = (long long)prefix[b] * ub, step = prefix[b + 1] - prefix[b];
    const long long rest = y - first, r = quotient(rest, step);
    return rest - r * step < step - sw ? y : first + (r + 1) * step;
  }
  // the part that holds tile t of unit r of batch entry b
  TQ_HOST_DEVICE long long part_of(int b, int r, int t) const {
    const long long step = prefix[b + 1] - prefix[b];
    return quotient(((long long)prefix[b] * ub + r * step + t + 1) * parts - 1, length);
  }
  // the unit at x and its tiles before `end`; n_hg row groups per kv-head
  TQ_HOST_DEVICE Seg find(long long x, long long end, int n_hg) const {
    Seg s;
    s.b = entry(x);
    const int step = prefix[s.b + 1] - prefix[s.b];
    const long long first = (long long)prefix[s.b] * ub;
    s.r = (int)quotient(x - first, step);
    s.kvh = s.r / n_hg;
    s.hg = s.r % n_hg;
    s.nt = step - sw;
    const long long begin = first + (long long)s.r * step;
    s.lo = (int)(x - begin);
    s.hi = end - begin < s.nt ? (int)(end - begin) : s.nt;
    return s;
  }
};

}  // namespace tree
}  // namespace tq
