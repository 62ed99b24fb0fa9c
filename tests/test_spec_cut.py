"""How the tree kernel's tiles are cut over its CTAs (csrc/tq_tree_cut.h), on the
CPU: every tile in one part, the parts of a unit found again, and parts of even
length whatever the batch's lengths are."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_decode_attention_tq_b200",
                    "csrc")
SWITCH = 3  # length of a unit's end, in tiles

# What a launch does: the prefix, then every part's walk.  A record per segment:
# part, entry, unit, kv-head, group, first and last tile, part_of the unit's first and last tile
SOURCE = """
#include <vector>
#include "tq_tree_cut.h"
using namespace tq::tree;
extern "C" int walk(const int* tiles, int batch, int ub, int n_hg, int grid, int* out, int room) {
  long long total = 0;
  for (int b = 0; b < batch; ++b) total += tiles[b];
  const int sw = switch_length(total * ub, grid);
  std::vector<int> prefix(batch + 1, 0);
  for (int b = 0; b < batch; ++b) prefix[b + 1] = prefix[b] + unit_length(tiles[b], sw);
  const Cut cut(prefix.data(), batch, ub, sw, grid);
  int n = 0;
  for (int c = 0; c < grid; ++c) {
    const long long begin = cut.start(c), end = c < cut.parts ? cut.start(c + 1) : begin;
    for (long long x = begin; x < end; ++n) {
      const Seg s = cut.find(x, end, n_hg);
      if (n >= room) return -1;
      const int r[9] = {c, s.b, s.r, s.kvh, s.hg, s.lo, s.hi - 1, (int)cut.part_of(s.b, s.r, 0),
                        (int)cut.part_of(s.b, s.r, s.nt - 1)};
      for (int i = 0; i < 9; ++i) out[9 * n + i] = r[i];
      x += s.nt - s.lo + sw;
    }
  }
  return n;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    d = tmp_path_factory.mktemp("cut")
    (d / "walk.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I" + CSRC, "-o", d / "walk.so", d / "walk.cpp"],
                   check=True)
    lib = ctypes.CDLL(str(d / "walk.so"))

    def call(tiles, ub, n_hg=1, grid=148):
        tiles = np.asarray(tiles, dtype=np.int32)
        out = np.zeros((grid + len(tiles) * ub + 1, 9), dtype=np.int32)
        n = lib.walk(ctypes.c_void_p(tiles.ctypes.data), len(tiles), ub, n_hg, grid, ctypes.c_void_p(out.ctypes.data),
                     len(out))
        assert n >= 0
        return out[:n]
    return call


def _check(seg, tiles, ub, n_hg, grid):
    """Every tile once and in order; what the join kernel relies on."""
    at = 0
    units = [(b, r) for b, n in enumerate(tiles) if n > 0 for r in range(ub)]
    parts = {}
    for c, b, r, kvh, hg, lo, hi, first, last in seg.tolist():
        assert (b, r) == units[at] and (kvh, hg) == (r // n_hg, r % n_hg)
        assert lo == parts.get((b, r), (0, 0))[1] and lo <= hi < tiles[b]
        f = parts.get((b, r), (c, 0))[0]
        assert first == f and (c == f if lo == 0 else c > f)  # the cut went through the unit
        assert (hi == tiles[b] - 1) == (c == last)
        parts[(b, r)] = (f, hi + 1)
        at += hi == tiles[b] - 1
    assert at == len(units)
    used = np.unique(seg[:, 0])
    assert np.array_equal(used, np.arange(min(grid, sum(tiles) * ub)))  # no part without a tile
    longest = np.bincount(seg[:, 0], weights=seg[:, 6] - seg[:, 5] + 1).max() if len(seg) else 0
    return int(longest)


@pytest.mark.parametrize("seed", range(40))
def test_every_tile_once(walk, seed):
    rng = np.random.default_rng(seed)
    batch, ub, grid = int(rng.integers(1, 40)), int(rng.integers(1, 20)), int(rng.choice([1, 2, 7, 148]))
    tiles = rng.integers(0, rng.choice([2, 5, 300, 4000]), batch) * (rng.random(batch) < rng.choice([0.1, 0.5, 1.0]))
    if grid > tiles.sum() * ub:
        grid = max(1, int(tiles.sum()) * ub)
    n_hg = 2 if ub % 2 == 0 else 1
    longest = _check(walk(tiles, ub, n_hg, grid), tiles.tolist(), ub, n_hg, grid)
    total, live = int(tiles.sum()) * ub, int((tiles > 0).sum()) * ub
    assert longest <= (total + SWITCH * live) / grid + 1 or total == 0


@pytest.mark.parametrize("slots,live", [(64, 1), (256, 1), (2048, 1), (64, 8), (64, 64)])
def test_empty_slots_take_no_part_of_the_work(walk, slots, live):
    """Live sequences of 256 tiles, 8 units each, spread over the slots: the
    longest part is that of the live sequences alone."""
    tiles = np.zeros(slots, dtype=int)
    tiles[np.linspace(0, slots - 1, live).astype(int)] = 256
    longest = _check(walk(tiles, 8), tiles.tolist(), 8, 1, 148)
    assert longest == _check(walk([256] * live, 8), [256] * live, 8, 1, 148)
    assert longest <= (256 + SWITCH) * 8 * live / 148 + 1


def test_long_lines(walk):
    _check(walk([2 ** 24, 0, 3, 2 ** 24 + 1], 16), [2 ** 24, 0, 3, 2 ** 24 + 1], 16, 1, 148)  # beyond 2^28 tiles
