"""Host side of the speculative-decoding operators (CPU only): declared symbols,
structures, the rotation's frequencies, tree masks, and the refusals of every
entry point before anything is launched."""
import ctypes
import os
import re

import numpy as np
import pytest

import quantized_decode_attention_tq_b200 as tq
from quantized_decode_attention_tq_b200 import _lib

from . import _spec_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GOOD = 0x7F0000000000  # an aligned address that no refused call dereferences
BAD, UNS, OK = _lib.TQ_ERR_INVALID_ARG, _lib.TQ_ERR_UNSUPPORTED, _lib.TQ_OK


def test_every_declared_symbol_is_bound():
    text = open(os.path.join(ROOT, "include", "tq_spec.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(tq_[a-z_0-9]+)\s*\(", text))
    assert names == set(_lib.SPEC_SIGNATURES)
    for n in names:
        assert hasattr(tq.lib(), n)


def test_struct_layouts():
    assert ctypes.sizeof(_lib.Rope) == 16 + 8 * 256 and _lib.Rope.turns.offset == 16
    assert ctypes.sizeof(_lib.Rows) == 56 and _lib.Rows.batch_stride.offset == 32
    assert ctypes.sizeof(_lib.CacheBufs) == 48 and _lib.CacheBufs.outliers.offset == 40


@pytest.mark.parametrize("rot", [2, 6, 96, 128, 512])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 32.0)])
def test_rope_frequencies(rot, scaling, factor):
    r = tq.make_rope(rot, base=500000.0, scaling=scaling, factor=factor, orig_ctx=8192, interleaved=True)
    f, gain = R.frequencies(rot, 500000.0, scaling, factor, 8192)
    turns = np.array([int(t) for t in r.turns], dtype=object)
    assert all(t == 0 for t in turns[rot // 2:])
    # the reference's f is good to a few parts in 2^52 (pow, a product, a sum)
    want = f / (2 * np.pi)
    got = np.array([float(t) for t in turns[:rot // 2]]) / 2.0 ** 64
    assert np.all(np.abs(got - want) <= 16 * 2.0 ** -52 * want + 2.0 ** -64)
    assert r.rot_dim == rot and r.interleaved == 1 and r.gain == np.float32(gain)


def test_rope_refusals():
    f, r = tq.lib().tq_make_rope, _lib.Rope()
    p = ctypes.byref(r)
    assert f(128, 0, 1e4, 0, 1.0, 4096, 32, 1, None) == BAD
    assert f(127, 0, 1e4, 0, 1.0, 4096, 32, 1, p) == BAD
    assert f(-2, 0, 1e4, 0, 1.0, 4096, 32, 1, p) == BAD
    assert f(514, 0, 1e4, 0, 1.0, 4096, 32, 1, p) == UNS
    assert f(128, 0, 1e4, 4, 1.0, 4096, 32, 1, p) == UNS
    assert f(128, 0, 1.0, 0, 1.0, 4096, 32, 1, p) == BAD
    assert f(128, 0, float("nan"), 0, 1.0, 4096, 32, 1, p) == BAD
    assert f(128, 0, 1e4, 1, 0.5, 4096, 32, 1, p) == BAD
    assert f(128, 0, 1e4, 3, 2.0, 0, 32, 1, p) == BAD
    assert f(128, 0, 1e4, 3, 2.0, 4096, 1, 32, p) == BAD
    assert f(0, 0, 1e4, 3, 2.0, 4096, 32, 1, p) == OK
    with pytest.raises(ValueError):
        tq.make_rope(128, scaling="other")


def _rows(heads=4, stride=512, addr=GOOD, weight=None):
    return _lib.Rows(addr, GOOD, weight, heads, stride, stride, 128)


def test_norm_rope_refusals():
    f, rope = tq.lib().tq_qk_norm_rope, tq.make_rope(128)

    def call(rope=rope, batch=2, seq=3, dim=128, q=_rows(), k=None, v=None, it=1, wt=1, ot=1, norm=1, eps=1e-6,
             bias=0.0, pos=GOOD, n_tok=None):
        ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
        return f(ref(rope), batch, seq, dim, ref(q), ref(k), ref(v), it, wt, ot, norm, eps, bias, pos, n_tok, None)

    assert call(seq=0) == OK  # a no-op
    assert call(batch=0) == BAD and call(seq=-1) == BAD and call(q=None) == BAD
    assert call(it=3) == BAD and call(wt=-1) == BAD and call(ot=9) == BAD
    assert call(dim=96) == UNS and call(dim=640) == UNS
    assert call(rope=tq.make_rope(256)) == BAD  # wider than the row
    assert call(pos=None) == BAD and call(pos=GOOD + 2) == BAD and call(n_tok=GOOD + 1) == BAD
    assert call(eps=-1.0) == BAD and call(eps=float("nan")) == BAD and call(bias=float("inf")) == BAD
    assert call(q=_rows(heads=0)) == BAD and call(q=_rows(addr=GOOD + 8)) == BAD
    assert call(q=_rows(stride=4)) == BAD and call(q=_rows(stride=-128)) == BAD
    assert call(q=_rows(weight=GOOD + 1)) == BAD
    assert call(batch=1 << 20, seq=1 << 12) == UNS


def test_tree_masks():
    #       -1
    #      0    1
    #     2 3   4
    #     5
    m, d = tq.tree_masks([-1, -1, 0, 0, 1, 2])
    assert [int(x) for x in m] == [1, 2, 5, 9, 18, 37] and list(d) == [0, 0, 1, 1, 1, 2]
    m, d = tq.tree_masks([[-1] + list(range(63))] * 2)  # a chain of 64
    assert m.shape == (2, 64) and m[1, 63] == -1 and d[1, 63] == 63
    for bad in ([0], [-2], [-1, 1], [-1] * 65, []):
        with pytest.raises((tq.TQError, ValueError)):
            tq.tree_masks(bad)


def test_tree_attention_refusals():
    d = tq.kv_desc(2, 2, 128, 64, 3, 2)
    cbs = {b: tq.make_codebook(b) for b in (2, 3)}
    need = tq.tree_workspace_size(d, 8, 5)
    assert need > 0
    assert tq.tree_workspace_size(d, 7, 5) == 0 and tq.tree_workspace_size(d, 8, 0) == 0
    assert tq.tree_workspace_size(d, 8, 65) == 0
    assert tq.tree_workspace_size(tq.kv_desc(2, 2, 384, 64, 3, 2), 8, 5) == 0

    def call(d=d, kb=3, hq=8, n=5, q=GOOD, qt=1, kc=GOOD, lens=GOOD, nodes=None, tree=GOOD, scale=0.1, out=GOOD, ot=1,
             ws=GOOD, wsb=need):
        return tq.lib().tq_decode_attention_tree(ctypes.byref(d), ctypes.byref(cbs[kb]), ctypes.byref(cbs[2]), hq, n, q,
                                                 qt, kc, GOOD, GOOD, GOOD, lens, nodes, tree, scale, out, ot, ws, wsb,
                                                 None, None)

    assert call(n=0) == BAD and call(n=65) == BAD and call(hq=7) == BAD and call(kb=2) == BAD
    assert call(qt=3) == BAD and call(ot=0) == BAD and call(scale=0.0) == BAD and call(scale=float("inf")) == BAD
    assert call(q=None) == BAD and call(kc=GOOD + 8) == BAD and call(lens=None) == BAD and call(out=GOOD + 2) == BAD
    assert call(tree=None) == BAD and call(tree=GOOD + 4) == BAD and call(nodes=GOOD + 2) == BAD
    assert call(d=tq.kv_desc(2, 2, 384, 64, 3, 2)) == UNS and call(d=tq.kv_desc(2, 2, 128, 63, 3, 2)) == UNS
    assert call(d=tq.kv_desc(4096, 2, 128, 64, 3, 2)) == UNS
    assert call(ws=None) == _lib.TQ_ERR_WORKSPACE and call(ws=GOOD + 16) == _lib.TQ_ERR_WORKSPACE
    assert call(wsb=need - 1) == _lib.TQ_ERR_WORKSPACE


def _bufs(**kw):
    c = dict(k_codes=GOOD, k_norms=GOOD, v_codes=GOOD, v_norms=GOOD, values=None, outliers=0)
    c.update(kw)
    return _lib.CacheBufs(**c)


BAD_BUFS = [dict(k_codes=None), dict(v_norms=None), dict(v_codes=GOOD + 8), dict(k_norms=GOOD + 2), dict(outliers=17),
            dict(outliers=-1), dict(outliers=3), dict(values=GOOD), dict(values=GOOD + 8, outliers=3)]


def test_compact_refusals():
    d = tq.kv_desc(2, 2, 128, 64, 3, 2)

    def call(d=d, c=_bufs(), keep=GOOD, m=4, n=GOOD, start=None, lens=None):
        return tq.lib().tq_cache_compact(ctypes.byref(d), ctypes.byref(c), keep, m, n, start, lens, None, None)

    assert call(m=0) == OK
    for kw in BAD_BUFS:
        assert call(c=_bufs(**kw)) == BAD, kw
    assert call(d=tq.kv_desc(2, 2, 100, 64, 3, 2)) == UNS and call(d=tq.kv_desc(2, 0, 128, 64, 3, 2)) == BAD
    assert call(keep=None) == BAD and call(n=None) == BAD and call(m=-1) == BAD
    assert call(keep=GOOD + 1) == BAD and call(n=GOOD + 2) == BAD and call(start=GOOD + 2) == BAD
    assert call(lens=GOOD + 2) == BAD
    far = GOOD + (1 << 20)
    assert call(start=far, lens=far) == BAD and call(n=far, lens=far + 4) == BAD  # written while they are read
    assert call(keep=far, lens=far + 28) == BAD and call(m=0, n=far, lens=far - 4) == BAD


def test_copy_refusals():
    d = tq.kv_desc(2, 2, 128, 64, 3, 2)

    def call(d=d, e=d, c=_bufs(), x=_bufs(), n=2, ss=GOOD, ds=GOOD, sp=None, dp=None, rows=GOOD, m=8):
        return tq.lib().tq_cache_copy(ctypes.byref(d), ctypes.byref(c), ctypes.byref(e), ctypes.byref(x), n, ss, ds, sp,
                                      dp, rows, m, None, None)

    assert call(n=0) == OK and call(m=0) == OK
    for kw in BAD_BUFS:
        assert call(c=_bufs(**kw)) == BAD and call(x=_bufs(**kw)) == BAD, kw
    for e in ((2, 4, 128, 64, 3, 2), (2, 2, 256, 64, 3, 2), (2, 2, 128, 64, 2, 2), (2, 2, 128, 64, 3, 3)):
        assert call(e=tq.kv_desc(*e)) == BAD
    assert call(e=tq.kv_desc(2, 2, 128, 64, 3, 2, sign_seed=1)) == BAD
    assert call(x=_bufs(values=GOOD, outliers=4)) == BAD  # the outlier counts differ
    assert call(n=-1) == BAD and call(m=-1) == BAD and call(ss=None) == BAD and call(rows=None) == BAD
    assert call(ss=GOOD + 1) == BAD and call(ds=GOOD + 2) == BAD and call(sp=GOOD + 2) == BAD


def test_binding_refuses_before_the_library():
    import torch
    x = torch.zeros(1, 1, 1, 128)
    with pytest.raises(ValueError):
        tq.qk_norm_rope(None, q=x, q_out=x)  # not on a GPU
    with pytest.raises(ValueError):
        tq.qk_norm_rope(None)


def test_binding_refuses_max_rows_that_its_int_cannot_hold():
    with pytest.raises(ValueError, match="max_rows"):
        tq.cache_copy(None, None, None, None, None, 2 ** 32)


def test_the_two_plain_forms_of_tree_attention_agree():
    rng = np.random.default_rng(0)
    cache = R.random_cache(rng, 3, 2, 40, 256, 3, 2)
    q = rng.standard_normal((3, 4, 6, 256))
    masks = np.array([[1, 3, 0, 9], [1, 2, 5, 8], [0, 2, 4, 8]], dtype=np.int64)
    args = (q, cache, 3, 2, [40, 4, 0], [4, 3, 2], masks, 0.0625, 5)
    for x, y in zip(R.tree_attention(*args), R.tree_attention_by_head(*args)):
        assert np.array_equal(np.isnan(x), np.isnan(y))
        live = ~np.isnan(x)
        assert np.allclose(x[live], y[live], rtol=1e-12, atol=1e-12)


def test_norm_rope_of_no_tokens_is_a_no_op_without_addresses():
    """Empty tensors have a null address."""
    f, rows = tq.lib().tq_qk_norm_rope, _lib.Rows(None, None, None, 4, 0, 0, 0)
    rope = tq.make_rope(64)
    args = [ctypes.byref(rope), 2, 0, 128, ctypes.byref(rows), None, None, 1, 1, 1, 1, 1e-6, 0.0, None, None, None]
    assert f(*args) == OK
    assert f(*args[:3], 96, *args[4:]) == UNS and f(*args[:7], 3, *args[8:]) == BAD  # the rest is still checked
    assert f(*args[:2], 1, *args[3:]) == BAD


def test_binding_refuses_max_rows_below_zero():
    for n in (-1, -2 ** 32 + 5):  # the second's lower bits are 5
        with pytest.raises(ValueError, match="max_rows"):
            tq.cache_copy(None, None, None, None, None, n)


def test_packed_structures_are_the_declared_ones():
    """The binding packs tq_rows and tq_cache_bufs; their fields lie where the structures have them."""
    from quantized_decode_attention_tq_b200 import spec
    rows = _lib.Rows.from_buffer_copy(spec._ROWS.pack(1, 2, 3, 4, 5, 6, 7))
    assert [getattr(rows, n) for n, _ in _lib.Rows._fields_] == [1, 2, 3, 4, 5, 6, 7]
    bufs = _lib.CacheBufs.from_buffer_copy(spec._BUFS.pack(1, 2, 3, 4, 5, 6))
    assert [getattr(bufs, n) for n, _ in _lib.CacheBufs._fields_] == [1, 2, 3, 4, 5, 6]
    assert spec._ROWS.size == ctypes.sizeof(_lib.Rows) and spec._BUFS.size == ctypes.sizeof(_lib.CacheBufs)
