"""GPU parity of the speculative-decoding operators against plain fp64
references, and a run of them together as a serving loop uses them."""
import itertools

import numpy as np
import pytest

import quantized_decode_attention_tq_b200 as tq
from oracle import tq_oracle as O

from . import _spec_ref as R
from ._parity import to_dev, torch_mod

pytestmark = pytest.mark.gpu


def _dt(name):
    return getattr(torch_mod(), name)


def _np(t):
    return t.detach().double().cpu().numpy()


# ---------------------------------------------------------------- norm + rope --

def _rope_case(rng, batch, tokens, hq, hk, dim, rot, interleaved, scaling, factor, norm, src, dst, ragged=False,
               start=1000, joint=True, weights=True, bias=0.0):
    torch = torch_mod()
    rope = tq.make_rope(rot, scaling=scaling, factor=factor, interleaved=interleaved) if rot else None
    qkv = torch.from_numpy(rng.standard_normal((batch, tokens, (hq + 2 * hk) * dim))).to(_dt(src)).cuda()
    q, k, v = (x.unflatten(2, (-1, dim)) for x in qkv.split([hq * dim, hk * dim, hk * dim], 2))
    if not joint:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    qw, kw = ((torch.from_numpy(1 + 0.1 * rng.standard_normal(dim)).to(_dt(src)).cuda() if weights else None)
              for _ in range(2))
    pos = to_dev((start + rng.integers(-50, 50, (batch, tokens))).astype(np.int32))
    n_tok = to_dev(rng.integers(0, tokens + 1, batch).astype(np.int32)) if ragged else None
    outs = [torch.full(s, 7.0, dtype=_dt(dst), device="cuda")
            for s in ((batch, tokens, hq, dim), (batch, hk, tokens, dim), (batch, hk, tokens, dim))]
    tq.qk_norm_rope(rope, q, k, v, pos, *outs, norm=norm, q_weight=qw, k_weight=kw, weight_bias=bias, n_tok=n_tok)
    torch.cuda.synchronize()
    f, gain = R.frequencies(rot, 10000.0, scaling, factor) if rot else (np.zeros(0), 1.0)
    count = np.full(batch, tokens) if n_tok is None else n_tok.cpu().numpy()
    live = np.arange(tokens)[None] < count[:, None]
    # Half a step of the output; 32 roundings of fp32 before it: at most 21 in
    # the mean of squares (half of them after the root), 4 in the norm's
    # quotient and products, and in the rotation 2 in cos or sin each, their
    # gain, two products and a sum, against the pair's length r.
    u_out, u32 = torch.finfo(_dt(dst)).eps / 2, 2.0 ** -24
    floor = {"float16": 2.0 ** -25}.get(dst, 0.0)
    for i, (x, w) in enumerate(((q, qw), (k, kw), (v, None))):
        ww = None if w is None else _np(w)
        if i < 2:
            y, r = R.norm_rope(_np(x), ww, pos.cpu().numpy(), f, gain, interleaved, norm, bias=bias)
        else:
            y, r = _np(x), np.zeros(x.shape)
        got = _np(outs[i]) if i == 0 else _np(outs[i]).transpose(0, 2, 1, 3)
        assert np.all(got[~live] == 7.0)
        err, allowed = np.abs(got - y), u_out * np.abs(y) * (1 + 2 ** -10) + 32 * u32 * r + floor
        assert np.all((err <= allowed)[live]), f"side {i}: {np.max((err / np.maximum(allowed, 1e-300))[live]):.3f}"


@pytest.mark.parametrize("dim,rot,interleaved", [(128, 128, False), (128, 128, True), (128, 64, False), (128, 36, False),
                                                 (128, 36, True), (128, 2, False), (256, 256, False), (256, 90, True),
                                                 (256, 16, False), (384, 384, False), (384, 200, True), (384, 50, False),
                                                 (512, 512, False), (512, 512, True), (512, 510, False), (128, 0, False)])
def test_rope_layouts(dim, rot, interleaved):
    rng = np.random.default_rng(dim + rot)
    _rope_case(rng, 2, 5, 4, 2, dim, rot, interleaved, "none", 1.0, True, "float32", "float32")
    _rope_case(rng, 3, 7, 3, 1, dim, rot, interleaved, "linear", 4.0, False, "bfloat16", "float16", ragged=True)


@pytest.mark.parametrize("src,dst", list(itertools.product(["float32", "float16", "bfloat16"], repeat=2)))
def test_rope_types(src, dst):
    _rope_case(np.random.default_rng(3), 2, 3, 8, 2, 128, 128, False, "yarn", 16.0, True, src, dst, bias=1.0)


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 8.0), ("ntk", 4.0), ("yarn", 32.0)])
def test_rope_far_and_negative_positions(scaling, factor):
    # the reference's angle is good to 2^-53 of itself: 2^31 rad * 2^-53 = 2.4e-7 rad, four of the 32 roundings
    for start in (2 ** 31 - 60, -(2 ** 31) + 60, 1000003, 0):
        _rope_case(np.random.default_rng(5), 1, 9, 2, 1, 128, 128, False, scaling, factor, False, "float32", "float32",
                   start=start)


@pytest.mark.parametrize("batch,tokens", [(1, 1), (1, 2500), (7, 431)])
def test_rope_sizes(batch, tokens):
    _rope_case(np.random.default_rng(6), batch, tokens, 5, 1, 128, 128, False, "none", 1.0, True, "bfloat16", "float16",
               ragged=batch > 1, joint=False, weights=False)


def test_rope_sides_alone_and_special_values():
    torch = torch_mod()
    rope = tq.make_rope(32)
    x = torch.randn(2, 3, 2, 128, device="cuda", dtype=torch.float16)
    x[0, 0, 0, 100], x[0, 1, 0, 3] = float("inf"), float("nan")
    pos = torch.arange(6, device="cuda", dtype=torch.int32).reshape(2, 3)
    a, b = torch.zeros_like(x), torch.zeros(2, 2, 3, 128, device="cuda", dtype=torch.float16)
    tq.qk_norm_rope(rope, q=x, positions=pos, q_out=a, norm=False)
    tq.qk_norm_rope(rope, k=x, positions=pos, k_out=b, norm=False)
    b2 = torch.zeros_like(b)
    tq.qk_norm_rope(None, v=x, v_out=b2)
    torch.cuda.synchronize()
    same = lambda s, t: torch.equal(s.nan_to_num(9.0), t.nan_to_num(9.0))  # noqa: E731
    assert same(a.transpose(1, 2), b) and same(x.transpose(1, 2), b2)
    # an infinity outside the rotated part stays where it is, a NaN in its pair
    assert torch.isinf(a).nonzero().tolist() == [[0, 0, 0, 100]]
    assert torch.isnan(a).nonzero().tolist() == [[0, 1, 0, 3], [0, 1, 0, 19]]


# ---------------------------------------------------------------------- tree --

def _dev_cache(cache, desc):
    kc, kn, vc, vn = cache
    return tq.Cache(desc, to_dev(kc), to_dev(kn.view(np.int16)), to_dev(vc), to_dev(vn.view(np.int16)))


def _random_tree(rng, n, roots=2):
    par = [-1 if j < roots else int(rng.integers(0, j)) for j in range(n)]
    return tq.tree_masks(par)[0]


def _tree_case(seed, batch, hq, hk, dim, kb, vb, cap, lens, n_q, counts=None, masks=None, src="float16", dst="float16",
               scale=None, cache=None, sign_seed=0, q=None, v_levels=1.0):
    torch = torch_mod()
    rng = np.random.default_rng(seed)
    cache = cache or R.random_cache(rng, batch, hk, cap, dim, kb, vb)
    desc = tq.kv_desc(batch, hk, dim, cap, kb, vb, sign_seed)
    dc = _dev_cache(cache, desc)
    if q is None:
        q = rng.standard_normal((batch, n_q, hq, dim))
    qd = torch.from_numpy(np.asarray(q)).to(_dt(src)).cuda()
    if masks is None:
        masks = np.stack([_random_tree(rng, n_q, min(2, n_q)) for _ in range(batch)])
    lens = np.asarray(lens, dtype=np.int32)
    cnt = np.full(batch, n_q) if counts is None else np.asarray(counts)
    out = torch.full((batch, n_q, hq, dim), 3.0, dtype=_dt(dst), device="cuda")
    ws = tq.alloc_tree_workspace(desc, hq, n_q)
    ws.fill_(255)  # NaN everywhere: any content is allowed
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    scale = dim ** -0.5 if scale is None else scale
    v_cb = tq.make_codebook(vb)
    for i in range(1 << vb):  # the sum over V is linear in its levels
        v_cb.centroids[i] *= v_levels
    tq.decode_attention_tree(dc, tq.make_codebook(kb), v_cb, qd, to_dev(lens), to_dev(masks), scale, out, ws,
                             n_nodes=None if counts is None else to_dev(cnt.astype(np.int32)), status=status)
    torch.cuda.synchronize()
    assert tq.read_device_status(status) == 0
    ref, spread, score = R.tree_attention(_np(qd), cache, kb, vb, lens, cnt, masks, scale, sign_seed)
    got = _np(out)
    past = np.isnan(ref)
    assert np.all(got[past] == 3.0)
    got = got / v_levels
    R.check_tree(got, ref, spread, score, torch.finfo(_dt(dst)).eps)
    return got, ref


@pytest.mark.parametrize("kb,vb", list(itertools.product([2, 3, 4], repeat=2)))
def test_tree_bits(kb, vb):
    _tree_case(kb * 4 + vb, 2, 8, 2, 128, kb, vb, 300, [300, 131], 7)
    _tree_case(kb * 4 + vb, 1, 4, 2, 256, kb, vb, 200, [197], 5, src="bfloat16", dst="bfloat16")


@pytest.mark.parametrize("dim,bits", [(128, 4), (128, 3), (256, 4), (256, 3), (256, 2)])
@pytest.mark.parametrize("v_levels", [1.0, 1.25])
def test_tree_wide_groups_with_equal_and_unequal_codebooks(dim, bits, v_levels):
    # 130 rows: the widest row groups and the fullest shared memory; K and V share a table or not
    _tree_case(dim + bits, 1, 10, 1, dim, bits, bits, 400, [390], 13, v_levels=v_levels)


@pytest.mark.parametrize("hq,hk,n_q", [(1, 1, 1), (1, 1, 2), (4, 4, 3), (8, 2, 4), (8, 1, 5), (12, 4, 16), (32, 8, 8),
                                       (4, 1, 33), (2, 2, 64), (16, 2, 16), (8, 2, 64), (6, 1, 64), (20, 1, 13)])
def test_tree_rows(hq, hk, n_q):
    _tree_case(n_q, 1, hq, hk, 128, 3, 3, 260, [257], n_q)


@pytest.mark.parametrize("dim", [128, 256])
@pytest.mark.parametrize("length", [1, 2, 127, 128, 129, 255, 256, 257, 1000])
def test_tree_lengths(dim, length):
    n = min(length, 5)
    _tree_case(length, 2, 4, 2, dim, 3, 2, 1000, [length, max(n, length - 64)], n)


def test_tree_empty_sequences_rows_and_nodes():
    masks = np.array([[0, 1, 2, 4], [1, 3, 0, 9], [15, 15, 15, 15], [0, 0, 0, 0]], dtype=np.int64)
    # sequence 0 is its nodes alone: row 0 sees nothing; sequence 1 has no node 3;
    # sequence 2 is empty (its nodes do not exist); sequence 3 is padded away
    got, _ = _tree_case(1, 4, 2, 1, 128, 4, 4, 64, [4, 40, 0, 9], 4, counts=[4, 3, 0, 0], masks=masks)
    assert np.all(got[0, 0] == 0.0) and np.all(got[2] == 3.0) and np.all(got[3] == 3.0)


def test_tree_nodes_before_the_cache():
    # two positions cached, four nodes named: nodes 0 and 1 do not exist
    masks = np.array([[1, 3, 7, 15]], dtype=np.int64)
    torch = torch_mod()
    rng = np.random.default_rng(0)
    cache = R.random_cache(rng, 1, 1, 16, 128, 3, 3)
    desc = tq.kv_desc(1, 1, 128, 16, 3, 3)
    q = torch.randn(1, 4, 1, 128, device="cuda", dtype=torch.float16)
    out = torch.full_like(q, 3.0)
    tq.decode_attention_tree(_dev_cache(cache, desc), tq.make_codebook(3), tq.make_codebook(3), q,
                             to_dev(np.array([2], dtype=np.int32)), to_dev(masks), 0.09, out,
                             tq.alloc_tree_workspace(desc, 1, 4))
    got = _np(out)
    assert np.all(got[0, :2] == 0.0)
    v = O.dequantize(cache[2], cache[3], 3, O.codebook_f32(3)[0], O.sign_vector(0))
    # row 2 sees position 0 alone: its V, off by the fp16 weight, centroid and output (3 * 2^-11)
    assert np.linalg.norm(got[0, 2, 0] - v[0, 0, 0]) <= 3.1 * 2 ** -11 * np.linalg.norm(v[0, 0, 0])


def test_tree_is_causal_multi_for_a_chain():
    """A chain of nodes is decode_attention_multi's case."""
    torch = torch_mod()
    rng = np.random.default_rng(2)
    cache = R.random_cache(rng, 2, 2, 512, 128, 3, 3)
    desc = tq.kv_desc(2, 2, 128, 512, 3, 3)
    dc, cb = _dev_cache(cache, desc), tq.make_codebook(3)
    q = torch.randn(2, 16, 8, 128, device="cuda", dtype=torch.float16)
    lens = to_dev(np.array([512, 300], dtype=np.int32))
    masks = np.stack([tq.tree_masks([-1] + list(range(15)))[0]] * 2)
    out = torch.zeros_like(q)
    tq.decode_attention_tree(dc, cb, cb, q, lens, to_dev(masks), 0.0884, out, tq.alloc_tree_workspace(desc, 8, 16))
    multi = torch.zeros(q.shape, device="cuda")
    tq.decode_attention_multi(dc, cb, cb, q, lens, 0.0884, multi, tq.alloc_workspace(desc, 8 * 16))
    ref, spread, score = R.tree_attention(_np(q), cache, 3, 3, [512, 300], [16, 16], masks, 0.0884)
    R.check_tree(_np(out), ref, spread, score, 2.0 ** -10)
    R.check_tree(_np(multi), ref, spread, score, 2.0 ** -23)


@pytest.mark.parametrize("scale,norm", [(0.5, 11.3), (3.0, 11.3), (0.0884, 0.002), (0.0884, 3000.0), (1e-4, 60000.0)])
def test_tree_peaked_scores_and_value_sizes(scale, norm):
    """Near one-hot weights, V of any size fp16 norms hold.  q is scaled so that the scores stay those of norm 11.3."""
    rng = np.random.default_rng(9)
    cache = R.random_cache(rng, 1, 2, 700, 128, 4, 3, norm=11.3)
    cache[3] = np.minimum(cache[3].astype(np.float64) * norm / 11.3, 65000).astype(np.float16)
    _tree_case(3, 1, 4, 2, 128, 4, 3, 700, [700], 6, scale=scale, cache=cache, src="float32", dst="bfloat16")


def test_tree_norms_that_grow_along_the_sequence():
    rng = np.random.default_rng(10)
    cache = R.random_cache(rng, 1, 1, 900, 128, 3, 3)
    grow = np.exp(np.linspace(np.log(1e-3), np.log(5e4), 900)).astype(np.float16)
    cache[3][0, 0, :, 0] = grow
    _tree_case(4, 1, 4, 1, 128, 3, 3, 900, [900], 4, cache=cache, dst="bfloat16")
    cache[3][0, 0, :, 0] = grow[::-1]
    cache[1][0, 0, :, 0] = (11.3 * np.linspace(0.1, 4, 900)).astype(np.float16)  # later keys score higher
    _tree_case(5, 1, 4, 1, 128, 3, 3, 900, [900], 4, cache=cache, dst="bfloat16")


def test_tree_small_values_behind_large_ones_of_no_weight():
    """The first 128 positions hold V 2^17 times larger than the rest, at weights
    around e^-15 of theirs: the sum is that of the small ones."""
    rng = np.random.default_rng(17)
    cache = R.random_cache(rng, 1, 1, 700, 128, 4, 4)
    cache[1][0, 0, :, 0], cache[1][0, 0, :128, 0] = 60.0, 0.5
    cache[3][0, 0, :, 0], cache[3][0, 0, :128, 0] = 0.015, 2000.0
    _tree_case(6, 1, 4, 1, 128, 4, 4, 700, [700], 4, cache=cache, dst="bfloat16")


@pytest.mark.parametrize("bad", [np.inf, np.nan])
def test_tree_hidden_values_do_not_reach_a_row(bad):
    torch = torch_mod()
    rng = np.random.default_rng(11)
    n, L = 6, 300
    cache = R.random_cache(rng, 1, 1, 400, 128, 3, 3)
    clean = [x.copy() for x in cache]
    for norms in (cache[1], cache[3]):
        norms[0, 0, L - n + 2] = bad  # node 2
        norms[0, 0, L:] = bad         # behind the sequence
    masks = np.array([[1, 3, 7, 9, 19, 33]], dtype=np.int64)  # only row 2 sees node 2
    desc = tq.kv_desc(1, 1, 128, 400, 3, 3)
    q = torch.randn(1, n, 2, 128, device="cuda", dtype=torch.float16)
    outs = []
    for c in (cache, clean):
        out = torch.zeros_like(q)
        tq.decode_attention_tree(_dev_cache(c, desc), tq.make_codebook(3), tq.make_codebook(3), q,
                                 to_dev(np.array([L], dtype=np.int32)), to_dev(masks), 0.0884, out,
                                 tq.alloc_tree_workspace(desc, 2, n))
        outs.append(out)
    torch.cuda.synchronize()
    others = [0, 1, 3, 4, 5]
    ref, spread, score = R.tree_attention(_np(q), clean, 3, 3, [L], [n], masks, 0.0884)
    got = _np(outs[0])[:, others]
    R.check_tree(got, ref[:, others], spread[:, others], score[:, others], 2.0 ** -10)
    assert torch.isnan(outs[0][0, 2]).any()


def test_tree_bad_query_rows_stay_alone():
    torch = torch_mod()
    rng = np.random.default_rng(12)
    cache = R.random_cache(rng, 1, 1, 300, 128, 3, 3)
    q = rng.standard_normal((1, 5, 4, 128))
    ref, spread, score = R.tree_attention(q.astype(np.float16).astype(np.float64), cache, 3, 3, [300], [5],
                                          [tq.tree_masks([-1, 0, 0, 1, 1])[0]], 0.0884)
    q[0, 1, 2, 7], q[0, 3, 0, 0], q[0, 4, 1] = np.nan, np.inf, 0.0
    desc = tq.kv_desc(1, 1, 128, 300, 3, 3)
    qd = torch.from_numpy(q).to(torch.float16).cuda()
    out = torch.zeros_like(qd)
    tq.decode_attention_tree(_dev_cache(cache, desc), tq.make_codebook(3), tq.make_codebook(3), qd,
                             to_dev(np.array([300], dtype=np.int32)),
                             to_dev(tq.tree_masks([[-1, 0, 0, 1, 1]])[0]), 0.0884, out,
                             tq.alloc_tree_workspace(desc, 4, 5))
    got = _np(out)
    assert np.isnan(got[0, 1, 2]).all() and np.isnan(got[0, 3, 0]).all()
    assert np.isfinite(got[0, 4, 1]).all()  # a zero query: even weights
    for j, h in ((1, 2), (3, 0), (4, 1)):
        got[0, j, h] = ref[0, j, h] = np.nan
    live = ~np.isnan(ref)
    R.check_tree(np.where(live, got, 0.0), ref, spread, score, 2.0 ** -10)


def test_tree_many_uneven_sequences():
    rng = np.random.default_rng(13)
    lens = rng.integers(0, 400, 37)
    counts = np.minimum(rng.integers(0, 4, 37), lens)
    _tree_case(14, 37, 4, 2, 128, 2, 3, 400, lens, 3, counts=counts, sign_seed=77)


def test_tree_long_uneven_sequences_cut_between_units():
    # enough 128-position tiles (1856) for cuts that weigh the units' ends, an
    # empty sequence among them
    lens = [10000, 0, 9130, 3001, 7200]
    _tree_case(21, 5, 8, 8, 128, 3, 3, 10000, lens, 2, counts=[2, 0, 1, 2, 2])


def test_tree_lengths_out_of_range_are_clamped():
    torch = torch_mod()
    rng = np.random.default_rng(15)
    cache = R.random_cache(rng, 3, 1, 64, 128, 3, 3)
    desc = tq.kv_desc(3, 1, 128, 64, 3, 3)
    dc, cb = _dev_cache(cache, desc), tq.make_codebook(3)
    q = torch.randn(3, 2, 2, 128, device="cuda", dtype=torch.float16)
    masks = to_dev(np.array([[1, 3]] * 3, dtype=np.int64))
    res = []
    for lens, counts in (([-5, 1000, 20], [2, 2, 9]), ([0, 64, 20], [2, 2, 2])):
        out, st = torch.zeros_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
        tq.decode_attention_tree(dc, cb, cb, q, to_dev(np.array(lens, dtype=np.int32)), masks, 0.0884, out,
                                 tq.alloc_tree_workspace(desc, 2, 2), n_nodes=to_dev(np.array(counts, dtype=np.int32)),
                                 status=st)
        res.append((out, tq.read_device_status(st)))
    assert res[0][1] == tq.TQ_DEV_LEN_RANGE and res[1][1] == 0
    assert torch.equal(res[0][0], res[1][0]) and torch.all(res[1][0][0] == 0)


def test_tree_repeats_bit_for_bit_and_replays_in_a_graph():
    torch = torch_mod()
    rng = np.random.default_rng(16)
    cache = R.random_cache(rng, 3, 2, 3000, 128, 3, 3)
    desc = tq.kv_desc(3, 2, 128, 3000, 3, 3)
    dc, cb = _dev_cache(cache, desc), tq.make_codebook(3)
    q = torch.randn(3, 9, 8, 128, device="cuda", dtype=torch.bfloat16)
    lens = to_dev(np.array([3000, 2999, 1201], dtype=np.int32))
    masks = to_dev(np.stack([_random_tree(rng, 9) for _ in range(3)]))
    ws = tq.alloc_tree_workspace(desc, 8, 9)
    outs = [torch.zeros_like(q) for _ in range(4)]

    def call(o):
        tq.decode_attention_tree(dc, cb, cb, q, lens, masks, 0.0884, o, ws)
    call(outs[0])
    call(outs[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(side):
        for o in outs[2:]:  # two graphs share the workspace
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                call(o)
            graphs.append(g)
        for _ in range(3):
            for g in graphs:
                g.replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


def test_tree_calls_at_once_on_two_streams():
    torch = torch_mod()
    rng = np.random.default_rng(18)
    cache = R.random_cache(rng, 2, 2, 2000, 128, 3, 3)
    desc = tq.kv_desc(2, 2, 128, 2000, 3, 3)
    dc, cb = _dev_cache(cache, desc), tq.make_codebook(3)
    lens = to_dev(np.array([2000, 1777], dtype=np.int32))
    masks = to_dev(np.stack([_random_tree(rng, 5) for _ in range(2)]))
    qs = [torch.randn(2, 5, 8, 128, device="cuda", dtype=torch.float16) for _ in range(2)]
    wss = [tq.alloc_tree_workspace(desc, 8, 5) for _ in range(2)]
    want = []
    for q in qs:
        o = torch.zeros_like(q)
        tq.decode_attention_tree(dc, cb, cb, q, lens, masks, 0.0884, o, wss[0])
        want.append(o)
    outs = [torch.zeros_like(q) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for q, ws, o, s in zip(qs, wss, outs, streams):
            tq.decode_attention_tree(dc, cb, cb, q, lens, masks, 0.0884, o, ws, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


# --------------------------------------------------------------- cache rows --

def _full_cache(rng, batch, hk, cap, dim, kb, vb, outliers=0):
    torch = torch_mod()
    cache = R.random_cache(rng, batch, hk, cap, dim, kb, vb)
    dc = _dev_cache(cache, tq.kv_desc(batch, hk, dim, cap, kb, vb))
    vo = None
    if outliers:
        ch = torch.arange(outliers, dtype=torch.int32, device="cuda").repeat(hk, 1)
        vo = tq.alloc_outliers(dc.desc, ch)
        vo.values.copy_(torch.from_numpy(rng.integers(-30000, 30000, tuple(vo.values.shape)).astype(np.int16)))
    return dc, vo


def _arrays(dc, vo):
    return [x.cpu().numpy().copy() for x in (dc.k_codes, dc.k_norms, dc.v_codes, dc.v_norms)] + \
        ([vo.values.cpu().numpy().copy()] if vo is not None else [])


def _compact_case(seed, batch, hk, cap, dim, kb, vb, keep, n_keep, start, outliers=0):
    torch = torch_mod()
    dc, vo = _full_cache(np.random.default_rng(seed), batch, hk, cap, dim, kb, vb, outliers)
    before = _arrays(dc, vo)
    keep, n_keep = np.asarray(keep, dtype=np.int32), np.asarray(n_keep, dtype=np.int32)
    lens, st = (torch.full((n,), 0, dtype=torch.int32, device="cuda") for n in (batch, 1))
    tq.cache_compact(dc, to_dev(keep), to_dev(n_keep), None if start is None else to_dev(np.array(start, dtype=np.int32)),
                     lens, vo, status=st)
    torch.cuda.synchronize()
    bits = 0
    for got, old in zip(_arrays(dc, vo), before):
        want = old.copy()
        for b in range(batch):
            n, s0 = min(max(int(n_keep[b]), 0), keep.shape[1]), 0 if start is None else int(start[b])
            bits |= tq.TQ_DEV_LEN_RANGE if n != n_keep[b] else 0
            if s0 < 0:
                bits |= tq.TQ_DEV_POS_RANGE
                continue
            for i in range(n):
                if s0 + i <= keep[b, i] < cap:
                    want[b, :, s0 + i] = old[b, :, keep[b, i]]
                else:
                    bits |= tq.TQ_DEV_POS_RANGE
        assert np.array_equal(got, want)
    s0 = np.zeros(batch, dtype=np.int64) if start is None else np.asarray(start)
    assert np.array_equal(lens.cpu().numpy(), np.clip(s0 + np.clip(n_keep, 0, keep.shape[1]), 0, cap))
    assert tq.read_device_status(st) == bits


def _ascending(rng, batch, lo, hi, n):
    return np.stack([lo + np.sort(rng.permutation(hi - lo)[:n]) for _ in range(batch)])


@pytest.mark.parametrize("dim,kb,vb,outliers", [(128, 3, 3, 0), (128, 2, 4, 3), (256, 3, 2, 0), (256, 4, 4, 16),
                                                (384, 2, 3, 8), (512, 4, 4, 16)])
@pytest.mark.parametrize("n", [1, 5, 33, 300, 2500])
def test_compact_sizes(dim, kb, vb, outliers, n):
    rng = np.random.default_rng(n + dim)
    cap = 2 * n + 40
    keep = _ascending(rng, 2, 7, cap, n)
    _compact_case(n, 2, 2, cap, dim, kb, vb, keep, [n, n - n // 3], [7, 3], outliers)


def test_compact_identity_repeats_and_all_rows():
    n = 1500
    _compact_case(1, 1, 1, n, 128, 3, 3, [np.arange(n)], [n], None)
    _compact_case(2, 1, 1, n, 128, 3, 3, [np.full(n, n - 1)], [n], None)           # the same row everywhere
    _compact_case(3, 1, 2, n, 128, 3, 3, [np.arange(n)[::-1]], [n // 2], None)     # not ascending, still above
    _compact_case(4, 2, 1, 64, 128, 3, 3, [[5, 6], [9, 9]], [0, 2], [2, 8])


def test_compact_skips_and_reports_what_it_cannot_do():
    keep = [[3, 1, 40, -2, 63, 64], [10, 11, 12, 13, 14, 15], [0, 1, 2, 3, 4, 5]]
    _compact_case(5, 3, 2, 64, 128, 3, 2, keep, [6, 9, -1], [1, 10, 0])
    _compact_case(6, 3, 2, 64, 128, 3, 2, keep, [6, 6, 6], [-1, 2 ** 31 - 1, 63])


@pytest.mark.parametrize("dim,kb,vb,outliers", [(128, 3, 3, 0), (128, 4, 2, 5), (256, 2, 3, 16), (512, 4, 4, 0)])
@pytest.mark.parametrize("rows", [1, 3, 130, 1777])
def test_copy_sizes(dim, kb, vb, outliers, rows):
    rng = np.random.default_rng(rows + dim)
    src, svo = _full_cache(rng, 3, 2, rows + 9, dim, kb, vb, outliers)
    dst, dvo = _full_cache(rng, 5, 2, rows + 31, dim, kb, vb, outliers)
    # a fork to three slots, one ragged copy at odd positions, one empty
    _copy_case(src, svo, dst, dvo, [1, 1, 1, 2, 0], [0, 4, 2, 3, 1], [0, 0, 0, 5, 0], [1, 1, 1, 30, 0],
               [rows, rows, rows // 2, rows, 0], rows)


def _copy_case(src, svo, dst, dvo, ss, ds, sp, dp, n, max_rows):
    torch = torch_mod()
    a, b = _arrays(src, svo), _arrays(dst, dvo)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda x: None if x is None else to_dev(np.asarray(x, dtype=np.int32))  # noqa: E731
    tq.cache_copy(src, dst, i32(ss), i32(ds), i32(n), max_rows, i32(sp), i32(dp), svo, dvo, status=st)
    torch.cuda.synchronize()
    want, bits = [x.copy() for x in b], 0
    caps, caps_d = src.desc.seq_cap, dst.desc.seq_cap
    for c in range(len(ss)):
        p, d = 0 if sp is None else sp[c], 0 if dp is None else dp[c]
        m = min(max(n[c], 0), max_rows)
        bits |= tq.TQ_DEV_LEN_RANGE if m != n[c] else 0
        if not (0 <= ss[c] < src.desc.batch and 0 <= ds[c] < dst.desc.batch and p >= 0 and d >= 0):
            bits |= tq.TQ_DEV_POS_RANGE
            continue
        room = max(0, min(caps - p, caps_d - d))
        if m > room:
            bits |= tq.TQ_DEV_POS_RANGE
            m = room
        for w, x in zip(want, a):
            w[ds[c], :, d:d + m] = x[ss[c], :, p:p + m]
    for got, w in zip(_arrays(dst, dvo), want):
        assert np.array_equal(got, w)
    assert tq.read_device_status(st) == bits


def test_copy_inside_one_cache_and_out_of_range():
    rng = np.random.default_rng(8)
    c, _ = _full_cache(rng, 6, 2, 100, 128, 3, 3)
    _copy_case(c, None, c, None, [0, 0, 1], [2, 3, 4], None, None, [100, 77, 100], 100)
    _copy_case(c, None, c, None, [0, 9, 1, 1], [2, 3, -1, 4], [90, 0, 0, -1], None, [50, 5, 5, 5], 60)
    _copy_case(c, None, c, None, [0, 1, 1], [3, 4, 5], [0, 3, 100], [95, 120, 0], [70, -4, 3], 60)


def test_copied_rows_attend_like_their_source():
    torch = torch_mod()
    c, _ = _full_cache(np.random.default_rng(9), 4, 2, 600, 128, 3, 3)
    i32 = lambda *x: to_dev(np.array(x, dtype=np.int32))  # noqa: E731
    tq.cache_copy(c, c, i32(0, 0, 0), i32(1, 2, 3), i32(555, 555, 555), 555)
    q = torch.randn(1, 8, 128, device="cuda", dtype=torch.float16).repeat(4, 1, 1)
    out, ws = torch.zeros(4, 8, 128, device="cuda"), tq.alloc_workspace(c.desc, 8)
    cb = tq.make_codebook(3)
    tq.decode_attention(c, cb, cb, q, i32(555, 555, 555, 555), 0.0884, out, ws)
    # a sequence's split over the CTAs may differ from its neighbour's: fp32
    # partials of 555 positions, and the fp16 weights' reference maximum
    assert torch.allclose(out, out[:1].expand_as(out), rtol=0, atol=2e-3 * out.abs().max().item())


# ----------------------------------------------------------------- together --

def test_a_speculative_round():
    """Prompt, fork, draft a tree, verify, compact, go on: the cache after the
    round is the one that the accepted tokens alone would have left, and
    attention over it agrees with the reference."""
    torch = torch_mod()
    torch.manual_seed(0)
    B, hq, hk, D, cap, prompt, n = 3, 8, 2, 128, 256, 100, 6
    desc = tq.kv_desc(B, hk, D, cap, 3, 3)
    cache, plain = tq.alloc_cache(desc), tq.alloc_cache(desc)
    cb = tq.make_codebook(3)
    rope = tq.make_rope(D, scaling="yarn", factor=4.0)
    qw, kw = (1 + 0.1 * torch.randn(D, device="cuda") for _ in range(2))

    def rows(qkv, pos):
        t = qkv.shape[1]
        q, k, v = (x.unflatten(2, (-1, D)) for x in qkv.split([hq * D, hk * D, hk * D], 2))
        o = [torch.empty(s, dtype=torch.float16, device="cuda")
             for s in ((qkv.shape[0], t, hq, D), (qkv.shape[0], hk, t, D), (qkv.shape[0], hk, t, D))]
        tq.qk_norm_rope(rope, q, k, v, pos, *o, q_weight=qw, k_weight=kw)
        return o
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    width = (hq + 2 * hk) * D
    # one prompt, encoded into slot 0, forked to the others
    _, k, v = rows(torch.randn(1, prompt, width, device="cuda"), i32(np.arange(prompt)[None]))
    for c in (cache, plain):
        one = tq.Cache(tq.kv_desc(1, hk, D, cap, 3, 3), *(x[:1] for x in (c.k_codes, c.k_norms, c.v_codes, c.v_norms)))
        tq.encode_kv(one, cb, cb, k, v)
        tq.cache_copy(c, c, i32([0] * 2), i32([1, 2]), i32([prompt] * 2), prompt)
    # the drafted tree of each sequence
    masks, depths = tq.tree_masks([[-1, 0, 0, 1, 2, 2], [-1, 0, 1, 2, 3, 4], [-1, -1, 0, 1, 3, 0]])
    draft = torch.randn(B, n, width, device="cuda")
    q, k, v = rows(draft, i32(prompt + depths))
    tq.encode_kv(cache, cb, cb, k, v, start_pos=i32([prompt] * B))
    lens = i32([prompt + n] * B)
    out = torch.zeros_like(q)
    ws = tq.alloc_tree_workspace(desc, hq, n)
    tq.decode_attention_tree(cache, cb, cb, q, lens, to_dev(masks), D ** -0.5, out, ws)
    host = [cache.k_codes.cpu().numpy(), cache.k_norms.cpu().numpy().view(np.float16), cache.v_codes.cpu().numpy(),
            cache.v_norms.cpu().numpy().view(np.float16)]
    ref, spread, score = R.tree_attention(_np(q), host, 3, 3, [prompt + n] * B, [n] * B, masks, D ** -0.5)
    R.check_tree(_np(out), ref, spread, score, 2.0 ** -10)
    # accept a path in each, move it to the front, and compare with its tokens encoded in order
    paths = [[0, 2, 5], [0, 1, 2, 3, 4, 5], [1]]
    keep = np.zeros((B, n), dtype=np.int32)
    for b, path in enumerate(paths):
        keep[b, :len(path)] = prompt + np.array(path)
    tq.cache_compact(cache, to_dev(keep), i32([len(p) for p in paths]), i32([prompt] * B), new_lens=lens)
    assert lens.tolist() == [prompt + len(p) for p in paths]
    for b, path in enumerate(paths):
        one = tq.Cache(tq.kv_desc(1, hk, D, cap, 3, 3), *(x[b:b + 1] for x in (plain.k_codes, plain.k_norms, plain.v_codes, plain.v_norms)))
        tq.encode_kv(one, cb, cb, k[b:b + 1, :, path].contiguous(), v[b:b + 1, :, path].contiguous(),
                     start_pos=i32([prompt]))
    for x, y in ((cache.k_codes, plain.k_codes), (cache.k_norms, plain.k_norms), (cache.v_codes, plain.v_codes),
                 (cache.v_norms, plain.v_norms)):
        for b, path in enumerate(paths):
            assert torch.equal(x[b, :, :prompt + len(path)], y[b, :, :prompt + len(path)])
    # the next token of every sequence
    q1 = torch.randn(B, hq, D, device="cuda", dtype=torch.float16)
    got, dws = torch.zeros(B, hq, D, device="cuda"), tq.alloc_workspace(desc, hq)
    tq.decode_attention(cache, cb, cb, q1, lens, D ** -0.5, got, dws)
    want = torch.zeros_like(got)
    tq.decode_attention(plain, cb, cb, q1, lens, D ** -0.5, want, dws)
    assert torch.equal(got, want)


def test_calls_follow_a_side_stream():
    torch = torch_mod()
    c, _ = _full_cache(np.random.default_rng(20), 2, 1, 64, 128, 3, 3)
    s = torch.cuda.Stream()
    i32 = lambda *x: to_dev(np.array(x, dtype=np.int32))  # noqa: E731
    a, b, n = i32(0), i32(1), i32(64)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        c.k_codes[0].fill_(1)
        torch.cuda._sleep(2_000_000)
        c.k_codes[0].fill_(9)
        tq.cache_copy(c, c, a, b, n, 64)
    s.synchronize()
    assert torch.all(c.k_codes[1] == 9)
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        c.k_codes[0].fill_(4)
    tq.cache_copy(c, c, a, b, n, 64, stream=s)
    s.synchronize()
    assert torch.all(c.k_codes[1] == 4)


def test_rope_of_no_tokens():
    torch = torch_mod()
    q, k = (torch.empty(2, 0, h, 128, device="cuda", dtype=torch.float16) for h in (4, 2))
    tq.qk_norm_rope(tq.make_rope(64), q, k, k, torch.empty(2, 0, device="cuda", dtype=torch.int32), torch.empty_like(q),
                    k.transpose(1, 2).contiguous(), k.transpose(1, 2).contiguous())
