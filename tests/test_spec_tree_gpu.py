"""The tree kernel's pipeline over many tiles: several tiles in every CTA (stage
and phase reuse, rescaling, cuts inside units), and waits that run out."""
import os
import subprocess
import sys

import numpy as np
import pytest

import quantized_decode_attention_tq_b200 as tq

from . import _spec_ref as R
from ._parity import to_dev, torch_mod

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

def _tiles(lens, hq, hk, n_q, dim, columns):
    """128-position tiles of all units, `columns` rows at a time."""
    groups = -(-(hq // hk) * n_q // columns)
    return sum(-(-int(x) // 128) for x in lens) * hk * groups


def _sms():
    return torch_mod().cuda.get_device_properties(0).multi_processor_count


def _run(desc, cache, hq, n_q, lens, counts, masks, q, dst="float16", v_levels=1.0):
    """decode_attention_tree over numpy inputs, as fp64; rows that are left alone hold 3."""
    torch = torch_mod()
    kc, kn, vc, vn = cache
    dc = tq.Cache(desc, to_dev(kc), to_dev(kn.view(np.int16)), to_dev(vc), to_dev(vn.view(np.int16)))
    v_cb = tq.make_codebook(desc.v_bits)
    for i in range(1 << desc.v_bits):
        v_cb.centroids[i] *= v_levels
    qd = torch.from_numpy(q).to(torch.float16).cuda()
    out = torch.full(q.shape, 3.0, dtype=getattr(torch, dst), device="cuda")
    ws = tq.alloc_tree_workspace(desc, hq, n_q)
    ws.fill_(255)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tq.decode_attention_tree(dc, tq.make_codebook(desc.k_bits), v_cb, qd, to_dev(np.asarray(lens, dtype=np.int32)),
                             to_dev(masks), desc.head_dim ** -0.5, out, ws,
                             n_nodes=to_dev(np.asarray(counts, dtype=np.int32)), status=status)
    assert tq.read_device_status(status) == 0
    return out.double().cpu().numpy() / v_levels, qd.double().cpu().numpy()


def _trees(rng, batch, n):
    return np.stack([tq.tree_masks([-1] + [int(rng.integers(-1, j)) for j in range(1, n)])[0] for _ in range(batch)])


def test_mostly_empty_batches():
    """Two live sequences among 24 slots, with enough tiles for cuts that weigh the units' ends."""
    rng = np.random.default_rng(1)
    B, hk, hq, cap, n, live = 24, 16, 32, 7500, 3, {5: 7499, 17: 7400}
    small = R.random_cache(rng, 2, hk, cap, 128, 3, 3)
    cache = [np.zeros((B,) + x.shape[1:], x.dtype) for x in small]
    for x, y in zip(cache, small):
        x[list(live)] = y
    lens, counts = [live.get(b, 0) for b in range(B)], [n if b in live or b == 9 else 0 for b in range(B)]
    assert _tiles(lens, hq, hk, n, 128, 16) > 12 * _sms()
    masks, q = _trees(rng, B, n), rng.standard_normal((B, n, hq, 128))
    got, q = _run(tq.kv_desc(B, hk, 128, cap, 3, 3), cache, hq, n, lens, counts, masks, q)
    at = list(live)
    ref, spread, score = R.tree_attention_by_head(q[at], small, 3, 3, [lens[b] for b in at], [n] * 2, masks[at], 128 ** -0.5)
    R.check_tree(got[at], ref, spread, score, 2.0 ** -10)
    for b in range(B):
        if b not in live:
            assert np.all(got[b] == (0.0 if b == 9 else 3.0))  # slot 9 drafts over nothing: its rows see nothing


RUN_OUT = """
import numpy as np, torch
import quantized_decode_attention_tq_b200 as tq
from quantized_decode_attention_tq_b200._lib import TQ_DEV_INTERNAL
from tests import _spec_ref as R
dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
rng, n, states = np.random.default_rng(0), 6, set()
for hq, hk, dim in ((8, 4, 128), (32, 2, 256), (64, 4, 128)):
    kc, kn, vc, vn = R.random_cache(rng, 4, hk, 6000, dim, 3, 3)
    desc = tq.kv_desc(4, hk, dim, 6000, 3, 3)
    cache = tq.Cache(desc, dev(kc), dev(kn.view(np.int16)), dev(vc), dev(vn.view(np.int16)))
    cb = tq.make_codebook(3)
    q = torch.randn(4, n, hq, dim, device="cuda", dtype=torch.float16)
    masks = dev(np.stack([tq.tree_masks([-1, 0, 0, 1, 2, 4])[0]] * 4))
    lens = dev(np.array([6000, 5999, 130, 4000], dtype=np.int32))
    out, ws = torch.zeros_like(q), tq.alloc_tree_workspace(desc, hq, n)
    for _ in range(10):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        tq.decode_attention_tree(cache, cb, cb, q, lens, masks, dim ** -0.5, out, ws, status=status)
        states.add(tq.read_device_status(status))
    # the context is usable: a chain of nodes by the other kernel, against the reference's first row
    multi = torch.zeros(q.shape, device="cuda")
    tq.decode_attention_multi(cache, cb, cb, q, lens, dim ** -0.5, multi, tq.alloc_workspace(desc, hq * n))
    chain = np.stack([tq.tree_masks([-1, 0, 1, 2, 3, 4])[0]] * 4)
    ref, spread, score = R.tree_attention_by_head(q[:, :1].double().cpu().numpy(), (kc, kn, vc, vn), 3, 3,
                                                  (lens - n + 1).tolist(), [1] * 4, chain[:, :1], dim ** -0.5)
    R.check_tree(multi[:, :1].double().cpu().numpy(), ref, spread, score, 2.0 ** -23)
assert states <= {0, TQ_DEV_INTERNAL}, states
print("states", sorted(states))
"""


def test_waits_that_run_out_are_reported_and_leave_the_context_usable():
    """The first wait for a score product takes longer than one try: the kernel
    reports it, drains what it issued and returns."""
    for tries, want in (("1", "states [8]"), ("1000000", "states [0]")):
        r = subprocess.run([sys.executable, "-c", RUN_OUT], cwd=ROOT, env={**os.environ, "TQ_TREE_WAIT_TRIES": tries},
                           capture_output=True, text=True, timeout=300)
        assert r.returncode == 0 and want in r.stdout, (tries, r.stdout, r.stderr[-2000:])


def test_empty_slots_cost_little():
    """One live sequence among 64 slots against the same alone; rows of empty
    slots are zeros to write, 8 MB here.  Twice the time would show work for slots
    that hold nothing (it was 3.5 times when their rows were written one by one)."""
    torch = torch_mod()

    def best(slots):
        desc = tq.kv_desc(slots, 8, 128, 32768, 3, 3)
        cache, cb = tq.alloc_cache(desc), tq.make_codebook(3)
        q = torch.randn(slots, 16, 32, 128, device="cuda", dtype=torch.float16)
        lens = torch.zeros(slots, dtype=torch.int32, device="cuda")
        lens[-1] = 32768
        masks = torch.ones(slots, 16, dtype=torch.int64, device="cuda")
        out, ws = torch.full_like(q, 3.0), tq.alloc_tree_workspace(desc, 32, 16)
        times = []
        for _ in range(8):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda._sleep(1_000_000)
            a.record()
            for _ in range(10):
                tq.decode_attention_tree(cache, cb, cb, q, lens, masks, 0.0884, out, ws)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        assert torch.all(out[:-1] == 0)
        return min(times[2:])
    assert best(64) <= 2 * best(1)


@pytest.mark.parametrize("hq,dim", [(8, 128), (64, 128), (8, 256)])
def test_small_v_norms_behind_zeros(hq, dim):
    """The first 128 positions have V norms of zero and most of the weight, the
    others 1 to 3 times the smallest norm that fp16 holds: they keep their
    precision wherever a CTA's part starts.  Outputs are compared 2^24 times as large, so that the bound's
    absolute term does not hide them."""
    rng = np.random.default_rng(hq + dim)
    B, hk, cap, n = 16, 8, 2048, 2
    cache = R.random_cache(rng, B, hk, cap, dim, 3, 3)
    cache[3][:] = (rng.integers(1, 4, cache[3].shape) * 2.0 ** -24).astype(np.float16)
    cache[3][:, :, :128] = 0
    cache[1][:, :, :128] *= 3
    cache[2][:] = cache[2][:, :, :1]  # V of one direction: nothing cancels
    lens = [cap] * B
    assert _tiles(lens, hq, hk, n, dim, 16) > 12 * _sms()
    masks, q = _trees(rng, B, n), rng.standard_normal((B, n, hq, dim))
    got, q = _run(tq.kv_desc(B, hk, dim, cap, 3, 3), cache, hq, n, lens, [n] * B, masks, q, dst="bfloat16")
    ref, spread, score = R.tree_attention_by_head(q, cache, 3, 3, lens, [n] * B, masks, dim ** -0.5)
    R.check_tree(got * 2.0 ** 24, ref * 2.0 ** 24, spread * 2.0 ** 24, score, 2.0 ** -7)


# rows of a kv-head: the columns of their row group (16 to 128, or 64 for heads of 256) and 104 to 200 rows in two
ROWS = [(128, 1, 9, 16), (128, 4, 7, 32), (128, 8, 7, 64), (128, 8, 13, 128), (128, 8, 25, 128),
        (256, 1, 9, 16), (256, 4, 7, 32), (256, 8, 7, 64), (256, 4, 25, 64)]


@pytest.mark.parametrize("norms", ["even", "growing", "falling", "mixed"])
@pytest.mark.parametrize("dim,group,n,columns", ROWS)
def test_parts_of_many_tiles(dim, group, n, columns, norms):
    """More than four tiles in every CTA, sequences of uneven lengths and trees.
    Growing K norms let late scores exceed early ones by far more than 2^6, so the
    references move and the sums are rescaled inside a part; growing V norms move
    their scale; falling ones leave both; mixed ones change from tile to tile."""
    rng = np.random.default_rng(dim + 8 * n + group)
    hk = 4
    units = 4 * hk * (2 if group * n > columns else 1)  # of four sequences
    B, cap = 4, 2 * (4 * _sms() * 128 // units // 2) + 600
    lens = [cap, cap - 129, cap - 511, cap - 300]
    counts = [n, n - 1, max(1, n // 2), n]
    kb, vb = {"even": (3, 3), "growing": (4, 2), "falling": (2, 4), "mixed": (3, 2)}[norms]
    cache = R.random_cache(rng, B, hk, cap, dim, kb, vb)
    ramp = np.linspace(0, 1, cap)[None, None, :, None]
    if norms == "mixed":
        ramp = np.repeat(rng.random((B, hk, -(-cap // 128), 1)), 128, axis=2)[:, :, :cap]
    if norms != "even":
        t = 1 - ramp if norms == "falling" else ramp
        cache[1] = (cache[1].astype(np.float64) * (0.1 + 3.9 * t)).astype(np.float16)
        cache[3] = (cache[3].astype(np.float64) * 10 ** (-4 + 7 * t)).astype(np.float16)
    hq = group * hk
    assert _tiles(lens, hq, hk, n, dim, columns) > 4 * _sms()
    masks, q = _trees(rng, B, n), rng.standard_normal((B, n, hq, dim))
    got, q = _run(tq.kv_desc(B, hk, dim, cap, kb, vb), cache, hq, n, lens, counts, masks, q, dst="bfloat16")
    ref, spread, score = R.tree_attention_by_head(q, cache, kb, vb, lens, counts, masks, dim ** -0.5)
    assert np.all(got[np.isnan(ref)] == 3.0)
    R.check_tree(got, ref, spread, score, 2.0 ** -7)


@pytest.mark.parametrize("v_levels", [1.0, 1.25])
@pytest.mark.parametrize("bits", [2, 3, 4])
@pytest.mark.parametrize("dim,group,n,columns", [(128, 8, 13, 128), (256, 8, 13, 64)])
def test_parts_of_many_tiles_with_the_fullest_shared_memory(dim, group, n, columns, bits, v_levels):
    """104 rows, K and V of one width: one code table for both or two (the V sum is
    linear in its levels), fewer stages and slots the fuller the memory."""
    rng = np.random.default_rng(dim + bits)
    B, hk, cap = 2, 4, 2 * (4 * _sms() * 128 // 16) + 400
    lens = [cap, cap - 200]
    cache = R.random_cache(rng, B, hk, cap, dim, bits, bits)
    hq = group * hk
    assert _tiles(lens, hq, hk, n, dim, 128) > 2 * _sms()
    masks, q = _trees(rng, B, n), rng.standard_normal((B, n, hq, dim))
    got, q = _run(tq.kv_desc(B, hk, dim, cap, bits, bits), cache, hq, n, lens, [n] * B, masks, q, v_levels=v_levels)
    ref, spread, score = R.tree_attention_by_head(q, cache, bits, bits, lens, [n] * B, masks, dim ** -0.5)
    R.check_tree(got, ref, spread, score, 2.0 ** -10)


def test_a_captured_call_follows_slots_that_come_and_go():
    """One graph, replayed with other lengths and node counts in the same tensors:
    all slots empty, one live, short ones, long ones (cuts with and without ends)."""
    torch = torch_mod()
    rng = np.random.default_rng(3)
    B, hk, hq, cap, n = 24, 8, 16, 4000, 3
    cache = R.random_cache(rng, B, hk, cap, 128, 2, 3)
    desc = tq.kv_desc(B, hk, 128, cap, 2, 3)
    dc = tq.Cache(desc, *(to_dev(x if x.dtype == np.uint8 else x.view(np.int16)) for x in cache))
    k_cb, v_cb = tq.make_codebook(2), tq.make_codebook(3)
    q = torch.randn(B, n, hq, 128, device="cuda", dtype=torch.float16)
    masks = to_dev(_trees(rng, B, n))
    lens, counts = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    out, eager, ws = torch.zeros_like(q), torch.zeros_like(q), tq.alloc_tree_workspace(desc, hq, n)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(o):
        tq.decode_attention_tree(dc, k_cb, v_cb, q, lens, masks, 0.0884, o, ws, n_nodes=counts, status=status)
    call(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    long = rng.integers(3000, cap + 1, B)
    for live in (np.zeros(B, dtype=int), np.where(np.arange(B) == 13, cap, 0), rng.integers(0, 300, B),
                 long * (rng.random(B) < 0.5), long, np.zeros(B, dtype=int)):
        lens.copy_(torch.from_numpy(live))
        counts.copy_(torch.from_numpy(rng.integers(0, n + 1, B)))
        out.fill_(3.0), eager.fill_(3.0)
        graph.replay()
        call(eager)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
        nodes = counts.tolist()
        ref, spread, score = R.tree_attention_by_head(q.double().cpu().numpy(), cache, 2, 3, live, nodes,
                                                      masks.cpu().numpy(), 0.0884)
        got = out.double().cpu().numpy()
        assert np.all(got[np.isnan(ref)] == 3.0)
        R.check_tree(got, ref, spread, score, 2.0 ** -10)
    assert tq.read_device_status(status) == 0
