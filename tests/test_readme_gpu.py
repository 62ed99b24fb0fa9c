"""The README's Python example runs as it stands there."""
import os
import re

import numpy as np
import pytest

import quantized_decode_attention_tq_b200 as tq

from . import _spec_ref as R
from ._parity import torch_mod

pytestmark = pytest.mark.gpu


def test_the_speculative_round_of_the_readme():
    torch = torch_mod()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
    blocks = re.findall(r"```python\n(.*?)```", open(path).read(), flags=re.S)
    assert len(blocks) == 1
    B, hq, hk, D, cap, n, context = 2, 8, 2, 128, 256, 5, [100, 64]
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    rnd = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    desc = tq.kv_desc(B, hk, D, cap, 3, 3)
    cache, cb = tq.alloc_cache(desc), tq.make_codebook(3)
    tq.encode_kv(cache, cb, cb, rnd(B, hk, 120, D), rnd(B, hk, 120, D))
    half = lambda *s: torch.empty(s, dtype=torch.float16, device="cuda")  # noqa: E731
    names = dict(tq=tq, torch=torch, parents=[[-1, 0, 0, 1, 2], [-1, -1, 0, 1, 3]], ctx=i32(context), n=n, cache=cache,
                 k_cb=cb, v_cb=cb, q=rnd(B, n, hq, D), k=rnd(B, n, hk, D), v=rnd(B, n, hk, D), wq=rnd(D), wk=rnd(D),
                 q_rows=half(B, n, hq, D), k_rows=half(B, hk, n, D), v_rows=half(B, hk, n, D), out=half(B, n, hq, D),
                 scale=D ** -0.5, workspace=tq.alloc_tree_workspace(desc, hq, n), lens=i32([0, 0]),
                 accepted=i32([[100, 102, 104], [65, 67, 0]]), n_accepted=i32([3, 2]))
    before, _, after = blocks[0].partition("tq.cache_compact(")
    exec(before, names)
    host = [x.cpu().numpy() for x in (cache.k_codes, cache.k_norms, cache.v_codes, cache.v_norms)]
    host[1], host[3] = host[1].view(np.float16), host[3].view(np.float16)
    masks = tq.tree_masks(names["parents"])[0]
    ref, spread, score = R.tree_attention(names["q_rows"].double().cpu().numpy(), host, 3, 3, [c + n for c in context],
                                          [n] * B, masks, D ** -0.5)
    R.check_tree(names["out"].double().cpu().numpy(), ref, spread, score, 2.0 ** -10)
    exec("tq.cache_compact(" + after, names)
    assert names["lens"].tolist() == [103, 66]
    assert np.array_equal(cache.k_codes[0, :, 101].cpu().numpy(), host[0][0, :, 102])
