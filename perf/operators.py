"""Cases for the operators of a speculative-decoding round over the packed KV cache.

Four operators: `rope` (per-head RMS norm of q and k, position rotation and the
split into the layouts the cache takes, in one pass), `tree` (attention of a tree
of drafted tokens over the packed cache), `compact` (keeping a chosen set of rows
of every sequence, in place) and `copy` (copying row ranges between the slots of
a cache, for example to fork a prompt).

With `own` false, `run` computes them in elementary torch operations; with `own`
true it calls the package.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"float16": torch.float16, "bfloat16": torch.bfloat16, "float32": torch.float32}
BLOCK = 128


# ------------------------------------------------------------------ the cases --

def listed():
    return [
        # one decode step of a batch: 8 tokens, latency
        {"name": "rope step", "op": "rope", "batch": 8, "tokens": 1, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "layout": "half", "scaling": "none", "factor": 1.0, "norm": True, "start": 32767,
         "ragged": False, "src": "bfloat16", "dst": "float16"},
        # prompts of a batch, positions scaled for a long context
        {"name": "rope prompts", "op": "rope", "batch": 8, "tokens": 4096, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "layout": "half", "scaling": "yarn", "factor": 16.0, "norm": True, "start": 61440,
         "ragged": False, "src": "bfloat16", "dst": "float16"},
        # a padded batch of uneven chunks, part of each wide head rotated, neighbouring pairs
        {"name": "rope partial ragged", "op": "rope", "batch": 4, "tokens": 1001, "q_heads": 16, "kv_heads": 4,
         "dim": 256, "rot": 96, "layout": "interleaved", "scaling": "linear", "factor": 4.0, "norm": False,
         "start": 500000, "ragged": True, "src": "float32", "dst": "float32"},
        # a small tree over a short chat: latency
        {"name": "tree short", "op": "tree", "batch": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "k_bits": 3,
         "v_bits": 3, "cap": 1024, "len": 777, "nodes": 8, "ragged": False, "dtype": "bfloat16"},
        # the serving batch at full length, a 16-node tree for each sequence
        {"name": "tree batch 16", "op": "tree", "batch": 8, "q_heads": 32, "kv_heads": 8, "dim": 128, "k_bits": 3,
         "v_bits": 3, "cap": 32768, "len": 32768, "nodes": 16, "ragged": False, "dtype": "float16"},
        # one long context, the widest tree
        {"name": "tree long 64", "op": "tree", "batch": 1, "q_heads": 32, "kv_heads": 8, "dim": 128, "k_bits": 4,
         "v_bits": 2, "cap": 131072, "len": 131072, "nodes": 64, "ragged": False, "dtype": "bfloat16"},
        # uneven sequences and uneven trees, heads of two blocks
        {"name": "tree ragged wide heads", "op": "tree", "batch": 4, "q_heads": 16, "kv_heads": 4, "dim": 256,
         "k_bits": 3, "v_bits": 2, "cap": 65536, "len": 65011, "nodes": 25, "ragged": True, "dtype": "bfloat16"},
        # after a tree is verified: the accepted path moves to the front of the drafted rows, latency
        {"name": "compact accepted path", "op": "compact", "batch": 8, "kv_heads": 8, "dim": 128, "k_bits": 3,
         "v_bits": 3, "cap": 32768, "first": 32000, "span": 64, "keep": 9},
        # a long context thinned to half its rows
        {"name": "compact half of the rows", "op": "compact", "batch": 8, "kv_heads": 8, "dim": 128, "k_bits": 3,
         "v_bits": 3, "cap": 32768, "first": 16, "span": 32740, "keep": 16370},
        # a short prompt forked for two more samples, latency
        {"name": "copy short fork", "op": "copy", "batch": 4, "kv_heads": 8, "dim": 128, "k_bits": 4, "v_bits": 4,
         "cap": 2048, "copies": 2, "rows": 301, "fork": True},
        # a long prompt forked to the rest of the batch
        {"name": "copy long fork", "op": "copy", "batch": 8, "kv_heads": 8, "dim": 128, "k_bits": 3, "v_bits": 3,
         "cap": 32768, "copies": 7, "rows": 32768, "fork": True},
        # uneven row ranges between slots, at odd positions (a prefix put behind another)
        {"name": "copy ranges", "op": "copy", "batch": 8, "kv_heads": 4, "dim": 256, "k_bits": 3, "v_bits": 2,
         "cap": 16384, "copies": 4, "rows": 8001, "fork": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "tree", "tree", "compact", "copy"])
    dim = rng.choice([128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    if op == "rope":
        group = rng.choice([1, 4, 4, 8])
        width = (group + 2) * kv * dim
        total = _log(rng, 1, (1 << 27) // width)
        batch = min(total, rng.randint(1, 8))
        return {"op": op, "batch": batch, "tokens": max(1, total // batch), "q_heads": kv * group, "kv_heads": kv,
                "dim": dim, "rot": rng.choice([dim, dim, dim // 2, 2 * rng.randint(2, dim // 2)]),
                "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "ntk", "yarn"]), "factor": rng.choice([2.0, 4.0, 32.0]),
                "norm": rng.random() < 0.6, "start": _log(rng, 1, 1000000), "ragged": rng.random() < 0.3,
                "src": rng.choice(["float16", "bfloat16", "bfloat16", "float32"]),
                "dst": rng.choice(["float16", "float16", "bfloat16", "float32"])}
    k_bits, v_bits = rng.choice([2, 3, 3, 4]), rng.choice([2, 3, 3, 4])
    if op == "tree":
        group, nodes = rng.choice([1, 4, 4, 8]), _log(rng, 1, 64)
        # scores of one case stay below those of the largest listed one
        room = (1 << 28) // (kv * group * nodes * dim // 128)
        length = _log(rng, nodes + 1, max(nodes + 2, min(131072, room)))
        batch = max(1, min(rng.randint(1, 8), room // length))
        cap = length + rng.choice([0, 1, 77])
        return {"op": op, "batch": batch, "q_heads": kv * group, "kv_heads": kv, "dim": dim, "k_bits": k_bits,
                "v_bits": v_bits, "cap": cap + cap % 2, "len": length, "nodes": nodes,
                "ragged": rng.random() < 0.5, "dtype": rng.choice(["float16", "bfloat16", "bfloat16"])}
    batch = rng.randint(2, 8)
    rows = _log(rng, 4, 32768 * 1024 // (kv * batch * dim))
    if op == "compact":
        first = rng.choice([0, 4, 1001])
        cap = first + rows + rng.choice([0, 5])
        return {"op": op, "batch": batch, "kv_heads": kv, "dim": dim, "k_bits": k_bits, "v_bits": v_bits,
                "cap": cap + cap % 2, "first": first, "span": rows, "keep": rng.randint(1, rows)}
    cap = rows + rng.choice([0, 6, 64])
    return {"op": op, "batch": batch, "kv_heads": kv, "dim": dim, "k_bits": k_bits, "v_bits": v_bits,
            "cap": cap + cap % 2, "copies": rng.randint(1, batch // 2), "rows": rows, "fork": rng.random() < 0.5}


# ----------------------------------------------- codebook, signs, rotation --

_centroids = {}


def centroids(bits):
    """Lloyd-Max levels of the standard normal density, ascending."""
    if bits not in _centroids:
        half = 1 << (bits - 1)
        c = [(k + 0.5) * 2.0 / half for k in range(half)]
        pdf = lambda x: math.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)  # noqa: E731
        for _ in range(200000):
            edge = [0.0] + [(a + b) / 2 for a, b in zip(c, c[1:])]
            new = []
            for k in range(half):
                tail = edge[k + 1] if k + 1 < half else None
                mass = 0.5 * (math.erfc(edge[k] / math.sqrt(2)) - (math.erfc(tail / math.sqrt(2)) if tail else 0.0))
                new.append((pdf(edge[k]) - (pdf(tail) if tail else 0.0)) / mass)
            moved = max(abs(a - b) for a, b in zip(c, new))
            c = new
            if moved < 1e-15:
                break
        _centroids[bits] = [-x for x in reversed(c)] + c
    return _centroids[bits]


def signs(seed=0):
    """The +-1 diagonal: top bits of 128 SplitMix64 outputs."""
    out, state, m = [], seed, (1 << 64) - 1
    for _ in range(BLOCK):
        state = (state + 0x9E3779B97F4A7C15) & m
        z = state
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & m
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & m
        out.append(-1.0 if (z ^ (z >> 31)) >> 63 else 1.0)
    return out


def hadamard(dtype):
    """The 128 x 128 Sylvester matrix: the sign of entry (i, j) is the parity of i AND j."""
    i = torch.arange(BLOCK, device=DEV)
    x = i[:, None] & i[None, :]
    for s in (4, 2, 1):
        x = x ^ (x >> s)
    return (1 - 2 * (x & 1)).to(dtype)


def frequencies(rot, scaling, factor, base=10000.0, orig_ctx=4096):
    """Radians per position of each pair in 64 bits, and the factor on cos and sin."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":  # Peng et al. 2023: pairs of many turns in the original context keep f, of few get f / factor
        at = lambda turns: rot * math.log(orig_ctx / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0
    return f, 1.0


# ---------------------------------------------------------------- the inputs --

def make_cache(c, gen, n_batch):
    """A cache as the encoder leaves it: indices of N(0,1) coordinates, norms of 128 unit normals in fp16."""
    nb = c["dim"] // BLOCK
    base = (n_batch, c["kv_heads"], c["cap"], nb)
    made = {}
    for side, bits in (("k", c["k_bits"]), ("v", c["v_bits"])):
        level = centroids(bits)
        edge = torch.tensor([(a + b) / 2 for a, b in zip(level, level[1:])], device=DEV)
        codes = torch.empty(base + (16 * bits,), dtype=torch.uint8, device=DEV)
        for b in range(n_batch):
            u = torch.randn(base[1:] + (16, 8), device=DEV, generator=gen)
            idx = torch.bucketize(u, edge, out_int32=True)
            word = (idx << (bits * torch.arange(8, device=DEV, dtype=torch.int32))).sum(-1, dtype=torch.int32)
            byte = torch.stack([(word >> (8 * j)) & 255 for j in range(bits)], -1)  # 8 codes fill `bits` bytes
            codes[b] = byte.to(torch.uint8).reshape(base[1:] + (16 * bits,))
        norm = (11.3 + 0.7 * torch.randn(base, device=DEV, generator=gen)).abs()
        made[side + "_codes"], made[side + "_norms"] = codes, norm.to(torch.float16).view(torch.int16)
    return made


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rnd = lambda *s: torch.randn(s, device=DEV, generator=gen)  # noqa: E731
    ints = lambda hi, *s: torch.randint(0, max(1, hi), s, device=DEV, generator=gen)  # noqa: E731
    i32 = torch.int32
    s = {"case": c}
    if c["op"] == "rope":
        B, T, Hq, Hk, D = (c[k] for k in ("batch", "tokens", "q_heads", "kv_heads", "dim"))
        qkv = rnd(B, T, (Hq + 2 * Hk) * D).to(DT[c["src"]])  # one projection's output, q, k and v side by side
        s["q"], s["k"], s["v"] = (x.unflatten(2, (-1, D)) for x in qkv.split([Hq * D, Hk * D, Hk * D], 2))
        s["q_weight"], s["k_weight"] = ((1 + 0.1 * rnd(D)).to(DT[c["src"]]) if c["norm"] else None for _ in range(2))
        first = ints(c["start"] + 1, B, 1)
        s["positions"] = (first + torch.arange(T, device=DEV)).to(i32)
        s["n_tok"] = (1 + ints(T, B)).to(i32) if c["ragged"] else None
        s["q_out"] = torch.zeros(B, T, Hq, D, dtype=DT[c["dst"]], device=DEV)
        s["k_out"], s["v_out"] = (torch.zeros(B, Hk, T, D, dtype=DT[c["dst"]], device=DEV) for _ in range(2))
        if own:
            import quantized_decode_attention_tq_b200 as tq
            s["rope"] = tq.make_rope(c["rot"], scaling=c["scaling"], factor=c["factor"], orig_ctx=4096,
                                     interleaved=c["layout"] == "interleaved")
        return s
    s.update(make_cache(c, gen, c["batch"]))
    B, cap = c["batch"], c["cap"]
    if c["op"] == "tree":
        n = c["nodes"]
        parent = torch.where(torch.arange(n, device=DEV) > 0, (torch.rand(B, n, device=DEV, generator=gen)
                             * torch.arange(n, device=DEV)).long(), -1)  # node 0 is the root, parents come first
        seen = torch.eye(n, dtype=torch.bool, device=DEV).repeat(B, 1, 1)
        for j in range(1, n):
            seen[:, j] |= seen[torch.arange(B, device=DEV), parent[:, j]]
        bit = torch.ones((), dtype=torch.int64, device=DEV) << torch.arange(n, device=DEV)
        s["tree"] = (seen * bit).sum(-1)
        ragged = c["ragged"]
        s["n_nodes"] = (n - ints((n + 1) // 2, B)).to(i32) if ragged else None
        short = ints(max(1, (c["len"] - n) // 2), B) if ragged else 0
        s["seq_lens"] = (torch.full((B,), c["len"], device=DEV) - short).to(i32)
        s["q"] = rnd(B, n, c["q_heads"], c["dim"]).to(DT[c["dtype"]])
        s["scale"] = c["dim"] ** -0.5
        s["out"] = torch.zeros_like(s["q"])
    elif c["op"] == "compact":
        pick = torch.rand(B, c["span"], device=DEV, generator=gen).argsort(1)[:, : c["keep"]].sort(1).values
        s["keep"] = (c["first"] + pick).to(i32)
        s["n_keep"] = (c["keep"] - ints(max(1, c["keep"] // 4), B)).to(i32)
        s["start"] = torch.full((B,), c["first"], dtype=i32, device=DEV)
        s["new_lens"] = torch.zeros(B, dtype=i32, device=DEV)
    else:
        n, slot = c["copies"], torch.randperm(B, device=DEV, generator=gen)
        rows = torch.full((n,), c["rows"], device=DEV)
        s["dst_slot"] = slot[:n].to(i32)
        if c["fork"]:
            s["src_slot"] = slot[-1:].expand(n).to(i32)
            s["src_pos"], s["dst_pos"] = (torch.zeros(n, dtype=i32, device=DEV) for _ in range(2))
        else:
            s["src_slot"] = slot[-n:].to(i32)
            rows = rows - ints(c["rows"] // 2, n)
            s["src_pos"], s["dst_pos"] = (torch.minimum(ints(64, n), cap - rows).to(i32) for _ in range(2))
        s["n_rows"] = rows.to(i32)
        s["max_rows"] = c["rows"]
    if own:
        import quantized_decode_attention_tq_b200 as tq
        desc = tq.kv_desc(B, c["kv_heads"], c["dim"], cap, c["k_bits"], c["v_bits"])
        s["cache"] = tq.Cache(desc, s["k_codes"], s["k_norms"], s["v_codes"], s["v_norms"])
        if c["op"] == "tree":
            s["k_cb"], s["v_cb"] = tq.make_codebook(c["k_bits"]), tq.make_codebook(c["v_bits"])
            s["workspace"] = tq.alloc_tree_workspace(desc, c["q_heads"], c["nodes"])
    return s


# ------------------------------------------------------------------ one pass --

def norm_rows(x, weight, eps=1e-6):
    x = x.float()
    return x if weight is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight.float()


def rotate_rows(x, cos, sin, rot, layout):
    """Rotate the first `rot` entries of x [B, T, H, D] by the angles of [B, T, rot / 2]."""
    head, rest = x[..., :rot], x[..., rot:]
    pairs = head.unflatten(-1, (-1, 2)) if layout == "interleaved" else head.unflatten(-1, (2, -1)).transpose(-1, -2)
    a, b = pairs[..., 0], pairs[..., 1]
    cos, sin = cos[:, :, None], sin[:, :, None]
    out = torch.stack([a * cos - b * sin, b * cos + a * sin], -1)
    out = out.flatten(-2) if layout == "interleaved" else out.transpose(-1, -2).flatten(-2)
    return torch.cat([out, rest], -1)


def plain_rope(s):
    c = s["case"]
    f, gain = frequencies(c["rot"], c["scaling"], c["factor"])
    angle = s["positions"].double()[..., None] * f.to(DEV)  # far positions: angles in 64 bits
    cos, sin = (gain * angle.cos()).float(), (gain * angle.sin()).float()
    q = rotate_rows(norm_rows(s["q"], s["q_weight"]), cos, sin, c["rot"], c["layout"])
    k = rotate_rows(norm_rows(s["k"], s["k_weight"]), cos, sin, c["rot"], c["layout"])
    q, k, v = q.to(s["q_out"].dtype), k.to(s["k_out"].dtype), s["v"].to(s["v_out"].dtype)
    k, v = k.transpose(1, 2), v.transpose(1, 2)
    if s["n_tok"] is not None:  # tokens behind a row's count are left as they were
        live = torch.arange(c["tokens"], device=DEV)[None] < s["n_tok"][:, None]
        q = torch.where(live[:, :, None, None], q, s["q_out"])
        k, v = (torch.where(live[:, None, :, None], x, s[n]) for x, n in ((k, "k_out"), (v, "v_out")))
    s["q_out"].copy_(q), s["k_out"].copy_(k), s["v_out"].copy_(v)
    return s["q_out"], s["k_out"], s["v_out"]


def unpack(codes, bits):
    """Packed codes [..., 16 * bits] as indices [..., 128]."""
    byte = codes.unflatten(-1, (16, bits)).int()
    word = (byte << (8 * torch.arange(bits, device=DEV, dtype=torch.int32))).sum(-1, keepdim=True, dtype=torch.int32)
    return ((word >> (bits * torch.arange(8, device=DEV, dtype=torch.int32))) & ((1 << bits) - 1)).flatten(-2)


def levels(codes, norms, bits, rows):
    """Rotated-domain values of the first `rows` rows, [B, H, rows, nb, 128] in 32 bits."""
    table = torch.tensor(centroids(bits), dtype=torch.float32, device=DEV)
    return table[unpack(codes[:, :, :rows], bits)] * (norms[:, :, :rows].view(torch.float16).float() / BLOCK)[..., None]


def plain_tree(s):
    c = s["case"]
    B, n, Hq, Hk, D, S = c["batch"], c["nodes"], c["q_heads"], c["kv_heads"], c["dim"], c["len"]
    G = Hq // Hk
    had, sign = hadamard(torch.float32), torch.tensor(signs(), device=DEV)
    q = (s["q"].float().unflatten(-1, (-1, BLOCK)) * sign) @ had  # one block after another
    q = q.reshape(B, n, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, n * G, D)
    k = levels(s["k_codes"], s["k_norms"], c["k_bits"], S).flatten(-2)
    score = (q @ k.transpose(-1, -2)) * s["scale"]  # [B, Hk, n * G, S]
    del k
    count = torch.full((B,), n, device=DEV) if s["n_nodes"] is None else s["n_nodes"].long()
    context = s["seq_lens"].long() - count
    t = torch.arange(S, device=DEV)
    node = t[None] - context[:, None]  # [B, S]
    drafted = (node >= 0) & (t[None] < s["seq_lens"][:, None])
    bit = (s["tree"][:, :, None] >> node.clamp(0, 63)[:, None]) & 1  # [B, n, S]
    seen = (node < 0)[:, None] | (drafted[:, None] & (bit == 1))
    seen = seen[:, None, :, None].expand(B, 1, n, G, S).reshape(B, 1, n * G, S)
    score = torch.where(seen, score, torch.full((), -math.inf, device=DEV))
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    del score
    total = weight.sum(-1, keepdim=True)
    v = levels(s["v_codes"], s["v_norms"], c["v_bits"], S).flatten(-2)
    o = weight @ v / torch.where(total > 0, total, torch.ones_like(total))
    o = (o.unflatten(-1, (-1, BLOCK)) @ had * sign).reshape(B, Hk, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D)
    live = torch.arange(n, device=DEV)[None] < count[:, None]  # rows behind a tree's nodes are left as they were
    s["out"].copy_(torch.where(live[:, :, None, None], o.to(s["out"].dtype), s["out"]))
    return s["out"]


PARTS = ("k_codes", "k_norms", "v_codes", "v_norms")


def plain_compact(s):
    b, i = (torch.arange(s["keep"].shape[1], device=DEV)[None] < s["n_keep"][:, None]).nonzero(as_tuple=True)
    src, dst = s["keep"][b, i].long(), s["start"][b].long() + i
    for x in (s[p] for p in PARTS):
        x[b, :, dst] = x[b, :, src]
    s["new_lens"].copy_(s["start"] + s["n_keep"])
    return [s[p] for p in PARTS] + [s["new_lens"]]


def plain_copy(s):
    n, t = (torch.arange(s["max_rows"], device=DEV)[None] < s["n_rows"][:, None]).nonzero(as_tuple=True)
    src, dst = s["src_pos"][n].long() + t, s["dst_pos"][n].long() + t
    for x in (s[p] for p in PARTS):
        x[s["dst_slot"][n].long(), :, dst] = x[s["src_slot"][n].long(), :, src]
    return [s[p] for p in PARTS]


def run(s):
    op = s["case"]["op"]
    if own:
        import quantized_decode_attention_tq_b200 as tq
        if op == "rope":
            tq.qk_norm_rope(s["rope"], s["q"], s["k"], s["v"], s["positions"], s["q_out"], s["k_out"], s["v_out"],
                            norm=s["case"]["norm"], eps=1e-6, q_weight=s["q_weight"], k_weight=s["k_weight"],
                            n_tok=s["n_tok"])
            return s["q_out"], s["k_out"], s["v_out"]
        if op == "tree":
            return tq.decode_attention_tree(s["cache"], s["k_cb"], s["v_cb"], s["q"], s["seq_lens"], s["tree"],
                                            s["scale"], s["out"], s["workspace"], n_nodes=s["n_nodes"])
        if op == "compact":
            tq.cache_compact(s["cache"], s["keep"], s["n_keep"], start=s["start"], new_lens=s["new_lens"])
            return [s[p] for p in PARTS] + [s["new_lens"]]
        tq.cache_copy(s["cache"], s["cache"], s["src_slot"], s["dst_slot"], s["n_rows"], s["max_rows"],
                      src_pos=s["src_pos"], dst_pos=s["dst_pos"])
        return [s[p] for p in PARTS]
    return {"rope": plain_rope, "tree": plain_tree, "compact": plain_compact, "copy": plain_copy}[op](s)


# ------------------------------------------------------------ work and truth --

def work(case):
    c = case
    size = {"float16": 2, "bfloat16": 2, "float32": 4}
    if c["op"] == "rope":
        rows = c["batch"] * c["tokens"] * (c["q_heads"] + 2 * c["kv_heads"]) * (0.5 if c["ragged"] else 1.0)
        return {"bytes": rows * c["dim"] * (size[c["src"]] + size[c["dst"]]), "flops": 8 * rows * c["dim"]}
    row = c["kv_heads"] * (c["dim"] // BLOCK) * (16 * (c["k_bits"] + c["v_bits"]) + 4)  # one position's bytes
    if c["op"] == "tree":
        length = c["len"] - (0.25 * (c["len"] - c["nodes"]) if c["ragged"] else 0)
        nodes = c["nodes"] * (0.75 if c["ragged"] else 1.0)
        io = 2 * c["batch"] * nodes * c["q_heads"] * c["dim"] * size[c["dtype"]]
        return {"bytes": c["batch"] * length * row + io,
                "flops": 4.0 * c["batch"] * length * nodes * c["q_heads"] * c["dim"]}
    if c["op"] == "compact":
        return {"bytes": 2.0 * c["batch"] * (c["keep"] - c["keep"] // 8) * row, "flops": 0}
    moved = c["copies"] * c["rows"] * (1.0 if c["fork"] else 0.75)
    return {"bytes": (moved + (c["rows"] if c["fork"] else moved)) * row, "flops": 0}


def exact_rope(s):
    c = s["case"]
    B, T, D, rot = c["batch"], c["tokens"], c["dim"], c["rot"]
    f, gain = frequencies(rot, c["scaling"], c["factor"])
    turn = torch.polar(torch.full((B, T, 1, rot // 2), gain, dtype=torch.float64, device=DEV),
                       (s["positions"].to(torch.float64)[:, :, None] * f.to(DEV))[:, :, None])
    i = torch.arange(rot // 2, device=DEV)
    one, two = (2 * i, 2 * i + 1) if c["layout"] == "interleaved" else (i, i + rot // 2)
    out = []
    for name in ("q", "k", "v"):
        x = s[name].double()
        w = s.get(name + "_weight")
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
        y = x.clone()
        if name != "v":
            z = torch.complex(x[..., one], x[..., two]) * turn
            y[..., one], y[..., two] = z.real, z.imag
        live = torch.ones(B, T, device=DEV, dtype=torch.bool) if s["n_tok"] is None else \
            torch.arange(T, device=DEV) < s["n_tok"][:, None]
        y = y * live[:, :, None, None]
        out.append(y if name == "q" else y.transpose(1, 2))
    return tuple(out)


def exact_tree(s):
    """Attention on the cache turned back to K and V, one sequence and kv-head after another."""
    c = s["case"]
    G, n, D = c["q_heads"] // c["kv_heads"], c["nodes"], c["dim"]
    back = hadamard(torch.float64) * torch.tensor(signs(), dtype=torch.float64, device=DEV) / BLOCK
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b in range(c["batch"]):
        length = int(s["seq_lens"][b])
        count = n if s["n_nodes"] is None else int(s["n_nodes"][b])
        seen = torch.ones(count, length, dtype=torch.bool, device=DEV)
        word = s["tree"][b, :count]
        for i in range(count):
            seen[:, length - count + i] = (word >> i) % 2 == 1
        for h in range(c["kv_heads"]):
            kv = []
            for side in ("k", "v"):
                bits = c[side + "_bits"]
                table = torch.tensor(centroids(bits), dtype=torch.float64, device=DEV).float().double()
                byte = s[side + "_codes"][b, h, :length].to(torch.uint8)  # [len, nb, 16 * bits]
                stream = (byte[..., None] >> torch.arange(8, device=DEV, dtype=torch.uint8)) & 1
                digit = stream.flatten(-2).unflatten(-1, (BLOCK, bits)).long()
                idx = (digit << torch.arange(bits, device=DEV)).sum(-1)
                norm = s[side + "_norms"][b, h, :length].view(torch.float16).double()
                kv.append(((table[idx] @ back) * norm[..., None]).flatten(-2))
            q = s["q"][b, :count, h * G:(h + 1) * G].double()
            x = torch.einsum("jgd,td->jgt", q, kv[0]) * s["scale"]
            x = x.masked_fill(~seen[:, None], -math.inf)
            p = torch.softmax(x, -1)
            out[b, :count, h * G:(h + 1) * G] = torch.einsum("jgt,td->jgd", p, kv[1])
    return out


def exact(case, seed):
    if case["op"] not in ("rope", "tree"):
        return None  # bytes are moved: whole numbers
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return exact_rope(s) if case["op"] == "rope" else exact_tree(s)
