"""Plain fp64 references of the speculative-decoding operators (include/tq_spec.h)."""
from __future__ import annotations

import math

import numpy as np

from oracle import tq_oracle as O


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, orig_ctx=4096, fast=32.0, slow=1.0):
    """Radians per position of each pair, and the gain (see tq_make_rope)."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2 * i / rot) if rot else i
    if scaling == "linear":
        f = f / factor
    if scaling != "yarn":
        return f, 1.0

    def at(turns):
        return rot * math.log(orig_ctx / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = min(max(math.floor(at(fast)), 0), rot - 1), max(min(math.ceil(at(slow)), rot - 1), 0)
    w = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
    return f * (1 - w) + f / factor * w, 0.1 * math.log(factor) + 1.0


def norm_rope(x, weight, positions, f, gain, interleaved, norm, eps=1e-6, bias=0.0):
    """One side's rows x [B, T, H, D] in fp64: (y, r), r the length of each
    element's pair (its own size where it is not rotated)."""
    y = x.astype(np.float64)
    if norm:
        w = 1.0 if weight is None else weight.astype(np.float64)
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps) * (w + bias)
    r = np.abs(y)
    h = len(f)
    if h:
        i = np.arange(h)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        ang = positions.astype(np.float64)[..., None, None] * f
        c, s = np.cos(ang), np.sin(ang)
        ya, yb = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = gain * (ya * c - yb * s), gain * (yb * c + ya * s)
        r[..., a] = r[..., b] = gain * np.hypot(ya, yb)
    return y, r


def random_cache(rng, batch, kv_heads, cap, dim, k_bits, v_bits, norm=11.3):
    """Codes, norms [B, H, cap, nb(, 16 bits)] with every index equally likely."""
    nb = dim // 128
    out = []
    for bits in (k_bits, v_bits):
        out.append(rng.integers(0, 256, (batch, kv_heads, cap, nb, 16 * bits), dtype=np.uint8))
        out.append((norm * (1 + 0.1 * rng.standard_normal((batch, kv_heads, cap, nb)))).astype(np.float16))
    return out


def visible(length, n, masks):
    """[n, length] truth: which cached positions each node sees."""
    see = np.zeros((n, length), dtype=bool)
    ctx = length - n
    for j in range(n):
        for t in range(length):
            see[j, t] = t < ctx or ((int(masks[j]) >> (t - ctx)) & 1) == 1
    return see


def tree_attention(q, cache, k_bits, v_bits, lens, counts, masks, scale, seed=0):
    """(out, spread, score): out [B, n_q, Hq, D] fp64, NaN in rows past a tree's
    nodes; spread = sum_t w_t |v_t| per row and 128-block (the size that weight
    and value errors scale with); score = max_t scale |q| |k_t| of each row."""
    kc, kn, vc, vn = cache
    s = O.sign_vector(seed)
    k = O.dequantize(kc, kn, k_bits, O.codebook_f32(k_bits)[0].astype(np.float64), s)
    v = O.dequantize(vc, vn, v_bits, O.codebook_f32(v_bits)[0].astype(np.float64), s)
    B, n_q, hq, D = q.shape
    g = hq // k.shape[1]
    out = np.full(q.shape, np.nan)
    spread, score = np.zeros((B, n_q, hq, D // 128)), np.zeros((B, n_q, hq))
    for b in range(B):
        L, n = int(lens[b]), int(counts[b])
        see = visible(L, n, masks[b])
        for j in range(n):
            for h in range(hq):
                t = np.nonzero(see[j])[0]
                if t.size == 0:
                    out[b, j, h] = 0.0
                    continue
                kk, vv, qq = k[b, h // g, t], v[b, h // g, t], q[b, j, h].astype(np.float64)
                x = scale * (kk @ qq)
                w = np.exp(x - x.max())
                w /= w.sum()
                out[b, j, h] = w @ vv
                spread[b, j, h] = w @ np.linalg.norm(vv.reshape(t.size, D // 128, 128), axis=-1)
                score[b, j, h] = scale * np.linalg.norm(qq) * np.linalg.norm(kk, axis=-1).max()
    return out, spread, score


def tree_attention_by_head(q, cache, k_bits, v_bits, lens, counts, masks, scale, seed=0):
    """tree_attention, with the rows of one sequence and kv-head at a time."""
    kc, kn, vc, vn = cache
    s = O.sign_vector(seed)
    B, n_q, hq, D = q.shape
    hk = kc.shape[1]
    g = hq // hk
    out = np.full(q.shape, np.nan)
    spread, score = np.zeros((B, n_q, hq, D // 128)), np.zeros((B, n_q, hq))
    for b in range(B):
        L, n = int(lens[b]), int(counts[b])
        if n == 0:
            continue
        see = np.repeat(visible(L, n, masks[b]), g, axis=0)  # [n * g, L], node-major
        for h in range(hk):
            k, v = (O.dequantize(c[b, h, :L], m[b, h, :L], bits, O.codebook_f32(bits)[0].astype(np.float64), s)
                    for c, m, bits in ((kc, kn, k_bits), (vc, vn, v_bits)))
            qq = q[b, :n, h * g:(h + 1) * g].astype(np.float64).reshape(n * g, D)
            x = np.where(see, scale * (qq @ k.T), -np.inf) if L else np.zeros((n * g, 0))
            top = x.max(axis=1, initial=-np.inf, keepdims=True)
            w = np.exp(x - np.where(top > -np.inf, top, 0.0))
            w /= np.maximum(w.sum(axis=1, keepdims=True), 1e-300)
            rows = (b, slice(0, n), slice(h * g, (h + 1) * g))
            out[rows] = (w @ v).reshape(n, g, D)
            spread[rows] = (w @ np.linalg.norm(v.reshape(L, D // 128, 128), axis=-1)).reshape(n, g, D // 128)
            kmax = np.where(see, np.linalg.norm(k, axis=-1)[None], 0.0).max(axis=1, initial=0.0)
            score[rows] = (scale * np.linalg.norm(qq, axis=-1) * kmax).reshape(n, g)
    return out, spread, score


def check_tree(got, ref, spread, score, eps_out):
    """Every 128-block of every row, in the 2-norm (the inverse rotation keeps
    it).  With u = 2^-11, half a step of fp16: a score x = scale q.k is off by at
    most d = score * 2u (centroids and query in fp16, u each; fp32 sums are
    below u / 100), so a normalised weight by a factor within 1 + 2d, the fp16
    product of weight and norm by u, the fp16 V centroid by u; the output is
    rounded by eps_out / 2."""
    u = 2.0 ** -11
    B, n, h, D = got.shape
    live = ~np.isnan(ref)
    assert not np.any(np.isnan(got[live]))
    diff = np.where(live, got - np.where(live, ref, 0.0), 0.0).reshape(B, n, h, D // 128, 128)
    size = np.linalg.norm(np.where(live, ref, 0.0).reshape(diff.shape), axis=-1)
    d = 2 * u * score[..., None]
    allowed = spread * (np.expm1(2 * d) + 2.1 * u) * (1 + u) + size * eps_out / 2 * 1.01 + 1e-6
    err = np.linalg.norm(diff, axis=-1)
    assert np.all(err <= allowed), f"error {np.max(err / allowed):.3f} of the bound"
    return float(np.max(err / allowed))
