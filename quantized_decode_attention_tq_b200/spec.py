"""Binding of the speculative-decoding operators (include/tq_spec.h).

Argument marshalling only, like api.py: torch tensors supply device memory, and
the calls run on the tensors' device and its current stream.
"""
from __future__ import annotations

import ctypes

import numpy as np

from ._lib import (TQ_BF16, TQ_F16, TQ_F32, TQ_MAX_TREE_NODES, CacheBufs, Codebook, KVDesc, Rope, Rows, check, lib)
from .api import Cache, VOutliers

_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
_CODES = {}


def _code(dtype) -> int:
    if not _CODES:
        import torch
        _CODES.update({torch.float32: TQ_F32, torch.float16: TQ_F16, torch.bfloat16: TQ_BF16})
    try:
        return _CODES[dtype]
    except KeyError:
        raise ValueError(f"unsupported dtype {dtype}: fp32, fp16 or bf16") from None


class _On:
    """The device of a call's tensors: checks them, makes it current, gives the stream."""

    def __init__(self, first, name):
        if not first.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        self.device = first.device

    def ptr(self, t, name, contiguous=True):
        if t is None:
            return None
        if t.device != self.device:
            raise ValueError(f"{name} must be on {self.device}, like the other tensors of the call")
        if contiguous and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    def i32(self, t, name, shape):
        if t is None:
            return None
        import torch
        if t.dtype != torch.int32 or tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must be int32 of shape {tuple(shape)}")
        return self.ptr(t, name)

    def call(self, fn, stream, *args):
        import torch
        if stream is not None and stream.device != self.device:
            raise ValueError(f"stream must be on {self.device}, like the tensors of the call")
        f = getattr(lib(), fn)
        if torch.cuda.current_device() == self.device.index:
            s = (stream or torch.cuda.current_stream()).cuda_stream
            check(fn, f(*args, s))
        else:
            with torch.cuda.device(self.device):
                s = (stream or torch.cuda.current_stream()).cuda_stream
                check(fn, f(*args, s))


# ---- position rotation and per-head norms ----------------------------------

def make_rope(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0, orig_ctx: float = 4096,
              beta_fast: float = 32.0, beta_slow: float = 1.0, interleaved: bool = False) -> Rope:
    """A position rotation of the first rot_dim elements of a row (tq_make_rope; host)."""
    if scaling not in _SCALING:
        raise ValueError(f"unknown scaling {scaling!r}: one of {', '.join(_SCALING)}")
    r = Rope()
    check("tq_make_rope", lib().tq_make_rope(rot_dim, int(interleaved), base, _SCALING[scaling], factor, orig_ctx,
                                             beta_fast, beta_slow, ctypes.byref(r)))
    return r


def _rows(on, x, out, weight, name, head_first, dim):
    """The Rows struct of one side: x [B, T, H, D] with any batch, token and head strides."""
    if x is None:
        if out is not None:
            raise ValueError(f"{name}_out without {name}")
        return None
    if x.dim() != 4 or x.shape[3] != dim or (x.stride(3) != 1 and dim > 1):
        raise ValueError(f"{name} must be [B, T, heads, head_dim] with contiguous rows")
    b, t, h, _ = x.shape
    want = (b, h, t, dim) if head_first else (b, t, h, dim)
    if out is None or tuple(out.shape) != want:
        raise ValueError(f"{name}_out must have shape {want}")
    if weight is not None and tuple(weight.shape) != (dim,):
        raise ValueError(f"{name}_weight must have shape ({dim},)")
    # a stride of a dimension of one element says nothing
    s = [x.stride(i) if x.shape[i] > 1 else 0 for i in range(3)]
    return Rows(on.ptr(x, name, contiguous=False), on.ptr(out, name + "_out"), on.ptr(weight, name + "_weight"), h,
                s[0], s[1], s[2])


def qk_norm_rope(rope: Rope | None, q=None, k=None, v=None, positions=None, q_out=None, k_out=None, v_out=None,
                 norm: bool = True, eps: float = 1e-6, q_weight=None, k_weight=None, weight_bias: float = 0.0,
                 n_tok=None, stream=None) -> None:
    """Norm and rotate the rows of a projection and lay them out (tq_qk_norm_rope).

    q, k, v: [B, T, heads, D], any strides with contiguous rows (a split of a
    joint projection), one dtype; positions: int32 [B, T].  q_out: [B, T, Hq, D];
    k_out, v_out: [B, Hkv, T, D], as encode_kv takes them."""
    given = [(n, x, o) for n, x, o in (("q", q, q_out), ("k", k, k_out), ("v", v, v_out)) if x is not None]
    if not given:
        raise ValueError("q, k or v is required")
    name, first, out0 = given[0]
    on = _On(first, name)
    if first.dim() != 4:
        raise ValueError(f"{name} must be [B, T, heads, head_dim]")
    b, t, _, dim = first.shape
    for n, x, o in given:
        if tuple(x.shape[:2]) != (b, t) or x.dtype != first.dtype:
            raise ValueError("q, k and v must have the same batch, tokens and dtype")
        if o is None or o.dtype != out0.dtype:
            raise ValueError(f"{n}_out is required, all outputs of one dtype")
    weights = [w for w in (q_weight, k_weight) if w is not None]
    if any(w.dtype != weights[0].dtype for w in weights):
        raise ValueError("q_weight and k_weight must have the same dtype")
    sides = [_rows(on, q, q_out, q_weight, "q", False, dim), _rows(on, k, k_out, k_weight, "k", True, dim),
             _rows(on, v, v_out, None, "v", True, dim)]
    on.call("tq_qk_norm_rope", stream, None if rope is None else ctypes.byref(rope), b, t, dim,
            *(None if s is None else ctypes.byref(s) for s in sides), _code(first.dtype),
            _code(weights[0].dtype) if weights else TQ_F32, _code(out0.dtype), int(norm), eps, weight_bias,
            on.i32(positions, "positions", (b, t)), on.i32(n_tok, "n_tok", (b,)))


# ---- attention of a tree of drafted tokens ----------------------------------

def tree_masks(parents):
    """Ancestor masks (int64 bit patterns) and depths (int32) of one tree or of a
    batch of trees, [n] or [B, n] (tq_tree_masks; host).  parents[j] < j, -1 for a
    child of the context."""
    par = np.ascontiguousarray(np.asarray(parents, dtype=np.int32))
    flat = par.reshape(-1, par.shape[-1]) if par.ndim else par.reshape(0, 1)
    masks, depths = np.zeros(flat.shape, dtype=np.uint64), np.zeros(flat.shape, dtype=np.int32)
    for i in range(flat.shape[0]):
        check("tq_tree_masks", lib().tq_tree_masks(flat[i].ctypes.data, flat.shape[1], masks[i].ctypes.data,
                                                   depths[i].ctypes.data))
    return masks.view(np.int64).reshape(par.shape), depths.reshape(par.shape)


def tree_workspace_size(desc: KVDesc, q_heads: int, n_q: int) -> int:
    return int(lib().tq_tree_workspace_size(ctypes.byref(desc), q_heads, n_q))


def alloc_tree_workspace(desc: KVDesc, q_heads: int, n_q: int, device="cuda"):
    """A workspace of decode_attention_tree (any content)."""
    import torch
    n = tree_workspace_size(desc, q_heads, n_q)
    if n == 0:
        raise ValueError("invalid tree-attention configuration")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _cache_ptrs(on, cache: Cache):
    return [on.ptr(getattr(cache, n), n) for n in ("k_codes", "k_norms", "v_codes", "v_norms")]


def decode_attention_tree(cache: Cache, k_cb: Codebook, v_cb: Codebook, q, seq_lens, tree, scale: float, out, workspace,
                          n_nodes=None, status=None, stream=None):
    """Attention of a tree of drafted tokens over the packed cache
    (tq_decode_attention_tree).  q, out: [B, n_q, Hq, D] (out fp16 or bf16);
    tree: int64 [B, n_q] ancestor masks; the last n_nodes[b] (default n_q) of
    seq_lens[b] cached positions are the drafted nodes."""
    on = _On(q, "q")
    if q.dim() != 4 or out.shape != q.shape:
        raise ValueError("q and out must be [B, n_q, heads, head_dim], of one shape")
    b, n_q, heads, dim = q.shape
    if (b, dim) != (cache.desc.batch, cache.desc.head_dim):
        raise ValueError("q does not match the cache's batch and head_dim")
    import torch
    if tree.dtype not in (torch.int64, torch.uint64) or tuple(tree.shape) != (b, n_q):
        raise ValueError(f"tree must be int64 of shape {(b, n_q)}")
    on.call("tq_decode_attention_tree", stream, ctypes.byref(cache.desc), ctypes.byref(k_cb), ctypes.byref(v_cb), heads,
            n_q, on.ptr(q, "q"), _code(q.dtype), *_cache_ptrs(on, cache), on.i32(seq_lens, "seq_lens", (b,)),
            on.i32(n_nodes, "n_nodes", (b,)), on.ptr(tree, "tree"), scale, on.ptr(out, "out"), _code(out.dtype),
            on.ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(), on.ptr(status, "status"))
    return out


# ---- rows of the cache -------------------------------------------------------

def _bufs(on, cache: Cache, vo: VOutliers | None) -> CacheBufs:
    return CacheBufs(*_cache_ptrs(on, cache), None if vo is None else on.ptr(vo.values, "values"),
                     0 if vo is None else vo.k)


def cache_compact(cache: Cache, keep, n_keep, start=None, new_lens=None, vo: VOutliers | None = None, status=None,
                  stream=None) -> None:
    """Keep chosen rows of every sequence, in place (tq_cache_compact): row
    keep[b, i] becomes row start[b] + i for i < n_keep[b].  keep: int32
    [B, max_keep]; vo: the side data of a v3 cache."""
    on = _On(cache.k_codes, "k_codes")
    b = cache.desc.batch
    if keep.dim() != 2:
        raise ValueError("keep must be [B, max_keep]")
    on.call("tq_cache_compact", stream, ctypes.byref(cache.desc), ctypes.byref(_bufs(on, cache, vo)),
            on.i32(keep, "keep", (b, keep.shape[1])), keep.shape[1], on.i32(n_keep, "n_keep", (b,)),
            on.i32(start, "start", (b,)), on.i32(new_lens, "new_lens", (b,)), on.ptr(status, "status"))


def cache_copy(src: Cache, dst: Cache, src_slot, dst_slot, n_rows, max_rows: int, src_pos=None, dst_pos=None,
               src_vo: VOutliers | None = None, dst_vo: VOutliers | None = None, status=None, stream=None) -> None:
    """Copy row ranges between cache slots (tq_cache_copy): n_rows[c] rows from
    src_pos[c] of slot src_slot[c] to dst_pos[c] of slot dst_slot[c]."""
    on = _On(src.k_codes, "k_codes")
    n = src_slot.shape[0]
    on.call("tq_cache_copy", stream, ctypes.byref(src.desc), ctypes.byref(_bufs(on, src, src_vo)),
            ctypes.byref(dst.desc), ctypes.byref(_bufs(on, dst, dst_vo)), n, on.i32(src_slot, "src_slot", (n,)),
            on.i32(dst_slot, "dst_slot", (n,)), on.i32(src_pos, "src_pos", (n,)), on.i32(dst_pos, "dst_pos", (n,)),
            on.i32(n_rows, "n_rows", (n,)), max_rows, on.ptr(status, "status"))


__all__ = ["TQ_MAX_TREE_NODES", "alloc_tree_workspace", "cache_compact", "cache_copy", "decode_attention_tree",
           "make_rope", "qk_norm_rope", "tree_masks", "tree_workspace_size"]
