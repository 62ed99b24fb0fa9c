"""Binding of the speculative-decoding operators (include/tq_spec.h).

Argument marshalling only, like api.py: torch tensors supply device memory, and
the calls run on the tensors' device and its current stream.
"""
from __future__ import annotations

import ctypes
import struct

import numpy as np

from ._lib import TQ_BF16, TQ_F16, TQ_F32, TQ_MAX_TREE_NODES, Codebook, KVDesc, Rope, check, lib
from .api import Cache, VOutliers

_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
_ROWS = struct.Struct("PPPi4xqqq")  # tq_rows
_BUFS = struct.Struct("PPPPPi4x")   # tq_cache_bufs
_torch = _int32 = None
_codes = {}
_fns = {}


def _setup():
    global _torch, _int32
    import torch
    _int32 = torch.int32
    _codes.update({torch.float32: TQ_F32, torch.float16: TQ_F16, torch.bfloat16: TQ_BF16})
    _torch = torch
    return torch


def _code(dtype) -> int:
    code = _codes.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {dtype}: fp32, fp16 or bf16")
    return code


def _device(t, name) -> int:
    """The device index that every tensor of the call must have."""
    if _torch is None:
        _setup()
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return d


def _ptr(t, name, dev, contiguous=True):
    if t is None:
        return None
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, like the other tensors of the call")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _i32(t, name, dev, shape):
    if t is None:
        return None
    if t.dtype is not _int32 or t.shape != shape:
        raise ValueError(f"{name} must be int32 of shape {shape}")
    if t.get_device() != dev or not t.is_contiguous():
        return _ptr(t, name, dev)
    return t.data_ptr()


def _status(t, dev):
    if t is None:
        return None
    if t.element_size() != 4 or t.numel() < 1:
        raise ValueError("status must be a one-element int32 tensor")
    return _ptr(t, "status", dev)


def _call(fn, dev, stream, *args):
    """Run fn(*args, stream) with the tensors' device current."""
    f, cuda = _fns.get(fn), _torch.cuda
    if f is None:
        f = _fns[fn] = getattr(lib(), fn)
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"stream must be on cuda:{dev}, like the tensors of the call")
    if cuda.current_device() == dev:
        st = f(*args, (cuda.current_stream() if stream is None else stream).cuda_stream)
    else:
        with cuda.device(dev):
            st = f(*args, (cuda.current_stream() if stream is None else stream).cuda_stream)
    if st:
        check(fn, st)


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


def _rows(x, out, weight, name, dev, ref, head_first):
    """The tq_rows of one side, x [B, T, heads, D] with any batch, token and head
    strides; ref: (batch, tokens, D, dtype, output dtype) of the call."""
    if x is None:
        if out is not None:
            raise ValueError(f"{name}_out without {name}")
        return None
    if x.dim() != 4:
        raise ValueError(f"{name} must be [B, T, heads, head_dim]")
    b, t, h, d = x.shape
    sb, st, sh, sd = x.stride()
    batch, tokens, dim, dtype, out_dtype = ref
    if b != batch or t != tokens or d != dim or x.dtype is not dtype:
        raise ValueError("q, k and v must have the same batch, tokens, head_dim and dtype")
    if sd != 1:
        raise ValueError(f"{name} must have contiguous rows")
    want = (b, h, t, d) if head_first else (b, t, h, d)
    if out is None or out.shape != want or out.dtype is not out_dtype:
        raise ValueError(f"{name}_out must have shape {want}, all outputs one dtype")
    if weight is not None and weight.shape != (d,):
        raise ValueError(f"{name}_weight must have shape ({d},)")
    # the stride of a dimension of one element says nothing
    return _ROWS.pack(_ptr(x, name, dev, False), _ptr(out, name + "_out", dev),
                      _ptr(weight, name + "_weight", dev) or 0, h, sb if b > 1 else 0, st if t > 1 else 0,
                      sh if h > 1 else 0)


def qk_norm_rope(rope: Rope | None, q=None, k=None, v=None, positions=None, q_out=None, k_out=None, v_out=None,
                 norm: bool = True, eps: float = 1e-6, q_weight=None, k_weight=None, weight_bias: float = 0.0,
                 n_tok=None, stream=None) -> None:
    """Norm and rotate the rows of a projection and lay them out (tq_qk_norm_rope).

    q, k, v: [B, T, heads, D], any strides with contiguous rows (a split of a
    joint projection), one dtype; positions: int32 [B, T].  q_out: [B, T, Hq, D];
    k_out, v_out: [B, Hkv, T, D], as encode_kv takes them."""
    first, out0 = (q, q_out) if q is not None else (k, k_out) if k is not None else (v, v_out)
    if first is None or out0 is None:
        raise ValueError("q, k or v is required, with its output")
    dev = _device(first, "q" if q is not None else "k" if k is not None else "v")
    if first.dim() != 4:
        raise ValueError("q, k and v must be [B, T, heads, head_dim]")
    b, t, _, d = first.shape
    ref = (b, t, d, first.dtype, out0.dtype)
    w_dtype = TQ_F32
    if q_weight is not None or k_weight is not None:
        w = q_weight if q_weight is not None else k_weight
        if k_weight is not None and k_weight.dtype is not w.dtype:
            raise ValueError("q_weight and k_weight must have the same dtype")
        w_dtype = _code(w.dtype)
    _call("tq_qk_norm_rope", dev, stream, None if rope is None else ctypes.byref(rope), b, t, d,
          _rows(q, q_out, q_weight, "q", dev, ref, False), _rows(k, k_out, k_weight, "k", dev, ref, True),
          _rows(v, v_out, None, "v", dev, ref, True), _code(first.dtype), w_dtype, _code(out0.dtype), 1 if norm else 0,
          eps, weight_bias, _i32(positions, "positions", dev, (b, t)), _i32(n_tok, "n_tok", dev, (b,)))


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


def decode_attention_tree(cache: Cache, k_cb: Codebook, v_cb: Codebook, q, seq_lens, tree, scale: float, out, workspace,
                          n_nodes=None, status=None, stream=None):
    """Attention of a tree of drafted tokens over the packed cache
    (tq_decode_attention_tree).  q, out: [B, n_q, Hq, D] (out fp16 or bf16);
    tree: int64 [B, n_q] ancestor masks; the last n_nodes[b] (default n_q) of
    seq_lens[b] cached positions are the drafted nodes."""
    dev = _device(q, "q")
    if q.dim() != 4 or out.shape != q.shape:
        raise ValueError("q and out must be [B, n_q, heads, head_dim], of one shape")
    b, n_q, heads, dim = q.shape
    desc = cache.desc
    if b != desc.batch or dim != desc.head_dim:
        raise ValueError("q does not match the cache's batch and head_dim")
    if tree.element_size() != 8 or tree.is_floating_point() or tree.shape != (b, n_q):
        raise ValueError(f"tree must be int64 of shape {(b, n_q)}")
    _call("tq_decode_attention_tree", dev, stream, ctypes.byref(desc), ctypes.byref(k_cb), ctypes.byref(v_cb), heads,
          n_q, _ptr(q, "q", dev), _code(q.dtype), _ptr(cache.k_codes, "k_codes", dev),
          _ptr(cache.k_norms, "k_norms", dev), _ptr(cache.v_codes, "v_codes", dev),
          _ptr(cache.v_norms, "v_norms", dev), _i32(seq_lens, "seq_lens", dev, (b,)),
          _i32(n_nodes, "n_nodes", dev, (b,)), _ptr(tree, "tree", dev), scale, _ptr(out, "out", dev),
          _code(out.dtype), _ptr(workspace, "workspace", dev), workspace.numel() * workspace.element_size(),
          _status(status, dev))
    return out


# ---- rows of the cache -------------------------------------------------------

def _bufs(cache: Cache, vo: VOutliers | None, dev) -> bytes:
    """The tq_cache_bufs of a cache."""
    a, b, c, d = cache.k_codes, cache.k_norms, cache.v_codes, cache.v_norms
    if not (a.get_device() == b.get_device() == c.get_device() == d.get_device() == dev and a.is_contiguous()
            and b.is_contiguous() and c.is_contiguous() and d.is_contiguous()):
        for n in ("k_codes", "k_norms", "v_codes", "v_norms"):
            _ptr(getattr(cache, n), n, dev)
    values, k = (0, 0) if vo is None else (_ptr(vo.values, "values", dev), vo.k)
    return _BUFS.pack(a.data_ptr(), b.data_ptr(), c.data_ptr(), d.data_ptr(), values, k)


def cache_compact(cache: Cache, keep, n_keep, start=None, new_lens=None, vo: VOutliers | None = None, status=None,
                  stream=None) -> None:
    """Keep chosen rows of every sequence, in place (tq_cache_compact): row
    keep[b, i] becomes row start[b] + i for i < n_keep[b].  keep: int32
    [B, max_keep]; vo: the side data of a v3 cache."""
    dev = _device(cache.k_codes, "k_codes")
    b = cache.desc.batch
    if keep.dim() != 2:
        raise ValueError("keep must be [B, max_keep]")
    m = keep.shape[1]
    _call("tq_cache_compact", dev, stream, ctypes.byref(cache.desc), _bufs(cache, vo, dev),
          _i32(keep, "keep", dev, (b, m)), m, _i32(n_keep, "n_keep", dev, (b,)), _i32(start, "start", dev, (b,)),
          _i32(new_lens, "new_lens", dev, (b,)), _status(status, dev))


def cache_copy(src: Cache, dst: Cache, src_slot, dst_slot, n_rows, max_rows: int, src_pos=None, dst_pos=None,
               src_vo: VOutliers | None = None, dst_vo: VOutliers | None = None, status=None, stream=None) -> None:
    """Copy row ranges between cache slots (tq_cache_copy): n_rows[c] rows from
    src_pos[c] of slot src_slot[c] to dst_pos[c] of slot dst_slot[c]."""
    if not 0 <= max_rows < 2 ** 31:  # others would lose their upper bits on the way
        raise ValueError("max_rows must be in [0, 2^31)")
    dev = _device(src.k_codes, "k_codes")
    n = src_slot.shape[0]
    shape = (n,)
    a = _bufs(src, src_vo, dev)
    b = a if dst is src and dst_vo is src_vo else _bufs(dst, dst_vo, dev)
    _call("tq_cache_copy", dev, stream, ctypes.byref(src.desc), a, ctypes.byref(dst.desc), b, n,
          _i32(src_slot, "src_slot", dev, shape), _i32(dst_slot, "dst_slot", dev, shape),
          _i32(src_pos, "src_pos", dev, shape), _i32(dst_pos, "dst_pos", dev, shape),
          _i32(n_rows, "n_rows", dev, shape), max_rows, _status(status, dev))


__all__ = ["TQ_MAX_TREE_NODES", "alloc_tree_workspace", "cache_compact", "cache_copy", "decode_attention_tree",
           "make_rope", "qk_norm_rope", "tree_masks", "tree_workspace_size"]
