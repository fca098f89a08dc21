"""ctypes binding of the paged-cache entry points (``include/paged_attention.h``):
block tables and slot maps, cache writes, attention over chosen or all cached
positions, and the latent forms.  As in :mod:`binding`, torch tensors are
device memory and streams, every step of an operator runs in the HIP kernels,
and there is no fallback.

Outputs and workspaces that are not given are allocated by torch on the call's
stream.  Nothing is differentiable: where autograd is on, tensors that require
gradients are refused (call under ``torch.no_grad()``, or detach them).
"""

from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple

from . import binding
from .binding import _check

ROPE_DIM = 64
HEAD_DIM = 128
MAX_SPLITS = 128

# Every symbol include/paged_attention.h declares.
EXPORTED = (
    "paged_layout", "paged_append", "paged_attention", "paged_attention_workspace_size", "latent_attention",
    "latent_attention_workspace_size", "latent_prefill", "latent_prefill_workspace_size",
    "paged_debug_place", "paged_debug_split", "paged_fork", "paged_copy", "paged_free", "paged_free_workspace_size",
    "paged_compact", "paged_compact_workspace_size", "paged_bounds", "paged_block_select",
    "paged_block_select_workspace_size", "paged_block_attention", "paged_block_attention_workspace_size",
    "paged_prefix_attention", "paged_prefix_attention_workspace_size",
)

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class Part(ctypes.Structure):
    _fields_ = [("src", _vp), ("dst", _vp), ("scales", _vp), ("src_stride", _i64), ("dst_page_stride", _i64),
                ("dst_token_stride", _i64), ("dst_head_stride", _i64), ("width", _i32), ("head_width", _i32)]


class AttentionArgs(ctypes.Structure):
    _fields_ = [("q", _vp), ("k", _vp), ("v", _vp), ("k_scales", _vp), ("v_scales", _vp), ("block_table", _vp),
                ("lengths", _vp), ("chosen", _vp), ("out", _vp), ("lse", _vp), ("q_row_stride", _i64),
                ("q_head_stride", _i64), ("page_stride", _i64), ("token_stride", _i64), ("head_stride", _i64),
                ("table_stride", _i64), ("chosen_stride", _i64), ("num_rows", _i32), ("next_n", _i32),
                ("num_heads", _i32), ("num_kv_heads", _i32), ("head_dim", _i32), ("page_size", _i32),
                ("num_pages", _i32), ("table_width", _i32), ("num_chosen", _i32), ("softmax_scale", _f32),
                ("dtype", _i32), ("store", _i32), ("max_splits", _i32)]


class PrefillArgs(ctypes.Structure):
    _fields_ = [("q", _vp), ("cache", _vp), ("scale", _vp), ("w_k", _vp), ("w_v", _vp), ("block_table", _vp),
                ("starts", _vp), ("lengths", _vp), ("out", _vp), ("lse", _vp), ("q_row_stride", _i64),
                ("q_head_stride", _i64), ("page_stride", _i64), ("token_stride", _i64), ("table_stride", _i64),
                ("context_tokens", _i64), ("num_tokens", _i32), ("num_seqs", _i32), ("num_heads", _i32),
                ("latent_dim", _i32), ("page_size", _i32), ("num_pages", _i32), ("table_width", _i32),
                ("softmax_scale", _f32), ("dtype", _i32), ("store", _i32)]


class Layout(NamedTuple):
    """What a step's layout gives besides the block table."""

    slots: "torch.Tensor"  # noqa: F821  int32 [capacity], -1 where a token has no place and past the last token
    row_lengths: "torch.Tensor"  # noqa: F821  int32 [capacity], 0 past the last token
    row_seqs: "torch.Tensor"  # noqa: F821  int32 [capacity], -1 past the last token
    starts: "torch.Tensor"  # noqa: F821  int32 [num_seqs + 1]
    pages: "torch.Tensor"  # noqa: F821  int32 [1], pages the step needs


_lib = None
torch = None  # imported with the library, on the first call


def load() -> ctypes.CDLL:
    """The built library with these entry points' signatures set."""
    global _lib, torch, _CODES
    if _lib is None:
        import torch as _torch
        torch = _torch
        _CODES = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: _E4M3}
        lib = binding.load()
        lib.paged_layout.argtypes = [_vp, _vp, _i32, _vp, _i32, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp,
                                     _vp]
        lib.paged_append.argtypes = [_vp, _i32, ctypes.POINTER(Part), _i32, _i32, _i32, _i32, _i32, _vp]
        for name, args in (("paged_attention", AttentionArgs), ("latent_attention", AttentionArgs),
                           ("latent_prefill", PrefillArgs)):
            getattr(lib, name).argtypes = [ctypes.POINTER(args), _vp, _vp]
            getattr(lib, name + "_workspace_size").argtypes = [ctypes.POINTER(args), _vp,
                                                               ctypes.POINTER(ctypes.c_size_t)]
        size = ctypes.POINTER(ctypes.c_size_t)
        lib.paged_fork.argtypes = [_vp, _i64, _i32, _vp, _i32, _vp, _vp, _i32, _vp, _i32, _i32, _vp, _i64, _vp, _vp, _vp,
                                   _vp, _vp, _vp]
        lib.paged_copy.argtypes = [_vp, _vp, _vp, _i32, _vp, _i32, _i32, _vp]
        lib.paged_free.argtypes = [_vp, _i64, _i32, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp]
        lib.paged_compact.argtypes = [_vp, _i64, _i32, _vp, _i32, _i32, _i32, _i32, _vp, _i64, _vp, _vp, _vp, _vp, _vp,
                                      _vp]
        lib.paged_free_workspace_size.argtypes = lib.paged_compact_workspace_size.argtypes = [_i32, size]
        lib.paged_prefix_attention.argtypes = [_vp, _vp, _vp, _i32, _vp, _vp]
        lib.paged_prefix_attention_workspace_size.argtypes = [_vp, _i32, _vp, size]
        lib.paged_bounds.argtypes = [_vp, _vp]
        lib.paged_block_select.argtypes = [_vp, _vp, _vp]
        lib.paged_block_select_workspace_size.argtypes = [_vp, _vp, size]
        lib.paged_block_attention.argtypes = [_vp, _vp, _i64, _i64, _i32, _vp, _vp]
        lib.paged_block_attention_workspace_size.argtypes = [_vp, _i32, _vp, size]
        for name in EXPORTED:
            getattr(lib, name).restype = ctypes.c_int
        lib.paged_debug_place.argtypes = [_vp, _i32, _i32, _i64, _i64, _i32]
        lib.paged_debug_place.restype = _i64
        lib.paged_debug_split.argtypes = [_i32, _i32, _i32, _i32, _vp]
        lib.paged_debug_split.restype = None
        _lib = lib
    return _lib


# ---------------------------------------------------------------------------
# Argument checks.  A decode step makes these calls once a layer, so what a
# call costs on the host counts: devices are compared by index, no context is
# entered for the usual call, and outputs that the call itself allocates are
# not checked.
# ---------------------------------------------------------------------------
_E4M3 = 2
_CODES: dict = {}


def _elsewhere(x, stream) -> bool:
    """Whether the call has to enter another device or stream first."""
    return stream is not None or x.get_device() != torch._C._cuda_getDevice()


def _on(stream, x):
    """The call's stream made current (and its device), so that what torch
    allocates for the call belongs to it."""
    device = x.device
    if device.type != "cuda":
        raise TypeError("tensors must be on a GPU")
    if stream is None:
        return torch.cuda.device(device)
    if stream.device != device:
        raise ValueError("stream and tensors must be on the same device")
    return torch.cuda.stream(stream)


def _no_gradients(name: str) -> None:
    """Tensors whose gradients a call would drop without a word are refused;
    where autograd is off they are taken as they are."""
    if torch.is_grad_enabled():
        raise RuntimeError(f"{name} has no gradients: call it under torch.no_grad() or detach its tensors")


def _code(x, name: str, cache: bool = False) -> int:
    code = _CODES.get(x.dtype)
    if code is None or (code == _E4M3 and not cache):
        raise TypeError(f"{name} must be bfloat16 or float16" + (" or float8_e4m3fn" if cache else ""))
    return code


def _ints(x, name: str, dev: int, n: int) -> int:
    """Pointer of a contiguous int32 tensor of n entries."""
    if x.dtype is not torch.int32 or x.get_device() != dev:
        raise TypeError(f"{name} must be an int32 tensor on cuda:{dev}")
    if x.numel() != n or not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {n} entries")
    return x.data_ptr()


def _matrix(x, name: str, dev: int, rows: int) -> int:
    """Pointer of an int32 [rows, n >= 1] tensor whose rows may be strided."""
    if x.dtype is not torch.int32 or x.get_device() != dev or x.dim() != 2:
        raise TypeError(f"{name} must be a 2-D int32 tensor on cuda:{dev}")
    if x.shape[0] != rows or x.shape[1] < 1 or (x.stride(1) != 1 and x.shape[1] > 1):
        raise ValueError(f"{name} must be [{rows}, n] with n >= 1 and unit column stride")
    return x.data_ptr()


def _scales(x, name: str, dev: int, n: int, code: int):
    if x is None:
        return None
    if code != _E4M3:
        raise ValueError(f"{name} belongs to a float8_e4m3fn cache")
    if x.dtype is not torch.float32 or x.get_device() != dev or x.numel() != n or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of {n} on cuda:{dev}")
    if x.requires_grad:
        _no_gradients(name)
    return x.data_ptr()


def _output(x, name: str, dtype, shape, like):
    """x if it is given (and fits), else a new tensor."""
    if x is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    if x.dtype is not dtype or x.get_device() != like.get_device() or tuple(x.shape) != shape or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {like.device}")
    return x


def _launch(name: str, args, workspace, key, like, size_args=(), more=()) -> None:
    """Calls entry point `name` with a workspace large enough: `workspace`, or
    a new one.  key: what its size depends on; size_args, more: further arguments
    of the size's and of the call itself."""
    args = ctypes.byref(args)
    dev = like.get_device()
    stream = torch._C._cuda_getCurrentRawStream(dev)
    need = _sizes.get((name, dev, key))
    if need is None:
        size = ctypes.c_size_t(0)
        _check(getattr(_lib, name + "_workspace_size")(args, *size_args, stream, size), name)
        need = size.value
        if len(_sizes) >= 4096:
            _sizes.clear()
        _sizes[name, dev, key] = need
    ptr = None
    if need:
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
        elif (workspace.get_device() != dev or not workspace.is_contiguous()
              or workspace.numel() * workspace.element_size() < need):
            raise ValueError(f"workspace must be a contiguous tensor of {need} bytes or more on {like.device}")
        ptr = workspace.data_ptr()
    _check(getattr(_lib, name)(args, *more, ptr, stream), name)


_sizes: dict = {}  # workspace bytes by shape: a pure function of it


# ---------------------------------------------------------------------------
# Layout and append
# ---------------------------------------------------------------------------

def paged_layout(lengths, new_tokens, free_pages, block_table, *, page_size: int, capacity: int,
                 out: Layout | None = None, stream=None) -> Layout:
    """Block tables and slot maps of one step.

    lengths, new_tokens: int32 [num_seqs], each sequence's tokens after the
    step and how many of them are new.  block_table (int32 [num_seqs, width])
    is updated in place: the pages the new tokens need are taken from
    free_pages (int32) in order.  Returns a Layout of `capacity` rows; tokens
    past it are not written.  Where its pages are more than free_pages has (its
    entries, or paged_free's count, whose list is padded with -1), the list ran
    out and tokens have no place.  See paged_layout in paged_attention.h.
    """
    lib = load()
    if _elsewhere(lengths, stream):
        with _on(stream, lengths):
            return paged_layout(lengths, new_tokens, free_pages, block_table, page_size=page_size, capacity=capacity,
                                out=out)
    if capacity < 0:
        raise ValueError("capacity must be >= 0")
    dev, n = lengths.get_device(), lengths.numel()
    width = block_table.shape[-1]
    if out is None:
        whole = torch.empty(3 * capacity + n + 2, dtype=torch.int32, device=lengths.device)
        out = Layout(*whole.split_with_sizes([capacity, capacity, capacity, n + 1, 1]))
        at = whole.data_ptr()
        slots, rows, seqs, starts = at, at + 4 * capacity, at + 8 * capacity, at + 12 * capacity
        pages = starts + 4 * (n + 1)
    else:
        slots, rows, seqs = (_ints(x, name, dev, capacity) for x, name in
                             ((out.slots, "out.slots"), (out.row_lengths, "out.row_lengths"),
                              (out.row_seqs, "out.row_seqs")))
        starts, pages = _ints(out.starts, "out.starts", dev, n + 1), _ints(out.pages, "out.pages", dev, 1)
    _check(lib.paged_layout(_ints(lengths, "lengths", dev, n), _ints(new_tokens, "new_tokens", dev, n), n,
                            _ints(free_pages, "free_pages", dev, free_pages.numel()), free_pages.numel(),
                            _matrix(block_table, "block_table", dev, n), block_table.stride(0) if n > 1 else width,
                            width, page_size, capacity, starts, slots, rows, seqs, pages,
                            torch._C._cuda_getCurrentRawStream(dev)), "paged_layout")
    return out


def _part(x, name: str, cache, column: int, heads: int, dim: int, scales) -> Part:
    """x [tokens, heads, dim] (inner dims contiguous) into columns of cache
    [pages, page_size, heads, dim] or [pages, page_size, width]."""
    stride = x.stride()
    if stride[-1] != 1 or (len(stride) == 3 and stride[1] != dim and heads > 1):
        raise ValueError(f"{name}'s rows must be contiguous")
    to = cache.stride()
    return Part(x.data_ptr(), cache.data_ptr() + column * cache.element_size(), scales, stride[0], to[0], to[1],
                to[2] if len(to) == 4 else 0, heads * dim, dim)


def _append(slots, one: Part, two: Part, cache, tokens: int, code: int, store: int) -> None:
    dev = cache.get_device()
    shape = cache.shape
    _check(_lib.paged_append(_ints(slots, "slots", dev, tokens), tokens, (Part * 2)(one, two), 2, shape[1], shape[0],
                             code, store, torch._C._cuda_getCurrentRawStream(dev)), "paged_append")


def paged_append(slots, k, v, k_cache, v_cache, *, k_scale=None, v_scale=None, stream=None) -> None:
    """Writes keys and values [num_tokens, num_kv_heads, head_dim] (bfloat16
    or float16, rows may be strided) to their slots (int32 [num_tokens], -1 to
    drop a token) of the caches [num_pages, page_size, num_kv_heads, head_dim]
    of the same type or float8_e4m3fn, then as x / scale with float32
    [num_kv_heads] scales (None: 1).  No slot may occur twice."""
    load()
    if k.requires_grad or v.requires_grad or k_cache.requires_grad or v_cache.requires_grad:
        _no_gradients("paged_append")
    if _elsewhere(k_cache, stream):
        with _on(stream, k_cache):
            return paged_append(slots, k, v, k_cache, v_cache, k_scale=k_scale, v_scale=v_scale)
    dev = k_cache.get_device()
    code, store = _code(k, "k"), _code(k_cache, "k_cache", True)
    if v.dtype is not k.dtype or v_cache.dtype is not k_cache.dtype:
        raise TypeError("k and v, and k_cache and v_cache, must have the same type")
    if k.get_device() != dev or v.get_device() != dev or v_cache.get_device() != dev:
        raise ValueError("k, v and the caches must be on one device")
    shape = k_cache.shape
    if k.dim() != 3 or len(shape) != 4 or k.shape != v.shape or shape != v_cache.shape:
        raise ValueError("k and v must be [num_tokens, heads, dim], the caches [num_pages, page_size, heads, dim]")
    tokens, heads, dim = k.shape
    if shape[2] != heads or shape[3] != dim or k_cache.stride(3) != 1 or v_cache.stride(3) != 1:
        raise ValueError("the caches must have k's heads and dim and unit stride in their last dimension")
    _append(slots, _part(k, "k", k_cache, 0, heads, dim, _scales(k_scale, "k_scale", dev, heads, store)),
            _part(v, "v", v_cache, 0, heads, dim, _scales(v_scale, "v_scale", dev, heads, store)), k_cache, tokens,
            code, store)


def latent_append(slots, latent, rope, cache, *, scale=None, stream=None) -> None:
    """Writes latent vectors [num_tokens, latent_dim] and their rope parts
    [num_tokens, 64] to their slots of cache [num_pages, page_size, latent_dim
    + 64], as paged_append does; scale: float32 [1]."""
    load()
    if latent.requires_grad or rope.requires_grad or cache.requires_grad:
        _no_gradients("latent_append")
    if _elsewhere(cache, stream):
        with _on(stream, cache):
            return latent_append(slots, latent, rope, cache, scale=scale)
    dev = cache.get_device()
    code, store = _code(latent, "latent"), _code(cache, "cache", True)
    if rope.dtype is not latent.dtype:
        raise TypeError("latent and rope must have the same type")
    if latent.get_device() != dev or rope.get_device() != dev:
        raise ValueError("latent, rope and cache must be on one device")
    if latent.dim() != 2 or rope.dim() != 2 or cache.dim() != 3 or cache.stride(2) != 1:
        raise ValueError("latent and rope must be 2-D and cache 3-D with unit stride in its last dimension")
    tokens, dim = latent.shape
    if rope.shape[0] != tokens or rope.shape[1] != ROPE_DIM or cache.shape[2] != dim + ROPE_DIM:
        raise ValueError(f"rope must have {ROPE_DIM} columns and cache latent's and rope's together")
    by = _scales(scale, "scale", dev, 1, store)
    _append(slots, _part(latent, "latent", cache, 0, 1, dim, by), _part(rope, "rope", cache, dim, 1, ROPE_DIM, by),
            cache, tokens, code, store)


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------

def _attend(entry: str, q, k, v, scales, lengths, block_table, chosen, next_n, softmax_scale, kv: int, value_dim: int,
            out, lse, workspace, max_splits: int, key=(), size_args=(), more=()):
    """The attentions of rows after what differs between them: k (and v) a
    cache [num_pages, page_size, ..., dim], scales (name, tensor, size) of
    each; key, size_args, more: as for _launch."""
    dev = q.get_device()
    code, store = _code(q, "q"), _code(k, "the cache", True)
    if store != _E4M3 and store != code:
        raise TypeError("the cache must have q's type or float8_e4m3fn")
    if k.get_device() != dev:
        raise ValueError("q and the cache must be on the same device")
    kshape, kstride, qstride = k.shape, k.stride(), q.stride()
    dim = kshape[-1]
    if q.dim() != 3 or q.shape[2] != dim or qstride[2] != 1:
        raise ValueError(f"q must be [num_rows, num_heads, {dim}] with unit stride in its last dimension")
    if kstride[-1] != 1:
        raise ValueError("the cache must have unit stride in its last dimension")
    rows, heads, _ = q.shape
    if next_n is None:
        next_n = int(lengths.shape[1]) if lengths.dim() == 2 else 1
    if next_n < 1 or rows % next_n != 0:
        raise ValueError("next_n must be >= 1 and divide the rows")
    lengths_at = _ints(lengths, "lengths", dev, rows)
    table_at = _matrix(block_table, "block_table", dev, rows // next_n)
    width = block_table.shape[1]
    chosen_at, chosen_stride, num_chosen = None, 0, 0
    if chosen is not None:
        chosen_at = _matrix(chosen, "chosen", dev, rows)
        chosen_stride, num_chosen = chosen.stride(0), chosen.shape[1]
    by = [_scales(x, name, dev, n, store) for name, x, n in scales]
    out = _output(out, "out", q.dtype, (rows, heads, value_dim), q)
    lse = _output(lse, "lse", torch.float32, (rows, heads), q)
    args = AttentionArgs(q.data_ptr(), k.data_ptr(), None if v is None else v.data_ptr(), by[0],
                         by[1] if len(by) > 1 else None, table_at, lengths_at, chosen_at, out.data_ptr(),
                         lse.data_ptr(), qstride[0], qstride[1], kstride[0], kstride[1],
                         kstride[2] if v is not None else 0, block_table.stride(0), chosen_stride, rows, next_n, heads,
                         kv, value_dim, kshape[1], kshape[0], width, num_chosen, softmax_scale, code, store, max_splits)
    _launch(entry, args, workspace, (rows, next_n, heads, kv, value_dim, kshape[1], width, num_chosen, max_splits, *key),
            q, size_args, more)
    return out, lse


def _paged(entry: str, q, k_cache, v_cache, block_table, lengths, chosen, softmax_scale, k_scale, v_scale, next_n, out, lse,
           workspace, max_splits: int, more=()):
    """The attentions over a cache of keys and values.  more: further arguments
    of the entry point, the last of them its size's too."""
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.stride() != v_cache.stride():
        raise ValueError("k_cache and v_cache must be [num_pages, page_size, num_kv_heads, head_dim], alike")
    if v_cache.dtype is not k_cache.dtype or v_cache.get_device() != q.get_device():
        raise TypeError("k_cache and v_cache must have the same type and device")
    kv, dim = k_cache.shape[2], k_cache.shape[3]
    if kv < 1 or q.dim() != 3 or q.shape[1] % kv != 0:
        raise ValueError("q's heads must be a multiple of the cache's")
    return _attend(entry, q, k_cache, v_cache, (("k_scale", k_scale, kv), ("v_scale", v_scale, kv)), lengths, block_table,
                   chosen, next_n, dim ** -0.5 if softmax_scale is None else softmax_scale, kv, dim, out, lse, workspace,
                   max_splits, more[-1:], more[-1:], more)


def paged_attention(q, k_cache, v_cache, block_table, lengths, *, chosen=None, softmax_scale: float | None = None,
                    k_scale=None, v_scale=None, next_n: int | None = None, out=None, lse=None, workspace=None,
                    max_splits: int = 0, stream=None):
    """Attention of each row of q [num_rows, num_heads, head_dim] over the
    first lengths[r] cached positions of its sequence, or over chosen[r]
    (int32 [num_rows, n], as topk_ragged returns it).  Returns (out, lse).

    k_cache, v_cache: [num_pages, page_size, num_kv_heads, head_dim] with the
    same strides, of q's type (bfloat16 or float16) or float8_e4m3fn with
    float32 [num_kv_heads] scales (None: 1); head_dim 64 or 128.  block_table:
    int32 [num_sequences, width].  lengths: int32 [num_rows] or [batch,
    next_n].  softmax_scale: head_dim ** -0.5 if None.  Rows that see nothing
    get zeros and -inf.  workspace: a contiguous tensor for split rows' parts,
    which holds nothing between calls; one that is large enough for a batch is
    for the same call with fewer rows (None: a new one).
    """
    load()
    if (q.requires_grad or k_cache.requires_grad or v_cache.requires_grad
            or (out is not None and out.requires_grad) or (lse is not None and lse.requires_grad)):
        _no_gradients("paged_attention")
    if _elsewhere(q, stream):
        with _on(stream, q):
            return paged_attention(q, k_cache, v_cache, block_table, lengths, chosen=chosen,
                                   softmax_scale=softmax_scale, k_scale=k_scale, v_scale=v_scale, next_n=next_n,
                                   out=out, lse=lse, workspace=workspace, max_splits=max_splits)
    return _paged("paged_attention", q, k_cache, v_cache, block_table, lengths, chosen, softmax_scale, k_scale, v_scale,
                  next_n, out, lse, workspace, max_splits)


def paged_prefix_attention(q, k_cache, v_cache, block_table, lengths, group_starts, shared, *,
                           softmax_scale: float | None = None, k_scale=None, v_scale=None, next_n: int | None = None,
                           out=None, lse=None, workspace=None, max_splits: int = 0, stream=None):
    """paged_attention of sequences that share their first positions: sequences
    [group_starts[g], group_starts[g + 1]) (int32 [num_groups + 1], ascending)
    have the same table entries for their first shared[g] (int32 [num_groups])
    positions, which are read once for all of them.  Sequences that are shorter,
    or in no group, are attended by themselves.  Returns (out, lse); all other
    arguments as for paged_attention."""
    load()
    if (q.requires_grad or k_cache.requires_grad or v_cache.requires_grad
            or (out is not None and out.requires_grad) or (lse is not None and lse.requires_grad)):
        _no_gradients("paged_prefix_attention")
    if _elsewhere(q, stream):
        with _on(stream, q):
            return paged_prefix_attention(q, k_cache, v_cache, block_table, lengths, group_starts, shared,
                                          softmax_scale=softmax_scale, k_scale=k_scale, v_scale=v_scale, next_n=next_n,
                                          out=out, lse=lse, workspace=workspace, max_splits=max_splits)
    dev, groups = q.get_device(), shared.numel()
    return _paged("paged_prefix_attention", q, k_cache, v_cache, block_table, lengths, None, softmax_scale, k_scale, v_scale,
                  next_n, out, lse, workspace, max_splits,
                  (_ints(group_starts, "group_starts", dev, groups + 1), _ints(shared, "shared", dev, groups), groups))


def latent_attention(q, cache, block_table, lengths, *, softmax_scale: float, chosen=None, scale=None,
                     next_n: int | None = None, out=None, lse=None, workspace=None, max_splits: int = 0, stream=None):
    """The absorbed form of latent attention: every head of q [num_rows,
    num_heads, latent_dim + 64] reads the shared vectors of cache [num_pages,
    page_size, latent_dim + 64] as keys and their first latent_dim values as
    values; latent_dim 256 or 512.  Returns (out [num_rows, num_heads,
    latent_dim], lse).  Other arguments as for paged_attention; scale:
    float32 [1] of a float8_e4m3fn cache."""
    load()
    if (q.requires_grad or cache.requires_grad
            or (out is not None and out.requires_grad) or (lse is not None and lse.requires_grad)):
        _no_gradients("latent_attention")
    if _elsewhere(q, stream):
        with _on(stream, q):
            return latent_attention(q, cache, block_table, lengths, softmax_scale=softmax_scale, chosen=chosen,
                                    scale=scale, next_n=next_n, out=out, lse=lse, workspace=workspace,
                                    max_splits=max_splits)
    if cache.dim() != 3:
        raise ValueError("cache must be [num_pages, page_size, latent_dim + 64]")
    return _attend("latent_attention", q, cache, None, (("scale", scale, 1),), lengths, block_table, chosen, next_n,
                   softmax_scale, 1, cache.shape[2] - ROPE_DIM, out, lse, workspace, max_splits)


def latent_prefill(q, cache, block_table, starts, lengths, w_k, w_v, *, context_tokens: int, softmax_scale: float,
                   scale=None, out=None, lse=None, workspace=None, stream=None):
    """The expanded form for chunks of new tokens: causal attention of q
    [num_tokens, num_heads, 192] over each sequence's whole context, whose
    keys [w_k c, rope] and values w_v c are formed from the latent vectors in
    the paged cache.  starts: int32 [num_seqs + 1], lengths: int32 [num_seqs],
    both as paged_layout gives and takes them; w_k, w_v: [num_heads, 128,
    latent_dim]; context_tokens: at least the sum of the lengths.  Returns
    (out [num_tokens, num_heads, 128], lse).  How keys and values are rounded:
    latent_prefill in paged_attention.h."""
    load()
    if (q.requires_grad or cache.requires_grad or w_k.requires_grad or w_v.requires_grad
            or (out is not None and out.requires_grad) or (lse is not None and lse.requires_grad)):
        _no_gradients("latent_prefill")
    if _elsewhere(q, stream):
        with _on(stream, q):
            return latent_prefill(q, cache, block_table, starts, lengths, w_k, w_v, context_tokens=context_tokens,
                                  softmax_scale=softmax_scale, scale=scale, out=out, lse=lse, workspace=workspace)
    dev = q.get_device()
    code, store = _code(q, "q"), _code(cache, "cache", True)
    if store != _E4M3 and store != code:
        raise TypeError("cache must have q's type or float8_e4m3fn")
    if q.dim() != 3 or q.shape[2] != HEAD_DIM + ROPE_DIM or q.stride(2) != 1:
        raise ValueError(f"q must be [num_tokens, num_heads, {HEAD_DIM + ROPE_DIM}], its last stride 1")
    if cache.dim() != 3 or cache.stride(2) != 1 or cache.get_device() != dev:
        raise ValueError("cache must be [num_pages, page_size, latent_dim + 64] on q's device, its last stride 1")
    tokens, heads, dim = q.shape[0], q.shape[1], cache.shape[2] - ROPE_DIM
    for w, name in ((w_k, "w_k"), (w_v, "w_v")):
        _output(w, name, q.dtype, (heads, HEAD_DIM, dim), q)
    n = lengths.numel()
    table_at = _matrix(block_table, "block_table", dev, n)
    by = _scales(scale, "scale", dev, 1, store)
    starts_at, lengths_at = _ints(starts, "starts", dev, n + 1), _ints(lengths, "lengths", dev, n)
    out = _output(out, "out", q.dtype, (tokens, heads, HEAD_DIM), q)
    lse = _output(lse, "lse", torch.float32, (tokens, heads), q)
    args = PrefillArgs(q.data_ptr(), cache.data_ptr(), by, w_k.data_ptr(), w_v.data_ptr(), table_at, starts_at,
                       lengths_at, out.data_ptr(), lse.data_ptr(), q.stride(0), q.stride(1), cache.stride(0),
                       cache.stride(1), block_table.stride(0), context_tokens, tokens, n, heads, dim, cache.shape[1],
                       cache.shape[0], block_table.shape[1], softmax_scale, code, store)
    _launch("latent_prefill", args, workspace,
            (context_tokens, tokens, n, heads, dim, cache.shape[1], block_table.shape[1]), q)
    return out, lse
