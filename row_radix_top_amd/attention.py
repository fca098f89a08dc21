"""ctypes binding of the paged-cache entry points (``include/paged_attention.h``):
block tables and slot maps, cache writes, attention over chosen or all cached
positions, and the latent forms.  As in :mod:`binding`, torch tensors are
device memory and streams, every step of an operator runs in the HIP kernels,
and there is no fallback.

Outputs and workspaces that are not given are allocated by torch on the call's
stream.  Nothing is differentiable.
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
    "paged_debug_place", "paged_debug_split",
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


def load() -> ctypes.CDLL:
    """The built library with these entry points' signatures set."""
    global _lib
    if _lib is None:
        lib = binding.load()
        lib.paged_layout.argtypes = [_vp, _vp, _i32, _vp, _i32, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp,
                                     _vp]
        lib.paged_append.argtypes = [_vp, _i32, ctypes.POINTER(Part), _i32, _i32, _i32, _i32, _i32, _vp]
        for name, args in (("paged_attention", AttentionArgs), ("latent_attention", AttentionArgs),
                           ("latent_prefill", PrefillArgs)):
            if not hasattr(lib, name):
                continue
            getattr(lib, name).argtypes = [ctypes.POINTER(args), _vp, _vp]
            getattr(lib, name + "_workspace_size").argtypes = [ctypes.POINTER(args), _vp,
                                                               ctypes.POINTER(ctypes.c_size_t)]
        for name in EXPORTED:
            if hasattr(lib, name):
                getattr(lib, name).restype = ctypes.c_int
        lib.paged_debug_place.argtypes = [_vp, _i32, _i32, _i64, _i64, _i32]
        lib.paged_debug_place.restype = _i64
        lib.paged_debug_split.argtypes = [_i32, _i32, _i32, _i32, _vp]
        lib.paged_debug_split.restype = None
        _lib = lib
    return _lib


# ---------------------------------------------------------------------------
# Argument checks
# ---------------------------------------------------------------------------

def _dtypes():
    import torch
    return {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2}


_codes = None


def _code(x, name: str, cache: bool = False) -> int:
    global _codes
    if _codes is None:
        _codes = _dtypes()
    code = _codes.get(x.dtype)
    if code is None or (code == 2 and not cache):
        raise TypeError(f"{name} must be bfloat16 or float16" + (" or float8_e4m3fn" if cache else ""))
    return code


def _ints(x, name: str, device, shape=None):
    import torch
    if x.dtype != torch.int32 or x.device != device:
        raise TypeError(f"{name} must be an int32 tensor on {device}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(x.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}")
    return x.data_ptr()


def _matrix(x, name: str, device, rows: int):
    """An int32 [rows, n >= 1] tensor whose rows may be strided."""
    import torch
    if x.dtype != torch.int32 or x.device != device or x.dim() != 2:
        raise TypeError(f"{name} must be a 2-D int32 tensor on {device}")
    if x.shape[0] != rows or x.shape[1] < 1 or (x.stride(1) != 1 and x.shape[1] > 1):
        raise ValueError(f"{name} must be [{rows}, n] with n >= 1 and unit column stride")
    return x.data_ptr()


def _scales(x, name: str, device, n: int, code: int):
    import torch
    if x is None:
        return None
    if code != 2:
        raise ValueError(f"{name} belongs to a float8_e4m3fn cache")
    if x.dtype != torch.float32 or x.device != device or x.numel() != n or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of {n} on {device}")
    return x.data_ptr()


def _like(x, name: str, device, dtype, shape):
    if x.dtype != dtype or x.device != device or tuple(x.shape) != shape or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {device}")
    return x


_null = contextlib.nullcontext()


def _on(stream, device):
    """The call's stream made current (and its device), so that what torch
    allocates for the call belongs to it."""
    import torch
    if device.type != "cuda":
        raise TypeError("tensors must be on a GPU")
    if stream is not None:
        if stream.device != device:
            raise ValueError("stream and tensors must be on the same device")
        return torch.cuda.stream(stream)
    if torch.cuda.current_device() != device.index:
        return torch.cuda.device(device)
    return _null


def _stream(device) -> int:
    import torch
    return torch.cuda.current_stream(device).cuda_stream


def _workspace(fn, args, workspace, device, name: str, sp: int):
    """Pointer of a workspace large enough (and the tensor, to keep it)."""
    import torch
    need = ctypes.c_size_t(0)
    _check(fn(ctypes.byref(args), sp, ctypes.byref(need)), name)
    if need.value == 0:
        return None, None
    if workspace is None:
        workspace = torch.empty(need.value, dtype=torch.uint8, device=device)
    elif (workspace.device != device or not workspace.is_contiguous()
          or workspace.numel() * workspace.element_size() < need.value):
        raise ValueError(f"workspace must be a contiguous tensor of {need.value} bytes or more on {device}")
    return workspace.data_ptr(), workspace


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
    past it are not written.  See paged_layout in paged_attention.h.
    """
    import torch
    device = lengths.device
    with _on(stream, device):
        n = lengths.numel()
        args = (_ints(lengths, "lengths", device), _ints(new_tokens, "new_tokens", device, (n,)), n,
                _ints(free_pages, "free_pages", device), free_pages.numel(),
                _matrix(block_table, "block_table", device, n), block_table.stride(0) if n > 1 else block_table.shape[1],
                block_table.shape[1], page_size, capacity)
        if capacity < 0:
            raise ValueError("capacity must be >= 0")
        if out is None:
            rows = torch.empty((3, capacity), dtype=torch.int32, device=device)
            ends = torch.empty(n + 2, dtype=torch.int32, device=device)
            out = Layout(rows[0], rows[1], rows[2], ends[:n + 1], ends[n + 1:])
        ptrs = [_ints(x, f"out.{name}", device, (size,)) for x, name, size in
                ((out.starts, "starts", n + 1), (out.slots, "slots", capacity),
                 (out.row_lengths, "row_lengths", capacity), (out.row_seqs, "row_seqs", capacity),
                 (out.pages, "pages", 1))]
        _check(load().paged_layout(*args, *ptrs, _stream(device)), "paged_layout")
    return out


def _part(x, name: str, cache, cache_name: str, column: int, heads: int, dim: int, tokens: int, scales) -> Part:
    """x [tokens, heads, dim] (inner dims contiguous) into columns of cache
    [pages, page_size, heads, dim] or [pages, page_size, width]."""
    if x.device != cache.device:
        raise ValueError(f"{name} and {cache_name} must be on the same device")
    if x.shape[0] != tokens or (x.numel() > 0 and not x[0].is_contiguous()):
        raise ValueError(f"{name} must have one contiguous row for each slot")
    if cache.stride(-1) != 1:
        raise ValueError(f"{cache_name} must have unit stride in its last dimension")
    return Part(x.data_ptr(), cache.data_ptr() + column * cache.element_size(), scales, x.stride(0), cache.stride(0),
                cache.stride(1), cache.stride(2) if cache.dim() == 4 else 0, heads * dim, dim)


def _append(slots, parts, cache, code: int, store: int, stream) -> None:
    array = (Part * len(parts))(*parts)
    _check(load().paged_append(_ints(slots, "slots", cache.device), slots.numel(), array, len(parts), cache.shape[1],
                               cache.shape[0], code, store, stream), "paged_append")


def paged_append(slots, k, v, k_cache, v_cache, *, k_scale=None, v_scale=None, stream=None) -> None:
    """Writes keys and values [num_tokens, num_kv_heads, head_dim] (bfloat16
    or float16, rows may be strided) to their slots (int32 [num_tokens], -1 to
    drop a token) of the caches [num_pages, page_size, num_kv_heads, head_dim]
    of the same type or float8_e4m3fn, then as x / scale with float32
    [num_kv_heads] scales (None: 1).  No slot may occur twice."""
    device = k_cache.device
    with _on(stream, device):
        code, store = _code(k, "k"), _code(k_cache, "k_cache", True)
        if v.dtype != k.dtype or v_cache.dtype != k_cache.dtype:
            raise TypeError("k and v, and k_cache and v_cache, must have the same type")
        if k.dim() != 3 or k_cache.dim() != 4 or k.shape != v.shape or k_cache.shape != v_cache.shape:
            raise ValueError("k and v must be [num_tokens, heads, dim], the caches [num_pages, page_size, heads, dim]")
        tokens, heads, dim = k.shape
        if tuple(k_cache.shape[2:]) != (heads, dim) or v_cache.device != device:
            raise ValueError("the caches must have k's heads and dim and be on one device")
        if slots.numel() != tokens:
            raise ValueError("slots must hold one entry for each token")
        _append(slots, [_part(k, "k", k_cache, "k_cache", 0, heads, dim, tokens,
                              _scales(k_scale, "k_scale", device, heads, store)),
                        _part(v, "v", v_cache, "v_cache", 0, heads, dim, tokens,
                              _scales(v_scale, "v_scale", device, heads, store))],
                k_cache, code, store, _stream(device))


def latent_append(slots, latent, rope, cache, *, scale=None, stream=None) -> None:
    """Writes latent vectors [num_tokens, latent_dim] and their rope parts
    [num_tokens, 64] to their slots of cache [num_pages, page_size, latent_dim
    + 64], as paged_append does; scale: float32 [1]."""
    device = cache.device
    with _on(stream, device):
        code, store = _code(latent, "latent"), _code(cache, "cache", True)
        if rope.dtype != latent.dtype:
            raise TypeError("latent and rope must have the same type")
        if latent.dim() != 2 or rope.dim() != 2 or cache.dim() != 3:
            raise ValueError("latent and rope must be 2-D and cache 3-D")
        tokens, dim = latent.shape
        if rope.shape[1] != ROPE_DIM or cache.shape[2] != dim + ROPE_DIM:
            raise ValueError(f"rope must have {ROPE_DIM} columns and cache latent's and rope's together")
        if slots.numel() != tokens:
            raise ValueError("slots must hold one entry for each token")
        by = _scales(scale, "scale", device, 1, store)
        _append(slots, [_part(latent, "latent", cache, "cache", 0, 1, dim, tokens, by),
                        _part(rope, "rope", cache, "cache", dim, 1, ROPE_DIM, tokens, by)],
                cache, code, store, _stream(device))


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------

def _attention_args(q, k, lengths, block_table, chosen, next_n, softmax_scale, dim: int, value_dim: int, out, lse,
                    max_splits: int):
    import torch
    device = q.device
    code, store = _code(q, "q"), _code(k, "the cache", True)
    if store != 2 and k.dtype != q.dtype:
        raise TypeError("the cache must have q's type or float8_e4m3fn")
    if k.device != device:
        raise ValueError("q and the cache must be on the same device")
    if q.dim() != 3 or q.shape[2] != dim or q.stride(2) != 1:
        raise ValueError(f"q must be [num_rows, num_heads, {dim}] with unit stride in its last dimension")
    if k.stride(-1) != 1:
        raise ValueError("the cache must have unit stride in its last dimension")
    rows, heads = q.shape[0], q.shape[1]
    if next_n is None:
        next_n = int(lengths.shape[1]) if lengths.dim() == 2 else 1
    if lengths.numel() != rows:
        raise ValueError("lengths must hold one entry for each row of q")
    if next_n < 1 or rows % next_n != 0:
        raise ValueError("next_n must be >= 1 and divide the rows")
    a = AttentionArgs()
    a.q, a.k = q.data_ptr(), k.data_ptr()
    a.lengths = _ints(lengths, "lengths", device)
    a.block_table = _matrix(block_table, "block_table", device, rows // next_n)
    a.table_stride, a.table_width = block_table.stride(0), block_table.shape[1]
    if chosen is not None:
        a.chosen = _matrix(chosen, "chosen", device, rows)
        a.chosen_stride, a.num_chosen = chosen.stride(0), chosen.shape[1]
    if out is None:
        out = torch.empty((rows, heads, value_dim), dtype=q.dtype, device=device)
    else:
        _like(out, "out", device, q.dtype, (rows, heads, value_dim))
    if lse is None:
        lse = torch.empty((rows, heads), dtype=torch.float32, device=device)
    else:
        _like(lse, "lse", device, torch.float32, (rows, heads))
    a.out, a.lse = out.data_ptr(), lse.data_ptr()
    a.q_row_stride, a.q_head_stride = q.stride(0), q.stride(1)
    a.page_stride, a.token_stride = k.stride(0), k.stride(1)
    a.num_rows, a.next_n, a.num_heads, a.num_kv_heads, a.head_dim = rows, next_n, heads, 1, value_dim
    a.num_pages, a.page_size = k.shape[0], k.shape[1]
    a.softmax_scale, a.dtype, a.store, a.max_splits = softmax_scale, code, store, max_splits
    return a, out, lse


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
    get zeros and -inf.
    """
    device = q.device
    with _on(stream, device):
        if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.stride() != v_cache.stride():
            raise ValueError("k_cache and v_cache must be [num_pages, page_size, num_kv_heads, head_dim], alike")
        if v_cache.dtype != k_cache.dtype or v_cache.device != device:
            raise TypeError("k_cache and v_cache must have the same type and device")
        kv, dim = k_cache.shape[2], k_cache.shape[3]
        if kv < 1 or q.dim() != 3 or q.shape[1] % kv != 0:
            raise ValueError("q's heads must be a multiple of the cache's")
        a, out, lse = _attention_args(q, k_cache, lengths, block_table, chosen, next_n,
                                      dim ** -0.5 if softmax_scale is None else softmax_scale, dim, dim, out, lse,
                                      max_splits)
        a.v, a.num_kv_heads, a.head_stride = v_cache.data_ptr(), kv, k_cache.stride(2)
        a.k_scales = _scales(k_scale, "k_scale", device, kv, a.store)
        a.v_scales = _scales(v_scale, "v_scale", device, kv, a.store)
        lib, sp = load(), _stream(device)
        ws, _keep = _workspace(lib.paged_attention_workspace_size, a, workspace, device, "paged_attention", sp)
        _check(lib.paged_attention(ctypes.byref(a), ws, sp), "paged_attention")
    return out, lse


def latent_attention(q, cache, block_table, lengths, *, softmax_scale: float, chosen=None, scale=None,
                     next_n: int | None = None, out=None, lse=None, workspace=None, max_splits: int = 0, stream=None):
    """The absorbed form of latent attention: every head of q [num_rows,
    num_heads, latent_dim + 64] reads the shared vectors of cache [num_pages,
    page_size, latent_dim + 64] as keys and their first latent_dim values as
    values; latent_dim 256 or 512.  Returns (out [num_rows, num_heads,
    latent_dim], lse).  Other arguments as for paged_attention; scale:
    float32 [1] of a float8_e4m3fn cache."""
    device = q.device
    with _on(stream, device):
        if cache.dim() != 3:
            raise ValueError("cache must be [num_pages, page_size, latent_dim + 64]")
        dim = cache.shape[2]
        a, out, lse = _attention_args(q, cache, lengths, block_table, chosen, next_n, softmax_scale, dim,
                                      dim - ROPE_DIM, out, lse, max_splits)
        a.k_scales = _scales(scale, "scale", device, 1, a.store)
        lib, sp = load(), _stream(device)
        ws, _keep = _workspace(lib.latent_attention_workspace_size, a, workspace, device, "latent_attention", sp)
        _check(lib.latent_attention(ctypes.byref(a), ws, sp), "latent_attention")
    return out, lse


def latent_prefill(q, cache, block_table, starts, lengths, w_k, w_v, *, context_tokens: int, softmax_scale: float,
                   scale=None, out=None, lse=None, workspace=None, stream=None):
    """The expanded form for chunks of new tokens: causal attention of q
    [num_tokens, num_heads, 192] over each sequence's whole context, whose
    keys [w_k c, rope] and values w_v c are formed from the latent vectors in
    the paged cache.  starts: int32 [num_seqs + 1], lengths: int32 [num_seqs],
    both as paged_layout gives and takes them; w_k, w_v: [num_heads, 128,
    latent_dim]; context_tokens: at least the sum of the lengths.  Returns
    (out [num_tokens, num_heads, 128], lse).  See paged_attention.h."""
    import torch
    device = q.device
    with _on(stream, device):
        code, store = _code(q, "q"), _code(cache, "cache", True)
        if store != 2 and cache.dtype != q.dtype:
            raise TypeError("cache must have q's type or float8_e4m3fn")
        if q.dim() != 3 or q.shape[2] != HEAD_DIM + ROPE_DIM or q.stride(2) != 1:
            raise ValueError(f"q must be [num_tokens, num_heads, {HEAD_DIM + ROPE_DIM}], its last stride 1")
        if cache.dim() != 3 or cache.stride(2) != 1 or cache.device != device:
            raise ValueError("cache must be [num_pages, page_size, latent_dim + 64] on q's device, its last stride 1")
        tokens, heads, dim = q.shape[0], q.shape[1], cache.shape[2] - ROPE_DIM
        for w, name in ((w_k, "w_k"), (w_v, "w_v")):
            _like(w, name, device, q.dtype, (heads, HEAD_DIM, dim))
        n = lengths.numel()
        a = PrefillArgs()
        a.q, a.cache, a.w_k, a.w_v = q.data_ptr(), cache.data_ptr(), w_k.data_ptr(), w_v.data_ptr()
        a.lengths, a.starts = _ints(lengths, "lengths", device), _ints(starts, "starts", device, (n + 1,))
        a.block_table = _matrix(block_table, "block_table", device, n)
        a.scale = _scales(scale, "scale", device, 1, store)
        if out is None:
            out = torch.empty((tokens, heads, HEAD_DIM), dtype=q.dtype, device=device)
        else:
            _like(out, "out", device, q.dtype, (tokens, heads, HEAD_DIM))
        if lse is None:
            lse = torch.empty((tokens, heads), dtype=torch.float32, device=device)
        else:
            _like(lse, "lse", device, torch.float32, (tokens, heads))
        a.out, a.lse = out.data_ptr(), lse.data_ptr()
        a.q_row_stride, a.q_head_stride = q.stride(0), q.stride(1)
        a.page_stride, a.token_stride, a.table_stride = cache.stride(0), cache.stride(1), block_table.stride(0)
        a.context_tokens, a.num_tokens, a.num_seqs, a.num_heads, a.latent_dim = context_tokens, tokens, n, heads, dim
        a.num_pages, a.page_size, a.table_width = cache.shape[0], cache.shape[1], block_table.shape[1]
        a.softmax_scale, a.dtype, a.store = softmax_scale, code, store
        lib, sp = load(), _stream(device)
        ws, _keep = _workspace(lib.latent_prefill_workspace_size, a, workspace, device, "latent_prefill", sp)
        _check(lib.latent_prefill(ctypes.byref(a), ws, sp), "latent_prefill")
    return out, lse
