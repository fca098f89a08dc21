"""ctypes binding of attention over pages that a cheap score chooses: bounds of the
cache's pages, the choice, and the attention over the chosen pages
(``include/paged_attention.h``).  Checks, streams and allocation as in
:mod:`attention`.
"""

from __future__ import annotations

import ctypes

from . import attention as _pa
from .attention import _code, _elsewhere, _ints, _launch, _matrix, _no_gradients, _on, _paged, load
from .binding import _check

_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class BoundsArgs(ctypes.Structure):
    _fields_ = [("k", _vp), ("block_table", _vp), ("starts", _vp), ("lengths", _vp), ("bounds", _vp), ("scales", _vp),
                ("page_stride", _i64), ("token_stride", _i64), ("head_stride", _i64), ("bounds_page_stride", _i64),
                ("bounds_head_stride", _i64), ("scales_stride", _i64), ("table_stride", _i64), ("num_seqs", _i32),
                ("num_tokens", _i32), ("num_kv_heads", _i32), ("head_dim", _i32), ("page_size", _i32),
                ("num_pages", _i32), ("table_width", _i32), ("store", _i32)]


class SelectArgs(ctypes.Structure):
    _fields_ = [("q", _vp), ("bounds", _vp), ("scales", _vp), ("block_table", _vp), ("lengths", _vp), ("blocks", _vp),
                ("q_row_stride", _i64), ("q_head_stride", _i64), ("bounds_page_stride", _i64),
                ("bounds_head_stride", _i64), ("scales_stride", _i64), ("table_stride", _i64), ("num_rows", _i32),
                ("next_n", _i32), ("num_heads", _i32), ("num_kv_heads", _i32), ("head_dim", _i32), ("page_size", _i32),
                ("num_pages", _i32), ("table_width", _i32), ("num_blocks", _i32), ("first", _i32), ("last", _i32),
                ("dtype", _i32)]


def _bounds(bounds, scales, dev: int, pages: int | None, kv: int | None, dim: int):
    """Checks bounds [pages, kv, 2, dim] and scales [pages, kv]; their pointers and strides."""
    shape = bounds.shape
    if bounds.dtype is not _pa.torch.int8 or bounds.get_device() != dev or len(shape) != 4:
        raise TypeError(f"bounds must be a 4-D int8 tensor on cuda:{dev}")
    if scales.dtype is not _pa.torch.float32 or scales.get_device() != dev or scales.dim() != 2:
        raise TypeError(f"scales must be a 2-D float32 tensor on cuda:{dev}")
    stride = bounds.stride()
    if (shape[2:] != (2, dim) or (pages is not None and shape[:2] != (pages, kv)) or scales.shape != shape[:2]
            or stride[3] != 1 or stride[2] != dim or (scales.stride(1) != 1 and shape[1] > 1)):
        raise ValueError(f"bounds must be [num_pages, num_kv_heads, 2, {dim}] with contiguous pairs, scales "
                         "[num_pages, num_kv_heads] with unit column stride")
    if scales.requires_grad:
        _no_gradients("scales")
    return bounds.data_ptr(), scales.data_ptr(), stride[0], stride[1], scales.stride(0)


def paged_bounds(k_cache, block_table, starts, lengths, bounds, scales, *, num_tokens: int, stream=None) -> None:
    """Bounds of the pages that hold a step's new tokens, from all their tokens
    in k_cache [num_pages, page_size, num_kv_heads, head_dim] (bfloat16, float16
    or float8_e4m3fn; head_dim 64 or 128), into bounds (int8 [num_pages,
    num_kv_heads, 2, head_dim]: each dim's largest and smallest value, rounded
    outward) and scales (float32 [num_pages, num_kv_heads]).

    Called after the step's paged_append: starts (int32 [num_seqs + 1]) and
    lengths (int32 [num_seqs]) as paged_layout gives and takes them, num_tokens
    its capacity: new tokens past it count in no bounds.  See paged_bounds in
    paged_attention.h."""
    lib = load()
    if k_cache.requires_grad:
        _no_gradients("paged_bounds")
    if _elsewhere(k_cache, stream):
        with _on(stream, k_cache):
            return paged_bounds(k_cache, block_table, starts, lengths, bounds, scales, num_tokens=num_tokens)
    dev = k_cache.get_device()
    store = _code(k_cache, "k_cache", True)
    shape, stride = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or stride[3] != 1:
        raise ValueError("k_cache must be [num_pages, page_size, num_kv_heads, head_dim], its last stride 1")
    n = lengths.numel()
    at = _bounds(bounds, scales, dev, shape[0], shape[2], shape[3])
    args = BoundsArgs(k_cache.data_ptr(), _matrix(block_table, "block_table", dev, n), _ints(starts, "starts", dev, n + 1),
                      _ints(lengths, "lengths", dev, n), at[0], at[1], stride[0], stride[1], stride[2], at[2], at[3], at[4],
                      block_table.stride(0), n, num_tokens, shape[2], shape[3], shape[1], shape[0], block_table.shape[1],
                      store)
    _check(lib.paged_bounds(ctypes.byref(args), _pa.torch._C._cuda_getCurrentRawStream(dev)), "paged_bounds")


def paged_block_select(q, bounds, scales, block_table, lengths, *, page_size: int, num_blocks: int, first: int = 1,
                       last: int = 1, next_n: int | None = None, out=None, workspace=None, stream=None):
    """For each row of q [num_rows, num_heads, head_dim] and key-value head the
    num_blocks pages of its sequence (0 for its first page_size positions) with
    the largest score by bounds and scales, as paged_bounds keeps them: int32
    [num_rows, num_kv_heads, num_blocks], ascending, -1 past the last.

    A block's score is the largest, over the heads that share the key-value
    head, of what no key within its bounds can pass: a sum of whole numbers, q
    rounded to 8 bits too, so that choices repeat bit for bit.  The row's first
    `first` and last `last` blocks are always among them.  lengths and next_n as
    for paged_attention.  See paged_block_select in paged_attention.h."""
    load()
    if q.requires_grad:
        _no_gradients("paged_block_select")
    if _elsewhere(q, stream):
        with _on(stream, q):
            return paged_block_select(q, bounds, scales, block_table, lengths, page_size=page_size, num_blocks=num_blocks,
                                      first=first, last=last, next_n=next_n, out=out, workspace=workspace)
    dev, code = q.get_device(), _code(q, "q")
    if q.dim() != 3 or q.stride(2) != 1:
        raise ValueError("q must be [num_rows, num_heads, head_dim] with unit stride in its last dimension")
    rows, heads, dim = q.shape
    at = _bounds(bounds, scales, dev, None, None, dim)
    pages, kv = scales.shape
    if next_n is None:
        next_n = int(lengths.shape[1]) if lengths.dim() == 2 else 1
    if next_n < 1 or rows % next_n != 0:
        raise ValueError("next_n must be >= 1 and divide the rows")
    if num_blocks < 1:
        raise ValueError("num_blocks must be >= 1")
    table_at = _matrix(block_table, "block_table", dev, rows // next_n)
    width = block_table.shape[1]
    if out is None:
        out = _pa.torch.empty((rows, kv, num_blocks), dtype=_pa.torch.int32, device=q.device)
    elif out.shape != (rows, kv, num_blocks):
        raise ValueError(f"out must be [{rows}, {kv}, {num_blocks}]")
    args = SelectArgs(q.data_ptr(), at[0], at[1], table_at, _ints(lengths, "lengths", dev, rows),
                      _ints(out, "out", dev, rows * kv * num_blocks), q.stride(0), q.stride(1), at[2], at[3], at[4],
                      block_table.stride(0), rows, next_n, heads, kv, dim, page_size, pages, width, num_blocks, first, last,
                      code)
    _launch("paged_block_select", args, workspace, (rows, next_n, heads, kv, dim, width), q)
    return out


def paged_block_attention(q, k_cache, v_cache, block_table, lengths, blocks, *, softmax_scale: float | None = None,
                          k_scale=None, v_scale=None, next_n: int | None = None, out=None, lse=None, workspace=None,
                          max_splits: int = 0, stream=None):
    """paged_attention over chosen pages: row r and key-value head g read the
    positions below lengths[r] of the blocks blocks[r, g] (int32 [num_rows,
    num_kv_heads, n], as paged_block_select returns it; blocks outside the row
    are left out).  Returns (out, lse); all other arguments as for
    paged_attention."""
    load()
    if (q.requires_grad or k_cache.requires_grad or v_cache.requires_grad
            or (out is not None and out.requires_grad) or (lse is not None and lse.requires_grad)):
        _no_gradients("paged_block_attention")
    if _elsewhere(q, stream):
        with _on(stream, q):
            return paged_block_attention(q, k_cache, v_cache, block_table, lengths, blocks, softmax_scale=softmax_scale,
                                         k_scale=k_scale, v_scale=v_scale, next_n=next_n, out=out, lse=lse,
                                         workspace=workspace, max_splits=max_splits)
    rows, kv = q.shape[0], k_cache.shape[2] if k_cache.dim() == 4 else 0
    if blocks.dtype is not _pa.torch.int32 or blocks.get_device() != q.get_device() or blocks.dim() != 3:
        raise TypeError(f"blocks must be a 3-D int32 tensor on {q.device}")
    if blocks.shape[0] != rows or blocks.shape[1] != kv or blocks.shape[2] < 1 or (blocks.stride(2) != 1
                                                                                   and blocks.shape[2] > 1):
        raise ValueError(f"blocks must be [{rows}, {kv}, n] with n >= 1 and unit stride in its last dimension")
    return _paged("paged_block_attention", q, k_cache, v_cache, block_table, lengths, None, softmax_scale, k_scale,
                  v_scale, next_n, out, lse, workspace, max_splits,
                  (blocks.data_ptr(), blocks.stride(0), blocks.stride(1), blocks.shape[2]))
