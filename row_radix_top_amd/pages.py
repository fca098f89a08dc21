"""ctypes binding of the operators on pages that sequences share: forks, copies,
the free list, and moves that bring the held pages together
(``include/paged_attention.h``).  Checks, streams and allocation as in
:mod:`attention`.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

from . import attention as _pa
from .attention import _elsewhere, _ints, _matrix, _no_gradients, _on, load
from .binding import _check

COPY_CACHES = 32  # of one launch

_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class PagedPages(ctypes.Structure):
    _fields_ = [("data", _vp), ("page_stride", _i64), ("token_stride", _i64), ("outer_stride", _i64), ("tokens", _i32),
                ("outer", _i32), ("width", _i32)]


class Fork(NamedTuple):
    """The rows of a new batch and the pages to copy for them."""

    table: "torch.Tensor"  # noqa: F821  int32 [num_rows, width]
    lengths: "torch.Tensor"  # noqa: F821  int32 [num_rows]
    src: "torch.Tensor"  # noqa: F821  int32 [num_rows], -1 where nothing is copied
    dst: "torch.Tensor"  # noqa: F821  int32 [num_rows]
    tokens: "torch.Tensor"  # noqa: F821  int32 [num_rows], of the copied page
    pages: "torch.Tensor"  # noqa: F821  int32 [1], pages the call needs


class Pages(NamedTuple):
    """What of a pool is free."""

    free: "torch.Tensor"  # noqa: F821  int32 [num_pages], ascending, -1 past the last
    refs: "torch.Tensor"  # noqa: F821  int32 [num_pages], entries that hold each page
    count: "torch.Tensor"  # noqa: F821  int32 [1], free pages


class Compact(NamedTuple):
    """A table whose pages have moved, and the moves."""

    table: "torch.Tensor"  # noqa: F821  int32 [num_sequences, width]
    src: "torch.Tensor"  # noqa: F821  int32 [num_pages // 2], -1 past the last move
    dst: "torch.Tensor"  # noqa: F821  int32 [num_pages // 2]
    moves: "torch.Tensor"  # noqa: F821  int32 [1]
    live: "torch.Tensor"  # noqa: F821  int32 [1], pages that are held


def _new(x, *sizes):
    """int32 tensors of these sizes from one allocation on x's device."""
    whole = _pa.torch.empty(sum(sizes), dtype=_pa.torch.int32, device=x.device)
    return whole.split_with_sizes(list(sizes))


def _table_out(x, name: str, dev: int, rows: int, width: int):
    at = _matrix(x, name, dev, rows)
    if x.shape[1] != width:
        raise ValueError(f"{name} must be [{rows}, {width}]")
    return at


def paged_fork(block_table, lengths, parents, free_pages, *, page_size: int, keep=None, out: Fork | None = None,
               stream=None) -> Fork:
    """Rows of a new batch that go on from rows of the last one.

    Row i takes over the pages of row parents[i] (int32 [num_rows]; outside
    the table: an empty row) for its first keep[i] tokens (int32 [num_rows];
    None: all).  Full pages are shared.  A last page that is not full is the
    row's own: the parent's where no other row of the new batch needs it, else
    the next of free_pages (int32), to be filled with

        paged_copy(fork.src, fork.dst, caches, tokens=fork.tokens)

    block_table (int32 [num_sequences, width]) and lengths stay as they are;
    rows that nothing goes on from are given up (paged_free finds their pages).
    Where fork.pages is more than free_pages has (its entries, or paged_free's
    count, whose list is padded with -1), the list ran out: a row without its
    last page has -1 there.
    """
    lib = load()
    if _elsewhere(lengths, stream):
        with _on(stream, lengths):
            return paged_fork(block_table, lengths, parents, free_pages, page_size=page_size, keep=keep, out=out)
    dev, n, rows = lengths.get_device(), lengths.numel(), parents.numel()
    table_at = _matrix(block_table, "block_table", dev, n)
    width = block_table.shape[1]
    if out is None:
        table, *rest = _new(lengths, rows * width, rows, rows, rows, rows, 1)
        out = Fork(table.view(rows, width), *rest)
    out_at = _table_out(out.table, "out.table", dev, rows, width)
    _check(lib.paged_fork(table_at, block_table.stride(0) if n > 1 else width, width, _ints(lengths, "lengths", dev, n),
                          n, _ints(parents, "parents", dev, rows),
                          None if keep is None else _ints(keep, "keep", dev, rows), rows,
                          _ints(free_pages, "free_pages", dev, free_pages.numel()), free_pages.numel(), page_size, out_at,
                          out.table.stride(0) if rows > 1 else width, _ints(out.lengths, "out.lengths", dev, rows),
                          _ints(out.src, "out.src", dev, rows), _ints(out.dst, "out.dst", dev, rows),
                          _ints(out.tokens, "out.tokens", dev, rows), _ints(out.pages, "out.pages", dev, 1),
                          _pa.torch._C._cuda_getCurrentRawStream(dev)), "paged_fork")
    return out


def _pages_of(x, num_pages: int, tokens: bool, dev: int) -> PagedPages:
    """x [num_pages, (page_size,) ...] as rows of bytes: a token's dims come down to strided rows of one width."""
    if x.get_device() != dev:
        raise ValueError("src and the caches must be on one device")
    shape, stride, size = x.shape, x.stride(), x.element_size()
    if len(shape) < (2 if tokens else 1) or shape[0] != num_pages:
        raise ValueError(f"a cache must be [{num_pages}, {'page_size, ' if tokens else ''}...]")
    count, step = (shape[1], stride[1]) if tokens else (1, 0)
    width, outer, outer_step = 1, 1, 0
    for n, by in zip(reversed(shape[2 if tokens else 1:]), reversed(stride[2 if tokens else 1:])):
        if n == 1:
            continue
        if outer == 1 and by == width:
            width *= n
        elif outer == 1 or by == outer * outer_step:
            outer_step = by if outer == 1 else outer_step
            outer *= n
        else:
            raise ValueError("a cache's token must be contiguous, or rows of contiguous elements one stride apart")
    if num_pages > 0 and x.numel() == 0:
        raise ValueError("a cache must not be empty")
    if not x.is_contiguous():
        # Every step passes what lies within it.
        span = width
        for by, n in sorted(((outer_step, outer), (step, count), (stride[0], num_pages))):
            if n > 1 and by < span:
                raise ValueError("a cache's elements must not share memory")
            span += by * (n - 1)
    return PagedPages(x.data_ptr(), stride[0] * size, step * size, outer_step * size, count, outer, width * size)


def paged_copy(src, dst, caches, *, tokens=None, stream=None) -> None:
    """Copies pages src[i] to pages dst[i] (int32 [num_pairs]; -1: no pair) of
    every cache: a sequence of tensors [num_pages, page_size, ...] of any types,
    keys, values and layers alike.  tokens: int32 [num_pairs], how many of a
    page's tokens are copied (None: whole pages; the caches may then be
    [num_pages, ...] of anything, a page's bounds among it).  No page is the dst
    of two pairs, or of one and the src of another."""
    lib = load()
    if len(caches) == 0:
        return
    if any(x.requires_grad for x in caches):
        _no_gradients("paged_copy")
    if _elsewhere(src, stream):
        with _on(stream, src):
            return paged_copy(src, dst, caches, tokens=tokens)
    dev, pairs = src.get_device(), src.numel()
    src_at, dst_at = _ints(src, "src", dev, pairs), _ints(dst, "dst", dev, pairs)
    tokens_at = None if tokens is None else _ints(tokens, "tokens", dev, pairs)
    num_pages = caches[0].shape[0]
    parts = [_pages_of(x, num_pages, tokens is not None, dev) for x in caches]
    _check(lib.paged_copy(src_at, dst_at, tokens_at, pairs, (PagedPages * len(parts))(*parts), len(parts), num_pages,
                          _pa.torch._C._cuda_getCurrentRawStream(dev)), "paged_copy")


def _workspace(name: str, num_pages: int, workspace, like):
    need = ctypes.c_size_t(0)
    _check(getattr(_pa._lib, name + "_workspace_size")(num_pages, need), name)
    need = need.value
    if workspace is None:
        workspace = _pa.torch.empty(need, dtype=_pa.torch.uint8, device=like.device)
    elif (workspace.get_device() != like.get_device() or not workspace.is_contiguous()
          or workspace.numel() * workspace.element_size() < need):
        raise ValueError(f"workspace must be a contiguous tensor of {need} bytes or more on {like.device}")
    return workspace


def paged_free(block_table, lengths, *, page_size: int, num_pages: int, out: Pages | None = None, workspace=None,
               stream=None) -> Pages:
    """The pages of a pool of num_pages that no row of block_table (int32
    [num_sequences, width]) holds, in ascending order, as paged_layout and
    paged_fork take them.  A row holds the pages of its first lengths[s] tokens:
    rows that ended have length 0.  workspace: as for paged_attention; its size
    depends on num_pages alone."""
    lib = load()
    if _elsewhere(lengths, stream):
        with _on(stream, lengths):
            return paged_free(block_table, lengths, page_size=page_size, num_pages=num_pages, out=out,
                              workspace=workspace)
    if num_pages < 0:
        raise ValueError("num_pages must be >= 0")
    dev, n = lengths.get_device(), lengths.numel()
    table_at = _matrix(block_table, "block_table", dev, n)
    width = block_table.shape[1]
    workspace = _workspace("paged_free", num_pages, workspace, lengths)
    if out is None:
        out = Pages(*_new(lengths, num_pages, num_pages, 1))
    _check(lib.paged_free(table_at, block_table.stride(0) if n > 1 else width, width, _ints(lengths, "lengths", dev, n),
                          n, page_size, num_pages, _ints(out.free, "out.free", dev, num_pages),
                          _ints(out.refs, "out.refs", dev, num_pages), _ints(out.count, "out.count", dev, 1),
                          workspace.data_ptr(), _pa.torch._C._cuda_getCurrentRawStream(dev)), "paged_free")
    return out


def paged_compact(block_table, lengths, *, page_size: int, num_pages: int, limit: int | None = None,
                  out: Compact | None = None, workspace=None, stream=None) -> Compact:
    """Held pages from `limit` on (None: the number of held pages) move to free
    ones below it, in ascending order, for as long as there are both.  Returns
    the table with their new numbers (a new one, or out.table, which may be
    block_table itself) and the moves, for

        paged_copy(compact.src, compact.dst, caches)
    """
    lib = load()
    if _elsewhere(lengths, stream):
        with _on(stream, lengths):
            return paged_compact(block_table, lengths, page_size=page_size, num_pages=num_pages, limit=limit, out=out,
                                 workspace=workspace)
    if num_pages < 0:
        raise ValueError("num_pages must be >= 0")
    if limit is not None and limit < 0:
        raise ValueError("limit must be >= 0")
    dev, n = lengths.get_device(), lengths.numel()
    table_at = _matrix(block_table, "block_table", dev, n)
    width = block_table.shape[1]
    workspace = _workspace("paged_compact", num_pages, workspace, lengths)
    if out is None:
        table, *rest = _new(lengths, n * width, num_pages // 2, num_pages // 2, 1, 1)
        out = Compact(table.view(n, width), *rest)
    out_at = _table_out(out.table, "out.table", dev, n, width)
    _check(lib.paged_compact(table_at, block_table.stride(0) if n > 1 else width, width,
                             _ints(lengths, "lengths", dev, n), n, page_size, num_pages, -1 if limit is None else limit,
                             out_at, out.table.stride(0) if n > 1 else width,
                             _ints(out.src, "out.src", dev, num_pages // 2),
                             _ints(out.dst, "out.dst", dev, num_pages // 2), _ints(out.moves, "out.moves", dev, 1),
                             _ints(out.live, "out.live", dev, 1), workspace.data_ptr(),
                             _pa.torch._C._cuda_getCurrentRawStream(dev)), "paged_compact")
    return out
