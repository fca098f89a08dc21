"""Outputs and inputs of the page operators that share memory are refused, by
their ranges: the kernels write some outputs while other workgroups still read."""

from __future__ import annotations

import numpy as np
import pytest

import row_radix_top_amd as rrt
from row_radix_top_amd import binding
from tests.gpu_util import require_gpu
from tests.test_shared_refusals import COMPACT, COMPACT_BASE, EINVAL, FORK, FORK_BASE, FREE, FREE_BASE, _call

# Every array at a place of its own; three rows of four entries from two, eight free pages.
APART = dict(FORK_BASE, block_table=0x1000, lengths=0x2000, parents=0x3000, keep=0x4000, free_pages=0x5000, num_free=8,
             out_table=0x6000, out_lengths=0x7000, src=0x8000, dst=0x9000, tokens=0xa000, pages=0xb000)


@pytest.mark.parametrize("out", ["out_table", "out_lengths", "src", "dst", "tokens", "pages"])
@pytest.mark.parametrize("inp,last", [("block_table", 28), ("lengths", 4), ("parents", 8), ("keep", 8), ("free_pages", 28)])
def test_forks_over_what_they_read(out, inp, last):
    for at in (0, last):  # its first entry and its last
        assert _call("paged_fork", FORK, APART, {out: APART[inp] + at}) == EINVAL
        assert "goes on from" in binding.last_error()


@pytest.mark.parametrize("a,b", [("out_lengths", "src"), ("src", "dst"), ("dst", "tokens"), ("tokens", "out_table"),
                                 ("pages", "out_table"), ("out_lengths", "pages")])
def test_forks_over_their_own_outputs(a, b):
    assert _call("paged_fork", FORK, APART, {a: APART[b]}) == EINVAL
    assert "goes on from" in binding.last_error()


@pytest.mark.parametrize("changes", [dict(table_stride=20, out_stride=20, out_table=0x1000 + 4 * 3),
                                     dict(table_stride=20, out_stride=20, out_table=0x1000 + 4 * 17),
                                     dict(table_stride=9, out_stride=7, out_table=0x1000 - 4 * 9),
                                     dict(out_stride=9, out_table=0x2000 - 4 * 18)])
def test_strided_tables_that_meet(changes):
    assert _call("paged_fork", FORK, APART, changes) == EINVAL
    assert "goes on from" in binding.last_error()


POOL = dict(FREE_BASE, block_table=0x1000, lengths=0x2000, free_pages=0x3000, refs=0x4000, count=0x5000, workspace=0x6000)


@pytest.mark.parametrize("changes", [dict(free_pages=0x2000), dict(refs=0x1000), dict(count=0x2004), dict(workspace=0x1010),
                                     dict(refs=0x3020), dict(count=0x4020), dict(free_pages=0x1000 - 32)])
def test_free_lists_over_what_they_read(changes):
    assert _call("paged_free", FREE, POOL, changes) == EINVAL
    assert "overlap" in binding.last_error()


MOVES = dict(COMPACT_BASE, block_table=0x1000, lengths=0x2000, out_table=0x3000, src=0x4000, dst=0x5000, moves=0x6000,
             live=0x7000, workspace=0x8000)


@pytest.mark.parametrize("changes", [dict(out_table=0x1004), dict(out_table=0x1000 - 16), dict(src=0x2000), dict(dst=0x1010),
                                     dict(moves=0x2004), dict(live=0x101c), dict(workspace=0x1000), dict(src=0x5000),
                                     dict(live=0x6000), dict(out_table=0x2000), dict(src=0x3000),
                                     dict(out_table=0x1000, src=0x1008), dict(out_table=0x1000, lengths=0x1000),
                                     dict(out_table=0x1000, workspace=0x1010)])
def test_moves_over_what_they_read(changes):
    assert _call("paged_compact", COMPACT, MOVES, changes) == EINVAL
    assert "overlap" in binding.last_error()


@pytest.mark.gpu
def test_views_beside_one_another_are_taken():
    """Two tables side by side in one buffer, and all lists in one allocation."""
    import torch
    require_gpu()
    i32 = lambda x: torch.as_tensor(np.asarray(x), device="cuda").to(torch.int32)  # noqa: E731
    both = torch.full((3, 2, 4), 9, dtype=torch.int32, device="cuda")
    both[:2, 0] = i32([[3, 4, -1, -1], [5, 6, 7, -1]])
    lists = torch.zeros(25, dtype=torch.int32, device="cuda")
    lists[:2] = i32([20, 40])
    lists[2:5] = i32([0, 0, 1])
    lists[5:8] = i32([10, 11, 12])
    n, parents, free, lengths, src, dst, tokens, pages = lists[:21].split([2, 3, 3, 3, 3, 3, 3, 1])
    out = rrt.Fork(both[:, 1], lengths, src, dst, tokens, pages)
    rrt.paged_fork(both[:2, 0], n, parents, free, page_size=16, out=out)
    assert both[:, 1].tolist() == [[3, 4, -1, -1], [3, 10, -1, -1], [5, 6, 7, -1]]
    assert both[:2, 0].tolist() == [[3, 4, -1, -1], [5, 6, 7, -1]]
    assert (lengths.tolist(), src.tolist(), dst.tolist(), tokens.tolist()) == ([20, 20, 40], [-1, 4, -1], [-1, 10, -1], [0, 4, 0])
    moved = rrt.paged_compact(both[:, 1], lengths, page_size=16, num_pages=12,
                              out=rrt.Compact(both[:, 0], *(i32([0] * k) for k in (6, 6, 1, 1))))
    again = rrt.paged_compact(both[:, 1], lengths, page_size=16, num_pages=12)
    assert torch.equal(moved.table, again.table) and both[:, 1].tolist()[0] == [3, 4, -1, -1]
