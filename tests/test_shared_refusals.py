"""Arguments that the entry points on shared and chosen pages refuse, through
the C ABI and without a GPU: every check comes before anything touches a device."""

from __future__ import annotations

import ctypes

import pytest

from row_radix_top_amd import attention as pa
from row_radix_top_amd import binding, blocks, pages
from tests.test_paged_refusals import _attention, _header

EINVAL, EWORKSPACE = -1, -3


def _fields(name):
    import re
    body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", _header()).group(1)
    for decl in filter(None, (d.strip() for d in body.split(";"))):
        kind, names = re.match(r"((?:const )?\w+\s*\*?)\s*(.*)", decl, flags=re.S).groups()
        for n in names.split(","):
            yield n.strip().lstrip("*"), 8 if "*" in kind or n.strip().startswith("*") or "int64" in kind else 4


@pytest.mark.parametrize("struct,name", [(pages.PagedPages, "paged_pages")])
def test_ctypes_mirrors_follow_the_header(struct, name):
    fields = list(_fields(name))
    assert [n for n, _ in fields] == [f[0] for f in struct._fields_]
    assert [s for _, s in fields] == [ctypes.sizeof(f[1]) for f in struct._fields_]


def test_copies_of_a_launch():
    import re
    assert f"#define PAGED_COPY_CACHES {pages.COPY_CACHES}" in re.sub(r" +", " ", _header())


def _call(name, order, base, changes):
    args = dict(base, **changes)
    return getattr(pa.load(), name)(*(args[n] for n in order.split()))


FORK = "block_table table_stride table_width lengths num_seqs parents keep num_rows free_pages num_free page_size out_table out_stride out_lengths src dst tokens pages stream"
FORK_BASE = dict(block_table=256, table_stride=4, table_width=4, lengths=256, num_seqs=2, parents=256, keep=None,
                 num_rows=3, free_pages=256, num_free=4, page_size=16, out_table=256, out_stride=4, out_lengths=256,
                 src=256, dst=256, tokens=256, pages=256, stream=None)


@pytest.mark.parametrize("changes,text", [
    (dict(num_seqs=-1), "num_seqs"), (dict(num_rows=-1), "num_rows"), (dict(num_free=-1), "num_free"),
    (dict(page_size=0), "page_size"), (dict(table_width=0), "table_width"), (dict(table_stride=3), "table_stride"),
    (dict(out_stride=3), "out_stride"), (dict(block_table=None), "null"), (dict(lengths=None), "null"),
    (dict(parents=None), "null"), (dict(free_pages=None), "free_pages"), (dict(out_table=None), "null"),
    (dict(src=None), "null"), (dict(dst=None), "null"), (dict(tokens=None), "null"), (dict(pages=None), "pages"),
    (dict(out_lengths=None), "null"), (dict(keep=257), "4-byte"), (dict(block_table=258), "4-byte"),
])
def test_fork_refuses(changes, text):
    assert _call("paged_fork", FORK, FORK_BASE, changes) == EINVAL
    assert text in binding.last_error()


@pytest.mark.parametrize("changes", [dict(), dict(out_table=512), dict(out_lengths=512)])
def test_fork_refuses_to_write_over_what_it_reads(changes):
    assert _call("paged_fork", FORK, FORK_BASE, changes) == EINVAL
    assert "goes on from" in binding.last_error()


def _copy(pairs=2, num_pages=4, src=256, dst=256, tokens=None, count=1, **cache):
    q = pages.PagedPages(256, 1024, 64, 0, 16, 1, 64)
    for k, v in cache.items():
        setattr(q, k, v)
    return pa.load().paged_copy(src, dst, tokens, pairs, (pages.PagedPages * 2)(q, q), count, num_pages, None)


@pytest.mark.parametrize("changes,text", [
    (dict(pairs=-1), "num_pairs"), (dict(num_pages=-1), "num_pages"), (dict(count=-1), "num_caches"),
    (dict(src=None), "null"), (dict(dst=None), "null"), (dict(tokens=258), "4-byte"), (dict(src=257), "4-byte"),
    (dict(data=None), "null data"), (dict(width=0), "width"), (dict(outer=0), "outer"), (dict(page_stride=-1), "strides"),
    (dict(width=1 << 30, outer=2), "2^31"), (dict(width=1 << 27), "2^31"), (dict(**{"tokens": None}, outer=-1), "outer"),
])
def test_copy_refuses(changes, text):
    assert _copy(**changes) == EINVAL
    assert text in binding.last_error()


def test_copy_of_nothing():
    assert _copy(pairs=0, src=None) == 0
    assert _copy(num_pages=0) == 0
    assert _copy(count=0) == 0


FREE = "block_table table_stride table_width lengths num_seqs page_size num_pages free_pages refs count workspace stream"
FREE_BASE = dict(block_table=256, table_stride=4, table_width=4, lengths=256, num_seqs=2, page_size=16, num_pages=9,
                 free_pages=256, refs=256, count=256, workspace=256, stream=None)


@pytest.mark.parametrize("changes,text", [
    (dict(num_seqs=-1), "num_seqs"), (dict(page_size=0), "page_size"), (dict(table_width=0), "table_width"),
    (dict(table_stride=3), "table_stride"), (dict(num_pages=-1), "num_pages"), (dict(block_table=None), "null"),
    (dict(lengths=None), "null"), (dict(free_pages=None), "null"), (dict(refs=None), "null"), (dict(count=None), "null"),
    (dict(refs=257), "4-byte"), (dict(workspace=264), "aligned"),
])
def test_free_refuses(changes, text):
    assert _call("paged_free", FREE, FREE_BASE, changes) == EINVAL
    assert text in binding.last_error()


COMPACT = "block_table table_stride table_width lengths num_seqs page_size num_pages limit out_table out_stride src dst moves live workspace stream"
COMPACT_BASE = dict(block_table=256, table_stride=4, table_width=4, lengths=256, num_seqs=2, page_size=16, num_pages=9,
                    limit=-1, out_table=512, out_stride=4, src=256, dst=256, moves=256, live=256, workspace=256,
                    stream=None)


@pytest.mark.parametrize("changes,text", [
    (dict(num_seqs=-1), "num_seqs"), (dict(page_size=0), "page_size"), (dict(limit=-2), "limit"), (dict(limit=10), "limit"),
    (dict(out_stride=3), "out_stride"), (dict(out_table=None), "null out_table"),
    (dict(out_table=256, out_stride=5), "in place"), (dict(src=None), "null"), (dict(moves=None), "null"),
    (dict(live=None), "null"), (dict(out_table=257), "4-byte"), (dict(workspace=264), "aligned"),
])
def test_compact_refuses(changes, text):
    assert _call("paged_compact", COMPACT, COMPACT_BASE, changes) == EINVAL
    assert text in binding.last_error()


@pytest.mark.parametrize("name,order,base", [("paged_free", FREE, FREE_BASE), ("paged_compact", COMPACT, COMPACT_BASE)])
def test_pools_need_their_workspace(name, order, base):
    assert _call(name, order, base, dict(workspace=None)) == EWORKSPACE
    assert "workspace" in binding.last_error()
    size = ctypes.c_size_t(0)
    most = 0
    for n in list(range(300)) + [1 << 20, (1 << 31) - 1]:
        assert getattr(pa.load(), name + "_workspace_size")(n, size) == 0
        assert size.value >= most and size.value >= n // 8
        most = size.value
    assert getattr(pa.load(), name + "_workspace_size")(-1, size) == EINVAL


def test_tensors_that_require_gradients_are_refused():
    import torch

    import row_radix_top_amd as rrt
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(RuntimeError, match="paged_copy has no gradients"):
        rrt.paged_copy(i, i, [torch.zeros(2, 16, 4), torch.zeros(2, 16, 4, requires_grad=True)])


def _struct(kind, base, changes):
    a = kind()
    for k, v in dict(base, **changes).items():
        setattr(a, k, v)
    return ctypes.byref(a)


@pytest.mark.parametrize("struct,name", [(blocks.BoundsArgs, "paged_bounds_args"), (blocks.SelectArgs, "paged_select_args")])
def test_ctypes_mirrors_of_arguments_follow_the_header(struct, name):
    fields = list(_fields(name))
    assert [n for n, _ in fields] == [f[0] for f in struct._fields_]
    assert [s for _, s in fields] == [ctypes.sizeof(f[1]) for f in struct._fields_]


BOUNDS = dict(k=512, block_table=256, starts=256, lengths=256, bounds=256, scales=256, page_stride=16 * 256,
              token_stride=256, head_stride=128, bounds_page_stride=512, bounds_head_stride=256, scales_stride=2,
              table_stride=4, num_seqs=2, num_tokens=5, num_kv_heads=2, head_dim=128, page_size=16, num_pages=4,
              table_width=4, store=0)


@pytest.mark.parametrize("changes,text", [
    (dict(store=3), "store"), (dict(num_seqs=-1), "num_seqs"), (dict(num_tokens=-1), "num_tokens"),
    (dict(num_kv_heads=0), "num_kv_heads"), (dict(head_dim=96), "head_dim"), (dict(page_size=0), "page_size"),
    (dict(table_width=0), "table_width"), (dict(num_pages=0), "num_pages"), (dict(k=None), "null"),
    (dict(starts=None), "null"), (dict(lengths=None), "null"), (dict(bounds=None), "null"), (dict(scales=None), "null"),
    (dict(block_table=None), "null"), (dict(k=520), "16 bytes"), (dict(token_stride=129), "16 bytes"),
    (dict(bounds=264), "16 bytes"), (dict(bounds_page_stride=520), "16 bytes"), (dict(page_stride=-16), "strides"),
    (dict(starts=257), "4-byte"), (dict(store=2, head_stride=136), "16 bytes"),
])
def test_bounds_refuse(changes, text):
    assert pa.load().paged_bounds(_struct(blocks.BoundsArgs, BOUNDS, changes), None) == EINVAL
    assert text in binding.last_error()


def test_bounds_of_nothing():
    for changes in (dict(num_seqs=0, k=None), dict(num_tokens=0, bounds=None)):
        assert pa.load().paged_bounds(_struct(blocks.BoundsArgs, BOUNDS, changes), None) == 0


SELECT = dict(q=256, bounds=256, scales=256, block_table=256, lengths=256, blocks=256, q_row_stride=1024,
              q_head_stride=128, bounds_page_stride=512, bounds_head_stride=256, scales_stride=2, table_stride=4,
              num_rows=2, next_n=1, num_heads=8, num_kv_heads=2, head_dim=128, page_size=16, num_pages=4, table_width=4,
              num_blocks=3, first=1, last=1, dtype=0)


@pytest.mark.parametrize("changes,text", [
    (dict(dtype=2), "dtype"), (dict(num_rows=-1), "num_rows"), (dict(next_n=0), "next_n"),
    (dict(num_rows=3, next_n=2), "next_n"), (dict(num_heads=0), "num_heads"), (dict(num_kv_heads=3), "num_kv_heads"),
    (dict(head_dim=256), "head_dim"), (dict(page_size=0), "page_size"), (dict(table_width=0), "table_width"),
    (dict(table_width=32769), "table_width"), (dict(num_blocks=0), "num_blocks"), (dict(first=-1), "first"),
    (dict(first=2, last=2), "at most num_blocks"), (dict(first=2147483647, last=2147483647), "at most num_blocks"),
    (dict(num_pages=0), "num_pages"), (dict(num_rows=1 << 30), "2^31"), (dict(q=None), "null"),
    (dict(bounds=None), "null"), (dict(scales=None), "null"), (dict(lengths=None), "null"), (dict(blocks=None), "null"),
    (dict(block_table=None), "null"), (dict(q=264), "16 bytes"), (dict(q_head_stride=129), "16 bytes"),
    (dict(bounds_head_stride=8), "16 bytes"), (dict(table_stride=-1), "strides"), (dict(blocks=258), "4-byte"),
])
def test_select_refuses(changes, text):
    assert pa.load().paged_block_select(_struct(blocks.SelectArgs, SELECT, changes), None, None) == EINVAL
    assert text in binding.last_error()


def test_select_of_nothing():
    assert pa.load().paged_block_select(_struct(blocks.SelectArgs, SELECT, dict(num_rows=0, q=None)), None, None) == 0


def _block_attention(at=256, num_blocks=4, row=8, head=4, **changes):
    return pa.load().paged_block_attention(ctypes.byref(_attention(**changes)), at, row, head, num_blocks, None, None)


@pytest.mark.parametrize("changes,text", [
    (dict(chosen=256, num_chosen=4), "chosen must be NULL"), (dict(num_blocks=0), "num_blocks"),
    (dict(num_blocks=1 << 27), "2^30"), (dict(row=-1), "strides"), (dict(head=-1), "strides"), (dict(at=257), "4-byte"),
    (dict(at=None), "null blocks"), (dict(page_size=0), "page_size"), (dict(head_dim=96), "head_dim"),
    (dict(v=None), "null v"), (dict(num_kv_heads=3), "num_kv_heads"), (dict(q=264), "16 bytes"),
])
def test_block_attention_refuses(changes, text):
    assert _block_attention(**changes) == EINVAL
    assert text in binding.last_error()


def test_block_attention_of_nothing():
    assert _block_attention(num_rows=0, q=None, at=None) == 0


def _prefix(starts=256, shared=256, groups=2, **changes):
    return pa.load().paged_prefix_attention(ctypes.byref(_attention(**changes)), starts, shared, groups, None, None)


@pytest.mark.parametrize("changes,text", [
    (dict(groups=-1), "num_groups"), (dict(starts=None), "null group_starts"), (dict(shared=None), "null group_starts"),
    (dict(starts=257), "4-byte"), (dict(shared=258), "4-byte"), (dict(chosen=256, num_chosen=4), "chosen must be NULL"),
    (dict(head_dim=96), "head_dim"), (dict(v=None), "null v"), (dict(num_kv_heads=3), "num_kv_heads"),
    (dict(q=264), "16 bytes"), (dict(max_splits=129), "max_splits"), (dict(groups=0, head_dim=96), "head_dim"),
])
def test_prefix_attention_refuses(changes, text):
    assert _prefix(**changes) == EINVAL
    assert text in binding.last_error()


def test_prefix_attention_of_nothing():
    assert _prefix(num_rows=0, q=None) == 0
    assert _prefix(num_rows=0, q=None, groups=0, starts=None, shared=None) == 0
