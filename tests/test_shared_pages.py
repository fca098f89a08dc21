"""paged_fork, paged_copy, paged_free and paged_compact on the GPU against plain
Python, exactly: sizes from nothing to many rows, tables with bad entries, lists
that run out, strided tables, other streams and graphs."""

from __future__ import annotations

import numpy as np
import pytest

import row_radix_top_amd as rrt
from tests import shared_ref
from tests.gpu_util import note, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def dev(x):
    import torch
    return torch.as_tensor(np.asarray(x), device="cuda").to(torch.int32)


def host(x):
    return x.cpu().numpy()


def batch(rng, seqs, width, page, spare=20):
    """A table whose rows share leading pages in groups, lengths, and the pool's pages."""
    lengths = rng.integers(0, width * page + 1, size=seqs)
    pages = seqs * width + spare
    order = rng.permutation(pages)
    table = np.full((seqs, width), -1)
    at = 0
    for s in range(seqs):
        need = -(-lengths[s] // page)
        table[s, :need] = order[at:at + need]
        at += need
        if s > 0 and rng.random() < 0.5:  # goes on from the row before it
            same = min(lengths[s], lengths[s - 1]) // page
            table[s, :same] = table[s - 1, :same]
    return table, lengths, order[at:], pages


def check_fork(table, lengths, parents, keep, free, page, **kw):
    got = rrt.paged_fork(kw.pop("on_device", dev(table)), dev(lengths), dev(parents), dev(free), page_size=page,
                         keep=None if keep is None else dev(keep), **kw)
    exp = shared_ref.fork(table, lengths, parents, keep, free, page)
    for name, a, b in zip(got._fields, got, exp):
        np.testing.assert_array_equal(host(a), np.atleast_1d(b), err_msg=name)
    return got


@pytest.mark.parametrize("page", [1, 3, 16, 64])
@pytest.mark.parametrize("seqs,rows,width", [(1, 1, 1), (1, 7, 5), (9, 9, 4), (40, 133, 11), (300, 70, 2), (3, 1500, 3)])
@pytest.mark.parametrize("cut", [False, True])
def test_forks(page, seqs, rows, width, cut):
    rng = np.random.default_rng(seqs * 100 + rows + page)
    table, lengths, free, _ = batch(rng, seqs, width, page)
    parents = rng.integers(0, seqs, size=rows)
    keep = rng.integers(-2, width * page + 3, size=rows) if cut else None
    note(f"fork page={page} seqs={seqs} rows={rows} width={width} cut={cut}")
    check_fork(table, lengths, parents, keep, free, page)


def test_forks_of_bad_parents_lengths_and_entries():
    rng = np.random.default_rng(5)
    table, lengths, free, _ = batch(rng, 6, 5, 16)
    lengths[:3] = [2147483647, -4, 70]
    table[0] = [3, -1, 2147483647, -2147483648, 9]
    table[2, 4] = -7  # the last page of 70 tokens is none
    parents = [0, 0, -1, 6, 2147483647, 2, 2, 2, 1, 5, -2147483648, 0]
    check_fork(table, lengths, parents, None, free, 16)
    check_fork(table, lengths, parents, [70, 2147483647, 3, 3, 3, 65, 66, 64, 5, -1, 2, 79], free, 16)


@pytest.mark.parametrize("have", [0, 1, 3])
def test_forks_when_the_free_list_runs_out(have):
    table, lengths = np.array([[4, 5], [6, 7]]), np.array([20, 32])
    got = check_fork(table, lengths, [0, 0, 1, 0, 1, 0], [20, 19, 31, 18, 17, 16], list(range(10, 10 + have)), 16)
    assert int(got.pages) == 3
    # A list that is padded, as paged_free gives it.
    check_fork(table, lengths, [0, 0, 1, 0], None, [11, -1, -1], 16)


def test_fork_of_nothing():
    import torch
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    got = rrt.paged_fork(dev([[1, 2]]), dev([20]), empty, empty, page_size=16)
    assert int(got.pages) == 0 and got.table.shape == (0, 2)
    got = rrt.paged_fork(torch.empty(0, 3, dtype=torch.int32, device="cuda"), empty, dev([0, 1]), dev([5]), page_size=16)
    assert bool((got.table == -1).all()) and got.lengths.tolist() == [0, 0] and int(got.pages) == 0


def test_fork_of_strided_tables_into_given_outputs():
    import torch
    rng = np.random.default_rng(8)
    table, lengths, free, _ = batch(rng, 5, 6, 16)
    wide = torch.full((5, 11), 77, dtype=torch.int32, device="cuda")
    wide[:, 2:8] = dev(table)
    new = torch.full((7, 9), 55, dtype=torch.int32, device="cuda")
    ints = lambda n: torch.full((n,), 55, dtype=torch.int32, device="cuda")  # noqa: E731
    out = rrt.Fork(new[:, 1:7], ints(7), ints(7), ints(7), ints(7), ints(1))
    got = check_fork(table, lengths, [0, 0, 1, 2, 2, 4, 4], None, free, 16, on_device=wide[:, 2:8], out=out)
    assert got.table.data_ptr() == out.table.data_ptr()
    assert bool((new[:, 0] == 55).all()) and bool((new[:, 7:] == 55).all())


CACHES = [("bfloat16", (16, 2, 64)), ("float8_e4m3fn", (16, 3, 64)), ("float16", (16, 1, 3)), ("int8", (16, 5)),
          ("float32", (16, 7))]


@pytest.mark.parametrize("dtype,shape", CACHES)
@pytest.mark.parametrize("tokens", [None, [0, 1, 16, 7, 99, -3, 5]])
def test_copies(dtype, shape, tokens):
    import torch
    pages = 30
    src, dst = [1, 2, 3, -1, 5, 6, 29], [11, 12, 13, 14, 15, -1, 0]
    src, dst = src + [30, 8, 9], dst + [20, 30, 9]  # outside the pool, onto itself
    t = None if tokens is None else tokens + [16, 16, 16]
    torch.manual_seed(0)
    caches = [torch.randint(0, 100, (pages,) + shape, device="cuda").to(getattr(torch, dtype)) for _ in range(3)]
    before = [c.float().cpu().clone() for c in caches]
    note(f"copy {dtype} {shape} tokens={tokens}")
    rrt.paged_copy(dev(src), dev(dst), caches, tokens=None if t is None else dev(t))
    for a, b in zip(caches, before):
        for i, (x, y) in enumerate(zip(src, dst)):
            n = shape[0] if t is None else min(max(t[i], 0), shape[0])
            if 0 <= x < pages and 0 <= y < pages:
                b[y, :n] = b[x, :n].clone()
        assert torch.equal(a.float().cpu(), b)


def test_copies_of_other_layouts():
    """Heads before tokens, keys and values in one pool, many caches in a call,
    what has no tokens."""
    import torch
    torch.manual_seed(1)
    both = torch.randn(9, 2, 4, 16, 64, device="cuda").bfloat16()  # pages of [2, heads, tokens, dim]
    views = [both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)]
    exp = both.clone()
    exp[7, :, :, :5] = both[2, :, :, :5]
    rrt.paged_copy(dev([2]), dev([7]), views, tokens=dev([5]))
    assert torch.equal(both, exp)
    many = torch.randn(70, 6, 8, 2, 64, device="cuda").bfloat16()
    exp = many.clone()
    exp[:, [0, 5]] = many[:, [3, 1]]
    rrt.paged_copy(dev([3, 1]), dev([0, 5]), list(many.unbind(0)))
    assert torch.equal(many, exp)
    bounds, scales = torch.randint(-9, 9, (6, 2, 2, 64), device="cuda", dtype=torch.int8), torch.randn(6, 1, device="cuda")
    exp = bounds.clone(), scales.clone()
    for x in exp:
        x[4] = x[0]
    rrt.paged_copy(dev([0]), dev([4]), [bounds, scales])
    assert torch.equal(bounds, exp[0]) and torch.equal(scales, exp[1])
    rrt.paged_copy(dev([0]), dev([4]), [])
    wide = torch.randn(4, 16, 3, 128, device="cuda")
    part = wide[..., 32:64]
    exp = wide.clone()
    exp[1, :9, :, 32:64] = wide[3, :9, :, 32:64]
    rrt.paged_copy(dev([3]), dev([1]), [part], tokens=dev([9]))
    assert torch.equal(wide, exp)


def test_copies_past_32_bits():
    """Pages that lie past 2^32 bytes."""
    import torch
    x = torch.empty(40, 1 << 27, dtype=torch.uint8, device="cuda")
    x[38] = 7
    x[39] = 3
    rrt.paged_copy(dev([38]), dev([0]), [x])
    rrt.paged_copy(dev([39]), dev([37]), [x], tokens=dev([1 << 26]))
    assert bool((x[0] == 7).all()) and bool((x[37, :1 << 26] == 3).all())


def check_pool(table, lengths, page, pages, limit=None, **kw):
    t, n = kw.pop("on_device", dev(table)), dev(lengths)
    got = rrt.paged_free(t, n, page_size=page, num_pages=pages)
    refs = shared_ref.refs(table, lengths, page, pages)
    free = np.nonzero(refs == 0)[0]
    np.testing.assert_array_equal(host(got.refs), refs)
    np.testing.assert_array_equal(host(got.free), shared_ref.padded(free, pages))
    assert int(got.count) == len(free)
    c = rrt.paged_compact(t, n, page_size=page, num_pages=pages, limit=limit, **kw)
    new, moves, live = shared_ref.compact(table, lengths, page, pages, limit)
    assert (int(c.moves), int(c.live)) == (len(moves), live)
    np.testing.assert_array_equal(host(c.src), shared_ref.padded([a for a, _ in moves], pages // 2))
    np.testing.assert_array_equal(host(c.dst), shared_ref.padded([b for _, b in moves], pages // 2))
    np.testing.assert_array_equal(host(c.table), new)
    return c


@pytest.mark.parametrize("page", [1, 16, 24])
@pytest.mark.parametrize("seqs,width,spare", [(1, 1, 0), (1, 1, 1), (5, 3, 2), (60, 30, 300), (900, 2, 63), (3, 2500, 1)])
def test_free_pages_and_moves(page, seqs, width, spare):
    rng = np.random.default_rng(seqs + width)
    table, lengths, _, pages = batch(rng, seqs, width, page, spare)
    note(f"free and compact page={page} seqs={seqs} width={width} pages={pages}")
    check_pool(table, lengths, page, pages)
    lengths[rng.random(seqs) < 0.5] = 0
    for limit in {None, 0, 1, pages // 3, pages - 1, pages}:
        check_pool(table, lengths, page, pages, limit)


def test_pools_of_every_small_size():
    rng = np.random.default_rng(3)
    for pages in [0, 1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1023, 1025]:
        table = rng.integers(-2, pages + 2, size=(4, 9))
        note(f"pool of {pages}")
        check_pool(table, [9, 4, 0, 2], 1, pages)
        check_pool(table, [9, 4, 0, 2], 1, pages, pages // 2)


def test_bad_entries_lengths_and_strides():
    import torch
    rng = np.random.default_rng(4)
    table = rng.integers(0, 50, size=(5, 7))
    table[1] = [-1, 50, 2147483647, -2147483648, 3, 3, 49]
    lengths = [2147483647, 100, -1, 17, 0]
    wide = torch.full((5, 10), 1, dtype=torch.int32, device="cuda")
    wide[:, 3:] = dev(table)
    c = check_pool(table, lengths, 16, 50, on_device=wide[:, 3:])
    # In place: the same, and nothing beside the table changes.
    ints = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    out = rrt.Compact(wide[:, 3:], ints(25), ints(25), ints(1), ints(1))
    again = rrt.paged_compact(wide[:, 3:], dev(lengths), page_size=16, num_pages=50, out=out)
    assert torch.equal(again.table, c.table) and bool((wide[:, :3] == 1).all())
    assert torch.equal(again.src, c.src) and torch.equal(again.dst, c.dst)


def test_no_rows_hold_nothing():
    import torch
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    t = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    got = rrt.paged_free(t, empty, page_size=16, num_pages=70)
    assert got.free.tolist() == list(range(70)) and int(got.count) == 70 and int(got.refs.sum()) == 0
    c = rrt.paged_compact(t, empty, page_size=16, num_pages=70, limit=9)
    assert int(c.moves) == 0 and int(c.live) == 0 and bool((c.src == -1).all())


def test_a_large_pool():
    """A million pages: the bitmap is 128 KB, and every workgroup counts it."""
    import torch
    rng = np.random.default_rng(6)
    pages, seqs, width = 1 << 20, 64, 3000
    table = rng.permutation(pages)[:seqs * width].reshape(seqs, width)
    lengths = rng.integers(0, width * 16, size=seqs)
    held = np.zeros(pages, dtype=bool)
    for s in range(seqs):
        held[table[s, :-(-lengths[s] // 16)]] = True
    got = rrt.paged_free(dev(table), dev(lengths), page_size=16, num_pages=pages)
    free = np.nonzero(~held)[0]
    np.testing.assert_array_equal(host(got.free), shared_ref.padded(free, pages))
    live = int(held.sum())
    c = rrt.paged_compact(dev(table), dev(lengths), page_size=16, num_pages=pages)
    src, dst = np.nonzero(held[live:])[0] + live, np.nonzero(~held[:live])[0]
    np.testing.assert_array_equal(host(c.src), shared_ref.padded(src, pages // 2))
    np.testing.assert_array_equal(host(c.dst), shared_ref.padded(dst, pages // 2))
    after = rrt.paged_free(c.table, dev(lengths), page_size=16, num_pages=pages)
    assert torch.equal(after.free[:pages - live], torch.arange(live, pages, device="cuda", dtype=torch.int32))


def test_streams_and_graphs():
    import torch
    rng = np.random.default_rng(9)
    table, lengths, free, pages = batch(rng, 8, 6, 16)
    t, n, p, f = dev(table), dev(lengths), dev([0, 0, 3, 4, 4, 4, 7, 1]), dev(free)
    cache = torch.randn(pages, 16, 2, 64, device="cuda").bfloat16()

    def step():
        fork = rrt.paged_fork(t, n, p, f, page_size=16)
        rrt.paged_copy(fork.src, fork.dst, [cache], tokens=fork.tokens)
        pool = rrt.paged_free(fork.table, fork.lengths, page_size=16, num_pages=pages)
        c = rrt.paged_compact(fork.table, fork.lengths, page_size=16, num_pages=pages, limit=pages // 2)
        return [*fork, *pool, *c]

    first = [x.clone() for x in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = rrt.paged_fork(t, n, p, f, page_size=16, stream=s)
    b = rrt.paged_free(a.table, a.lengths, page_size=16, num_pages=pages, stream=s)
    rrt.paged_copy(a.src, a.dst, [cache], tokens=a.tokens, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, [*a, *b]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        p.copy_(dev(rng.integers(-1, 8, size=8)))
        n.copy_(dev(np.minimum(lengths, 16 * k + 7)))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        assert all(torch.equal(x, y) for x, y in zip(got, step()))


def test_refusals_of_tensors():
    import torch
    t, n, p, f = dev([[1, 2], [3, 4]]), dev([20, 9]), dev([0, 1, 1]), dev([5, 6])
    c = torch.zeros(8, 16, 2, 64, device="cuda")
    for call, err in [
        (lambda: rrt.paged_fork(t.long(), n, p, f, page_size=16), TypeError),
        (lambda: rrt.paged_fork(t, n[:1], p, f, page_size=16), ValueError),
        (lambda: rrt.paged_fork(t, n, p, f, page_size=16, keep=dev([1])), ValueError),
        (lambda: rrt.paged_fork(t, n, p.cpu(), f, page_size=16), TypeError),
        (lambda: rrt.paged_fork(t, n, p, f, page_size=0), rrt.TopKError),
        (lambda: rrt.paged_copy(p, p[:2], [c]), ValueError),
        (lambda: rrt.paged_copy(p, p, [c, c[:7]]), ValueError),
        (lambda: rrt.paged_copy(p, p, [c.cpu()]), ValueError),
        (lambda: rrt.paged_copy(p, p, [c[:, :, :, :32:2]], tokens=p), ValueError),
        (lambda: rrt.paged_copy(p, p, [c[:, :, :1, :1].expand(8, 16, 2, 64)]), ValueError),
        (lambda: rrt.paged_copy(p, p, [c[:, :0]]), ValueError),
        (lambda: rrt.paged_copy(p, p, [c[:, 0, 0, 0]], tokens=p), ValueError),
        (lambda: rrt.paged_free(t, n, page_size=16, num_pages=-1), ValueError),
        (lambda: rrt.paged_free(t, n, page_size=16, num_pages=300, workspace=c.view(-1)[:9]), ValueError),
        (lambda: rrt.paged_free(t.float(), n, page_size=16, num_pages=3), TypeError),
        (lambda: rrt.paged_compact(t, n, page_size=16, num_pages=9, limit=10), rrt.TopKError),
        (lambda: rrt.paged_compact(t, n, page_size=16, num_pages=9, limit=-1), ValueError),
    ]:
        with pytest.raises(err):
            call()


@pytest.mark.parametrize("pages", [8190, 8191, 8192, 8193])
def test_pools_about_what_one_workgroup_takes(pages):
    rng = np.random.default_rng(pages)
    table = rng.integers(-2, pages + 2, size=(5, 700))
    note(f"pool of {pages}")
    for limit in (None, 0, 1500, pages - 1, pages):
        check_pool(table, [700, 4, 0, 699, 64], 1, pages, limit)


@pytest.mark.parametrize("width", [4095, 4096, 4097])
def test_tables_about_what_one_workgroup_takes(width):
    rng = np.random.default_rng(width)
    for pages in (0, 1, 33, 64, 257, 1025):
        table = rng.integers(-2, pages + 2, size=(4, width))
        note(f"pool of {pages} width={width}")
        for limit in {None, 0, pages // 2, pages}:
            check_pool(table, [9, 4, 0, width], 1, pages, limit)


@pytest.mark.parametrize("rows,width", [(63, 7), (64, 7), (65, 7), (64, 256), (64, 257), (1, 16384), (1, 16385)])
@pytest.mark.parametrize("cut", [False, True])
def test_forks_about_what_one_workgroup_takes(rows, width, cut):
    rng = np.random.default_rng(rows + width)
    table, lengths, free, _ = batch(rng, 9, width, 3)
    parents = rng.integers(-1, 10, size=rows)
    keep = rng.integers(-2, width * 3 + 3, size=rows) if cut else None
    note(f"fork rows={rows} width={width} cut={cut}")
    check_fork(table, lengths, parents, keep, free, 3)
    check_fork(table, lengths, parents, keep, free[:2], 3)
