"""paged_prefix_attention on the GPU against 64-bit sums: group sizes on either
side of every tile, types, head layouts, shared lengths from nothing to all,
sequences that take no part, bad pages, and places that must not count."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest

import row_radix_top_amd as rrt
from row_radix_top_amd import attention as pa
from row_radix_top_amd import binding
from tests import paged_ref, shared_ref
from tests.gpu_util import note, require_gpu
from tests.test_workspaces import _attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def dev(x):
    import torch
    return torch.as_tensor(np.asarray(x), device="cuda").to(torch.int32)


class Case:
    """groups: (shared positions, [lengths of each sequence's rows]).  Every
    place that no row may read holds NaN."""

    def __init__(self, groups, *, heads=8, kv=2, dim=128, dtype="bfloat16", store="same", page=16, width=None, seed=0,
                 spread=1.0, before=(), after=()):
        import torch
        rng = np.random.default_rng(seed)
        rows = [r for r in before] + [r for _, g in groups for r in g] + [r for r in after]
        self.rows2d = np.asarray([np.atleast_1d(r) for r in rows], dtype=np.int64)
        self.lengths = self.rows2d if self.rows2d.shape[1] > 1 else self.rows2d[:, 0]
        self.next_n = self.rows2d.shape[1]
        self.starts = len(before) + np.concatenate([[0], np.cumsum([len(g) for _, g in groups])])
        self.shared = np.array([s for s, _ in groups], dtype=np.int64)
        self.page = page
        seqs = len(rows)
        most = np.maximum(self.rows2d.max(axis=1), 0)
        need = -(-most // page)
        self.width = width or max(1, int(need.max()))
        need = np.minimum(need, self.width)
        self.pages = int(need.sum()) + 3
        order = rng.permutation(self.pages)
        self.table = np.full((seqs, self.width), -1, dtype=np.int64)
        at = 0
        for s in range(seqs):
            self.table[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
        # Shared pages: those of the first sequence that is long enough.  One that
        # shares part of a page holds the same keys and values there.
        self.reader = np.arange(seqs)
        for g, n in enumerate(self.shared):
            inside = [s for s in range(self.starts[g], self.starts[g + 1]) if (self.rows2d[s] >= n).all()]
            for s in inside:
                self.table[s, :n // page] = self.table[inside[0], :n // page]
                self.reader[s] = inside[0]
        self.heads, self.kv, self.dim = heads, kv, dim
        self.dt = getattr(torch, dtype)
        self.st = self.dt if store == "same" else getattr(torch, store)
        torch.manual_seed(seed)
        self.q = (torch.randn(self.rows2d.size, heads, dim, device="cuda") * spread).to(self.dt)
        self.k, self.v = (torch.randn(self.pages, page, kv, dim, device="cuda").to(self.st) for _ in range(2))
        self.ks = self.vs = None
        if self.st == torch.float8_e4m3fn:
            self.ks, self.vs = (torch.rand(kv, device="cuda") + 0.5 for _ in range(2))
        self.scale = dim ** -0.5
        self.poison()

    def poison(self):
        import torch
        used = np.zeros(self.pages * self.page, dtype=bool)
        for r in range(self.rows2d.size):
            s = self.slots(r)
            used[s[s >= 0]] = True
        bad = torch.as_tensor(~used, device="cuda")
        for c in (self.k, self.v):
            flat = c.view(-1, self.kv, self.dim)
            bits = flat.view(torch.uint8) if self.st == torch.float8_e4m3fn else flat.view(torch.int16)
            bits[bad] = 0x7f if self.st == torch.float8_e4m3fn else 0x7fff

    def slots(self, r):
        """The slots that row r reads: the shared ones through its group's reader."""
        s = r // self.next_n
        p = np.arange(shared_ref.clamp(self.rows2d.reshape(-1)[r], self.width * self.page))
        own = paged_ref.slots_of(self.table[s], p, self.page, self.pages)
        g = np.searchsorted(self.starts, s, side="right") - 1
        if 0 <= g < len(self.shared) and s < self.starts[g + 1] and (self.rows2d[s] >= self.shared[g]).all():
            n = shared_ref.clamp(self.shared[g], len(p))
            own[:n] = paged_ref.slots_of(self.table[self.reader[s]], p[:n], self.page, self.pages)
        return own

    def run(self, **kw):
        return rrt.paged_prefix_attention(self.q, self.k, self.v, dev(self.table), dev(self.lengths), dev(self.starts),
                                          dev(self.shared), k_scale=self.ks, v_scale=self.vs, softmax_scale=self.scale, **kw)

    def expected(self):
        q, k, v = (x.double().cpu().numpy() for x in (self.q, self.k, self.v))
        if self.ks is not None:
            k, v = k * self.ks.double().cpu().numpy()[:, None], v * self.vs.double().cpu().numpy()[:, None]
        k, v = k.reshape(-1, self.kv, self.dim), v.reshape(-1, self.kv, self.dim)
        u, fp16, group = paged_ref.half_step(self.dt), "float16" == str(self.dt)[6:], self.heads // self.kv
        rows = q.shape[0]
        res = [np.zeros((rows, self.heads, self.dim)), np.zeros((rows, self.heads)),
               np.zeros((rows, self.heads, self.dim)), np.zeros((rows, self.heads))]
        for r in range(rows):
            s = self.slots(r)
            s = s[s >= 0]
            for h in range(self.heads):
                for dst, x in zip(res, paged_ref.attend(q[r, h], k[s, h // group], v[s, h // group], self.scale, u, fp16)):
                    dst[r, h] = x
        return res

    def check(self, what, **kw):
        note(f"prefix attention {what} rows={self.rows2d.shape} heads={self.heads}/{self.kv} dim={self.dim} {self.dt} "
             f"{self.st} page={self.page} groups={self.starts.tolist()[:9]} shared={self.shared.tolist()[:9]} {kw}")
        out, lse = self.run(**kw)
        exp, elog, tol, tlog = self.expected()
        paged_ref.check(out.double().cpu().numpy(), exp, tol, f"{what} out")
        paged_ref.check(lse.double().cpu().numpy(), elog, tlog, f"{what} lse")
        return out, lse


GROUPS = [(0, [5, 1]), (64, [64, 65, 100]), (300, [300]), (257, [400, 256, 258, 0, 700])]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv", [(1, 1), (8, 2), (40, 4), (20, 1), (48, 1)])
def test_types_and_heads(dtype, store, dim, heads, kv):
    """1 to 48 columns a sequence: one, two and four wavefronts along them."""
    Case(GROUPS, heads=heads, kv=kv, dim=dim, dtype=dtype, store=store).check("types")


@pytest.mark.parametrize("rows", [1, 2, 3, 5, 9, 17])
@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
def test_numbers_of_columns(rows, store):
    """8 columns a row: 8 to 136 of them, on either side of 32, 64 and 128."""
    rng = np.random.default_rng(rows)
    for dim in (64, 128):
        Case([(600, list(600 + rng.integers(0, 90, size=rows)))], heads=8, kv=1, dim=dim, store=store, seed=rows).check("columns")


@pytest.mark.parametrize("shared", [1, 15, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513, 1000])
def test_shared_lengths(shared):
    for rows in (1, 3, 6):
        Case([(shared, [shared + 16 * i for i in range(rows)])], heads=32, kv=2, page=16 if shared % 16 == 0 else 1,
             seed=shared).check("shared")


@pytest.mark.parametrize("page", [1, 5, 24, 64, 100])
@pytest.mark.parametrize("splits", [0, 1, 3, 32, 128])
def test_pages_and_splits(page, splits):
    Case([(1200 // page * page, [1300, 1200, 3000]), (page, [page, 2 * page + 1, 1])], page=page, heads=24, kv=2,
         seed=page).check("splits", max_splits=splits)


def test_parts_of_pages_that_are_shared_too():
    """70 positions of 16 a page: the last page of the shared part is the first
    sequence's; those of the others hold other keys there, which no row reads."""
    Case([(70, [70, 75, 200]), (9, [9, 30])], heads=8, kv=2, seed=1).check("part of a page")


@pytest.mark.parametrize("heads,kv", [(8, 2), (32, 1), (4, 4)])
@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
def test_several_rows_a_sequence(heads, kv, store):
    groups = [(160, [[160, 161, 162], [200, 199, 300], [159, 161, 170], [0, 0, 0]]), (48, [[48, 48, 48], [60, 49, 50]]),
              (0, [[1, 2, 3]])]
    Case(groups, heads=heads, kv=kv, store=store, seed=3).check("multi-token")


def test_sequences_outside_every_group():
    Case([(96, [100, 96]), (48, [60])], before=[70, 0], after=[33, 200, 1], seed=4).check("outside")


def test_groups_without_sequences_and_first_ones_that_take_no_part():
    Case([(64, []), (64, [0, 10, 80, 64]), (32, []), (500, [100, 200]), (16, [])], seed=5).check("empty groups")


def test_many_groups():
    """More than the lanes of a wavefront, of one to three sequences each."""
    rng = np.random.default_rng(6)
    for count in (63, 64, 65, 150):
        groups = [(int(n), [int(n + m) for m in rng.integers(-3, 20, size=rng.integers(0, 4))])
                  for n in rng.integers(0, 6, size=count) * 16]
        Case(groups, heads=4, kv=1, dim=64, seed=count).check("many groups")


def test_bad_pages_are_left_out():
    c = Case([(160, [300, 200, 161]), (64, [64, 90])], seed=7)
    c.table[:3, [0, 4, 9]] = [-1, c.pages, 2147483647]
    c.table[3:, 1] = -2147483648
    c.table[1, 11] = c.pages + 5
    c.k.normal_(), c.v.normal_()
    c.check("bad pages")
    c.table[:] = -1  # nothing left
    c.check("no pages")


def test_lengths_and_sizes_out_of_range_are_clamped():
    c = Case([(64, [64, 64, 3])], seed=8, width=4)
    c.rows2d = np.array([[2147483647], [-5], [2147483647]])
    c.lengths = c.rows2d[:, 0]
    c.table[:] = [0, 1, 2, 3]
    c.reader[:] = 0
    c.k.normal_(), c.v.normal_()
    c.check("clamped")
    c.shared = np.array([2147483647])  # all of the table
    c.check("shared past the table")
    c.shared = np.array([-9])
    c.check("nothing shared")


def test_starts_that_make_no_sense():
    """No read or write out of range: the inputs are as before, rows behind untouched."""
    import torch
    c = Case([(64, [64, 80, 90])], seed=9)
    c.k.normal_(), c.v.normal_()
    k, v = c.k.clone(), c.v.clone()
    buf = torch.full((6, c.heads, c.dim), 7.0, device="cuda", dtype=c.dt)
    for starts in ([5, 2, -1, 9], [2147483647, -2147483648, 3, 0], [-7, -7, 2147483647, 1]):
        rrt.paged_prefix_attention(c.q, c.k, c.v, dev(c.table), dev(c.lengths), dev(starts), dev([64, 64, 64]), out=buf[:3])
        torch.cuda.synchronize()
    assert bool((buf[3:] == 7).all()) and torch.equal(k, c.k) and torch.equal(v, c.v)


def test_large_scores_and_scales_of_either_sign():
    Case([(600, [600, 650, 700])], heads=24, kv=2, spread=60.0, seed=10).check("large scores")
    for scale in (-0.1, 0.0, 1e-30):
        c = Case([(300, [300, 333])], heads=24, kv=2, seed=11)
        c.scale = scale
        c.check(f"scale {scale}")
        c = Case([(300, [300, 333])], heads=24, kv=2, store="float8_e4m3fn", seed=11)
        c.scale = scale
        c.ks[0] *= -1
        c.check(f"scale {scale} of e4m3")


def test_small_weights_beside_a_large_one():
    """fp16 holds nothing below 2^-24: many weights of e^-17 together count."""
    import torch
    for rows in (1, 3, 6):
        c = Case([(4096, [4096] * rows)], heads=32, kv=2, dim=64, dtype="float16", seed=12)
        c.q.zero_()
        c.q[..., 0] = 1.0
        c.k.zero_(), c.v.zero_()
        slots = torch.as_tensor(c.slots(0), device="cuda")
        c.k.view(-1, 2, 64)[slots, :, 0] = -17.0
        c.k.view(-1, 2, 64)[slots[1000], :, 0] = 0.0
        c.v.view(-1, 2, 64)[slots] = 1.0
        c.v.view(-1, 2, 64)[slots[1000]] = 0.0
        c.scale = 1.0
        out, _ = c.run()
        n = 4095 * np.exp(-17.0)
        exp = n / (1 + n)
        # The sum is rounded once to fp16: half of its spacing at 1.7e-4, 2^-24.
        assert float((out.double() - exp).abs().max()) <= 2.0 ** -24


def test_far_pages():
    """A pool whose pages lie past 2^32 elements."""
    import torch
    pages, page = 1 << 15, 512  # x 2 heads x 128 = 2^32 elements each
    k = torch.empty(pages + 8, page, 2, 128, device="cuda", dtype=torch.bfloat16)
    v = torch.empty_like(k)
    for heads in (2, 40):
        c = Case([(512, [900, 512, 1000])], heads=heads, page=page, seed=13)
        order = {int(p): pages + i for i, p in enumerate(sorted({int(x) for x in c.table.reshape(-1) if x >= 0}))}
        table = np.array([[order.get(int(x), -1) for x in row] for row in c.table])
        for a, b in order.items():
            k[b], v[b] = c.k[a], c.v[a]
        near = c.run()
        far = rrt.paged_prefix_attention(c.q, k, v, dev(table), dev(c.lengths), dev(c.starts), dev(c.shared),
                                         softmax_scale=c.scale)
        assert torch.equal(near[0], far[0]) and torch.equal(near[1], far[1])


def test_strided_views():
    import torch
    c = Case([(64, [200, 64]), (0, [3])], seed=14)
    out, lse = c.check("plain")
    wide = torch.empty(3, 24, 128, device="cuda", dtype=c.dt)
    wide[:, 8:16] = c.q
    both = torch.stack([c.k, c.v], dim=1).transpose(2, 3).contiguous()  # pages of [2, heads, tokens, dim]
    table = torch.full((3, c.width + 5), -1, device="cuda", dtype=torch.int32)
    table[:, :c.width] = dev(c.table)
    again = rrt.paged_prefix_attention(wide[:, 8:16], both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2),
                                       table[:, :c.width], dev(c.lengths), dev(c.starts), dev(c.shared),
                                       softmax_scale=c.scale)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_no_groups_is_paged_attention():
    import torch
    c = Case([(0, [200, 64, 3])], seed=15)
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    a = rrt.paged_prefix_attention(c.q, c.k, c.v, dev(c.table), dev(c.lengths), dev([0]), empty, softmax_scale=c.scale)
    b = rrt.paged_attention(c.q, c.k, c.v, dev(c.table), dev(c.lengths), softmax_scale=c.scale)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a = rrt.paged_prefix_attention(c.q[:0], c.k, c.v, dev(c.table)[:0], dev([]), dev([0, 0]), dev([9]), softmax_scale=c.scale)
    assert a[0].shape == (0, 8, 128)


def test_streams_graphs_and_rows_behind():
    import torch
    c = Case([(400, [900, 500, 400]), (64, [70])], heads=24, kv=2, seed=16)
    out, lse = c.check("eager")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = c.run(stream=s)
    s.synchronize()
    assert torch.equal(other[0], out) and torch.equal(other[1], lse)
    lengths, table, starts, shared = dev(c.lengths), dev(c.table), dev(c.starts), dev(c.shared)
    graphs = []
    for splits in (0, 2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = rrt.paged_prefix_attention(c.q, c.k, c.v, table, lengths, starts, shared, softmax_scale=c.scale,
                                             max_splits=splits)
        graphs.append((g, res, splits))
    for step in range(4):
        lengths.copy_(dev([900 - 100 * step, 500, 400 - step, 70]))
        shared.copy_(dev([400 - 16 * step, 64 - 16 * step]))
        for g, _, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, res, splits in graphs:
            now = rrt.paged_prefix_attention(c.q, c.k, c.v, table, lengths, starts, shared, softmax_scale=c.scale,
                                             max_splits=splits)
            assert torch.equal(res[0], now[0]) and torch.equal(res[1], now[1])
    buf = torch.full((6, c.heads, c.dim), 7.0, device="cuda", dtype=c.dt)
    log = torch.full((6, c.heads), 7.0, device="cuda")
    c.run(out=buf[:4], lse=log[:4], workspace=torch.full((1 << 26,), 0xff, dtype=torch.uint8, device="cuda"))
    assert torch.equal(buf[:4], out) and bool((buf[4:] == 7).all()) and bool((log[4:] == 7).all())


def _size(args, groups):
    need = ctypes.c_size_t(0)
    assert pa.load().paged_prefix_attention_workspace_size(ctypes.byref(args), groups, None, need) == 0, binding.last_error()
    return need.value


@pytest.mark.parametrize("changes", [dict(), dict(num_heads=64, num_kv_heads=8), dict(next_n=2), dict(max_splits=3),
                                     dict(table_width=16)], ids=str)
def test_a_size_holds_for_fewer_rows_groups_and_shorter_ones(changes):
    n = changes.get("next_n", 1)
    for groups in (1, 4, 700):
        most = 0
        for rows in [n * r for r in range(1, 300)] + [n * 5000]:
            need = _size(_attention("paged_attention", rows, **changes), groups)
            assert need >= most
            most = need
        for width in (1, 7, 64, 300, 2047):
            short = _attention("paged_attention", 64 * n, **dict(changes, table_width=min(width, changes.get("table_width", width))))
            assert _size(short, groups) <= _size(_attention("paged_attention", 64 * n, **changes), groups)
    for rows in (1, 7, 64):
        a = _attention("paged_attention", rows * n, **changes)
        sizes = {_size(a, g) for g in (1, 2, 5, 64, 1000)}
        assert len(sizes) == 1


def test_sizes_of_a_workspace():
    import torch
    c = Case([(1500, [1600, 1501, 1500])], heads=24, kv=2, seed=17)
    pa._sizes.clear()
    out, lse = c.run()
    (need,) = pa._sizes.values()
    assert need > 0
    exact = torch.full((need + 64,), 0xff, dtype=torch.uint8, device="cuda")
    again = c.run(workspace=exact[:need])
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1]) and bool((exact[need:] == 0xff).all())
    with pytest.raises(ValueError, match="workspace"):
        c.run(workspace=exact[:need - 1])
    with pytest.raises(rrt.TopKError, match="aligned"):
        c.run(workspace=exact[8:8 + need])


def test_refusals_of_tensors():
    import torch
    c = Case([(16, [20, 30])], seed=18)
    t, n, s, m = dev(c.table), dev(c.lengths), dev(c.starts), dev(c.shared)
    for args, err in [((c.q.float(), c.k, c.v, t, n, s, m), TypeError), ((c.q, c.k.half(), c.v.half(), t, n, s, m), TypeError),
                      ((c.q, c.k, c.v, t, n, s[:1], m), ValueError), ((c.q, c.k, c.v, t, n, s.long(), m), TypeError),
                      ((c.q, c.k, c.v, t, n, s, m.cpu()), TypeError), ((c.q, c.k, c.v[:-1], t, n, s, m), ValueError),
                      ((c.q[:, :7], c.k, c.v, t, n, s, m), ValueError), ((c.q, c.k, c.v, t[:1], n, s, m), ValueError),
                      ((c.q.clone().requires_grad_(), c.k, c.v, t, n, s, m), RuntimeError)]:
        with pytest.raises(err):
            rrt.paged_prefix_attention(*args)
    with pytest.raises(ValueError):
        c.run(out=c.q[:1])
