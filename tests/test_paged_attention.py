"""paged_attention on the GPU against 64-bit sums, over head layouts, types,
ragged lengths, chosen positions, bad pages and places that must not count."""

from __future__ import annotations

import math

import numpy as np
import pytest

import row_radix_top_amd as rrt
from tests import paged_ref
from tests.gpu_util import note, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


class Case:
    """A paged cache with shuffled pages, every place that no row may read
    filled with NaN."""

    def __init__(self, lengths, *, heads=8, kv=2, dim=128, dtype="bfloat16", store="same", page_size=16, width=None,
                 chosen=None, seed=0, poison=True, spread=1.0):
        import torch
        rng = np.random.default_rng(seed)
        self.lengths = np.asarray(lengths, dtype=np.int32)
        rows2d = self.lengths if self.lengths.ndim == 2 else self.lengths[:, None]
        self.next_n = rows2d.shape[1]
        seqs, rows = rows2d.shape[0], rows2d.size
        most = np.maximum(rows2d.max(axis=1), 0)
        need = -(-most // page_size)
        self.page_size, self.width = page_size, width or max(1, int(need.max()))
        need = np.minimum(need, self.width)
        self.pages = int(need.sum()) + 3
        order = rng.permutation(self.pages)
        self.table = np.full((seqs, self.width), -1, dtype=np.int32)
        at = 0
        for s in range(seqs):
            self.table[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
        self.heads, self.kv, self.dim = heads, kv, dim
        self.dt = getattr(torch, dtype)
        self.st = self.dt if store == "same" else getattr(torch, store)
        torch.manual_seed(seed)
        self.q = (torch.randn(rows, heads, dim, device="cuda") * spread).to(self.dt)
        self.k, self.v = (torch.randn(self.pages, page_size, kv, dim, device="cuda").to(self.st) for _ in range(2))
        self.ks = self.vs = None
        if self.st == torch.float8_e4m3fn:
            self.ks, self.vs = (torch.rand(kv, device="cuda") + 0.5 for _ in range(2))
        self.chosen = None if chosen is None else np.asarray(chosen, dtype=np.int32)
        self.scale = dim ** -0.5
        if poison:
            used = np.zeros(self.pages * page_size, dtype=bool)
            for r in range(rows):
                s = self.row_slots(r)
                used[s[s >= 0]] = True
            bad = torch.as_tensor(~used, device="cuda")
            for c in (self.k, self.v):
                flat = c.view(-1, kv, dim)
                bits = flat.view(torch.uint8) if self.st == torch.float8_e4m3fn else flat.view(torch.int16)
                bits[bad] = 0x7f if self.st == torch.float8_e4m3fn else 0x7fff

    def row_slots(self, r):
        c = None if self.chosen is None else self.chosen[r]
        p = paged_ref.row_positions(self.lengths.reshape(-1)[r], self.width * self.page_size, c)
        return paged_ref.slots_of(self.table[r // self.next_n], p, self.page_size, self.pages)

    def run(self, **kw):
        import torch
        dev = lambda x: torch.as_tensor(x, device="cuda")  # noqa: E731
        kw.setdefault("chosen", None if self.chosen is None else dev(self.chosen))
        return rrt.paged_attention(self.q, self.k, self.v, dev(self.table), dev(self.lengths), k_scale=self.ks,
                                   v_scale=self.vs, softmax_scale=self.scale, **kw)

    def expected(self):
        import torch
        q, k, v = (x.double().cpu().numpy() for x in (self.q, self.k, self.v))
        if self.ks is not None:
            k = k * self.ks.double().cpu().numpy()[:, None]
            v = v * self.vs.double().cpu().numpy()[:, None]
        k, v = k.reshape(-1, self.kv, self.dim), v.reshape(-1, self.kv, self.dim)
        u, fp16 = paged_ref.half_step(self.dt), self.dt == torch.float16
        rows = q.shape[0]
        res = [np.zeros((rows, self.heads, self.dim)), np.zeros((rows, self.heads)),
               np.zeros((rows, self.heads, self.dim)), np.zeros((rows, self.heads))]
        group = self.heads // self.kv
        for r in range(rows):
            s = self.row_slots(r)
            s = s[s >= 0]
            for h in range(self.heads):
                got = paged_ref.attend(q[r, h], k[s, h // group], v[s, h // group], self.scale, u, fp16)
                for dst, x in zip(res, got):
                    dst[r, h] = x
        return res

    def check(self, what, **kw):
        note(f"paged_attention {what} rows={self.q.shape[0]} heads={self.heads}/{self.kv} dim={self.dim} "
             f"{self.dt} {self.st} page={self.page_size} chosen={self.chosen is not None} {kw}")
        out, lse = self.run(**kw)
        exp, elog, tol, tlog = self.expected()
        paged_ref.check(out.double().cpu().numpy(), exp, tol, f"{what} out")
        paged_ref.check(lse.double().cpu().numpy(), elog, tlog, f"{what} lse")
        return out, lse


LENGTHS = [0, 1, 2, 31, 32, 33, 127, 128, 129, 255, 511, 700]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv", [(1, 1), (8, 2), (40, 4), (20, 1)])
def test_dense(dtype, store, dim, heads, kv):
    Case(LENGTHS, heads=heads, kv=kv, dim=dim, dtype=dtype, store=store).check("dense")


@pytest.mark.parametrize("page_size", [1, 5, 24, 64])
@pytest.mark.parametrize("splits", [0, 1, 2, 5, 128])
def test_pages_and_splits(page_size, splits):
    Case([3000, 1, 0, 1290, 257], page_size=page_size, seed=page_size).check("splits", max_splits=splits)


@pytest.mark.parametrize("heads,kv", [(8, 2), (12, 2), (32, 1), (4, 4)])
@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
def test_multi_token_rows(heads, kv, store):
    """Rows of a sequence see different lengths; what only the later ones see
    is finite for them and NaN for none."""
    lengths = [[64, 65, 66], [0, 1, 2], [33, 200, 31], [0, 0, 0], [700, 1, 640], [95, 96, 97]]
    Case(lengths, heads=heads, kv=kv, store=store, seed=3).check("multi-token")


def test_later_tokens_that_are_not_finite_do_not_reach_earlier_rows():
    import torch
    c = Case([[40, 41, 42]], heads=8, kv=2, seed=5)
    s = paged_ref.slots_of(c.table[0], [40, 41], c.page_size, c.pages)
    for cache, value in ((c.k, float("inf")), (c.v, float("nan"))):
        cache.view(-1, c.kv, c.dim)[torch.as_tensor(s, device="cuda")] = value
    out, lse = c.run()
    exp, elog, tol, tlog = c.expected()
    paged_ref.check(out[:1].double().cpu().numpy(), exp[:1], tol[:1], "first row")
    paged_ref.check(lse[:1].double().cpu().numpy(), elog[:1], tlog[:1], "first row lse")
    assert bool(out[1:].isnan().all())


@pytest.mark.parametrize("next_n", [1, 2])
@pytest.mark.parametrize("n", [64, 65, 150])
def test_many_ragged_rows(n, next_n):
    """Rows run longest first, 64 groups at a time: each exactly once."""
    rng = np.random.default_rng(n)
    last = rng.integers(0, 300, size=n)
    lengths = last if next_n == 1 else np.stack([np.maximum(last - 1, 0), last], axis=1)
    Case(lengths, heads=2, kv=1, dim=64, seed=n).check("many rows")
    Case(lengths, heads=2, kv=1, dim=64, seed=n).check("many rows", max_splits=3)


def _choose(rng, lengths, k, keep=1.0):
    rows = []
    for n in lengths:
        pick = np.sort(rng.permutation(n)[:min(k, n)]) if n > 0 else np.empty(0, np.int64)
        rows.append(np.concatenate([pick, np.full(k - len(pick), -1)]))
    return np.stack(rows)


@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("k", [1, 33, 512, 700])
def test_chosen(store, dim, k):
    rng = np.random.default_rng(k)
    lengths = [1, 40, 0, 512, 900, 2000]
    Case(lengths, dim=dim, store=store, chosen=_choose(rng, lengths, k), seed=k).check("chosen")


def test_chosen_in_any_order_twice_and_out_of_range():
    rng = np.random.default_rng(1)
    c = rng.integers(-3, 90, size=(4, 300))  # repeated, unordered, some past the length
    c[1] = -1
    c[2, :10] = [2147483647, -2147483648, 70, 70, 70, 0, 0, 69, 71, 72]
    Case([70, 50, 72, 0], chosen=c, seed=2).check("chosen")


def test_chosen_multi_token():
    rng = np.random.default_rng(7)
    lengths = np.array([[500, 501], [3, 4], [0, 1]])
    Case(lengths, heads=40, kv=4, chosen=_choose(rng, lengths.reshape(-1), 128), seed=7).check("chosen multi-token")


@pytest.mark.parametrize("chosen", [False, True])
def test_bad_pages_are_left_out(chosen):
    rng = np.random.default_rng(4)
    lengths = [300, 90, 33]
    c = Case(lengths, chosen=_choose(rng, lengths, 64) if chosen else None, seed=4, poison=False)
    c.table[0, [0, 7, 18]] = [-1, c.pages, 2147483647]
    c.table[1, :] = -2147483648  # nothing left
    c.table[2, 2] = c.pages + 5
    c.check("bad pages")


def test_lengths_out_of_range_are_clamped():
    c = Case([100, 50], seed=8, width=4)
    c.lengths = np.array([2147483647, -5], dtype=np.int32)
    c.table[0, :] = [0, 1, 2, 3]
    c.k.normal_(), c.v.normal_()
    c.check("clamped")


def test_strided_views():
    import torch
    c = Case([200, 64, 3], heads=8, kv=2, seed=9)
    wide = torch.empty(3, 3 * 8, 128, device="cuda", dtype=c.dt)
    wide[:, 8:16] = c.q
    c.q = wide[:, 8:16]
    both = torch.stack([c.k, c.v], dim=1).transpose(2, 3).contiguous()  # pages of [2, heads, tokens, dim]
    c.k, c.v = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    out, lse = c.run()
    k, v = c.k.contiguous(), c.v.contiguous()
    c.k, c.v = k, v
    exp, elog, tol, tlog = c.expected()
    paged_ref.check(out.double().cpu().numpy(), exp, tol, "strided")
    table = torch.full((3, c.width + 5), -1, device="cuda", dtype=torch.int32)
    table[:, :c.width] = torch.as_tensor(c.table, device="cuda")
    again, _ = rrt.paged_attention(c.q, c.k, c.v, table[:, :c.width], torch.as_tensor(c.lengths, device="cuda"),
                                   softmax_scale=c.scale)
    assert torch.equal(again, out)


def test_large_scores_and_far_offsets():
    """Scores of some hundreds (weights down to zero), and a pool whose far
    pages lie past 2^32 elements."""
    import torch
    Case([600, 37], spread=60.0, seed=10).check("large scores")
    pages, page_size = 1 << 15, 512  # x 2 heads x 128 = 2^32 elements each
    k = torch.empty(pages + 8, page_size, 2, 128, device="cuda", dtype=torch.bfloat16)
    v = torch.empty_like(k)
    table = np.array([[pages + 7, pages + 1]], dtype=np.int32)
    c = Case([900], page_size=page_size, seed=11, poison=False)
    k[table[0]] = c.k[c.table[0]]
    v[table[0]] = c.v[c.table[0]]
    near = c.run()
    out = rrt.paged_attention(c.q, k, v, torch.as_tensor(table, device="cuda"),
                              torch.as_tensor(c.lengths, device="cuda"), softmax_scale=c.scale)
    assert torch.equal(out[0], near[0]) and torch.equal(out[1], near[1])


def test_outputs_of_other_streams_graphs_and_rows_behind():
    import torch
    c = Case([[900, 901], [40, 41]], seed=12)
    out, lse = c.check("eager")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = c.run(stream=s)
    s.synchronize()
    assert torch.equal(other[0], out) and torch.equal(other[1], lse)
    # Two graphs with workspaces of their own, replayed in turn on new lengths.
    lengths = torch.as_tensor(c.lengths, device="cuda")
    table = torch.as_tensor(c.table, device="cuda")
    graphs = []
    for splits in (2, 5):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = rrt.paged_attention(c.q, c.k, c.v, table, lengths, softmax_scale=c.scale, max_splits=splits)
        graphs.append((g, res, splits))
    for step in range(3):
        now = torch.tensor([[900 - 200 * step, 901], [40 - step, 41 - step]], dtype=torch.int32, device="cuda")
        lengths.copy_(now)
        for g, _, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, res, splits in graphs:
            eager = rrt.paged_attention(c.q, c.k, c.v, table, now, softmax_scale=c.scale, max_splits=splits)
            assert torch.equal(res[0], eager[0]) and torch.equal(res[1], eager[1])
    # Rows of the output buffer behind the batch stay as they were.
    buf = torch.full((6, c.heads, c.dim), 7.0, device="cuda", dtype=c.dt)
    log = torch.full((6, c.heads), 7.0, device="cuda")
    c.run(out=buf[:4], lse=log[:4])
    assert torch.equal(buf[:4], out) and bool((buf[4:] == 7).all()) and bool((log[4:] == 7).all())


def test_refusals_of_tensors():
    import torch
    c = Case([5, 6], seed=13)
    t, n = torch.as_tensor(c.table, device="cuda"), torch.as_tensor(c.lengths, device="cuda")
    for args, err in [((c.q.float(), c.k, c.v, t, n), TypeError), ((c.q, c.k.half(), c.v.half(), t, n), TypeError),
                      ((c.q[:, :7], c.k, c.v, t, n), ValueError), ((c.q, c.k, c.v[:-1], t, n), ValueError),
                      ((c.q, c.k, c.v, t[:1], n), ValueError), ((c.q, c.k, c.v, t, n[:1]), ValueError),
                      ((c.q, c.k, c.v, t.long(), n), TypeError), ((c.q, c.k, c.v, t, n.cpu()), TypeError),
                      ((c.q[:, :, ::2], c.k[..., ::2], c.v[..., ::2], t, n), ValueError)]:
        with pytest.raises(err):
            rrt.paged_attention(*args)
    with pytest.raises(ValueError):
        c.run(workspace=torch.empty(1, device="cuda"), max_splits=2) if c.width > 40 else c.run(out=c.q[:1])
    with pytest.raises(ValueError):
        rrt.paged_attention(c.q, c.k, c.v, t, n, k_scale=torch.ones(2, device="cuda"))
    assert math.isclose(128 ** -0.5, c.scale)
