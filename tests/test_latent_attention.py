"""latent_attention on the GPU against 64-bit sums."""

from __future__ import annotations

import numpy as np
import pytest

import row_radix_top_amd as rrt
from tests import paged_ref
from tests.gpu_util import note, require_gpu

pytestmark = pytest.mark.gpu

ROPE = 64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


class Case:
    """A latent cache with shuffled pages, every place that no row may read
    filled with NaN."""

    def __init__(self, lengths, *, heads=20, dim=512, dtype="bfloat16", store="same", page_size=16, chosen=None, seed=0,
                 poison=True, spread=1.0, rising=False):
        import torch
        rng = np.random.default_rng(seed)
        self.lengths = np.asarray(lengths, dtype=np.int32)
        rows2d = self.lengths if self.lengths.ndim == 2 else self.lengths[:, None]
        self.next_n, self.chosen = rows2d.shape[1], None if chosen is None else np.asarray(chosen, dtype=np.int32)
        seqs, rows = rows2d.shape[0], rows2d.size
        need = -(-np.maximum(rows2d.max(axis=1), 0) // page_size)
        self.page_size, self.width, self.pages = page_size, max(1, int(need.max())), int(need.sum()) + 3
        order, at = rng.permutation(self.pages), 0
        self.table = np.full((seqs, self.width), -1, dtype=np.int32)
        for s in range(seqs):
            self.table[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
        self.heads, self.dim = heads, dim
        self.dt = getattr(torch, dtype)
        self.st = self.dt if store == "same" else getattr(torch, store)
        torch.manual_seed(seed)
        self.q = (torch.randn(rows, heads, dim + ROPE, device="cuda") * spread).to(self.dt)
        c = torch.randn(self.pages, page_size, dim + ROPE, device="cuda")
        if rising:  # scores that grow along the row, so that the softmax's reference has to follow
            for s in range(seqs):
                slots = paged_ref.slots_of(self.table[s], np.arange(int(rows2d[s].max())), page_size, self.pages)
                up = torch.linspace(0, 3, len(slots), device="cuda")[:, None]
                c.view(-1, dim + ROPE)[torch.as_tensor(slots, device="cuda")] += up * self.q[s * self.next_n, 0].float()
        self.c = c.to(self.st)
        self.by = torch.full((1,), 0.75, device="cuda") if self.st == torch.float8_e4m3fn else None
        self.scale = (128 + ROPE) ** -0.5
        if poison:
            used = np.zeros(self.pages * page_size, dtype=bool)
            for r in range(rows):
                s = self.row_slots(r)
                used[s[s >= 0]] = True
            flat = self.c.view(-1, dim + ROPE)
            bits = flat.view(torch.uint8) if self.st == torch.float8_e4m3fn else flat.view(torch.int16)
            bits[torch.as_tensor(~used, device="cuda")] = 0x7f if self.st == torch.float8_e4m3fn else 0x7fff

    def row_slots(self, r):
        c = None if self.chosen is None else self.chosen[r]
        p = paged_ref.row_positions(self.lengths.reshape(-1)[r], self.width * self.page_size, c)
        return paged_ref.slots_of(self.table[r // self.next_n], p, self.page_size, self.pages)

    def run(self, **kw):
        import torch
        dev = lambda x: torch.as_tensor(x, device="cuda")  # noqa: E731
        return rrt.latent_attention(self.q, self.c, dev(self.table), dev(self.lengths), softmax_scale=self.scale,
                                    chosen=None if self.chosen is None else dev(self.chosen), scale=self.by, **kw)

    def expected(self):
        import torch
        q, c = self.q.double().cpu().numpy(), self.c.double().cpu().numpy().reshape(-1, self.dim + ROPE)
        if self.by is not None:
            c = c * float(self.by)
        u, fp16 = paged_ref.half_step(self.dt), self.dt == torch.float16
        rows = q.shape[0]
        res = [np.zeros((rows, self.heads, self.dim)), np.zeros((rows, self.heads)),
               np.zeros((rows, self.heads, self.dim)), np.zeros((rows, self.heads))]
        for r in range(rows):
            s = self.row_slots(r)
            k = c[s[s >= 0]]
            for h in range(self.heads):
                got = paged_ref.attend(q[r, h], k, k[:, :self.dim], self.scale, u, fp16)
                for dst, x in zip(res, got):
                    dst[r, h] = x
        return res

    def check(self, what, **kw):
        note(f"latent_attention {what} rows={self.q.shape[0]} heads={self.heads} dim={self.dim} {self.dt} {self.st} "
             f"page={self.page_size} chosen={self.chosen is not None} {kw}")
        out, lse = self.run(**kw)
        exp, elog, tol, tlog = self.expected()
        paged_ref.check(out.double().cpu().numpy(), exp, tol, f"{what} out")
        paged_ref.check(lse.double().cpu().numpy(), elog, tlog, f"{what} lse")
        return out, lse


@pytest.mark.parametrize("splits", [0, 2])
def test_many_ragged_rows(splits):
    """Rows run longest first, 64 at a time: each exactly once."""
    rng = np.random.default_rng(6)
    Case(rng.integers(0, 400, size=70), heads=2, dim=256, seed=6).check("many rows", max_splits=splits)


def _choose(rng, lengths, k):
    rows = []
    for n in lengths:
        pick = np.sort(rng.permutation(n)[:min(k, n)]) if n > 0 else np.empty(0, np.int64)
        rows.append(np.concatenate([pick, np.full(k - len(pick), -1)]))
    return np.stack(rows)


LENGTHS = [0, 1, 31, 32, 33, 63, 64, 65, 130, 300]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
@pytest.mark.parametrize("dim", [256, 512])
@pytest.mark.parametrize("heads", [1, 16, 20, 33, 64, 128, 130])
def test_dense(dtype, store, dim, heads):
    Case(LENGTHS, heads=heads, dim=dim, dtype=dtype, store=store, seed=heads).check("dense")


@pytest.mark.parametrize("page_size", [1, 5, 24, 64])
@pytest.mark.parametrize("splits", [0, 1, 2, 5, 128])
def test_pages_and_splits(page_size, splits):
    Case([1500, 1, 0, 700, 129], heads=12, page_size=page_size, seed=page_size).check("splits", max_splits=splits)


@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
@pytest.mark.parametrize("heads", [8, 40, 128])
@pytest.mark.parametrize("k", [1, 33, 200])
def test_chosen(store, heads, k):
    rng = np.random.default_rng(k)
    lengths = [1, 40, 0, 200, 900]
    Case(lengths, heads=heads, store=store, chosen=_choose(rng, lengths, k), seed=k).check("chosen")


@pytest.mark.parametrize("dim", [256, 512])
def test_chosen_in_any_order_twice_and_out_of_range(dim):
    rng = np.random.default_rng(1)
    c = rng.integers(-3, 90, size=(4, 150))
    c[1] = -1
    c[2, :10] = [2147483647, -2147483648, 70, 70, 70, 0, 0, 69, 71, 72]
    Case([70, 50, 72, 0], dim=dim, heads=33, chosen=c, seed=2).check("chosen")


@pytest.mark.parametrize("heads", [16, 32, 64, 128])
def test_multi_token_rows_and_rising_scores(heads):
    Case([[64, 65, 66], [0, 1, 2], [300, 1, 290]], heads=heads, seed=3).check("multi-token")
    Case([500, 333], heads=heads, seed=4, rising=True).check("rising", max_splits=1)
    Case([500, 333], heads=heads, seed=5, rising=True, store="float8_e4m3fn").check("rising e4m3", max_splits=2)


def test_later_tokens_that_are_not_finite_do_not_reach_earlier_rows():
    import torch
    c = Case([[40, 41, 42]], heads=20, seed=5)
    s = paged_ref.slots_of(c.table[0], [40, 41], c.page_size, c.pages)
    c.c.view(-1, c.dim + ROPE)[torch.as_tensor(s, device="cuda")] = float("nan")
    out, lse = c.run()
    exp, elog, tol, tlog = c.expected()
    paged_ref.check(out[:1].double().cpu().numpy(), exp[:1], tol[:1], "first row")
    paged_ref.check(lse[:1].double().cpu().numpy(), elog[:1], tlog[:1], "first row lse")
    assert bool(out[1:].isnan().all())


@pytest.mark.parametrize("chosen", [False, True])
@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
def test_bad_pages_are_left_out(chosen, store):
    rng = np.random.default_rng(4)
    lengths = [300, 90, 33]
    c = Case(lengths, chosen=_choose(rng, lengths, 64) if chosen else None, store=store, seed=4, poison=False)
    c.table[0, [0, 7, 18]] = [-1, c.pages, 2147483647]
    c.table[1, :] = -2147483648
    c.table[2, 2] = c.pages + 5
    c.check("bad pages")


def test_strides_streams_graphs_and_large_scores():
    import torch
    Case([600, 37], spread=40.0, seed=10).check("large scores")
    c = Case([400, 64, 3], heads=20, seed=9)
    out, lse = c.check("contiguous")
    wide = torch.zeros(3, 20 + 8, c.dim + ROPE + 64, device="cuda", dtype=c.dt)
    wide[:, 8:, 64:] = c.q
    cache = torch.full((c.pages, 2, c.page_size, c.dim + ROPE + 8), float("nan"), device="cuda", dtype=c.dt)
    cache[:, 1, :, :c.dim + ROPE] = c.c
    c.q, c.c = wide[:, 8:, 64:], cache[:, 1, :, :c.dim + ROPE]
    again = c.run()
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = c.run(stream=s)
    s.synchronize()
    assert torch.equal(other[0], out)
    lengths, table = torch.as_tensor(c.lengths, device="cuda"), torch.as_tensor(c.table, device="cuda")
    graphs = []
    for splits in (1, 3):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = rrt.latent_attention(c.q, c.c, table, lengths, softmax_scale=c.scale, max_splits=splits)
        graphs.append((g, res, splits))
    for step in range(3):
        now = torch.tensor([400 - 130 * step, 64 - step, 3 - step], dtype=torch.int32, device="cuda")
        lengths.copy_(now)
        for g, _, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, res, splits in graphs:
            eager = rrt.latent_attention(c.q, c.c, table, now, softmax_scale=c.scale, max_splits=splits)
            assert torch.equal(res[0], eager[0]) and torch.equal(res[1], eager[1])


def test_offsets_past_32_bits():
    import torch
    c = Case([130], heads=8, dim=256, page_size=64, seed=11, poison=False)
    near = c.run()
    pages = (1 << 32) // (64 * 320) + 4
    cache = torch.empty(pages, 64, 320, device="cuda", dtype=c.dt)
    table = torch.tensor([[pages - 1, 0, pages - 3]], dtype=torch.int32, device="cuda")
    cache[table[0].long()] = c.c[torch.as_tensor(c.table[0], device="cuda").long()]
    far = rrt.latent_attention(c.q, cache, table, torch.as_tensor(c.lengths, device="cuda"), softmax_scale=c.scale)
    assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])
