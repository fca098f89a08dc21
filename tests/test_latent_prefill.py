"""latent_prefill on the GPU against 64-bit sums: ragged chunks over paged
contexts, in the expanded form."""

from __future__ import annotations

import math

import numpy as np
import pytest

import row_radix_top_amd as rrt
from tests import paged_ref
from tests.gpu_util import note, require_gpu

pytestmark = pytest.mark.gpu

ROPE, HEAD = 64, 128


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


TWO_PARTS = 1024  # a sequence's first tokens, whose keys are kept to twice the bits


class Case:
    def __init__(self, lengths, new, *, heads=3, dim=256, dtype="bfloat16", store="same", page_size=16, seed=0, gap=0,
                 poison=True, spread=1.0):
        import torch
        rng = np.random.default_rng(seed)
        self.lengths, self.new = np.asarray(lengths, dtype=np.int32), np.asarray(new)
        self.starts = np.concatenate([[gap], gap + np.cumsum(self.new)]).astype(np.int32)
        self.tokens = int(self.starts[-1]) + gap
        need = -(-np.maximum(self.lengths, 0) // page_size)
        self.page_size, self.width, self.pages = page_size, max(1, int(need.max())), int(need.sum()) + 3
        order, at = rng.permutation(self.pages), 0
        self.table = np.full((len(lengths), self.width), -1, dtype=np.int32)
        for s in range(len(lengths)):
            self.table[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
        self.heads, self.dim = heads, dim
        self.dt = getattr(torch, dtype)
        self.st = self.dt if store == "same" else getattr(torch, store)
        torch.manual_seed(seed)
        self.q = (torch.randn(self.tokens, heads, HEAD + ROPE, device="cuda") * spread).to(self.dt)
        self.wk, self.wv = ((torch.randn(heads, HEAD, dim, device="cuda") / math.sqrt(dim)).to(self.dt) for _ in range(2))
        self.c = torch.randn(self.pages, page_size, dim + ROPE, device="cuda").to(self.st)
        self.by = torch.full((1,), 0.75, device="cuda") if self.st == torch.float8_e4m3fn else None
        self.scale = (HEAD + ROPE) ** -0.5
        if poison:
            used = np.zeros(self.pages * page_size, dtype=bool)
            for s in range(len(lengths)):
                slots = self.slots(s)
                used[slots[slots >= 0]] = True
            self.poison(~used)

    def poison(self, mask):
        import torch
        flat = self.c.view(-1, self.dim + ROPE)
        bits = flat.view(torch.uint8) if self.st == torch.float8_e4m3fn else flat.view(torch.int16)
        bits[torch.as_tensor(mask, device="cuda")] = 0x7f if self.st == torch.float8_e4m3fn else 0x7fff

    def slots(self, s):
        n = min(max(int(self.lengths[s]), 0), self.width * self.page_size)
        return paged_ref.slots_of(self.table[s], np.arange(n), self.page_size, self.pages)

    def run(self, context=None, **kw):
        import torch
        dev = lambda x: torch.as_tensor(x, device="cuda")  # noqa: E731
        if context is None:
            context = int(np.clip(self.lengths, 0, self.width * self.page_size).sum())
        return rrt.latent_prefill(self.q, self.c, dev(self.table), dev(self.starts), dev(self.lengths), self.wk, self.wv,
                                  context_tokens=context, softmax_scale=self.scale, scale=self.by, **kw)

    def expected(self):
        """Sums in 64 bits, and their bounds: those of paged_ref.attend, with
        the keys and values rounded to the 16-bit type on top.  A key off by u
        relative to each of its 128 formed dims moves a score by at most u
        sum |q k| scale, which changes the weight by twice that; a value off by
        u |v| moves the output by u A.  Keys of a sequence's first 1024 tokens
        come in two parts and are off by u^2 only, with 128 more products to
        sum, each within 2^-24 of the sum.  The products W c themselves are sums of
        dim fp32 terms: (dim + 2) 2^-24 of their absolute sum, which moves a
        score by that of sum |q| (|W| |c|) and an output by that of p |W| |c|."""
        import torch
        q, c = self.q.double().cpu().numpy(), self.c.double().cpu().numpy().reshape(-1, self.dim + ROPE)
        wk, wv = self.wk.double().cpu().numpy(), self.wv.double().cpu().numpy()
        if self.by is not None:
            c = c * float(self.by)
        u, fp16, f = paged_ref.half_step(self.dt), self.dt == torch.float16, paged_ref.F32
        shape = (self.tokens, self.heads)
        out, lse = np.zeros(shape + (HEAD,)), np.zeros(shape)
        tol, tlog = np.zeros(shape + (HEAD,)), np.zeros(shape)
        for s in range(len(self.lengths)):
            slots = self.slots(s)
            n = len(slots)
            x = c[np.maximum(slots, 0)]
            for j in range(int(self.new[s])):
                t = int(self.starts[s]) + j
                keep = (np.arange(n) <= n - int(self.new[s]) + j) & (slots >= 0)
                for h in range(self.heads):
                    y = x[keep]
                    kn, v = y[:, :self.dim] @ wk[h].T, y[:, :self.dim] @ wv[h].T
                    k = np.concatenate([kn, y[:, self.dim:]], axis=1)
                    o, lg, to, tl = paged_ref.attend(q[t, h], k, v, self.scale, u, fp16)
                    if keep.any():
                        aq = np.abs(q[t, h, :HEAD])
                        ak, av = np.abs(y[:, :self.dim]) @ np.abs(wk[h]).T, np.abs(y[:, :self.dim]) @ np.abs(wv[h]).T
                        grow = (self.dim + 2) * f
                        # keys below the 16-bit type's normal range round by an absolute 2^-25 in fp16
                        ku = np.where(np.flatnonzero(keep) < TWO_PARTS, u * u + 130 * f, u)[:, None]
                        e = float(((np.abs(kn) * ku + ak * grow + (2.0 ** -25 if fp16 else 0)) @ aq).max() * abs(self.scale))
                        p = np.exp(k @ q[t, h] * self.scale - lg)
                        to = to + p @ (np.abs(v) * (u + 2 * e * (1 + u)) + av * grow + (2.0 ** -25 if fp16 else 0))
                        tl = tl + e
                    out[t, h], lse[t, h], tol[t, h], tlog[t, h] = o, lg, to, tl
        return out, lse, tol, tlog

    def check(self, what, **kw):
        note(f"latent_prefill {what} tokens={self.tokens} heads={self.heads} dim={self.dim} {self.dt} {self.st} "
             f"page={self.page_size} lengths={self.lengths.tolist()} new={self.new.tolist()}")
        out, lse = self.run(**kw)
        exp, elog, tol, tlog = self.expected()
        a, b = int(self.starts[0]), int(self.starts[-1])
        paged_ref.check(out[a:b].double().cpu().numpy(), exp[a:b], tol[a:b], f"{what} out")
        paged_ref.check(lse[a:b].double().cpu().numpy(), elog[a:b], tlog[a:b], f"{what} lse")
        return out, lse


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
@pytest.mark.parametrize("dim", [256, 512])
@pytest.mark.parametrize("page_size", [5, 16])
def test_ragged_chunks(dtype, store, dim, page_size):
    Case([1, 64, 65, 200, 3, 129, 300], [1, 64, 1, 130, 0, 129, 33], dim=dim, dtype=dtype, store=store,
         page_size=page_size, seed=dim).check("ragged")


@pytest.mark.parametrize("n,new", [(1, 1), (63, 63), (64, 1), (127, 127), (128, 128), (129, 129), (257, 200)])
def test_one_sequence(n, new):
    Case([n], [new], heads=2, seed=n).check("one sequence")


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
def test_past_the_tokens_kept_in_two_parts(dtype, store):
    Case([1025, 1100, 2100, 1024], [2, 40, 3, 1], heads=2, dtype=dtype, store=store, seed=9).check("two parts")


@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
def test_few_rows_share_out_their_contexts(store):
    """Long contexts are split and joined; short ones beside them are not, and rows outside are left alone."""
    import torch
    c = Case([5000, 70, 1500, 2600, 0, 3900], [3, 70, 130, 1, 4, 2], heads=2, store=store, gap=5, seed=14)  # 3900: some parts are empty
    out = torch.full((c.tokens, c.heads, HEAD), 3.0, device="cuda", dtype=c.dt)
    lse = torch.full((c.tokens, c.heads), 3.0, device="cuda")
    c.check("split", out=out, lse=lse)
    for x in (out, lse):
        assert bool((x[:5] == 3).all()) and bool((x[-5:] == 3).all())
    c.table[0, 3:40] = -1  # a part whose tokens are mostly missing
    c.table[3, 100:] = -1
    c.check("split, missing pages")


@pytest.mark.parametrize("by", [0.0, -0.04, 448.0])
def test_scales_of_the_cache(by):
    c = Case([70, 9], [70, 3], heads=2, store="float8_e4m3fn", seed=10)
    c.by.fill_(by)
    c.check("cache scale")


def test_softmax_scales_of_zero_and_below():
    for scale in (0.0, -0.05):
        c = Case([200, 9], [70, 3], heads=2, seed=11)
        c.scale = scale
        c.check("softmax scale")


def test_many_sequences():
    rng = np.random.default_rng(3)
    lengths = rng.integers(0, 20, size=150)
    new = np.array([rng.integers(0, n + 1) for n in lengths])
    Case(lengths, new, heads=1, page_size=4, seed=3).check("many sequences")


def test_more_new_tokens_than_context():
    """The first rows of such a chunk see nothing."""
    out, lse = Case([10, 0], [25, 7], heads=2, seed=4).check("short context")
    assert bool((out[:15] == 0).all()) and bool((lse[25:] == -math.inf).all())


def test_rows_outside_every_sequence_are_left_alone():
    import torch
    c = Case([40, 30], [20, 30], gap=7, seed=5)
    out = torch.full((c.tokens, c.heads, HEAD), 3.0, device="cuda", dtype=c.dt)
    lse = torch.full((c.tokens, c.heads), 3.0, device="cuda")
    c.check("gap", out=out, lse=lse)
    for x in (out, lse):
        assert bool((x[:7] == 3).all()) and bool((x[-7:] == 3).all())


def test_bad_pages_and_clamped_lengths():
    c = Case([100, 70, 50], [60, 70, 10], seed=6, poison=False)
    c.table[0, [0, 3]] = [-1, c.pages]
    c.table[1, :] = -2147483648
    c.table[2, 1] = 2147483647
    c.check("bad pages")
    c = Case([64, 40], [20, 40], seed=7, poison=False)
    c.lengths[0] = 2147483647  # the table holds 64
    c.check("clamped")


@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
def test_later_tokens_that_are_not_finite_do_not_reach_earlier_rows(store):
    import torch
    c = Case([150], [100], heads=2, store=store, seed=8)
    bad = np.zeros(c.pages * c.page_size, dtype=bool)
    bad[c.slots(0)[[120, 149]]] = True
    c.poison(bad)
    out, lse = c.run()
    exp, elog, tol, tlog = c.expected()
    k = 120 - 50
    paged_ref.check(out[:k].double().cpu().numpy(), exp[:k], tol[:k], "earlier rows")
    paged_ref.check(lse[:k].double().cpu().numpy(), elog[:k], tlog[:k], "earlier rows lse")
    assert bool(out[k:].isnan().all()) and bool(lse[k:].isnan().all())


def test_values_past_the_range_reach_the_rows_that_see_them():
    """A value that fp16 does not hold is an infinity in the rows that see it, whole tiles and others."""
    import torch
    c = Case([260], [260], heads=2, dtype="float16", seed=12)
    c.wv[:, 0] = 200.0
    flat = c.c.view(-1, c.dim + ROPE)
    slot = int(c.slots(0)[5])
    flat[torch.as_tensor(c.slots(0), device="cuda"), :c.dim] -= flat[torch.as_tensor(c.slots(0), device="cuda"), :c.dim].mean(
        dim=1, keepdim=True)  # values of dim 0 near 0
    flat[slot, :c.dim] += 3.0
    out, lse = c.run()
    assert bool((out[5:, :, 0] == math.inf).all()) and bool(out[:5].isfinite().all())
    assert bool(out[:, :, 1:].isfinite().all()) and bool(lse.isfinite().all())


def test_context_tokens_too_small():
    """Sequences that do not fit give NaN; those before them are right."""
    c = Case([100, 500, 90], [10, 20, 30], heads=2, seed=9)
    out, lse = c.run(context=200)
    whole, wlse = c.run()
    assert torch_equal(out[:10], whole[:10]) and torch_equal(lse[:10], wlse[:10])
    assert bool(out[10:].isnan().all()) and bool(lse[10:].isnan().all())


def torch_equal(a, b):
    import torch
    return torch.equal(a, b)


def test_strides_streams_and_graphs():
    import torch
    Case([130, 64], [100, 64], spread=30.0, seed=10).check("large scores")
    c = Case([200, 64, 3], [150, 1, 3], heads=4, seed=11)
    out, lse = c.check("contiguous")
    wide = torch.zeros(c.tokens, c.heads + 2, HEAD + ROPE + 64, device="cuda", dtype=c.dt)
    wide[:, 2:, 64:] = c.q
    cache = torch.full((c.pages, 2, c.page_size, c.dim + ROPE + 8), float("nan"), device="cuda", dtype=c.dt)
    cache[:, 1, :, :c.dim + ROPE] = c.c
    c.q, c.c = wide[:, 2:, 64:], cache[:, 1, :, :c.dim + ROPE]
    again = c.run()
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = c.run(stream=s)
    s.synchronize()
    assert torch.equal(other[0], out)
    lengths, starts, table = (torch.as_tensor(x, device="cuda") for x in (c.lengths, c.starts, c.table))

    def call():
        return rrt.latent_prefill(c.q, c.c, table, starts, lengths, c.wk, c.wv, context_tokens=400, softmax_scale=c.scale)

    g, h = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        one = call()
    with torch.cuda.graph(h):
        two = call()
    for step in range(3):
        lengths.copy_(torch.tensor([200 - 20 * step, 64, 3], dtype=torch.int32))
        starts.copy_(torch.tensor([0, 150 - 20 * step, 151 - 20 * step, 154 - 20 * step], dtype=torch.int32))
        end = 154 - 20 * step
        g.replay(), h.replay()
        torch.cuda.synchronize()
        eager = call()
        for res in (one, two):
            assert torch.equal(res[0][:end], eager[0][:end]) and torch.equal(res[1][:end], eager[1][:end])
