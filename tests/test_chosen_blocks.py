"""paged_bounds, paged_block_select and paged_block_attention on the GPU: the
first two exactly against their definition in whole numbers, the third against
64-bit sums."""

from __future__ import annotations

import numpy as np
import pytest

import row_radix_top_amd as rrt
from tests import paged_ref, shared_ref
from tests.gpu_util import note, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def dev(x):
    import torch
    return torch.as_tensor(np.asarray(x), device="cuda").to(torch.int32)


def floats(x):
    return x.float().cpu().numpy()


class Keys:
    """A key cache with shuffled pages, its bounds, and rows over it."""

    def __init__(self, lengths, *, heads=8, kv=2, dim=128, dtype="bfloat16", store="same", page=16, width=None, seed=0):
        import torch
        self.rng = np.random.default_rng(seed)
        torch.manual_seed(seed)
        self.lengths = np.asarray(lengths, dtype=np.int64)
        self.rows2d = self.lengths if self.lengths.ndim == 2 else self.lengths[:, None]
        self.seqs, self.next_n = self.rows2d.shape
        self.ctx = np.maximum(self.rows2d.max(axis=1), 0)
        need = -(-self.ctx // page)
        self.page, self.width = page, width or max(1, int(need.max()))
        need = np.minimum(need, self.width)
        self.pages = int(need.sum()) + 3
        order = self.rng.permutation(self.pages)
        self.table = np.full((self.seqs, self.width), -1, dtype=np.int64)
        at = 0
        for s in range(self.seqs):
            self.table[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
        self.heads, self.kv, self.dim = heads, kv, dim
        self.dt = getattr(torch, dtype)
        self.store = dtype if store == "same" else store
        self.st = getattr(torch, self.store)
        rows = self.rows2d.size
        self.q = torch.randn(rows, heads, dim, device="cuda").to(self.dt)
        self.k = torch.randn(self.pages, page, kv, dim, device="cuda").to(self.st)
        self.bounds = torch.randint(-127, 128, (self.pages, kv, 2, dim), device="cuda", dtype=torch.int8)
        self.scales = torch.rand(self.pages, kv, device="cuda") + 0.5

    def update(self, new, **kw):
        starts = np.concatenate([[0], np.cumsum(new)])
        rrt.paged_bounds(self.k, dev(self.table), dev(starts), dev(self.ctx), self.bounds, self.scales,
                         num_tokens=kw.pop("num_tokens", int(starts[-1])), **kw)

    def expected_bounds(self, new):
        b, s = self.bounds.cpu().numpy().astype(np.int64), self.scales.cpu().numpy().copy()
        k = floats(self.k)
        for q in range(self.seqs):
            n = min(int(self.ctx[q]), self.width * self.page)
            fresh = min(int(new[q]), n)
            for j in range((n - fresh) // self.page, -(-n // self.page) if fresh else 0):
                p = self.table[q, j]
                if not 0 <= p < self.pages:
                    continue
                for h in range(self.kv):
                    b[p, h], s[p, h] = shared_ref.bounds(k[p, :min(self.page, n - j * self.page), h],
                                                         shared_ref.LARGEST[self.store])
        return b, s

    def check_bounds(self, new, **kw):
        note(f"bounds {self.store} dim={self.dim} kv={self.kv} page={self.page} ctx={self.ctx.tolist()[:8]} new={list(new)[:8]}")
        exp = self.expected_bounds(new)
        self.update(new, **kw)
        np.testing.assert_array_equal(self.bounds.cpu().numpy(), exp[0])
        np.testing.assert_array_equal(self.scales.cpu().numpy(), exp[1])

    def select(self, k, **kw):
        return rrt.paged_block_select(self.q, self.bounds, self.scales, dev(self.table), dev(self.lengths),
                                      page_size=self.page, num_blocks=k, **kw)

    def check_select(self, k, first=1, last=1, **kw):
        note(f"select {self.dt} heads={self.heads}/{self.kv} dim={self.dim} page={self.page} rows={self.rows2d.shape} "
             f"width={self.width} k={k} first={first} last={last}")
        got = self.select(k, first=first, last=last, **kw)
        q, b, s = floats(self.q), self.bounds.cpu().numpy(), self.scales.cpu().numpy()
        group = self.heads // self.kv
        most = min(self.width * self.page, 1 << 30)
        exp = np.full((self.rows2d.size, self.kv, k), -1)
        for r, n in enumerate(self.rows2d.reshape(-1)):
            have = -(-shared_ref.clamp(n, most) // self.page)
            p = self.table[r // self.next_n, :have]
            there = (p >= 0) & (p < self.pages)
            at = np.where(there, p, 0)
            for h in range(self.kv):
                x = shared_ref.scores(q[r, h * group:(h + 1) * group], b[at, h], s[at, h],
                                      shared_ref.LARGEST["bfloat16" if "bf" in str(self.dt) else "float16"])
                exp[r, h] = shared_ref.choose(x, there, k, first, last)
        np.testing.assert_array_equal(got.cpu().numpy(), exp)
        return got


LENGTHS = [0, 1, 15, 16, 17, 160, 161, 700]


@pytest.mark.parametrize("dtype,store", [("bfloat16", "same"), ("float16", "same"), ("float16", "float8_e4m3fn")])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kv", [1, 3])
@pytest.mark.parametrize("page", [1, 5, 16, 64])
def test_bounds(dtype, store, dim, kv, page):
    c = Keys(LENGTHS, kv=kv, heads=kv, dim=dim, dtype=dtype, store=store, page=page)
    for new in ([0, 1, 1, 1, 1, 1, 1, 1], [0, 0, 15, 7, 2, 160, 0, 700], c.ctx):
        c.check_bounds(new)


@pytest.mark.parametrize("seqs", [1, 63, 64, 65, 300])
def test_bounds_of_many_sequences(seqs):
    rng = np.random.default_rng(seqs)
    c = Keys(rng.integers(0, 90, size=seqs), kv=1, heads=1, dim=64, seed=seqs)
    c.check_bounds(np.minimum(rng.integers(0, 40, size=seqs) * (rng.random(seqs) < 0.7), c.ctx))
    c.check_bounds(np.minimum(1, c.ctx), num_tokens=5000)  # room for more


def test_bounds_of_extraordinary_keys():
    import torch
    for store in ("bfloat16", "float16", "float8_e4m3fn"):
        c = Keys([40, 16], kv=1, heads=1, store=store, dtype="float16" if store != "bfloat16" else store, seed=2)
        k = c.k.float()
        p = c.table[0, :3]
        k[p[0]] = 0.0  # nothing but zeros
        k[p[1], 3, 0, 5], k[p[1], :, 0, 6] = float("nan"), float("nan")
        k[p[2], 0, 0, :4] = torch.tensor([1e-30, -1e-30, 3e-5, -6e-8])
        c.k.copy_(k.to(c.st))
        if store != "float8_e4m3fn":
            c.k[c.table[1, 0], 2, 0, 9] = float("-inf")
        c.k[p[2], 8:] = float("nan")  # behind the last token
        c.check_bounds([40, 16])
        assert not bool(c.scales[c.table[0, :3].tolist() + [c.table[1, 0]]].isnan().any())


def test_bounds_of_bad_pages_and_strides():
    import torch
    c = Keys([100, 70, 40], kv=2, heads=2, seed=3)
    c.table[0, [0, 3]] = [-1, c.pages]
    c.table[1, 4] = 2147483647
    c.check_bounds(c.ctx)
    both = torch.zeros(c.pages, 2, 3, 2, 128, device="cuda", dtype=torch.int8)
    wide = torch.zeros(c.pages, 5, device="cuda")
    flat, scales = c.bounds, c.scales
    c.k = c.k.transpose(1, 2).contiguous().transpose(1, 2)
    c.bounds, c.scales = both[:, 1, 1:], wide[:, 2:4]
    c.update(c.ctx)
    real = [int(p) for p in c.table.reshape(-1) if 0 <= p < c.pages]
    assert torch.equal(c.bounds[real], flat[real]) and torch.equal(c.scales[real], scales[real])
    assert not bool(both[:, 0].any()) and not bool(both[:, 1, 0].any()) and not bool(wide[:, :2].any())


def test_bounds_of_starts_that_make_no_sense():
    """Nothing is read or written out of range; pages of sequences in order are right."""
    c = Keys([100, 70, 40], seed=4)
    before = c.bounds.clone(), c.scales.clone()
    for starts in ([0, -5, 3, 2], [2147483647, 0, 2147483647, -2147483648], [-2147483648, 2147483647, 0, 9]):
        rrt.paged_bounds(c.k, dev(c.table), dev(starts), dev([2147483647, -1, 40]), c.bounds, c.scales, num_tokens=64)
    c.bounds.copy_(before[0]), c.scales.copy_(before[1])
    c.check_bounds([100, 70, 40])


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv", [(1, 1), (6, 2), (8, 1), (20, 1), (40, 1), (80, 1), (12, 4)])
def test_choices(dtype, dim, heads, kv):
    c = Keys([0, 1, 16, 17, 300, 801, 800, 640], heads=heads, kv=kv, dim=dim, dtype=dtype, seed=heads)
    c.update(c.ctx)
    for k, first, last in ((2, 1, 1), (7, 0, 0), (16, 3, 2), (50, 1, 1), (64, 64, 0)):
        c.check_select(k, first, last)


@pytest.mark.parametrize("heads,kv,next_n", [(8, 1, 3), (4, 2, 9), (1, 1, 70), (3, 1, 5), (32, 1, 2)])
def test_choices_of_several_rows(heads, kv, next_n):
    rng = np.random.default_rng(next_n)
    last = np.array([0, 5, 260, 1000])
    rows = np.maximum(0, last[:, None] - next_n + 1 + np.arange(next_n))
    rows[3] = rng.integers(0, 1001, size=next_n)
    rows[3, 0] = 1000
    c = Keys(rows, heads=heads, kv=kv, dim=64, seed=next_n)
    c.update(c.ctx)
    c.check_select(9)


@pytest.mark.parametrize("have", [255, 256, 257, 511, 1023, 1025, 4095, 4096, 4097, 9000])
def test_choices_of_long_rows(have):
    """One page a position: each number of blocks on either side of what the
    kernels hold in registers, alone (split) and beside many others (not)."""
    rng = np.random.default_rng(have)
    for others in (0, 140):
        c = Keys([have] + [3] * others, heads=2, kv=2, dim=64, page=1, seed=have)
        c.bounds.copy_(c.bounds.clamp(-20, 20))
        c.check_select(int(rng.integers(2, have)))
        c.check_select(have - 1)
    c.check_select(have + 5)


@pytest.mark.parametrize("heads,kv,seqs,have", [(33, 33, 2, 4096), (136, 17, 4, 4096), (136, 17, 4, 2049)])
def test_choices_whose_scores_fill_a_workgroup(heads, kv, seqs, have):
    """Nine rows a sequence, of one page a position: eight of them share a workgroup, with up to 128 KB of scores."""
    rng = np.random.default_rng(have + heads)
    rows = rng.integers(have - 150, have + 1, size=(seqs, 9))
    rows[0, 0], rows[-1, 3], rows[-1, -1] = have, 0, 7
    c = Keys(rows, heads=heads, kv=kv, dim=64, page=1, width=have, seed=heads)
    c.check_select(33)


def test_the_most_blocks_there_are():
    c = Keys([32768, 32001], heads=1, kv=1, dim=64, page=1, seed=7)
    c.check_select(2000)
    with pytest.raises(rrt.TopKError, match="table_width"):
        Keys([32769], heads=1, kv=1, dim=64, page=1).select(4)


@pytest.mark.parametrize("next_n,have", [(1, 300), (1, 2000), (4, 300), (1, 6000)])
def test_ties_go_to_the_lower_block(next_n, have):
    for levels in (1, 3):
        c = Keys([[have] * next_n] * 2, heads=2, kv=2, dim=64, page=1, seed=levels)
        c.bounds.copy_((c.bounds[:1] // 4).expand_as(c.bounds))
        c.scales.copy_(c.scales[0, 0] * (c.scales * 7).int().remainder(levels).float().add(1))
        for k in (2, 40, have - 3):
            c.check_select(k)
            c.check_select(k, 0, 0)


def test_choices_where_pages_are_none():
    c = Keys([640, 100, 64], heads=4, kv=2, seed=8)
    c.update(c.ctx)
    c.table[0, [0, 3, 39]] = [-1, c.pages, 2147483647]
    c.table[1] = -2147483648
    for k in (2, 5, 38, 39, 60):
        c.check_select(k)


def test_choices_of_extraordinary_queries_and_lengths():
    c = Keys([640, 640, 640, 640, 50], heads=4, kv=2, seed=9)
    c.update(c.ctx)
    c.q[0] = 0
    c.q[1, :, 3], c.q[1, 2, 5] = float("inf"), float("nan")
    c.q[2, 1] = float("nan")
    c.q[3] = 1e-38
    c.scales[int(c.table[0, 5])] = 0
    c.bounds[int(c.table[0, 5])] = 0
    c.check_select(7)
    c.lengths = np.array([2147483647, -3, 641, 17, 0])
    c.rows2d = c.lengths[:, None]
    c.check_select(7)


def test_choices_on_other_streams_in_graphs_and_in_one_buffer():
    import torch
    c = Keys([[900, 901], [40, 41]], heads=6, kv=2, page=1, seed=12)
    out = c.check_select(33)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = c.select(33, stream=s)
    s.synchronize()
    assert torch.equal(out, other)
    lengths, table = dev(c.lengths), dev(c.table)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rrt.paged_block_select(c.q, c.bounds, c.scales, table, lengths, page_size=1, num_blocks=33)
    for n in (901, 500, 20, 0):
        lengths.copy_(dev(np.minimum(c.lengths, n)))
        graph.replay()
        torch.cuda.synchronize()
        now = got.clone()
        c.lengths, c.rows2d = np.minimum(c.lengths, n), np.minimum(c.rows2d, n)
        assert torch.equal(now, c.check_select(33))
    # A workspace of a large batch's size serves smaller ones; anything may be in it.
    big = Keys([1500] * 60, heads=4, kv=2, dim=64, page=1, seed=13)
    buffer = torch.full((60 * 2 * 1504 * 4,), 0xff, dtype=torch.uint8, device="cuda")
    table, lengths = dev(big.table), dev(big.lengths)
    for rows in (60, 30, 7, 1):
        args = dict(page_size=1, num_blocks=9)
        a = rrt.paged_block_select(big.q[:rows], big.bounds, big.scales, table[:rows], lengths[:rows], **args)
        b = rrt.paged_block_select(big.q[:rows], big.bounds, big.scales, table[:rows], lengths[:rows], workspace=buffer, **args)
        assert torch.equal(a, b)


class Blocks(Keys):
    """Keys and values, every place that no row may read filled with NaN."""

    def __init__(self, lengths, blocks, **kw):
        import torch
        super().__init__(lengths, **kw)
        self.v = torch.randn(self.pages, self.page, self.kv, self.dim, device="cuda").to(self.st)
        self.ks = self.vs = None
        if self.st == torch.float8_e4m3fn:
            self.ks, self.vs = (torch.rand(self.kv, device="cuda") + 0.5 for _ in range(2))
        rows = self.rows2d.size
        if isinstance(blocks, int):
            made = np.full((rows, self.kv, blocks), -1)
            for r, n in enumerate(self.rows2d.reshape(-1)):
                have = -(-shared_ref.clamp(n, self.width * self.page) // self.page)
                for h in range(self.kv):
                    pick = np.sort(self.rng.permutation(have)[:blocks])
                    made[r, h, :len(pick)] = pick
            blocks = made
        self.blocks = np.asarray(blocks)
        used = np.zeros((self.pages * self.page, self.kv), dtype=bool)
        for r in range(rows):
            for h in range(self.kv):
                s = self.slots(r, h)
                used[s, h] = True
        bad = torch.as_tensor(~used, device="cuda")
        for x in (self.k, self.v):
            flat = x.view(-1, self.kv, self.dim)
            bits = flat.view(torch.uint8) if self.st == torch.float8_e4m3fn else flat.view(torch.int16)
            bits[bad] = 0x7f if self.st == torch.float8_e4m3fn else 0x7fff
        self.scale = self.dim ** -0.5

    def slots(self, r, h):
        """Slots that row r and key-value head h read, as often as they do."""
        n = shared_ref.clamp(self.rows2d.reshape(-1)[r], self.width * self.page)
        out = []
        for b in self.blocks[r, h]:
            if 0 <= b < self.width and b * self.page < n:
                page = self.table[r // self.next_n, b]
                if 0 <= page < self.pages:
                    out.extend(page * self.page + np.arange(min(self.page, n - b * self.page)))
        return np.array(out, dtype=np.int64)

    def run(self, **kw):
        return rrt.paged_block_attention(self.q, self.k, self.v, dev(self.table), dev(self.lengths), dev(self.blocks),
                                         k_scale=self.ks, v_scale=self.vs, softmax_scale=self.scale, **kw)

    def check(self, what, **kw):
        import torch
        note(f"block attention {what} rows={self.rows2d.shape} heads={self.heads}/{self.kv} dim={self.dim} {self.dt} "
             f"{self.st} page={self.page} blocks={self.blocks.shape[2]} {kw}")
        out, lse = self.run(**kw)
        q, k, v = (x.double().cpu().numpy() for x in (self.q, self.k, self.v))
        if self.ks is not None:
            k, v = k * self.ks.double().cpu().numpy()[:, None], v * self.vs.double().cpu().numpy()[:, None]
        k, v = k.reshape(-1, self.kv, self.dim), v.reshape(-1, self.kv, self.dim)
        u, fp16 = paged_ref.half_step(self.dt), self.dt == torch.float16
        rows, group = q.shape[0], self.heads // self.kv
        res = [np.zeros((rows, self.heads, self.dim)), np.zeros((rows, self.heads)),
               np.zeros((rows, self.heads, self.dim)), np.zeros((rows, self.heads))]
        for r in range(rows):
            for h in range(self.heads):
                s = self.slots(r, h // group)
                for dst, x in zip(res, paged_ref.attend(q[r, h], k[s, h // group], v[s, h // group], self.scale, u, fp16)):
                    dst[r, h] = x
        paged_ref.check(out.double().cpu().numpy(), res[0], res[2], f"{what} out")
        paged_ref.check(lse.double().cpu().numpy(), res[1], res[3], f"{what} lse")
        return out, lse


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv", [(1, 1), (8, 2), (40, 4), (20, 1)])
def test_attention(dtype, store, dim, heads, kv):
    Blocks([0, 1, 16, 31, 200, 700], 9, heads=heads, kv=kv, dim=dim, dtype=dtype, store=store).check("types")


@pytest.mark.parametrize("page", [1, 5, 24, 64, 200])
@pytest.mark.parametrize("splits", [0, 1, 3, 128])
def test_attention_of_pages_and_splits(page, splits):
    Blocks([3000, 1, 0, 1290, 257], 700 // page + 2, page=page, seed=page).check("splits", max_splits=splits)


def test_attention_of_one_block():
    Blocks([1, 16, 17, 100], 1, seed=1).check("one block")


def test_attention_of_several_rows():
    Blocks([[64, 65, 66], [0, 1, 2], [33, 200, 31]], 4, heads=12, kv=2, seed=2).check("multi-token")


def test_attention_of_blocks_in_any_order_twice_and_outside():
    rng = np.random.default_rng(3)
    b = rng.integers(-3, 12, size=(4, 2, 9))
    b[1] = -1
    b[2, :, :6] = [2147483647, -2147483648, 3, 3, 4, 1 << 27]
    c = Blocks([70, 50, 72, 0], b, seed=3)
    c.check("any blocks")
    wide = Blocks([70, 50], np.array([[[4, 6, 5]] * 2] * 2), seed=4, width=9)  # inside the table, behind the row
    wide.check("behind the row")


def test_attention_where_pages_are_none():
    c = Blocks([300, 90, 33], 8, seed=5)
    c.table[0, [0, 7, 18]] = [-1, c.pages, 2147483647]
    c.table[1] = -2147483648
    c.k.normal_(), c.v.normal_()
    c.check("bad pages")


def test_attention_of_strided_blocks_and_lengths_out_of_range():
    import torch
    c = Blocks([200, 64, 3], 5, seed=6)
    out, _ = c.check("plain")
    wide = torch.full((3, 2, 9), 1, dtype=torch.int32, device="cuda")
    wide[..., 2:7] = dev(c.blocks)
    again, _ = rrt.paged_block_attention(c.q, c.k, c.v, dev(c.table), dev(c.lengths), wide[..., 2:7], softmax_scale=c.scale)
    assert torch.equal(out, again)
    one = wide[:, :1, 2:7].expand(3, 2, 5)  # the same blocks for all heads
    c.blocks = one.cpu().numpy()
    c.k.normal_(), c.v.normal_()
    exp, _ = c.check("shared")
    again, _ = rrt.paged_block_attention(c.q, c.k, c.v, dev(c.table), dev(c.lengths), one, softmax_scale=c.scale)
    assert torch.equal(exp, again)
    c.lengths = np.array([2147483647, -5, 3])
    c.rows2d = c.lengths[:, None]
    c.table[0] = np.where(c.table[0] < 0, 0, c.table[0])
    c.check("clamped")


def test_all_blocks_are_all_positions():
    """With every block chosen the result is paged_attention's, up to the order of sums."""
    c = Blocks([500, 33, 16, 0], np.tile(np.arange(32), (4, 2, 1)), seed=7)
    out, lse = c.run()
    exp, log = rrt.paged_attention(c.q, c.k, c.v, dev(c.table), dev(c.lengths), softmax_scale=c.scale)
    assert float((out.float() - exp.float()).abs().max()) <= 2 * paged_ref.half_step(c.dt) * 4 * float(c.v.float().nan_to_num().abs().max())
    fine = log.isfinite()
    assert torch_equal_inf(lse, log, fine)


def torch_equal_inf(a, b, fine):
    import torch
    return torch.equal(a[~fine], b[~fine]) and float((a - b)[fine].abs().max()) < 1e-5


def test_attention_on_other_streams_in_graphs_and_buffers():
    import torch
    c = Blocks([900, 40], 30, seed=12)
    out, lse = c.check("eager")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = c.run(stream=s)
    s.synchronize()
    assert torch.equal(other[0], out) and torch.equal(other[1], lse)
    lengths, table, blocks = dev(c.lengths), dev(c.table), dev(c.blocks)
    graphs = []
    for splits in (2, 3):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = rrt.paged_block_attention(c.q, c.k, c.v, table, lengths, blocks, softmax_scale=c.scale, max_splits=splits)
        graphs.append((g, res, splits))
    for n in (900, 600, 17):
        lengths.copy_(dev(np.minimum(c.lengths, n)))
        for g, _, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, res, splits in graphs:
            now = rrt.paged_block_attention(c.q, c.k, c.v, table, lengths, blocks, softmax_scale=c.scale, max_splits=splits)
            assert torch.equal(res[0], now[0]) and torch.equal(res[1], now[1])
    buf = torch.full((5, c.heads, c.dim), 7.0, device="cuda", dtype=c.dt)
    log = torch.full((5, c.heads), 7.0, device="cuda")
    big = torch.full((1 << 24,), 0xff, dtype=torch.uint8, device="cuda")
    c.run(out=buf[:2], lse=log[:2], workspace=big)
    assert torch.equal(buf[:2], out) and bool((buf[2:] == 7).all()) and bool((log[2:] == 7).all())


def test_refusals_of_tensors():
    import torch
    c = Blocks([40, 6], 3, seed=13)
    t, n, b = dev(c.table), dev(c.lengths), dev(c.blocks)
    s = dev([0, 40, 46])
    for call, err in [
        (lambda: rrt.paged_bounds(c.k.float(), t, s, n, c.bounds, c.scales, num_tokens=46), TypeError),
        (lambda: rrt.paged_bounds(c.k, t, s[:2], n, c.bounds, c.scales, num_tokens=46), ValueError),
        (lambda: rrt.paged_bounds(c.k, t, s, n, c.bounds[:-1], c.scales, num_tokens=46), ValueError),
        (lambda: rrt.paged_bounds(c.k, t, s, n, c.bounds.short(), c.scales, num_tokens=46), TypeError),
        (lambda: rrt.paged_bounds(c.k, t, s, n, c.bounds, c.scales.double(), num_tokens=46), TypeError),
        (lambda: rrt.paged_bounds(c.k, t, s, n, c.bounds, c.scales, num_tokens=-1), rrt.TopKError),
        (lambda: rrt.paged_block_select(c.q.float(), c.bounds, c.scales, t, n, page_size=16, num_blocks=3), TypeError),
        (lambda: rrt.paged_block_select(c.q, c.bounds, c.scales, t, n, page_size=16, num_blocks=0), ValueError),
        (lambda: rrt.paged_block_select(c.q, c.bounds, c.scales, t, n, page_size=16, num_blocks=2, first=2), rrt.TopKError),
        (lambda: rrt.paged_block_select(c.q, c.bounds, c.scales, t, n, page_size=0, num_blocks=2), rrt.TopKError),
        (lambda: rrt.paged_block_select(c.q, c.bounds, c.scales, t[:1], n, page_size=16, num_blocks=3), ValueError),
        (lambda: rrt.paged_block_select(c.q[..., :64], c.bounds, c.scales, t, n, page_size=16, num_blocks=3), ValueError),
        (lambda: rrt.paged_block_select(c.q[:, :7], c.bounds, c.scales, t, n, page_size=16, num_blocks=3), rrt.TopKError),
        (lambda: c.select(3, out=b[:1]), ValueError),
        (lambda: rrt.paged_block_attention(c.q, c.k, c.v, t, n, b.long()), TypeError),
        (lambda: rrt.paged_block_attention(c.q, c.k, c.v, t, n, b[:, :1]), ValueError),
        (lambda: rrt.paged_block_attention(c.q, c.k, c.v, t, n, b[..., :0]), ValueError),
        (lambda: rrt.paged_block_attention(c.q, c.k, c.v[:-1], t, n, b), ValueError),
        (lambda: rrt.paged_block_attention(c.q.clone().requires_grad_(), c.k, c.v, t, n, b), RuntimeError),
        (lambda: rrt.paged_block_select(c.q.clone().requires_grad_(), c.bounds, c.scales, t, n, page_size=16, num_blocks=3),
         RuntimeError),
    ]:
        with pytest.raises(err):
            call()
