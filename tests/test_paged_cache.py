"""Block tables, slot maps and appends on the GPU, against plain loops."""

from __future__ import annotations

import numpy as np
import pytest

import row_radix_top_amd as rrt
from tests import paged_ref
from tests.gpu_util import note, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _dev(x, dtype=None):
    import torch
    t = torch.as_tensor(np.asarray(x), device="cuda")
    return t if dtype is None else t.to(dtype)


def _layout_case(lengths, new, page_size, width, short=0, extra=3, stride=None, seed=0):
    """Runs paged_layout on a table that holds the earlier tokens' pages and
    checks every output, the entries it has to leave alone included."""
    import torch
    rng = np.random.default_rng(seed)
    n = len(lengths)
    clamped = np.clip(lengths, 0, width * page_size)
    fresh = np.clip(new, 0, clamped)
    held = -(-(clamped - fresh) // page_size)
    take = int((-(-clamped // page_size) - held).sum())
    table = rng.integers(-5, 1 << 20, size=(n, stride or width)).astype(np.int32)  # arbitrary past the held pages
    free = (rng.permutation(take + 5) + 1000)[:max(0, take - short)].astype(np.int32)
    capacity = int(fresh.sum()) + extra
    note(f"layout n={n} page={page_size} width={width} tokens={int(fresh.sum())} take={take} short={short}")
    whole = _dev(table.copy())
    view = whole[:, :width]
    out = rrt.paged_layout(_dev(lengths, torch.int32), _dev(new, torch.int32), _dev(free), view, page_size=page_size,
                           capacity=capacity)
    exp, slots, row_lengths, row_seqs, starts, taken = paged_ref.layout(lengths, new, free, table[:, :width], page_size,
                                                                        capacity)
    got = whole.cpu().numpy()
    np.testing.assert_array_equal(got[:, :width], exp)
    np.testing.assert_array_equal(got[:, width:], table[:, width:])
    np.testing.assert_array_equal(out.slots.cpu().numpy(), slots)
    np.testing.assert_array_equal(out.row_lengths.cpu().numpy(), row_lengths)
    np.testing.assert_array_equal(out.row_seqs.cpu().numpy(), row_seqs)
    np.testing.assert_array_equal(out.starts.cpu().numpy(), starts)
    assert int(out.pages) == taken


@pytest.mark.parametrize("page_size", [1, 5, 16, 64])
@pytest.mark.parametrize("n", [1, 3, 64, 255, 256, 257, 700])
def test_layout_random(n, page_size):
    rng = np.random.default_rng(n * 100 + page_size)
    width = 9
    lengths = rng.integers(0, width * page_size + 1, size=n)
    new = np.where(rng.random(n) < 0.6, 1, rng.integers(0, width * page_size + 1, size=n))
    _layout_case(lengths, new, page_size, width, seed=n)


@pytest.mark.parametrize("n", [1023, 2048, 2049, 5000])
def test_layout_of_many_sequences(n):
    rng = np.random.default_rng(n)
    _layout_case(rng.integers(0, 81, size=n), rng.integers(0, 4, size=n), 16, 5, seed=n)
    _layout_case(rng.integers(0, 81, size=n), np.where(rng.random(n) < 0.01, 80, 0), 16, 5, seed=n)


def test_layout_of_more_tokens_than_32_bits_count():
    """The sum of the lengths stops at 2^31 - 1; the tokens before that are laid out."""
    import torch
    n, page, width, capacity = 5, 1 << 20, 1024, 40
    new = _dev([7] + [1 << 30] * (n - 1), torch.int32)
    table = torch.full((n, width), -7, dtype=torch.int32, device="cuda")
    out = rrt.paged_layout(torch.full((n,), 1 << 30, dtype=torch.int32, device="cuda"), new,
                           _dev(np.arange(100, 600, dtype=np.int32)), table, page_size=page, capacity=capacity)
    first = (1 << 30) - 7
    assert out.row_lengths.tolist() == list(range(first + 1, first + 8)) + list(range(1, capacity - 6))
    assert out.row_seqs.tolist() == [0] * 7 + [1] * (capacity - 7)
    assert out.slots.tolist() == [-1] * 7 + [100 * page + i for i in range(capacity - 7)]
    assert out.starts.tolist() == [0, 7, 7 + (1 << 30), (1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 1]
    assert int(out.pages) == 4 * width
    taken = torch.arange(4 * width, dtype=torch.int32, device="cuda") + 100
    assert bool((table[0] == -7).all())
    assert torch.equal(table[1:].reshape(-1), torch.where(taken < 600, taken, -1))


def test_layout_of_a_page_past_the_slots():
    """A page whose slots do not fit 32 bits has none."""
    import torch
    table = _dev([[1 << 20, 5], [(1 << 31) // 3000, 5]], torch.int32)
    out = rrt.paged_layout(_dev([8, 8], torch.int32), _dev([1, 1], torch.int32), _dev(np.zeros(0, np.int32)),
                           table, page_size=3000, capacity=2)
    last = (1 << 31) // 3000 * 3000 + 7
    assert out.slots.tolist() == [-1, last if last < 1 << 31 else -1]


def test_layout_decode_and_prefill_extremes():
    _layout_case([0, 0, 0], [0, 0, 0], 16, 4)
    _layout_case([0], [5], 16, 4)  # no more new tokens than tokens
    _layout_case([-3, 1000, 7], [2, 2000, -1], 16, 4)  # clamped
    _layout_case([64, 64], [64, 64], 16, 4, extra=0)
    _layout_case([17, 33], [1, 1], 16, 4, stride=11)
    _layout_case([20000], [20000], 16, 1250)  # one sequence owns every token
    _layout_case([0] * 300 + [900] + [0] * 300, [0] * 300 + [900] + [0] * 300, 7, 200)


@pytest.mark.parametrize("short", [1, 5, 10 ** 6])
def test_layout_with_too_few_pages(short):
    _layout_case([40, 100, 3, 64], [30, 100, 3, 1], 16, 8, short=short)


def test_layout_capacity_below_the_tokens():
    import torch
    lengths, new = _dev([10, 20], torch.int32), _dev([10, 20], torch.int32)
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    out = rrt.paged_layout(lengths, new, _dev(np.arange(9, dtype=np.int32)), table, page_size=8, capacity=12)
    exp, slots, *_ = paged_ref.layout([10, 20], [10, 20], np.arange(9), np.full((2, 4), -1), 8, 12)
    np.testing.assert_array_equal(table.cpu().numpy(), exp)
    np.testing.assert_array_equal(out.slots.cpu().numpy(), slots)
    assert out.starts.tolist() == [0, 10, 30] and int(out.pages) == 5


def test_layout_of_no_sequences():
    import torch
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    out = rrt.paged_layout(none, none, none, torch.empty((0, 4), dtype=torch.int32, device="cuda"), page_size=8,
                           capacity=5)
    assert out.slots.tolist() == [-1] * 5 and out.row_lengths.tolist() == [0] * 5 and out.starts.tolist() == [0]
    assert int(out.pages) == 0


# ---------------------------------------------------------------------------
# Append
# ---------------------------------------------------------------------------

def _special(x, rng):
    """Values next to and past the 8-bit range, NaN and infinities."""
    flat = x.view(-1)
    at = rng.choice(flat.numel(), size=min(flat.numel(), 24), replace=False)
    vals = [0.0, -0.0, 448.0, 464.0, 465.0, -449.0, 1e4, -1e4, float("inf"), float("-inf"), float("nan"), 2.0 ** -9,
            2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -6, 0.0625, 17.0, 18.0, 19.0, 21.0, 2.0 ** -7, 1.0625, 1.1875, -1.3]
    for i, v in zip(at, vals):
        flat[int(i)] = v


def _rounded(x, scale, dtype):
    """What the cache has to hold, by the 64-bit quotient where it is exact to
    tell (ties of the 8-bit grid are exact in 32 bits too)."""
    import torch
    if dtype != torch.float8_e4m3fn:
        return x
    y = x.float() / scale
    return torch.where(y.isnan(), y, y.clamp(-448.0, 448.0)).to(dtype)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
@pytest.mark.parametrize("tokens,heads,dim,page_size", [(1, 1, 64, 16), (37, 3, 128, 5), (130, 2, 72, 16), (9, 2, 20, 4),
                                                        (64, 8, 128, 32)])
def test_paged_append(dtype, store, tokens, heads, dim, page_size):
    import torch
    rng = np.random.default_rng(tokens)
    dt = getattr(torch, dtype)
    st = dt if store == "same" else getattr(torch, store)
    pages = -(-tokens // page_size) + 2
    torch.manual_seed(tokens)
    qkv = torch.randn(tokens, 3 * heads, dim, device="cuda").to(dt)
    k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    base = qkv.cpu()
    _special(base, rng)
    qkv.copy_(base)
    both = torch.randint(0, 120, (pages, 2, page_size, heads, dim), device="cuda").float().to(st)
    kc, vc = both[:, 0], both[:, 1]  # caches that share pages: strided
    slots = rng.permutation(pages * page_size)[:tokens].astype(np.int32)
    if tokens > 4:
        slots[[1, 3]] = [-1, pages * page_size]  # dropped
    ks = vs = None
    if st == torch.float8_e4m3fn:
        ks, vs = torch.rand(heads, device="cuda") + 0.3, torch.rand(heads, device="cuda") + 0.3
    exp = both.clone()
    for t, s in enumerate(slots):
        if 0 <= s < pages * page_size:
            exp[s // page_size, 0, s % page_size] = _rounded(k[t], 1 if ks is None else ks[:, None], st)
            exp[s // page_size, 1, s % page_size] = _rounded(v[t], 1 if vs is None else vs[:, None], st)
    note(f"append {dtype} {store} tokens={tokens} heads={heads} dim={dim} page={page_size}")
    rrt.paged_append(_dev(slots), k, v, kc, vc, k_scale=ks, v_scale=vs)
    bits = torch.uint8 if st == torch.float8_e4m3fn else torch.int16
    same = (both.view(bits) == exp.view(bits)) | (both.float().isnan() & exp.float().isnan())
    assert bool(same.all()), f"{int((~same).sum())} values differ"


@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
@pytest.mark.parametrize("dim", [256, 512])
def test_latent_append(store, dim):
    import torch
    st = torch.bfloat16 if store == "same" else torch.float8_e4m3fn
    torch.manual_seed(dim)
    tokens, page_size, pages = 33, 16, 4
    latent = torch.randn(tokens, dim, device="cuda").bfloat16()
    rope = torch.randn(tokens, 2, 64, device="cuda").bfloat16()[:, 1]  # strided rows
    cache = torch.zeros(pages, page_size, dim + 64, device="cuda").to(st)
    slots = torch.randperm(pages * page_size, device="cuda")[:tokens].int()
    scale = torch.full((1,), 0.37, device="cuda") if st != torch.bfloat16 else None
    note(f"latent append {store} dim={dim}")
    rrt.latent_append(slots, latent, rope, cache, scale=scale)
    exp = torch.zeros_like(cache, dtype=torch.float32)
    rows = _rounded(torch.cat([latent, rope], 1), 0 if scale is None else scale, st).float()
    exp.view(-1, dim + 64)[slots.long()] = rows
    assert torch.equal(cache.float(), exp)


def test_append_replayed_in_a_graph():
    import torch
    torch.manual_seed(0)
    k, v = (torch.randn(8, 2, 64, device="cuda").half() for _ in range(2))
    kc, vc = (torch.zeros(4, 16, 2, 64, device="cuda").half() for _ in range(2))
    slots = torch.arange(8, device="cuda", dtype=torch.int32)
    rrt.paged_append(slots, k, v, kc, vc)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rrt.paged_append(slots, k, v, kc, vc)
    for step in range(3):
        k.normal_()
        slots.copy_(torch.arange(8, device="cuda", dtype=torch.int32) * 5 + step)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(kc.view(-1, 2, 64)[slots.long()], k)
        assert torch.equal(vc.view(-1, 2, 64)[slots.long()], v)
