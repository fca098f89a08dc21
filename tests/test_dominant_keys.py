"""latent_prefill where one key outweighs a row's others: nothing averages that
key's rounding away, so the log-sum-exp is as exact as the key is kept.  Keys of a
sequence's first 1024 tokens are kept in two parts; the others to half a step of
fp16, 2^-11, in each of their 128 formed dims, whatever the 16-bit type."""

from __future__ import annotations

import numpy as np
import pytest

import row_radix_top_amd as rrt
from tests import paged_ref
from tests.gpu_util import note, require_gpu
from tests.test_latent_prefill import HEAD, ROPE, TWO_PARTS, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _bounds(c, row, h, n):
    """The 64-bit log-sum-exp, its bound and the largest weight.  Scores off by
    e_j each move it by log(sum p e^e) <= sum p (e^e - 1): of a key of 192 dims
    the sums' own error and, of its formed ones, the rounding as it is kept."""
    import torch
    q, x = c.q[row, h].double().cpu().numpy(), c.c.double().cpu().numpy().reshape(-1, c.dim + ROPE)[c.slots(0)][:n]
    if c.by is not None:
        x = x * float(c.by)
    wk = c.wk[h].double().cpu().numpy()
    u, f, fp16 = 2.0 ** -11, paged_ref.F32, c.dt == torch.float16
    kn = x[:, :c.dim] @ wk.T
    k = np.concatenate([kn, x[:, c.dim:]], axis=1)
    s = k @ q * c.scale
    lse = s.max() + np.log(np.exp(s - s.max()).sum())
    p = np.exp(s - lse)
    aq = np.abs(q)
    sums = ((np.abs(k) @ aq) * (k.shape[1] + 130) + (np.abs(x[:, :c.dim]) @ np.abs(wk).T @ aq[:HEAD]) * (c.dim + 2)) * f
    kept = np.where(np.arange(n) < TWO_PARTS, u * u, u) * (np.abs(kn) @ aq[:HEAD]) + (2.0 ** -25 * aq[:HEAD].sum() if fp16 else 0)
    own = (n + 16) * 2 * f + 4 * f * (abs(lse) + 1)
    return lse, float(p @ np.expm1((sums + kept) * c.scale)) + own, p.max()


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
@pytest.mark.parametrize("place", [0, 500, 1023, 1024, 3000])
def test_one_key_above_the_others(dtype, store, place):
    import torch
    c = Case([3500], [2], heads=2, dtype=dtype, store=store, seed=place + 1)
    # The place's vector along what the first row's first head asks for, its
    # score some 20 above the others'.
    want = c.wk[0].double().T @ c.q[0, 0, :HEAD].double()
    by = 1.0 if c.by is None else float(c.by)
    want *= 20 / c.scale / float((c.wk[0].double() @ want) @ c.q[0, 0, :HEAD].double()) / by
    c.c.view(-1, c.dim + ROPE)[int(c.slots(0)[place]), :c.dim] = want.to(torch.float32).to(c.st)
    out, lse = c.check(f"dominant key at {place}")
    exp, tol, p = _bounds(c, 0, 0, 3499)
    off = abs(float(lse[0, 0]) - exp)
    note(f"log-sum-exp {exp:.3f}, weight {p:.4f}, off by {off:.2e}, bound {tol:.2e}")
    assert p > 0.9 and off <= tol


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("place", [500, 1024, 3000])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -30, 2.0 ** 40])
def test_a_key_whose_roundings_agree(dtype, place, size):
    """Every formed dim of the far key is size (1 + 0.99 2^-8), which bf16 rounds
    by nearly half a step, all in one direction; queries ask for it with a score
    of 20.  Keys are kept to at least fp16's half step, 2^-11, at any size."""
    import torch
    if dtype == "float16" and size != 1.0:
        size = 2.0 ** -10 if size < 1 else 2.0 ** 13
    dt, n = getattr(torch, dtype), 3500
    pages = torch.randperm(n // 16 + 1, device="cuda").to(torch.int32)[None, :].contiguous()
    c = torch.zeros(n // 16 + 1, 16, 256 + ROPE, device="cuda")
    at = (int(pages[0, place // 16]), place % 16)
    c[at][0], c[at][1] = size, size * 0.99 * 2.0 ** -8
    c = c.to(dt)
    w = torch.zeros(2, 1, HEAD, 256, device="cuda", dtype=dt)
    w[0, :, :, :2], w[1, :, :, 0] = 1.0, 1.0
    q = torch.zeros(1, 1, HEAD + ROPE, device="cuda", dtype=dt)
    q[:, :, :HEAD] = 1.0
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    scale = 20.0 / (HEAD * size)
    note(f"key with roundings that agree, {dtype} at {place}, size {size}")
    out, lse = rrt.latent_prefill(q, c, pages, ints(0, 1), ints(n), w[0], w[1], context_tokens=n, softmax_scale=scale)
    key = float(c[at][0].double() + c[at][1].double())
    score = HEAD * key * float(np.float32(scale))
    exp = score + np.log1p((n - 1) * np.exp(-score))
    tol = score * (2.0 ** -11 + (HEAD + ROPE + 130 + 4) * paged_ref.F32) * 1.01 + (n + 16) * 2 * paged_ref.F32 + 4 * paged_ref.F32 * 21
    if place < TWO_PARTS:
        tol = score * (2.0 ** -17 + (HEAD + ROPE + 130 + 4) * paged_ref.F32) * 1.01 + (n + 16) * 2 * paged_ref.F32 + 4 * paged_ref.F32 * 21
    off = abs(float(lse) - exp)
    note(f"log-sum-exp {exp:.4f}, off by {off:.2e}, bound {tol:.2e}")
    assert off <= tol


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("keys,ropes", [(0, 30), (30, 0), (-20, 20), (20, -20), (60, 60), (100, -30), (-60, -60)])
def test_keys_and_rope_parts_of_other_sizes(dtype, keys, ropes):
    """Formed keys about 2^keys, rope parts about 2^ropes, both asked for alike: what is kept of
    one does not cost the other."""
    import torch
    if dtype == "float16":
        keys, ropes = (max(-6, min(6, x)) for x in (keys, ropes))
    c = Case([300, 70], [40, 70], heads=2, dtype=dtype, seed=31)
    c.wk *= 2.0 ** (keys / 2)
    c.c[:, :, :c.dim] *= 2.0 ** (keys / 2)
    c.wv *= 2.0 ** (-keys / 2)
    c.c[:, :, c.dim:] *= 2.0 ** ropes
    c.q[:, :, :HEAD] *= 2.0 ** -keys
    c.q[:, :, HEAD:] *= 2.0 ** -ropes
    c.check(f"keys 2^{keys}, rope parts 2^{ropes}")


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
def test_a_large_token_does_not_cost_its_neighbours(dtype, store):
    """Tokens whose keys and rope parts are far larger, in the middle of tiles: rows before them are as
    exact as without, rows that see them too."""
    import torch
    c = Case([400, 70], [300, 70], heads=2, dtype=dtype, store=store, seed=41)
    exp, elog, tol, tlog = c.expected()
    large = {"bfloat16": 2.0 ** 60, "float16": 2.0 ** 9}[dtype] if store == "same" else 64.0
    for token in (130, 390):
        row = c.c.view(-1, c.dim + ROPE)[int(c.slots(0)[token])]
        row.copy_((row.float() * large).clamp(-448, 448).to(c.st) if store != "same" else row * large)
    out, lse = c.run()
    for rows in (slice(0, 130 - 100), slice(300, 370)):  # row j sees positions up to 100 + j
        paged_ref.check(out[rows].double().cpu().numpy(), exp[rows], tol[rows], "rows without the large token")
        paged_ref.check(lse[rows].double().cpu().numpy(), elog[rows], tlog[rows], "their lse")
    if large < 2.0 ** 10:
        c.check("all rows")


@pytest.mark.parametrize("keys,ropes", [(0, 0), (40, 30), (-30, 20)])
def test_other_sizes_in_split_contexts_and_beside_what_is_not_finite(keys, ropes):
    """Contexts that are shared out, some of their tokens of other sizes than the rest; and a later token
    that is not finite, which earlier rows do not see."""
    import torch

    def sized(c):
        c.wk *= 2.0 ** keys
        c.c[::2, :, c.dim:] *= 2.0 ** ropes  # every other page
        c.q[:, :, :HEAD] *= 2.0 ** -keys
        return c

    sized(Case([3000, 1200], [2, 3], heads=2, seed=51)).check("split, other sizes")
    c = sized(Case([260], [200], heads=2, seed=52))
    bad = np.zeros(c.pages * c.page_size, dtype=bool)
    bad[c.slots(0)[[150, 259]]] = True
    c.poison(bad)
    out, lse = c.run()
    exp, elog, tol, tlog = c.expected()
    k = 150 - 60
    paged_ref.check(out[:k].double().cpu().numpy(), exp[:k], tol[:k], "earlier rows")
    paged_ref.check(lse[:k].double().cpu().numpy(), elog[:k], tlog[:k], "earlier rows' lse")
    assert bool(out[k:].isnan().all())


def test_rows_and_tokens_of_other_sizes_among_the_ordinary():
    """Some rows and some tokens alone take the other way through the tiles."""
    c = Case([700, 130], [300, 130], heads=2, seed=61)
    c.q[5, :, HEAD:] *= 2.0 ** -20
    c.q[200, :, :HEAD] *= 2.0 ** -25
    c.q[201] *= 2.0 ** 60
    c.check("rows")
    c.q[201] *= 2.0 ** -60
    flat = c.c.view(-1, c.dim + ROPE)
    for token, by in ((70, 2.0 ** -12), (300, 2.0 ** 9), (511, 2.0 ** -30)):
        flat[int(c.slots(0)[token])] *= by
    c.check("rows and tokens")
