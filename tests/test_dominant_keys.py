"""latent_prefill where one key outweighs a row's others: nothing averages that
key's rounding away, so the log-sum-exp is as exact as the key is kept.  Keys of a
sequence's first 1024 tokens are kept in two parts; the others to half a step of
the 16-bit type, u in each of their 128 formed dims."""

from __future__ import annotations

import numpy as np
import pytest

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
    u, f, fp16 = paged_ref.half_step(c.dt), paged_ref.F32, c.dt == torch.float16
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
