"""Scores of 2^40 and more: the largest takes the whole row, whatever fp32 can
tell of the others' distance to it."""

from __future__ import annotations

import numpy as np
import pytest

from tests import paged_ref
from tests.gpu_util import note, require_gpu
from tests.test_latent_attention import Case as LatentCase
from tests.test_latent_prefill import Case as PrefillCase
from tests.test_paged_attention import Case as PagedCase

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _check(what, got, rows, scale, u):
    """rows: (row, head, q, keys, values) in 64 bits.  A score is off by no more
    than 2^-11 of its terms' sum for each (the keys' rounding) and as much for its
    sums: rows whose largest score leads by less say nothing."""
    out, lse = (x.double().cpu().numpy() for x in got)
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    said = 0
    for r, h, q, k, v in rows:
        s = (k @ q) * scale
        off = 2 * (np.abs(k) @ np.abs(q)).max() * abs(scale) * 2.0 ** -11
        order = np.argsort(s)
        assert abs(lse[r, h] - s[order[-1]]) <= off + 1e-3
        if len(s) > 1 and s[order[-1]] - s[order[-2]] < 2 * off + 200:
            continue
        said += 1
        best = v[order[-1]]
        assert (np.abs(out[r, h] - best) <= 3 * u * np.abs(best) + 1e-4).all(), (what, r, h)
    note(f"{what}: {said} rows of {len(rows)} have one winner")
    assert said > 0.5 * len(rows)


SCALES = [2.0 ** 40, -(2.0 ** 60), 2.0 ** 28]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("scale", SCALES)
def test_paged_attention(dtype, scale):
    c = PagedCase([1, 40, 300, 900], heads=4, kv=2, dtype=dtype, seed=1)
    c.scale = scale
    q, k, v = (x.double().cpu().numpy() for x in (c.q, c.k, c.v))
    rows = [(r, h, q[r, h], k.reshape(-1, 2, 128)[c.row_slots(r), h // 2], v.reshape(-1, 2, 128)[c.row_slots(r), h // 2])
            for r in range(4) for h in range(4)]
    _check("paged_attention", c.run(), rows, scale, paged_ref.half_step(c.dt))


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("scale", SCALES)
def test_latent_attention(dtype, scale):
    c = LatentCase([1, 40, 300, 900], heads=4, dim=256, dtype=dtype, seed=2)
    c.scale = scale
    q, k = c.q.double().cpu().numpy(), c.c.double().cpu().numpy().reshape(-1, 320)
    rows = [(r, h, q[r, h], k[c.row_slots(r)], k[c.row_slots(r), :256]) for r in range(4) for h in range(4)]
    _check("latent_attention", c.run(), rows, scale, paged_ref.half_step(c.dt))


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("lengths,new", [([400, 70], [300, 70]), ([3000], [3])])
def test_latent_prefill(dtype, scale, lengths, new):
    c = PrefillCase(lengths, new, heads=2, dtype=dtype, seed=3)
    c.scale = scale
    q, x = c.q.double().cpu().numpy(), c.c.double().cpu().numpy().reshape(-1, 320)
    wk, wv = c.wk.double().cpu().numpy(), c.wv.double().cpu().numpy()
    rows = []
    for s in range(len(lengths)):
        y = x[c.slots(s)]
        for h in range(2):
            k, v = np.concatenate([y[:, :256] @ wk[h].T, y[:, 256:]], axis=1), y[:, :256] @ wv[h].T
            for j in range(int(c.new[s])):
                n = len(y) - int(c.new[s]) + j + 1
                rows.append((int(c.starts[s]) + j, h, q[int(c.starts[s]) + j, h], k[:n], v[:n]))
    _check("latent_prefill", c.run(), rows, scale, paged_ref.half_step(c.dt))
