"""Bounds of keys so small that their scale is subnormal, and how far outside its
bounds a key may lie.

A scale is top * fl(1 / 127), each rounded once: off by at most 2^-23 of itself
(two half steps of 2^-24), or, where it is below 2^-126, by half of 2^-149 more.
The smallest bfloat16 is 2^-133, whose scale is 516 times 2^-149: 2^-10 of it.  A
quotient that passes 127 for that reason is clamped, so the key lies by as much
outside; all others are rounded outward."""

from __future__ import annotations

import numpy as np
import pytest

from tests.gpu_util import require_gpu
from tests.test_chosen_blocks import Keys

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("store,tiny", [("bfloat16", 2.0 ** -133), ("float16", 2.0 ** -24), ("float8_e4m3fn", 2.0 ** -9)])
@pytest.mark.parametrize("most", [1, 2, 3, 126, 127])
def test_the_smallest_keys(store, tiny, most):
    import torch
    c = Keys([64, 40], kv=2, heads=2, store=store, dtype="float16" if store != "bfloat16" else store, seed=most)
    whole = torch.randint(-most, most + 1, c.k.shape, device="cuda")
    c.k.copy_((whole.double() * tiny).to(c.st))
    c.k[c.table[0, 1]] = 0
    c.check_bounds([64, 40])
    for s in range(2):
        for j in range(-(-int(c.ctx[s]) // 16)):
            p = int(c.table[s, j])
            zero = s == 0 and j == 1
            assert bool((c.scales[p] == 0).all()) == zero
            if zero:
                assert not bool(c.bounds[p].any())


@pytest.mark.parametrize("store,size,off", [("bfloat16", 1.0, 2.0 ** -23), ("float16", 1.0, 2.0 ** -23),
                                            ("float8_e4m3fn", 1.0, 2.0 ** -23), ("bfloat16", 2.0 ** -128, 2.0 ** -10)])
def test_keys_lie_within_their_bounds(store, size, off):
    c = Keys([900], kv=3, heads=3, dim=64, store=store, dtype="float16" if store != "bfloat16" else store, seed=1)
    c.k.copy_((c.k.double() * size).to(c.st))
    c.update(c.ctx)
    for j in range(-(-900 // 16)):
        p = int(c.table[0, j])
        k = c.k[p, :min(16, 900 - 16 * j)].double().cpu().numpy()  # [tokens, heads, dim]
        hi, lo = (c.bounds[p, :, i].double().cpu().numpy() * c.scales[p].double().cpu().numpy()[:, None] for i in range(2))
        top = np.abs(k).max(axis=(0, 2))[:, None]
        assert (k.max(axis=0) <= hi + top * off).all() and (k.min(axis=0) >= lo - top * off).all()
