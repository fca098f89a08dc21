"""Rows of chosen positions that are split over several workgroups and joined:
by the library's own rule, as 2048 chosen positions of a small batch are, and by
max_splits."""

from __future__ import annotations

import numpy as np
import pytest

from tests.gpu_util import require_gpu
from tests.test_latent_attention import Case as LatentCase
from tests.test_paged_attention import Case as PagedCase

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _chosen(seed, lengths, k):
    """Distinct positions, ascending, -1 behind them; rows of fewer positions
    than k have parts of nothing but -1.  The last row's are out of order, some
    twice, some out of range."""
    rng = np.random.default_rng(seed)
    rows = []
    for n in lengths:
        pick = np.sort(rng.permutation(n)[:min(k, n)])
        rows.append(np.concatenate([pick, np.full(k - len(pick), -1)]))
    rows[-1] = rng.integers(-5, max(1, lengths[-1]) + 20, size=k)
    return np.stack(rows).astype(np.int64)


LENGTHS = [2300, 0, 1, 600, 513, 2048, 1100]  # seven rows: not a multiple of the eight that are numbered together
PAIRS = [[2299, 2300], [0, 1], [600, 601], [1023, 1024], [40, 41]]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
@pytest.mark.parametrize("k", [1024, 1500, 2048])
@pytest.mark.parametrize("splits", [0, 2, 3, 16])
def test_paged_attention(dtype, store, k, splits):
    PagedCase(LENGTHS, heads=4, kv=2, dim=64, dtype=dtype, store=store, chosen=_chosen(k, LENGTHS, k),
              seed=k).check("chosen, split", max_splits=splits)


@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
@pytest.mark.parametrize("splits", [0, 3])
def test_paged_attention_multi_token(store, splits):
    flat = [n for p in PAIRS for n in p]
    PagedCase(PAIRS, heads=20, kv=1, dim=128, store=store, chosen=_chosen(5, flat, 1500), seed=5,
              page_size=24).check("chosen, split, two rows a sequence", max_splits=splits)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
@pytest.mark.parametrize("dim,heads", [(256, 33), (512, 4)])
@pytest.mark.parametrize("k,splits", [(130, 2), (300, 2), (1024, 0), (1500, 3), (2048, 0), (2048, 2), (2048, 16)])
def test_latent_attention(dtype, store, dim, heads, k, splits):
    LatentCase(LENGTHS, heads=heads, dim=dim, dtype=dtype, store=store, chosen=_chosen(k, LENGTHS, k),
               seed=k).check("chosen, split", max_splits=splits)


@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
@pytest.mark.parametrize("splits", [0, 3])
def test_latent_attention_multi_token(store, splits):
    flat = [n for p in PAIRS for n in p]
    LatentCase(PAIRS, heads=20, dim=256, store=store, chosen=_chosen(6, flat, 1500), seed=6,
               page_size=24).check("chosen, split, two rows a sequence", max_splits=splits)
