"""paged_copy with lists of far more pairs than are real, as paged_compact gives
them: as many entries as half the pool has pages, -1 past the last move."""

from __future__ import annotations

import numpy as np
import pytest

import row_radix_top_amd as rrt
from tests.gpu_util import note, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def lists(pairs, real, pages, rng):
    """`real` moves at random places of a list of `pairs`, some others out of range or onto themselves."""
    import torch
    at = rng.permutation(pairs)[:real]
    order = rng.permutation(pages)[:2 * real]
    src, dst = np.full(pairs, -1), np.full(pairs, -1)
    src[at], dst[at] = order[:real], order[real:]
    odd = np.setdiff1d(rng.integers(0, pairs, size=9), at)
    src[odd], dst[odd] = 3, np.where(odd % 2, 3, pages)
    i32 = lambda x: torch.as_tensor(x, device="cuda").to(torch.int32)  # noqa: E731
    return i32(src), i32(dst), order[:real], order[real:], at


@pytest.mark.parametrize("pairs", [1 << 19, (1 << 19) + 77, 70001])
@pytest.mark.parametrize("count,dtype,shape", [(32, "bfloat16", (16, 8)), (33, "int8", (4, 3)), (1, "float32", (16, 4, 128)),
                                               (2, "uint8", (1, 70000))])
def test_few_moves_in_a_long_list(pairs, count, dtype, shape):
    """Up to 2^19 pairs of 32 caches, a workgroup for each of which would be 2^32 threads."""
    import torch
    rng = np.random.default_rng(pairs + count)
    pages, real = 300, 120
    src, dst, a, b, at = lists(pairs, real, pages, rng)
    note(f"copy of {pairs} pairs, {count} caches {dtype} {shape}")
    torch.manual_seed(count)
    whole = torch.randint(0, 100, (count, pages) + shape, device="cuda").to(getattr(torch, dtype))
    exp = whole.clone()
    exp[:, b.tolist()] = whole[:, a.tolist()]
    rrt.paged_copy(src, dst, list(whole.unbind(0)))
    assert torch.equal(whole, exp)


def test_tokens_of_a_long_list():
    import torch
    rng = np.random.default_rng(5)
    pairs, pages, real = 200003, 4000, 1900
    src, dst, a, b, at = lists(pairs, real, pages, rng)
    tokens = rng.integers(-2, 20, size=pairs)
    torch.manual_seed(5)
    cache = torch.randint(0, 100, (pages, 16, 2, 32), device="cuda").half()
    exp = cache.clone()
    for x, y, n in zip(a, b, tokens[at]):
        n = min(max(int(n), 0), 16)
        exp[y, :n] = cache[x, :n]
    rrt.paged_copy(src, dst, [cache], tokens=torch.as_tensor(tokens, device="cuda").to(torch.int32))
    assert torch.equal(cache, exp)


def test_the_moves_of_a_large_pool():
    """A pool of 2^20 pages and the whole list of its compaction, over 32 caches."""
    import torch
    rng = np.random.default_rng(6)
    pages, seqs, width = 1 << 20, 16, 100
    table = rng.permutation(pages)[:seqs * width].reshape(seqs, width)
    i32 = lambda x: torch.as_tensor(x, device="cuda").to(torch.int32)  # noqa: E731
    lengths = rng.integers(1, width + 1, size=seqs)
    caches = torch.randint(0, 1 << 30, (32, pages, 1), device="cuda", dtype=torch.int32)
    held = i32(np.concatenate([table[s, :n] for s, n in enumerate(lengths)])).long()
    before = caches[:, held].clone()
    moved = rrt.paged_compact(i32(table), i32(lengths), page_size=1, num_pages=pages)
    rrt.paged_copy(moved.src, moved.dst, list(caches.unbind(0)))
    now = torch.cat([moved.table[s, :n] for s, n in enumerate(lengths)]).long()
    assert int(now.max()) == len(now) - 1 and torch.equal(caches[:, now], before)
