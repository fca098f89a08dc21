"""How a server sees that the pool ran out of pages, with paged_free's own list:
a step needs more than its count, and exactly then something has no page."""

from __future__ import annotations

import numpy as np
import pytest

import row_radix_top_amd as rrt
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("spare", [0, 1, 2, 3, 4, 9])
def test_pages_against_the_count(spare):
    import torch
    i32 = lambda x: torch.as_tensor(np.asarray(x), device="cuda").to(torch.int32)  # noqa: E731
    table, lengths = i32([[4, 5, -1], [0, 7, 2]]), i32([20, 40])
    pool = rrt.paged_free(table, lengths, page_size=16, num_pages=8)
    assert int(pool.count) == 3 and pool.free.tolist() == [1, 3, 6, -1, -1, -1, -1, -1]
    parents = [0] + [0] * min(spare, 3) + [1] * max(spare - 2, 1)  # a copy for each but the first of either
    fork = rrt.paged_fork(table, lengths, i32(parents), pool.free, page_size=16)
    last = (fork.lengths - 1) // 16
    got = fork.table.gather(1, last.long()[:, None])
    assert (int(fork.pages) > int(pool.count)) == bool((got < 0).any())
    new = i32([12 + 16 * (spare // 3), spare])  # tokens for rows of a new batch, of pages that are not there yet
    width = torch.full((2, 6), -1, dtype=torch.int32, device="cuda")
    rows = rrt.paged_layout(new, new, pool.free, width, page_size=16, capacity=64)
    tokens = int(rows.starts[-1])
    assert (int(rows.pages) > int(pool.count)) == bool((rows.slots[:tokens] < 0).any())
