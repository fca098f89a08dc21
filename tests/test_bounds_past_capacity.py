"""paged_bounds of a step with more new tokens than it has room for: the tokens
past num_tokens were never written, so they count in no page's bounds."""

from __future__ import annotations

import numpy as np
import pytest

import row_radix_top_amd as rrt
from tests import shared_ref
from tests.gpu_util import note, require_gpu
from tests.test_chosen_blocks import Keys, dev, floats

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def expected(c, new, room):
    """Bounds after a step of `new` tokens of which the first `room` have a place."""
    b, s = c.bounds.cpu().numpy().astype(np.int64), c.scales.cpu().numpy().copy()
    k, start = floats(c.k), 0
    for q in range(c.seqs):
        n, fresh = int(c.ctx[q]), int(new[q])
        there = min(fresh, max(room - start, 0))
        start += fresh
        end = n - fresh + there
        for j in range((n - fresh) // c.page, -(-end // c.page) if there else 0):
            p = c.table[q, j]
            for h in range(c.kv):
                b[p, h], s[p, h] = shared_ref.bounds(k[p, :min(c.page, end - j * c.page), h], shared_ref.LARGEST[c.store])
    return b, s


@pytest.mark.parametrize("page,dim,kv", [(16, 128, 2), (1, 64, 1), (5, 64, 3)])
@pytest.mark.parametrize("room", [1, 9, 10, 11, 15, 16, 17, 41, 42, 43, 57, 58, 59, 74, 75, 80])
def test_tokens_past_the_room(page, dim, kv, room):
    new = [10, 0, 32, 16, 1, 16]  # 75 tokens
    c = Keys([26, 40, 70, 16, 33, 100], kv=kv, heads=kv, dim=dim, page=page, seed=room)
    note(f"bounds page={page} dim={dim} kv={kv} room={room}")
    exp = expected(c, new, room)
    c.update(new, num_tokens=room)
    np.testing.assert_array_equal(c.bounds.cpu().numpy(), exp[0])
    np.testing.assert_array_equal(c.scales.cpu().numpy(), exp[1])


def test_a_step_that_is_too_long():
    """As a server runs it: layout and append leave out what has no room, and so do the bounds.  The pages' other tokens
    are NaN, which bounds pass over, or far too large, which they would not."""
    import torch
    c = Keys([40, 70, 90], kv=2, heads=2, seed=1)
    c.k.fill_(1e4)
    lengths, new = dev([40, 70, 90]), dev([40, 70, 90])
    table = torch.full((3, c.width), -1, dtype=torch.int32, device="cuda")
    rows = rrt.paged_layout(lengths, new, dev(np.arange(c.pages)), table, page_size=16, capacity=64)
    k = torch.randn(64, 2, 128, device="cuda").bfloat16()
    rrt.paged_append(rows.slots, k, k, c.k, c.k.clone())
    bounds, scales = c.bounds.clone(), c.scales.clone()
    rrt.paged_bounds(c.k, table, rows.starts, lengths, c.bounds, c.scales, num_tokens=64)
    t = table.cpu().numpy()
    written = [*t[0, :3], *t[1, :2]]  # 40 and 24 tokens
    others = [p for p in range(c.pages) if p not in written]
    assert torch.equal(c.bounds[others], bounds[others]) and torch.equal(c.scales[others], scales[others])
    assert float(c.scales[written].max()) < 10 / 127
