"""One workspace for a server's steps with and without groups of sequences."""

from __future__ import annotations

import numpy as np
import pytest

import row_radix_top_amd as rrt
from tests.gpu_util import require_gpu
from tests.test_shared_prefixes import _size, dev
from tests.test_workspaces import _attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("changes", [dict(), dict(num_heads=64, num_kv_heads=8), dict(next_n=2), dict(max_splits=3),
                                     dict(max_splits=128), dict(table_width=16)], ids=str)
def test_a_size_holds_for_no_groups(changes):
    n = changes.get("next_n", 1)
    for rows in [n * r for r in range(1, 200)] + [n * 5000]:
        a = _attention("paged_attention", rows, **changes)
        assert _size(a, 0) <= _size(a, 3), rows


def test_a_step_with_groups_and_one_without_in_one_buffer():
    import torch
    rng = np.random.default_rng(2)
    rows, width = 2, 2048
    k, v = (torch.randn(rows * width, 16, 1, 64, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(rows, 2, 64, device="cuda").bfloat16()
    table = rng.permutation(rows * width).reshape(rows, width)
    table[1, :100] = table[0, :100]
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    steps = [(dev([0, 2]), dev([1600])), (dev([0]), none)]
    buffer = torch.full((_size(_attention("paged_attention", rows, num_heads=2, num_kv_heads=1, head_dim=64, page_size=16,
                                          table_width=width), 1),), 0xff, dtype=torch.uint8, device="cuda")
    for starts, shared in steps:
        args = (q, k, v, dev(table), dev([30000, 32768]), starts, shared)
        a, b = rrt.paged_prefix_attention(*args), rrt.paged_prefix_attention(*args, workspace=buffer)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
