"""Launches count their threads in 32 bits: what would need more is refused by
the host's own check, before anything touches a device."""

from __future__ import annotations

import pytest

from row_radix_top_amd import attention as pa
from row_radix_top_amd import binding, blocks
from tests.test_shared_refusals import BOUNDS, EINVAL, _struct


# Workgroups of 256 threads take four (page, head) each: 2^30 of them, and the first number past the limit.
@pytest.mark.parametrize("changes", [dict(num_tokens=2147483647, page_size=1, num_kv_heads=2),
                                     dict(num_tokens=(1 << 26) - 4, page_size=1, num_kv_heads=1)])
def test_more_threads_than_a_launch_takes(changes):
    assert pa.load().paged_bounds(_struct(blocks.BoundsArgs, BOUNDS, changes), None) == EINVAL
    assert "more than one launch takes" in binding.last_error()
