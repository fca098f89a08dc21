"""Choices of pages whose scores pass the range of fp32: the first and last pages
of a row still come before all others and places without a page after them."""

from __future__ import annotations

import numpy as np
import pytest

from tests.gpu_util import require_gpu
from tests.test_chosen_blocks import Keys

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


# In one launch, by one wavefront a row: 40 pages.  Several rows of a sequence.  One head
# a key-value head, several sixteens of them, and several passes of those.  A row of pages
# that is scored in parts, and one that is picked by a whole workgroup.
FORMS = [dict(lengths=[640, 640, 50], heads=8, kv=2), dict(lengths=[[638, 639, 640], [50, 51, 52]], heads=4, kv=2),
         dict(lengths=[640, 33], heads=2, kv=2, dim=64), dict(lengths=[640, 33], heads=40, kv=1),
         dict(lengths=[640, 33], heads=80, kv=1), dict(lengths=[2000], heads=8, kv=2, page=1),
         dict(lengths=[6000, 4200], heads=8, kv=2, page=1, dim=64)]


@pytest.mark.parametrize("form", range(len(FORMS)))
def test_infinite_queries_keep_the_first_and_last_pages(form):
    c = Keys(seed=form, **FORMS[form])
    c.update(c.ctx)
    c.q[:, :, 3] = float("inf")
    got = c.check_select(7, 2, 3).cpu().numpy()
    for r, n in enumerate(c.rows2d.reshape(-1)):
        have = -(-int(n) // c.page)
        for b in {0, 1, have - 3, have - 2, have - 1}:
            if 0 <= b < have:
                assert (got[r] == b).any(axis=1).all(), (r, b)


def test_infinite_keys_keep_the_last_page():
    c = Keys([640, 640], heads=8, kv=2, seed=3)
    for page in (5, 7, 9, 11):
        c.k[c.table[0, page], 2, :, 4] = float("inf")
    c.update(c.ctx)
    got = c.check_select(5).cpu().numpy()
    for head in range(2):
        assert {0, 39} <= set(got[0, head].tolist())
        assert len({5, 7, 9, 11} & set(got[0, head].tolist())) == 3


@pytest.mark.parametrize("form", range(len(FORMS)))
def test_places_without_a_page_come_after_the_lowest_scores(form):
    c = Keys(seed=form, **FORMS[form])
    c.bounds.fill_(-50)
    c.q[:], c.q[:, :, 3] = 0, float("inf")
    absent = list(range(1, 31, 3))
    c.table[0, absent] = -1
    have = int(c.rows2d[0, 0] + c.page - 1) // c.page
    k = have - len(absent)
    got = c.check_select(k).cpu().numpy()
    for row in got[:c.next_n]:
        for chosen in row:
            assert not set(absent) & set(chosen.tolist())


def test_scales_that_are_no_numbers_rank_last_of_the_pages():
    c = Keys([640, 640], heads=8, kv=2, seed=5)
    c.update(c.ctx)
    strange = [3, 8, 20, 33]
    c.scales[c.table[0, strange].tolist()] = float("nan")
    c.table[0, [4, 5]] = -1
    got = c.check_select(34, 0, 0).cpu().numpy()
    assert not set(strange + [4, 5]) & set(got[0].reshape(-1).tolist())
    got = c.check_select(38, 0, 0).cpu().numpy()
    for head in range(2):
        np.testing.assert_array_equal(got[0, head], [b for b in range(40) if b not in (4, 5)])
