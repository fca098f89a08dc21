"""Long rows with one position far above the others: the others' weights are
each below what fp16 resolves next to 1, and together they are the output.

One position scores TOP, the other n - 1 score 0; its value is 0 and theirs
1, so the output is (n - 1) e^-TOP / (1 + (n - 1) e^-TOP).  e^-18 is below
half of fp16's smallest number, 2^-24; e^-17 rounds to it, 1.4 times too much.
(An e4m3 cache holds 17 as 16.)"""

from __future__ import annotations

import math

import numpy as np
import pytest

import row_radix_top_amd as rrt
from tests import paged_ref
from tests.gpu_util import note, require_gpu

pytestmark = pytest.mark.gpu

N, PAGE = 65536, 64
# A kernel that keeps its weights as multiples 2^LIFT of the definition's
# (relative to the row's maximum) rounds none by more than 2^-25 2^-LIFT
# beside the type's half step.  7: what a reference that lags behind the
# maximum by at most 2^8 can leave below fp16's largest number.
LIFT = 7


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _expected(top, dt):
    """Output and log-sum-exp, and paged_ref.attend's bounds with the floor
    of small weights at 2^-25 2^-LIFT each.  Scores are one product, 0 or top."""
    u, acc = paged_ref.half_step(dt), (N + 16) * 2 * paged_ref.F32
    rest = (N - 1) * math.exp(-top)
    out, lse = rest / (1 + rest), top + math.log1p(rest)
    e = top * 4 * paged_ref.F32
    return out, lse, u * out + (u + 2 * e + acc) * out + N * 2.0 ** (-25 - LIFT), e + acc + 4 * paged_ref.F32 * (lse + 1)


def _check(got, top, dt, what):
    note(f"small weights {what} top={top} {dt}")
    top = float(top)
    out, lse, tol, tlog = _expected(top, dt)
    o, lg = (x.double().cpu().numpy() for x in got)
    paged_ref.check(o, np.full(o.shape, out), np.full(o.shape, tol), f"{what} out")
    paged_ref.check(lg, np.full(lg.shape, lse), np.full(lg.shape, tlog), f"{what} lse")


def _table():
    import torch
    return torch.randperm(N // PAGE, device="cuda").to(torch.int32)[None, :].contiguous()


TYPES = [("bfloat16", "same"), ("float16", "same"), ("float16", "float8_e4m3fn")]


@pytest.mark.parametrize("dtype,store", TYPES)
@pytest.mark.parametrize("top", [17.0, 18.0])
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_paged_attention(dtype, store, top, splits):
    import torch
    dt = getattr(torch, dtype)
    st = dt if store == "same" else getattr(torch, store)
    table = _table()
    k, v = (torch.zeros(N // PAGE, PAGE, 1, 128, device="cuda") for _ in range(2))
    v.fill_(1.0)
    at = (int(table[0, 3]), 5)
    k[at][:, 0], v[at][:] = top, 0.0
    q = torch.zeros(1, 2, 128, device="cuda", dtype=dt)
    q[:, :, 0] = 1.0
    got = rrt.paged_attention(q, k.to(st), v.to(st), table, torch.tensor([N], dtype=torch.int32, device="cuda"),
                              softmax_scale=1.0, max_splits=splits)
    _check(got, k.to(st)[at][0, 0], dt, f"paged_attention {store} splits={splits}")


@pytest.mark.parametrize("dtype,store", TYPES)
@pytest.mark.parametrize("top", [17.0, 18.0])
@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("place", [(3, 5), (1000, 63)])
def test_latent_attention(dtype, store, top, splits, place):
    """The far position early, and late enough that a reference has long been set."""
    import torch
    dt = getattr(torch, dtype)
    st = dt if store == "same" else getattr(torch, store)
    table = _table()
    c = torch.ones(N // PAGE, PAGE, 256 + 64, device="cuda")
    c[:, :, 256] = 0.0
    at = (int(table[0, place[0]]), place[1])
    c[at][:256], c[at][256] = 0.0, top
    q = torch.zeros(1, 2, 256 + 64, device="cuda", dtype=dt)
    q[:, :, 256] = 1.0
    got = rrt.latent_attention(q, c.to(st), table, torch.tensor([N], dtype=torch.int32, device="cuda"),
                               softmax_scale=1.0, max_splits=splits)
    _check(got, c.to(st)[at][256], dt, f"latent_attention {store} splits={splits}")


@pytest.mark.parametrize("dtype,store", TYPES)
@pytest.mark.parametrize("top", [17.0, 18.0])
@pytest.mark.parametrize("place", [(3, 5), (20, 7)])
def test_latent_prefill(dtype, store, top, place):
    """The far position among the tokens that are kept in two parts, and behind them."""
    import torch
    dt = getattr(torch, dtype)
    st = dt if store == "same" else getattr(torch, store)
    table = _table()
    c = torch.zeros(N // PAGE, PAGE, 256 + 64, device="cuda")
    c[:, :, 1] = 1.0
    at = (int(table[0, place[0]]), place[1])
    c[at][0], c[at][1] = top, 0.0
    w = torch.zeros(2, 2, 128, 256, device="cuda", dtype=dt)
    w[0, :, 0, 0], w[1, :, :, 1] = 1.0, 1.0  # k[0] = c[0], v = c[1]
    q = torch.zeros(1, 2, 192, device="cuda", dtype=dt)
    q[:, :, 0] = 1.0
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    got = rrt.latent_prefill(q, c.to(st), table, ints(0, 1), ints(N), w[0], w[1], context_tokens=N, softmax_scale=1.0)
    _check(got, c.to(st)[at][0], dt, f"latent_prefill {store}")
