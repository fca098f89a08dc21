"""latent_prefill of an e4m3 cache whose scale is far from 1: what the kernel
keeps of keys and rope parts stays inside the 16-bit type's range."""

from __future__ import annotations

import numpy as np
import pytest

from tests import paged_ref
from tests.gpu_util import require_gpu
from tests.test_latent_prefill import HEAD, ROPE, TWO_PARTS, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _expected(c):
    """As Case.expected for rows that see no more than TWO_PARTS tokens, with
    fp16's absolute roundings where they are: a key is kept as the raw sum, to
    2^-25 of it; a value and an output as they are, to 2^-25."""
    import torch
    by = float(c.by)
    q, x = c.q.double().cpu().numpy(), c.c.double().cpu().numpy().reshape(-1, c.dim + ROPE)
    wk, wv = c.wk.double().cpu().numpy(), c.wv.double().cpu().numpy()
    u, fp16, f = paged_ref.half_step(c.dt), c.dt == torch.float16, paged_ref.F32
    floor = 2.0 ** -25 * abs(by)  # of a key, which bf16 rounds to fp16 too
    tiny = 2.0 ** -25 if fp16 else 0.0  # of a value or an output
    shape = (c.tokens, c.heads)
    out, lse, tol, tlog = np.zeros(shape + (HEAD,)), np.zeros(shape), np.zeros(shape + (HEAD,)), np.zeros(shape)
    for s in range(len(c.lengths)):
        y0 = x[c.slots(s)]
        n, new = len(y0), int(c.new[s])
        assert n <= TWO_PARTS
        for j in range(new):
            y, t = y0[:n - new + j + 1], int(c.starts[s]) + j
            for h in range(c.heads):
                kn, v = y[:, :c.dim] @ wk[h].T * by, y[:, :c.dim] @ wv[h].T * by
                k = np.concatenate([kn, y[:, c.dim:] * by], axis=1)
                o, lg, to, tl = paged_ref.attend(q[t, h], k, v, c.scale, u, fp16)
                aq = np.abs(q[t, h, :HEAD])
                ak = np.abs(y[:, :c.dim]) @ np.abs(wk[h]).T * abs(by)
                av = np.abs(y[:, :c.dim]) @ np.abs(wv[h]).T * abs(by)
                grow = (c.dim + 2) * f
                e = float(((np.abs(kn) * (u * u + 130 * f) + ak * grow + floor) @ aq).max() * abs(c.scale))
                p = np.exp(k @ q[t, h] * c.scale - lg)
                out[t, h], lse[t, h] = o, lg
                tol[t, h] = to + p @ (np.abs(v) * (u + 2 * e * (1 + u)) + av * grow + tiny) + tiny
                tlog[t, h] = tl + e
    return out, lse, tol, tlog


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("by", [2.0 ** -20, -3e-6, 2.0 ** -15, 0.003, 300.0, -700.0, 1e-30, 1e25])
def test_scales_far_from_one(dtype, by):
    import torch
    c = Case([70, 9, 300], [70, 3, 20], heads=2, dtype=dtype, store="float8_e4m3fn", seed=21)
    if abs(by) > 1:
        c.wv *= 1 / 64  # values and rope parts that are large ...
        c.c.view(-1, c.dim + ROPE)[:, c.dim:] = (c.c.view(-1, c.dim + ROPE)[:, c.dim:].float() * 100).clamp(-448, 448).to(c.st)
        c.q[:, :, HEAD:] /= 64  # ... with scores that are not
    c.by.fill_(by)
    by = float(c.by)
    c.scale = (HEAD + ROPE) ** -0.5 / abs(by)
    if by > 1e20 and dtype == "float16":
        c.wv.zero_()  # fp16 holds no such output
    out, lse = c.run()
    exp, elog, tol, tlog = _expected(c)
    a, b = int(c.starts[0]), int(c.starts[-1])
    paged_ref.check(lse[a:b].double().cpu().numpy(), elog[a:b], tlog[a:b], f"scale {by} lse")
    paged_ref.check(out[a:b].double().cpu().numpy(), exp[a:b], tol[a:b], f"scale {by} out")
