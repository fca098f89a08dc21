"""Plain 64-bit implementations of the paged-cache operators and the error
bounds that the tests hold the kernels to.

Bounds.  With u = eps / 2 of the 16-bit type (half a step) and f = 2^-24 (half
a step of fp32), an output o = sum p v has
  - its own rounding:                        u |o|
  - each weight rounded to 16 bits:          u A,  A = sum p |v|
  - scores in fp32: a dot product of d terms is off by at most (d + 2) f times
    its terms' absolute sum (the products of 16-bit values are exact in fp32,
    each addition and the scaling round once), and a score off by e changes
    its weight by a factor within 1 +- 2e (numerator and sum): 2 e A
  - exp2 and the sums of n terms:            (n + 16) 2 f A
  - a weight below 2^-14 in fp16 is off by at most 2^-25 instead of u times
    itself (the weights are relative to a maximum, so their sum is at least
    1): n 2^-25 max|v|.
The log-sum-exp is off by the scores' e, (n + 16) 2 f and its own rounding.
"""

from __future__ import annotations

import math

import numpy as np

F32 = 2.0 ** -24


def half_step(torch_dtype) -> float:
    import torch
    return float(torch.finfo(torch_dtype).eps) / 2


def slots_of(table_row, positions, page_size, num_pages):
    """Pool slots of positions, -1 where the table holds no page."""
    p = np.asarray(positions, dtype=np.int64)
    page = np.asarray(table_row, dtype=np.int64)[p // page_size]
    return np.where((page >= 0) & (page < num_pages), page * page_size + p % page_size, -1)


def row_positions(length, width_tokens, chosen=None):
    n = int(min(max(int(length), 0), width_tokens))
    if chosen is None:
        return np.arange(n, dtype=np.int64)
    c = np.asarray(chosen, dtype=np.int64)
    return c[(c >= 0) & (c < n)]


def attend(q, k, v, scale, u, fp16):
    """One head: q [d], k [n, d], v [n, e] in float64.  Returns out [e], lse
    and their bounds."""
    n = k.shape[0]
    if n == 0:
        return np.zeros(v.shape[1]), -math.inf, np.zeros(v.shape[1]), 0.0
    with np.errstate(invalid="ignore"):
        s = (k @ q) * scale
    e = float(np.max((np.abs(k) @ np.abs(q)) * abs(scale)) * (k.shape[1] + 2) * F32)
    top = s.max()
    p = np.exp(s - top)
    total = p.sum()
    p /= total
    out, a = p @ v, p @ np.abs(v)
    acc = (n + 16) * 2 * F32
    tol = u * np.abs(out) + (u + 2 * e + acc) * a * (1 + u)
    if fp16:
        tol = tol + n * 2.0 ** -25 * np.abs(v).max()
    lse = top + math.log(total)
    return out, lse, tol, e + acc + 4 * F32 * (abs(lse) + 1)


def check(got, exp, tol, what):
    """|got - exp| <= tol everywhere; infinities have to be equal."""
    got = np.asarray(got, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        same = (got == exp) | (np.abs(got - exp) <= tol)
    if not same.all():
        at = tuple(int(i[0]) for i in np.nonzero(~same))
        with np.errstate(invalid="ignore"):
            worst = np.nanmax(np.where(np.isfinite(exp), np.abs(got - exp) / np.maximum(tol, 1e-300), 0))
        raise AssertionError(f"{what}: {int((~same).sum())} of {same.size} off; first at {at}: got {got[at]}, expected "
                             f"{exp[at]} +- {np.broadcast_to(tol, exp.shape)[at]}; worst {worst:.3g} of the bound")


def layout(lengths, new_tokens, free, table, page_size, capacity):
    """Sequence by sequence, token by token."""
    table = np.array(table, dtype=np.int64)
    slots, row_lengths, row_seqs, starts, taken = [], [], [], [0], 0
    for s, (n, new) in enumerate(zip(lengths, new_tokens)):
        n = min(max(int(n), 0), table.shape[1] * page_size)
        new = min(max(int(new), 0), n)
        for j in range(-(-(n - new) // page_size), -(-n // page_size)):
            table[s, j] = free[taken] if taken < len(free) else -1
            taken += 1
        for p in range(n - new, n):
            page = table[s, p // page_size]
            slots.append(page * page_size + p % page_size if page >= 0 else -1)
            row_lengths.append(p + 1)
            row_seqs.append(s)
        starts.append(starts[-1] + new)

    def padded(x, fill):
        return np.array((x + [fill] * capacity)[:capacity], dtype=np.int64)

    return table, padded(slots, -1), padded(row_lengths, 0), padded(row_seqs, -1), np.array(starts), taken
