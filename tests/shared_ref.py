"""Plain implementations of the operators on shared pages, row by row and page by
page, in Python integers."""

from __future__ import annotations

import numpy as np


def clamp(x, most):
    return min(max(int(x), 0), int(most))


def fork(table, lengths, parents, keep, free, page):
    """(table, lengths, src, dst, tokens, pages) of the new batch."""
    table = np.asarray(table, dtype=np.int64)
    width = table.shape[1]
    most = min(width * page, 1 << 30)
    rows = []
    for i, p in enumerate(parents):
        m = 0
        if 0 <= p < len(lengths):
            m = clamp(lengths[p], most)
            if keep is not None:
                m = clamp(keep[i], m)
        rows.append(m)
    out = np.full((len(parents), width), -1, dtype=np.int64)
    for i, m in enumerate(rows):
        need = -(-m // page)
        if need:
            out[i, :need] = table[parents[i], :need]
    held = out.copy()
    src, dst, tokens, taken = [], [], [], 0
    for i, m in enumerate(rows):
        j = m // page
        last = int(held[i, j]) if m % page else -1
        shared = last >= 0 and any(
            r != i and rows[r] > j * page and held[r, j] == last and (rows[r] >= (j + 1) * page or r < i)
            for r in range(len(rows)))
        if not shared:
            src.append(-1), dst.append(-1), tokens.append(0)
            continue
        got = int(free[taken]) if taken < len(free) else -1
        taken += 1
        out[i, j] = got
        src.append(last), dst.append(got), tokens.append(m % page)
    return out, np.array(rows), np.array(src), np.array(dst), np.array(tokens), taken


def held(table, lengths, page, pages):
    """Every (row, place) that holds a page of the pool."""
    width = np.asarray(table).shape[1]
    for s, n in enumerate(lengths):
        for j in range(-(-clamp(n, min(width * page, 1 << 30)) // page)):
            if 0 <= table[s][j] < pages:
                yield s, j


def refs(table, lengths, page, pages):
    n = np.zeros(pages, dtype=np.int64)
    for s, j in held(table, lengths, page, pages):
        n[table[s][j]] += 1
    return n


def compact(table, lengths, page, pages, limit=None):
    """(table, moves as (from, to), held pages)."""
    n = refs(table, lengths, page, pages)
    live = int((n > 0).sum())
    limit = live if limit is None else limit
    movers = [p for p in range(limit, pages) if n[p]]
    holes = [p for p in range(limit) if not n[p]]
    moves = list(zip(movers, holes))
    to = dict(moves)
    out = np.array(table, dtype=np.int64)
    for s, j in held(table, lengths, page, pages):
        out[s, j] = to.get(int(out[s, j]), int(out[s, j]))
    return out, moves, live


def padded(x, n, fill=-1):
    return np.array(list(x) + [fill] * (n - len(x)), dtype=np.int64)


# ---------------------------------------------------------------------------
# Bounds and the choice of blocks: whole numbers and fp32 roundings as defined
# ---------------------------------------------------------------------------

OVER_127 = np.float32(1) / np.float32(127)
LARGEST = {"bfloat16": 3.3895313892515355e38, "float16": 65504.0, "float8_e4m3fn": 448.0}


def bounds(keys, largest):
    """keys [tokens, dim] in float32: (bounds [2, dim], scale)."""
    k = np.where(np.isnan(keys), np.nan, np.clip(keys, -largest, largest)).astype(np.float32)
    none = np.isnan(k).all(axis=0)
    hi = np.where(none, 0, np.nanmax(np.where(none, 0, k), axis=0)).astype(np.float32)
    lo = np.where(none, 0, np.nanmin(np.where(none, 0, k), axis=0)).astype(np.float32)
    scale = np.float32(max(np.abs(hi).max(), np.abs(lo).max())) * OVER_127
    by = scale if scale != 0 else np.float32(1)
    return np.stack([np.clip(np.ceil(hi / by), -127, 127), np.clip(np.floor(lo / by), -127, 127)]), scale


def scores(q, bound, scale, largest):
    """q [heads, dim] float32, bound [blocks, 2, dim] whole, scale [blocks] float32: a float32 score a block."""
    q = np.where(np.isnan(q), 0, np.clip(q, -largest, largest)).astype(np.float32)
    by = (np.abs(q).max(axis=1) * OVER_127).astype(np.float32)
    whole = np.clip(np.rint(q / np.where(by == 0, np.float32(1), by)[:, None]), -127, 127).astype(np.int64)
    hi, lo = bound[:, 0].astype(np.int64), bound[:, 1].astype(np.int64)
    total = np.maximum(whole, 0) @ hi.T + np.minimum(whole, 0) @ lo.T
    most = np.finfo(np.float32).max
    with np.errstate(over="ignore", invalid="ignore"):
        each = (total.astype(np.float32) * by[:, None]).astype(np.float32).max(axis=0)
        score = (each * scale.astype(np.float32)).astype(np.float32)
    return np.where(np.isnan(score), -most, np.clip(score, -most, most))


def choose(score, there, k, first, last):
    """The k best of one row's blocks, ascending, -1 past the last."""
    n = len(score)
    b = np.arange(n)
    rank = np.where(there, np.where((b < first) | (b >= n - last), 0, 1), 2)  # always taken; by its score; no page
    order = np.lexsort((b, np.where(rank == 1, -score, 0), rank))
    return padded(np.sort(order[:k]), k)
