"""Measured cases of the paged-cache operators for sequences that share pages
and for attention over chosen pages.

Five passes that a server makes: rows of a new batch that take over the pages
of earlier ones, with the copies of their last pages (``fork``), pages that no
row holds any more and the moves that close the gaps (``reclaim``), attention
of rows that share a prefix (``prefix``), bounds of the step's pages and the
choice of pages by them (``select``), and attention over each row's chosen
pages (``blocks``).

``run`` computes them in plain torch operations, or through the package's
entry points where ``own`` is true.
"""

from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZES = {"bf16": 2, "fp16": 2, "e4m3": 1}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # Four samples of each of two requests begin: the smallest call, all latency.
        {"name": "fork_samples", "op": "fork", "seqs": 2, "rows": 8, "min_len": 500, "max_len": 1500, "page": 16,
         "kv_heads": 8, "dim": 128, "store": "bf16", "layers": 1, "cut": False},
        # A step of beams over a large batch: rows go on from any other one, some from a part of it; all layers' last
        # pages are copied.
        {"name": "fork_beams", "op": "fork", "seqs": 512, "rows": 512, "min_len": 1, "max_len": 4096, "page": 64,
         "kv_heads": 4, "dim": 128, "store": "bf16", "layers": 4, "cut": True},
        # Some of a small batch's requests have ended.
        {"name": "reclaim_small", "op": "reclaim", "groups": 4, "fanout": 4, "min_len": 100, "max_len": 2000, "page": 16,
         "kv_heads": 2, "dim": 128, "store": "bf16", "layers": 1, "ended": 0.3},
        # A large pool after half of its requests have ended: thousands of pages move in an 8-bit cache.
        {"name": "reclaim_large", "op": "reclaim", "groups": 1024, "fanout": 2, "min_len": 1, "max_len": 4096,
         "page": 32, "kv_heads": 8, "dim": 128, "store": "e4m3", "layers": 1, "ended": 0.5},
        # Eight samples of one request a little after its prompt.
        {"name": "prefix_samples", "op": "prefix", "groups": 1, "min_rows": 8, "max_rows": 8, "min_shared": 2000,
         "max_shared": 2000, "max_own": 70, "heads": 32, "kv_heads": 8, "dim": 128, "dtype": "bf16", "store": "bf16",
         "page": 16},
        # A batch of 64 requests behind one long system prompt.
        {"name": "prefix_batch", "op": "prefix", "groups": 1, "min_rows": 64, "max_rows": 64, "min_shared": 32768,
         "max_shared": 32768, "max_own": 1024, "heads": 64, "kv_heads": 8, "dim": 128, "dtype": "bf16",
         "store": "bf16", "page": 64},
        # Twelve prompts with few or many samples each, an 8-bit cache, five heads a key-value head.
        {"name": "prefix_groups_e4m3", "op": "prefix", "groups": 12, "min_rows": 1, "max_rows": 32, "min_shared": 500,
         "max_shared": 12000, "max_own": 700, "heads": 40, "kv_heads": 8, "dim": 128, "dtype": "fp16", "store": "e4m3",
         "page": 32},
        # One token of each of 64 requests: the new tokens' pages, then 64 of up to 1024 pages for each row.
        {"name": "select_decode", "op": "select", "seqs": 64, "next_n": 1, "min_len": 1, "max_len": 32768, "heads": 64,
         "kv_heads": 8, "dim": 128, "dtype": "bf16", "store": "bf16", "page": 32, "blocks": 64},
        # Chunks of 256 new tokens over long contexts, each token with a choice of its own.
        {"name": "select_chunk", "op": "select", "seqs": 4, "next_n": 256, "min_len": 20000, "max_len": 50000,
         "heads": 32, "kv_heads": 4, "dim": 128, "dtype": "fp16", "store": "fp16", "page": 16, "blocks": 128},
        # One request with a very long context.
        {"name": "blocks_single", "op": "blocks", "seqs": 1, "next_n": 1, "min_len": 100001, "max_len": 100001,
         "heads": 32, "kv_heads": 8, "dim": 128, "dtype": "bf16", "store": "bf16", "page": 64, "blocks": 32},
        # A decode batch, 64 pages of 32 tokens for each row and key-value head.
        {"name": "blocks_decode", "op": "blocks", "seqs": 64, "next_n": 1, "min_len": 1, "max_len": 32768, "heads": 64,
         "kv_heads": 8, "dim": 128, "dtype": "bf16", "store": "bf16", "page": 32, "blocks": 64},
        # Two tokens a request over an 8-bit cache, heads of 64 dims, an odd number of pages.
        {"name": "blocks_e4m3", "op": "blocks", "seqs": 48, "next_n": 2, "min_len": 3000, "max_len": 16384, "heads": 24,
         "kv_heads": 8, "dim": 64, "dtype": "fp16", "store": "e4m3", "page": 64, "blocks": 37},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fork", "reclaim", "prefix", "prefix", "select", "blocks", "blocks"])
    page = rng.choice([16, 32, 64, 128])
    kv, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    store = rng.choice([dtype, dtype, "e4m3"])
    if op == "fork":
        seqs = _log(rng, 1, 256)
        return {"op": op, "seqs": seqs, "rows": rng.choice([seqs, min(512, _log(rng, seqs, 8 * seqs))]),
                "min_len": 1, "max_len": _log(rng, 64, 4096), "page": min(page, 64), "kv_heads": min(kv, 4), "dim": dim,
                "store": store, "layers": rng.choice([1, 2, 4]), "cut": rng.random() < 0.5}
    if op == "reclaim":
        groups = _log(rng, 1, 512)
        return {"op": op, "groups": groups, "fanout": rng.choice([1, 2, 3, 4]), "min_len": 1,
                "max_len": _log(rng, 64, 4096), "page": max(page, 32), "kv_heads": kv, "dim": dim, "store": "e4m3",
                "layers": 1, "ended": rng.choice([0.1, 0.5, 0.9])}
    heads = kv * rng.choice([1, 3, 4, 8])
    case = {"op": op, "heads": heads, "kv_heads": kv, "dim": dim, "dtype": dtype, "store": store, "page": page}
    if op == "prefix":
        groups = _log(rng, 1, 16)
        rows = _log(rng, 1, max(1, 64 // groups))
        hi = _log(rng, 128, max(129, 32768 // groups))
        return case | {"groups": groups, "min_rows": rng.choice([1, rows]), "max_rows": rows,
                       "min_shared": rng.choice([1, hi]), "max_shared": hi, "max_own": _log(rng, 1, 1000)}
    if rng.random() < 0.3:
        seqs, next_n, hi = 1, _log(rng, 8, 128), _log(rng, 1024, 16384)
    else:
        seqs, next_n = _log(rng, 1, 64), rng.choice([1, 1, 2, 3])
        hi = _log(rng, 64, min(131072, (1 << 20) // (seqs * next_n)))
    return case | {"seqs": seqs, "next_n": next_n, "min_len": rng.choice([1, hi // 2, hi]), "max_len": hi,
                   "blocks": rng.choice([4, 16, 31, 64])}


# ---------------------------------------------------------------------------
# What the case alone gives: lengths, who goes on from whom, who shares what
# ---------------------------------------------------------------------------

def _rng(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _contexts(case):
    """The context length of each sequence."""
    rng = _rng(case)
    return [rng.randint(case["min_len"], case["max_len"]) for _ in range(case["seqs"])]


def _rows(case):
    """[seqs, next_n]: how much of its context each row sees, 0 for rows before the first token."""
    n = case["next_n"]
    return np.maximum(0, np.asarray(_contexts(case))[:, None] - n + 1 + np.arange(n)[None, :]).astype(np.int32)


def _forks(case):
    """Lengths of the batch's rows, and of the new batch: the row that each goes on from, and the tokens it keeps."""
    ctx, rng = _contexts(case), _rng(case)
    seqs, rows = case["seqs"], case["rows"]
    # Samples: as many rows of each.  Beams: any row may be gone on from, some are given up.
    parents = [rng.randrange(seqs) if case["cut"] else r * seqs // rows for r in range(rows)]
    keep = [rng.randint(0, ctx[p]) if case["cut"] and rng.random() < 0.2 else ctx[p] for p in parents]
    return ctx, parents, keep


def _copies(case):
    """(row, tokens) of the new rows whose last page is copied."""
    ctx, parents, keep = _forks(case)
    page, users = case["page"], {}
    for r, (p, m) in enumerate(zip(parents, keep)):
        for j in {m // page} if m % page else set():
            users.setdefault((p, j), []).append(r)
    found = []
    for (p, j), rows in users.items():
        whole = any(q == p and m >= (j + 1) * page for q, m in zip(parents, keep))
        found += [(r, keep[r] % page) for r in (rows if whole else rows[1:])]
    return sorted(found)


def _held(case):
    """Rows of a pool part of whose requests have ended: for each its pages, in a pool that they and the ended ones
    filled; the tokens of each; the pages of the pool."""
    rng, page = _rng(case), case["page"]
    rows, lengths, used = [], [], 0
    for _ in range(case["groups"]):
        first = rng.randint(case["min_len"], case["max_len"])  # the request's prompt: its whole pages are shared
        shared = list(range(used, used + first // page))
        used += first // page
        for _ in range(case["fanout"]):
            n = first + rng.randint(0, case["page"] * 2)
            more = -(-n // page) - len(shared)
            rows.append(shared + list(range(used, used + more)))
            used += more
            lengths.append(0 if rng.random() < case["ended"] else n)
    return rows, lengths, used + 5


def _groups(case):
    """For each group of rows: the tokens that it shares (whole pages), and each row's length."""
    rng, found = _rng(case), []
    for _ in range(case["groups"]):
        shared = rng.randint(case["min_shared"], case["max_shared"]) // case["page"] * case["page"]
        rows = rng.randint(case["min_rows"], case["max_rows"])
        found.append((shared, [shared + rng.randint(1, case["max_own"]) for _ in range(rows)]))
    return found


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEVICE)


def _normal(gen, shape, dtype, by=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16 if dtype == torch.float8_e4m3fn else dtype, device=DEVICE)
    x.normal_(generator=gen)
    return (x * by).to(dtype) if by != 1.0 or dtype == torch.float8_e4m3fn else x


def _table(rows, pages, gen):
    """A block table from each row's page numbers, shuffled over the pool; -1 past a row's last."""
    width = max(1, max(len(r) for r in rows))
    at = np.full((len(rows), width), -1, dtype=np.int64)
    for r, x in enumerate(rows):
        at[r, :len(x)] = x
    order = torch.randperm(pages, generator=gen, device=DEVICE)
    at = torch.as_tensor(at, device=DEVICE)
    return torch.where(at >= 0, order[at.clamp(min=0)], -1).to(torch.int32).contiguous(), order


def _apart(lengths, page):
    """Pages of rows that share none."""
    rows, used = [], 0
    for n in lengths:
        need = -(-int(n) // page)
        rows.append(range(used, used + need))
        used += need
    return rows, used


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    op, page, kv, dim = case["op"], case["page"], case["kv_heads"], case["dim"]
    store = DTYPES[case["store"]]
    e4m3 = store == torch.float8_e4m3fn
    if op in ("fork", "reclaim"):
        if op == "fork":
            ctx, parents, keep = _forks(case)
            rows, used = _apart(ctx, page)
            spare = case["rows"] + 7
            table, order = _table(rows, used + spare, gen)
            state = {"table": table, "lengths": _i32(ctx), "parents": _i32(parents), "pages": used + spare,
                     "keep": _i32(keep) if case["cut"] else None, "free": order[used:].to(torch.int32)}
        else:
            rows, lengths, pages = _held(case)
            table, _ = _table(rows, pages, gen)
            state = {"table": table, "lengths": _i32(lengths), "pages": pages}
        # All layers' keys and values in one allocation, an entry of the list for each.
        caches = _normal(gen, (2 * case["layers"], state["pages"], page, kv, dim), store)
        return state | {"case": case, "caches": caches, "views": list(caches.unbind(0))}
    heads, dtype = case["heads"], DTYPES[case["dtype"]]
    if op == "prefix":
        groups, rows, used = _groups(case), [], 0
        for shared, lengths in groups:
            first, used = list(range(used, used + shared // page)), used + shared // page
            for n in lengths:
                more = -(-n // page) - len(first)
                rows.append(first + list(range(used, used + more)))
                used += more
        lengths = [n for _, x in groups for n in x]
        state = {"starts": _i32(np.cumsum([0] + [len(x) for _, x in groups])), "shared": _i32([s for s, _ in groups]),
                 "lengths": _i32(lengths), "most_shared": max(s for s, _ in groups),
                 "most_own": max(n - s for s, x in groups for n in x), "most_rows": max(len(x) for _, x in groups)}
        count = len(lengths)
    else:
        lengths = _rows(case)
        rows, used = _apart(_contexts(case), page)
        state = {"lengths": torch.as_tensor(lengths, device=DEVICE)}
        count = lengths.size
    pages = used + 3
    state |= {"case": case, "table": _table(rows, pages, gen)[0], "q": _normal(gen, (count, heads, dim), dtype),
              "k_cache": _normal(gen, (pages, page, kv, dim), store, 25.0 if e4m3 else 1.0)}
    if op == "select":
        ctx = np.asarray(_contexts(case))
        new = np.minimum(ctx, case["next_n"])
        # Keys of a page point one way more or less, so that some pages matter more than others.
        for k in state["k_cache"].split(4096):
            k.copy_((k.float() + _normal(gen, (k.shape[0], 1, kv, dim), dtype, 12.0 if e4m3 else 0.5).float()).to(store))
        bounds, scales = _bounds_of(state["k_cache"].amin(1).float(), state["k_cache"].amax(1).float()) if not e4m3 else \
            _bounds_of(*(torch.cat([f(k.float(), 1) for k in state["k_cache"].split(4096)]) for f in (torch.amin, torch.amax)))
        return state | {"contexts": _i32(ctx), "starts": _i32(np.concatenate([[0], np.cumsum(new)])),
                        "tokens": int(new.sum()), "bounds": bounds, "scales": scales, "page": page,
                        "most_new": int(new.max()) // page + 2}
    state |= {"v_cache": _normal(gen, (pages, page, kv, dim), store, 25.0 if e4m3 else 1.0),
              "k_scale": torch.rand(kv, generator=gen, device=DEVICE) * 0.02 + 0.03 if e4m3 else None,
              "v_scale": torch.rand(kv, generator=gen, device=DEVICE) * 0.02 + 0.03 if e4m3 else None,
              "softmax_scale": 1 / math.sqrt(dim)}
    if op == "blocks":
        # Distinct pages of each row's context, its last one among them, ascending, -1 past the last.
        flat = state["lengths"].reshape(-1, 1, 1)
        have = (flat + page - 1) // page
        width = max(state["table"].shape[1], case["blocks"])
        x = torch.rand((count, kv, width), generator=gen, device=DEVICE)
        b = torch.arange(width, device=DEVICE)
        x = torch.where(b == have - 1, 2.0, torch.where(b < have, x, -1.0))
        v, at = x.topk(case["blocks"], dim=2)
        at = torch.where(v >= 0, at, width).sort(dim=2).values
        state |= {"blocks": torch.where(at < have, at, -1).to(torch.int32).contiguous()}
    return state


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    if own:
        return _own(state)
    return {"fork": _fork, "reclaim": _reclaim, "prefix": _prefix, "select": _select,
            "blocks": _blocks}[state["case"]["op"]](state)


def _own(s):
    import row_radix_top_amd as rrt

    case = s["case"]
    op, page = case["op"], case["page"]
    if op == "fork":
        f = rrt.paged_fork(s["table"], s["lengths"], s["parents"], s["free"], page_size=page, keep=s["keep"])
        rrt.paged_copy(f.src, f.dst, s["views"], tokens=f.tokens)
        return {"table": f.table, "lengths": f.lengths, "src": f.src, "dst": f.dst, "tokens": f.tokens,
                "pages": f.pages, "caches": s["caches"]}
    if op == "reclaim":
        p = rrt.paged_free(s["table"], s["lengths"], page_size=page, num_pages=s["pages"])
        c = rrt.paged_compact(s["table"], s["lengths"], page_size=page, num_pages=s["pages"])
        rrt.paged_copy(c.src, c.dst, s["views"])
        return {"free": p.free, "refs": p.refs, "count": p.count, "table": c.table, "src": c.src, "dst": c.dst,
                "moves": c.moves, "live": c.live, "caches": s["caches"]}
    if op == "prefix":
        out, lse = rrt.paged_prefix_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["starts"],
                                              s["shared"], softmax_scale=s["softmax_scale"], k_scale=s["k_scale"],
                                              v_scale=s["v_scale"])
        return {"out": out, "lse": lse}
    if op == "select":
        rrt.paged_bounds(s["k_cache"], s["table"], s["starts"], s["contexts"], s["bounds"], s["scales"],
                         num_tokens=s["tokens"])
        blocks = rrt.paged_block_select(s["q"], s["bounds"], s["scales"], s["table"], s["lengths"], page_size=page,
                                        num_blocks=case["blocks"])
        return {"bounds": s["bounds"], "scales": s["scales"], "blocks": blocks}
    out, lse = rrt.paged_block_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["blocks"],
                                         softmax_scale=s["softmax_scale"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _copy_pages(caches, src, dst, tokens=None):
    """The first `tokens` tokens of pages src go to pages dst, in every cache."""
    real = dst >= 0
    src, dst = src[real].long(), dst[real].long()
    if tokens is None:
        caches[:, dst] = caches[:, src]
        return
    bits = caches.view(torch.uint8)
    goes = torch.arange(caches.shape[2], device=caches.device) < tokens[real][:, None]
    bits[:, dst] = torch.where(goes[None, :, :, None, None], bits[:, src], bits[:, dst])


def _fork(s):
    page, table, free = s["case"]["page"], s["table"], s["free"]
    n, width = s["parents"].numel(), table.shape[1]
    p = s["parents"].long()
    known = (p >= 0) & (p < table.shape[0])
    p = torch.where(known, p, 0)
    m = torch.where(known, s["lengths"].long()[p], 0)
    if s["keep"] is not None:
        m = torch.minimum(m, s["keep"].long().clamp(min=0))
    last, part = (m // page).clamp(max=width - 1), m % page
    j = torch.arange(width, device=table.device)
    rows = torch.where(j < ((m + page - 1) // page)[:, None], table[p], -1)
    held = rows.gather(1, last[:, None])
    others = rows[:, last].t()  # [row, another row's page at the same place]
    whole = m >= ((last + 1) * page)[:, None]
    earlier = torch.arange(n, device=table.device) < torch.arange(n, device=table.device)[:, None]
    copied = (part > 0) & (held[:, 0] >= 0) & ((others == held) & (whole | earlier)).any(1)
    order = copied.cumsum(0) - 1
    got = torch.where(copied & (order < free.numel()), free[order.clamp(0, free.numel() - 1)], -1)
    rows = torch.where(copied[:, None] & (j == last[:, None]), got[:, None], rows)
    src = torch.where(copied, held[:, 0], -1)
    tokens = torch.where(copied, part, 0).to(torch.int32)
    _copy_pages(s["caches"], src, got, tokens)
    return {"table": rows, "lengths": m.to(torch.int32), "src": src, "dst": got, "tokens": tokens,
            "pages": copied.sum().reshape(1).to(torch.int32), "caches": s["caches"]}


def _reclaim(s):
    page, table, pages = s["case"]["page"], s["table"].long(), s["pages"]
    need = (s["lengths"].long() + page - 1) // page
    held = (torch.arange(table.shape[1], device=table.device) < need[:, None]) & (table >= 0) & (table < pages)
    refs = torch.zeros(pages + 1, dtype=torch.int64, device=table.device)
    refs.index_add_(0, torch.where(held, table, pages).reshape(-1), held.reshape(-1).long())
    refs = refs[:pages]
    at = torch.arange(pages, device=table.device)
    free = refs == 0
    listed_first = torch.where(free, at, pages).sort().values
    live = pages - free.sum()
    movers = torch.where(~free & (at >= live), at, pages).sort().values[:pages // 2]
    holes = torch.where(free & (at < live), at, pages).sort().values[:pages // 2]
    goes = (movers < pages) & (holes < pages)
    src, dst = torch.where(goes, movers, -1), torch.where(goes, holes, -1)
    moved = torch.arange(pages + 1, device=table.device)
    moved[torch.where(goes, movers, pages)] = torch.where(goes, holes, pages)
    new = torch.where(held, moved[torch.where(held, table, 0)], table)
    _copy_pages(s["caches"].view(torch.uint8), src, dst)
    i32 = torch.int32
    return {"free": torch.where(listed_first < pages, listed_first, -1).to(i32), "refs": refs.to(i32),
            "count": free.sum().reshape(1).to(i32), "table": new.to(i32), "src": src.to(i32), "dst": dst.to(i32),
            "moves": goes.sum().reshape(1).to(i32), "live": live.reshape(1).to(i32), "caches": s["caches"]}


def _softmax(x):
    """Probabilities and log-sum-exp over the last axis; zeros and -inf where nothing is left."""
    top = x.amax(-1, keepdim=True)
    p = (x - torch.where(top == -math.inf, 0.0, top)).exp()
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, 1.0, total), (top + total.log()).squeeze(-1)


def _slots(table, pos, seen, page):
    """Slots of positions pos [n, m] of the table's rows, and whether each counts."""
    at = table.long().gather(1, torch.where(seen, pos, 0) // page)
    seen = seen & (at >= 0)
    return torch.where(seen, at * page + torch.where(seen, pos, 0) % page, 0), seen


def _keys_values(s, slots, seen):
    kv, dim = s["case"]["kv_heads"], s["case"]["dim"]
    k, v = (s[c].view(-1, kv, dim)[slots].float() for c in ("k_cache", "v_cache"))
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"][:, None], v * s["v_scale"][:, None]
    return k, torch.where(seen[..., None, None], v, 0.0)


def _prefix(s):
    """The shared part of each group at once, the rows' own parts beside it, one softmax over both."""
    page, kv, dim = s["case"]["page"], s["case"]["kv_heads"], s["case"]["dim"]
    table, lengths, shared, starts = s["table"], s["lengths"].long(), s["shared"].long(), s["starts"].long()
    rows, most, wide, dev = lengths.numel(), s["most_shared"], s["most_rows"], table.device
    row = torch.arange(rows, device=dev)
    group = torch.searchsorted(starts, row, right=True) - 1
    place = row - starts[group]
    q = s["q"].float().view(rows, kv, -1, dim)
    each = q.shape[2]
    together = q.new_zeros(shared.numel(), wide, kv, each, dim)
    together[group, place] = q
    pos = torch.arange(most, device=dev).expand(shared.numel(), -1)
    slots, seen = _slots(table[starts[:-1]], pos, pos < shared[:, None], page)
    k, v = _keys_values(s, slots, seen)
    x = torch.matmul(together.permute(0, 2, 1, 3, 4).reshape(-1, kv, wide * each, dim), k.permute(0, 2, 3, 1).contiguous())
    x = torch.where(seen[:, None, None], x * s["softmax_scale"], -math.inf)
    first = x.view(-1, kv, wide, each, most).permute(0, 2, 1, 3, 4)[group, place]
    pos = shared[group][:, None] + torch.arange(s["most_own"], device=dev)
    slots, own_seen = _slots(table, pos, pos < lengths[:, None], page)
    own_k, own_v = _keys_values(s, slots, own_seen)
    y = torch.matmul(q, own_k.permute(0, 2, 3, 1).contiguous()) * s["softmax_scale"]
    p, lse = _softmax(torch.cat([first, torch.where(own_seen[:, None, None], y, -math.inf)], dim=-1))
    weights = p.new_zeros(shared.numel(), wide, kv, each, most)
    weights[group, place] = p[..., :most]
    out = torch.matmul(weights.permute(0, 2, 1, 3, 4).reshape(-1, kv, wide * each, most), v.transpose(1, 2).contiguous())
    out = out.view(-1, kv, wide, each, dim).permute(0, 2, 1, 3, 4)[group, place]
    out = out + torch.matmul(p[..., most:], own_v.transpose(1, 2).contiguous())
    return {"out": out.reshape(rows, -1, dim).to(s["q"].dtype), "lse": lse.reshape(rows, -1)}


def _bounds_of(lo, hi):
    """Bounds [..., 2, dim] in 8 bits, the largest and the smallest, rounded outward; their scale."""
    scale = torch.maximum(lo.abs(), hi.abs()).amax(-1) / 127
    by = torch.where(scale == 0, 1.0, scale)[..., None]
    both = torch.stack([(hi / by).ceil(), (lo / by).floor()], dim=-2)
    return both.clamp(-127, 127).to(torch.int8), scale


def _select(s):
    case, page, table = s["case"], s["case"]["page"], s["table"].long()
    kv, dim, n = case["kv_heads"], case["dim"], case["next_n"]
    dev, contexts = table.device, s["contexts"].long()
    # Bounds of the pages that hold new tokens, from all their tokens.
    new = (s["starts"][1:] - s["starts"][:-1]).long()
    j = ((contexts - new) // page)[:, None] + torch.arange(s["most_new"], device=dev)
    touched = (j * page < contexts[:, None]) & (new > 0)[:, None]
    seq, j = touched.nonzero(as_tuple=True)[0], j[touched]
    at = table[seq, j]
    k = s["k_cache"][at].float()
    inside = (j[:, None] * page + torch.arange(page, device=dev) < contexts[seq][:, None])[..., None, None]
    bounds, scales = _bounds_of(torch.where(inside, k, math.inf).amin(1), torch.where(inside, k, -math.inf).amax(1))
    s["bounds"][at], s["scales"][at] = bounds, scales
    # Scores: the queries in 8 bits; sums of whole numbers are exact in any order.
    seqs, rows = table.shape[0], s["q"].shape[0]
    q = s["q"].float()
    by = q.abs().amax(-1) / 127
    q = (q / torch.where(by == 0, 1.0, by)[..., None]).round().clamp(-127, 127)
    q = torch.cat([q.clamp(min=0), q.clamp(max=0)], dim=-1).view(seqs, n, kv, -1, 2 * dim)
    each = q.shape[3]
    held = table.clamp(min=0)
    b = s["bounds"][held].view(seqs, -1, kv, 2 * dim).permute(0, 2, 3, 1).float().contiguous()
    x = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(seqs, kv, n * each, 2 * dim), b).view(seqs, kv, n, each, -1)
    x = (x * by.view(seqs, n, kv, each).permute(0, 2, 1, 3)[..., None]).amax(3)
    x = (x * s["scales"][held].permute(0, 2, 1)[:, :, None]).permute(0, 2, 1, 3).reshape(rows, kv, -1)
    # The first and the last page always, pages that are none never.
    block = torch.arange(x.shape[-1], device=dev)
    have = ((s["lengths"].reshape(-1).long() + page - 1) // page)[:, None, None]
    there = ((table >= 0).repeat_interleave(n, 0)[:, None] & (block < have)).expand(-1, kv, -1)
    x = torch.where((block < 1) | (block >= have - 1), math.inf, x)
    order = torch.where(there, x, -math.inf).sort(dim=-1, descending=True, stable=True).indices[..., :case["blocks"]]
    if order.shape[-1] < case["blocks"]:
        order = torch.cat([order, order.new_full((rows, kv, case["blocks"] - order.shape[-1]), x.shape[-1])], dim=-1)
    order = torch.where(order < have, order, 1 << 30).sort(dim=-1).values
    return {"bounds": s["bounds"], "scales": s["scales"],
            "blocks": torch.where(order < 1 << 30, order, -1).to(torch.int32)}


def _blocks(s):
    page, kv, dim = s["case"]["page"], s["case"]["kv_heads"], s["case"]["dim"]
    rows = s["q"].shape[0]
    lengths = s["lengths"].reshape(-1).long()[:, None]
    blocks = s["blocks"].long()
    pos = (blocks[..., None] * page + torch.arange(page, device=blocks.device)).view(rows, -1)
    seen = (blocks >= 0)[..., None].expand(-1, -1, -1, page).reshape(rows, -1) & (pos < lengths)
    slots, seen = _slots(s["table"].repeat_interleave(s["case"]["next_n"], 0), pos, seen, page)
    slots, seen = slots.view(rows, kv, -1), seen.view(rows, kv, -1)
    head = torch.arange(kv, device=slots.device)[:, None]
    k, v = (s[c].view(-1, kv, dim)[slots, head].float() for c in ("k_cache", "v_cache"))
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"][:, None, None], v * s["v_scale"][:, None, None]
    v = torch.where(seen[..., None], v, 0.0)
    x = torch.matmul(s["q"].float().view(rows, kv, -1, dim), k.transpose(2, 3).contiguous()) * s["softmax_scale"]
    p, lse = _softmax(torch.where(seen[:, :, None], x, -math.inf))
    return {"out": torch.matmul(p, v).reshape(rows, -1, dim).to(s["q"].dtype), "lse": lse.reshape(rows, -1)}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    page, op = case["page"], case["op"]
    token = case["kv_heads"] * case["dim"] * SIZES[case["store"]]  # keys, or values, of a token
    if op == "fork":
        ctx, _, keep = _forks(case)
        width = -(-max(ctx) // page)
        held = sum(-(-m // page) for m in keep)
        moved = sum(t for _, t in _copies(case))
        return {"bytes": 4 * (held + case["rows"] * (width + 6) + len(ctx)) + 4 * case["layers"] * moved * token,
                "flops": 0}
    if op == "reclaim":
        rows, lengths, pages = _held(case)
        width = max(len(r) for r in rows)
        live = len({p for r, n in zip(rows, lengths) if n for p in r})
        held = sum(-(-n // page) for n in lengths)
        # Shuffled over the pool, this share of the live pages lies past their number.
        moves = int(live * (pages - live) / pages)
        return {"bytes": 4 * (held + len(rows) * (1 + width) + 2 * pages + 2 * (pages // 2))
                + 4 * case["layers"] * moves * page * token, "flops": 0}
    item, heads, dim = SIZES[case["dtype"]], case["heads"], case["dim"]
    if op == "prefix":
        groups = _groups(case)
        rows = sum(len(x) for _, x in groups)
        read = sum(s + sum(n - s for n in x) for s, x in groups)
        pairs = sum(n for _, x in groups for n in x)
        return {"bytes": 2 * read * token + rows * heads * (2 * dim * item + 4) + 4 * read // page + 4 * rows,
                "flops": 4 * pairs * heads * dim}
    seen = _rows(case)
    have = -(-seen // page)
    rows = seen.size
    if op == "select":
        ctx = np.asarray(_contexts(case))
        new = np.minimum(ctx, case["next_n"])
        first = (ctx - new) // page
        fresh = int((-(-ctx // page) - first).sum())
        pages = int((-(-ctx // page)).sum())
        one = case["kv_heads"] * (2 * dim + 4)
        return {"bytes": int((ctx - first * page).sum()) * token + fresh * one + pages * (one + 4)
                + rows * (heads * dim * item + 4 + 4 * case["kv_heads"] * case["blocks"]),
                "flops": 4 * int(have.sum()) * heads * dim}
    took = np.minimum(have, case["blocks"])
    # Its last page among them, a row sees all but what that page lacks.
    pairs = int((took * page - (have * page - seen)).sum())
    # Rows of a sequence may choose the same pages: at least what one of them reads, at most what there is.
    read = int((took * page - (have * page - seen)).max(1).sum())
    return {"bytes": 2 * read * token + rows * heads * (2 * dim * item + 4) + 4 * rows * (1 + case["kv_heads"] * case["blocks"]),
            "flops": 4 * pairs * heads * dim}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _row_attention(q, k, v, scale):
    """Heads q [h, d] over their keys [n, d] and values [n, e], in 64 bits."""
    if k.shape[0] == 0:
        return q.new_zeros(q.shape[0], v.shape[1]), q.new_full((q.shape[0],), -math.inf)
    x = (q @ k.T) * scale
    lse = torch.logsumexp(x, dim=1)
    return torch.exp(x - lse[:, None]) @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "fork":
        return _exact_fork(s)
    if case["op"] == "reclaim":
        return _exact_reclaim(s)
    if case["op"] == "select":
        return _exact_select(s)
    page, kv, group = case["page"], case["kv_heads"], case["heads"] // case["kv_heads"]
    table = s["table"].cpu().numpy().astype(np.int64)
    outs, lses = [], []
    by = (1.0, 1.0) if s["k_scale"] is None else (s["k_scale"].double(), s["v_scale"].double())
    for r, n in enumerate(s["lengths"].reshape(-1).tolist()):
        own_table = table[r // case.get("next_n", 1)]
        out, lse = [], []
        for h in range(kv):
            pos = np.arange(n)
            if case["op"] == "blocks":
                pos = np.concatenate([np.arange(b * page, min(n, (b + 1) * page)) for b in s["blocks"][r, h].tolist() if b >= 0]
                                     or [pos[:0]])
            at = torch.as_tensor(own_table[pos // page] * page + pos % page, device=DEVICE)
            k, v = (s[c].view(-1, kv, case["dim"])[at, h].double() for c in ("k_cache", "v_cache"))
            if s["k_scale"] is not None:
                k, v = k * by[0][h], v * by[1][h]
            o, x = _row_attention(s["q"][r, h * group:(h + 1) * group].double(), k, v, s["softmax_scale"])
            out.append(o)
            lse.append(x)
        outs.append(torch.cat(out))
        lses.append(torch.cat(lse))
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}


def _exact_fork(s):
    """Row by row; a page may be written on by one row alone."""
    page, table, free = s["case"]["page"], s["table"].cpu().numpy(), s["free"].tolist()
    ctx, parents = s["lengths"].tolist(), s["parents"].tolist()
    m = [ctx[p] if s["keep"] is None else min(ctx[p], k) for p, k in
         zip(parents, parents if s["keep"] is None else s["keep"].tolist())]
    new = np.full((len(parents), table.shape[1]), -1, np.int32)
    full, held_by = set(), {}
    for r, p in enumerate(parents):
        need = -(-m[r] // page)
        new[r, :need] = table[p, :need]
        full.update(int(x) for x in new[r, :m[r] // page])
    src, dst, tokens, taken = [], [], [], 0
    caches = s["caches"].clone()
    for r, n in enumerate(m):
        last = int(new[r, n // page]) if n % page else -1
        if last < 0 or (last not in full and held_by.setdefault(last, r) == r):
            src.append(-1), dst.append(-1), tokens.append(0)
            continue
        to, taken = free[taken], taken + 1
        new[r, n // page] = to
        src.append(last), dst.append(to), tokens.append(n % page)
        caches.view(torch.uint8)[:, to, :n % page] = s["caches"].view(torch.uint8)[:, last, :n % page]
    i32 = np.int32
    return {"table": new, "lengths": np.asarray(m, i32), "src": np.asarray(src, i32), "dst": np.asarray(dst, i32),
            "tokens": np.asarray(tokens, i32), "pages": np.asarray([taken], i32), "caches": caches}


def _exact_reclaim(s):
    page, pages = s["case"]["page"], s["pages"]
    table, lengths = s["table"].cpu().numpy(), s["lengths"].tolist()
    refs = np.zeros(pages, np.int32)
    for row, n in zip(table, lengths):
        for p in row[:-(-n // page)]:
            refs[p] += 1
    free, live = [p for p in range(pages) if refs[p] == 0], int((refs > 0).sum())
    movers, holes = [p for p in range(live, pages) if refs[p]], [p for p in free if p < live]
    moved = dict(zip(movers, holes))
    new, caches = table.copy(), s["caches"].clone()
    for r, n in enumerate(lengths):
        new[r, :-(-n // page)] = [moved.get(p, p) for p in table[r, :-(-n // page)].tolist()]
    caches.view(torch.uint8)[:, list(moved.values())] = s["caches"].view(torch.uint8)[:, list(moved)]

    def padded(x, n):
        return np.asarray(list(x) + [-1] * (n - len(x)), np.int32)

    return {"free": padded(free, pages), "refs": refs, "count": np.asarray([len(free)], np.int32), "table": new,
            "src": padded(moved, pages // 2), "dst": padded(moved.values(), pages // 2),
            "moves": np.asarray([len(moved)], np.int32), "live": np.asarray([live], np.int32), "caches": caches}


def _exact_select(s):
    """The scales in 64 bits; the bounds and the choice are whole numbers."""
    page, table, scales = s["case"]["page"], s["table"].tolist(), s["scales"].double()
    starts = s["starts"].tolist()
    for b, n in enumerate(s["contexts"].tolist()):
        new = starts[b + 1] - starts[b]
        for j in range((n - new) // page, -(-n // page) if new else 0):
            k = s["k_cache"][table[b][j], :min(page, n - j * page)].double()
            scales[table[b][j]] = k.abs().amax((0, 2)) / 127
    return {"bounds": None, "scales": scales, "blocks": None}
