"""Measured cases of the paged-cache operators around the ragged top-K.

Five operators of one serving step over a paged cache: the block tables and
slot maps of the step (``layout``), the write of its new tokens (``append``),
attention of each row over its sequence's cached keys and values, all of them
or the positions a top-K chose (``attention``), the same over one shared latent
vector a token in the absorbed form (``latent``), and the expanded form for
chunks of new tokens (``prefill``).

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
E4M3_MAX = 448.0
NOPE, ROPE, VALUE = 128, 64, 128  # the expanded form's head: keys of NOPE + ROPE, values of VALUE


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One decode step of 64 requests, contexts up to 32768: the smallest call, all latency.
        {"name": "layout_decode", "op": "layout", "seqs": 64, "min_len": 1, "max_len": 32768, "new_min": 1,
         "new_max": 1, "page": 32, "short": False},
        # A large step that mixes single tokens with long chunks, its batch padded past the last token.
        {"name": "layout_mixed", "op": "layout", "seqs": 2048, "min_len": 1, "max_len": 16384, "new_min": 1,
         "new_max": 257, "page": 16, "short": False},
        # The new token of each of 64 requests, keys and values of 8 heads.
        {"name": "append_decode", "op": "append", "kind": "kv", "tokens": 64, "heads": 8, "dim": 128,
         "dtype": "bf16", "store": "bf16", "page": 32},
        # A prefill chunk's latent vectors, rounded to 8 bits on the way in.
        {"name": "append_latent_e4m3", "op": "append", "kind": "latent", "tokens": 16000, "heads": 1, "dim": 512,
         "dtype": "bf16", "store": "e4m3", "page": 64},
        # Four requests of exactly 8192 tokens: a small decode batch, split over the cache's length.
        {"name": "attention_small", "op": "attention", "seqs": 4, "next_n": 1, "min_len": 8192, "max_len": 8192,
         "heads": 32, "kv_heads": 8, "dim": 128, "dtype": "bf16", "store": "bf16", "page": 16, "top": 0},
        # A ragged decode batch, 64 requests of 1 to 32768 tokens: bound by reading the cache.
        {"name": "attention_ragged", "op": "attention", "seqs": 64, "next_n": 1, "min_len": 1, "max_len": 32768,
         "heads": 64, "kv_heads": 8, "dim": 128, "dtype": "bf16", "store": "bf16", "page": 32, "top": 0},
        # Two tokens a request, each over its own 2048 chosen positions of an 8-bit cache.
        {"name": "attention_chosen_e4m3", "op": "attention", "seqs": 32, "next_n": 2, "min_len": 16384,
         "max_len": 65536, "heads": 40, "kv_heads": 4, "dim": 128, "dtype": "bf16", "store": "e4m3", "page": 64,
         "top": 2048},
        # One request, an odd head count and an odd length: the smallest latent call.
        {"name": "latent_single", "op": "latent", "seqs": 1, "next_n": 1, "min_len": 8191, "max_len": 8191,
         "heads": 20, "dim": 512, "dtype": "fp16", "store": "fp16", "page": 16, "top": 0},
        # A decode step of 64 requests over 2048 chosen positions each.
        {"name": "latent_chosen", "op": "latent", "seqs": 64, "next_n": 1, "min_len": 1, "max_len": 32768,
         "heads": 128, "dim": 512, "dtype": "bf16", "store": "bf16", "page": 32, "top": 2048},
        # Two chunks of 512 new tokens, each token over 1024 chosen positions of an 8-bit cache.
        {"name": "latent_rows_e4m3", "op": "latent", "seqs": 2, "next_n": 512, "min_len": 12288, "max_len": 16384,
         "heads": 64, "dim": 512, "dtype": "bf16", "store": "e4m3", "page": 64, "top": 1024},
        # Ragged chunks over longer contexts.
        {"name": "prefill_chunks", "op": "prefill", "seqs": 3, "min_len": 1500, "max_len": 5000, "new_min": 1,
         "new_max": 1200, "heads": 24, "dim": 512, "dtype": "fp16", "store": "fp16", "page": 32},
        # One prompt of 8192 tokens: the largest call.
        {"name": "prefill_long", "op": "prefill", "seqs": 1, "min_len": 8192, "max_len": 8192, "new_min": 8192,
         "new_max": 8192, "heads": 32, "dim": 512, "dtype": "bf16", "store": "bf16", "page": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layout", "append", "attention", "attention", "latent", "latent", "prefill"])
    page = rng.choice([16, 32, 64, 128])
    if op == "layout":
        seqs = _log(rng, 1, 2048)
        hi = _log(rng, 64, min(131072, (1 << 24) // seqs))
        new = rng.choice([1, 2, 4, min(hi, max(1, 262144 // seqs))])
        return {"op": op, "seqs": seqs, "min_len": rng.choice([1, new, hi]) if hi >= new else 1, "max_len": hi,
                "new_min": 1, "new_max": min(new, hi), "page": page, "short": rng.random() < 0.2}
    dtype = rng.choice(["bf16", "fp16"])
    store = rng.choice([dtype, dtype, "e4m3"])
    if op == "append":
        kind = rng.choice(["kv", "latent"])
        return {"op": op, "kind": kind, "tokens": _log(rng, 1, 12000), "heads": rng.choice([1, 2, 4, 8]) if kind == "kv" else 1,
                "dim": rng.choice([64, 128]) if kind == "kv" else rng.choice([256, 512]), "dtype": dtype,
                "store": store, "page": page}
    if op == "prefill":
        seqs, heads = _log(rng, 1, 16), rng.choice([4, 8, 20, 32])
        hi = _log(rng, 64, max(65, int(8192 / math.sqrt(seqs))))
        return {"op": op, "seqs": seqs, "min_len": max(1, hi // 4), "max_len": hi, "new_min": 1,
                "new_max": _log(rng, 1, hi), "heads": heads, "dim": rng.choice([256, 512]), "dtype": dtype,
                "store": store, "page": page}
    top = rng.choice([0, 512, 1024, 2048])
    if top and rng.random() < 0.3:
        seqs, next_n, hi = 1, _log(rng, 16, 256), _log(rng, 1024, 16384)
    else:
        seqs, next_n = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 3])
        hi = _log(rng, 64, min(131072, (1 << 20) // (seqs * next_n)))
    case = {"op": op, "seqs": seqs, "next_n": next_n, "min_len": rng.choice([1, hi // 2, hi]), "max_len": hi}
    if op == "attention":
        kv = rng.choice([1, 2, 4, 8])
        case |= {"heads": kv * rng.choice([1, 3, 4, 8, 16]), "kv_heads": kv, "dim": rng.choice([64, 128])}
    else:
        case |= {"heads": rng.choice([8, 20, 32, 64, 128]), "dim": rng.choice([256, 512])}
    case |= {"dtype": dtype, "store": store, "page": page, "top": top}
    return case


def _lengths(case):
    """The context length of each sequence and its new tokens: a ragged batch that the case alone gives."""
    rng = random.Random("%d %d %d" % (case["seqs"], case["min_len"], case["max_len"]))
    ctx = [rng.randint(case["min_len"], case["max_len"]) for _ in range(case["seqs"])]
    if "next_n" in case:
        return ctx, [min(case["next_n"], c) for c in ctx]
    # Three in four of a mixed step's sequences decode one token.
    mixed = case["new_max"] > 8 and case["seqs"] > 64
    new = [1 if mixed and rng.random() < 0.75 else rng.randint(case["new_min"], case["new_max"]) for _ in ctx]
    return ctx, [min(a, b) for a, b in zip(new, ctx)]


def _rows(case):
    """[seqs, next_n]: how much of its context each row sees, 0 for rows before the first token."""
    ctx, _ = _lengths(case)
    n = case["next_n"]
    return np.maximum(0, np.asarray(ctx)[:, None] - n + 1 + np.arange(n)[None, :]).astype(np.int32)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEVICE)


def _pages(case, ctx, gen):
    """A block table of shuffled pages (-1 past a sequence's last) and the pool's page count."""
    need = [-(-c // case["page"]) for c in ctx]
    total, width = sum(need), max(1, -(-case["max_len"] // case["page"]))
    pages = torch.randperm(total + 2, generator=gen, device=DEVICE).to(torch.int32)
    at = torch.as_tensor(np.cumsum([0] + need[:-1]), device=DEVICE)[:, None] + torch.arange(width, device=DEVICE)
    inside = torch.arange(width, device=DEVICE) < _i32(need)[:, None]
    return torch.where(inside, pages[at.clamp(max=total + 1)], -1).to(torch.int32).contiguous(), total + 2


def _normal(gen, shape, dtype, by=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16 if dtype == torch.float8_e4m3fn else dtype, device=DEVICE)
    x.normal_(generator=gen)
    return (x * by).to(dtype) if by != 1.0 or dtype == torch.float8_e4m3fn else x


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    state = {"case": case}
    if case["op"] == "append":
        tokens, heads, dim, page = case["tokens"], case["heads"], case["dim"], case["page"]
        dtype, store = DTYPES[case["dtype"]], DTYPES[case["store"]]
        pages = -(-tokens // page) + 4
        slots = torch.randperm(pages * page, generator=gen, device=DEVICE)[:tokens].to(torch.int32)
        slots[tokens - tokens // 16:] = -1  # the batch's padding
        state |= {"slots": slots}
        if case["kind"] == "kv":
            qkv = _normal(gen, (tokens, 3 * heads, dim), dtype, 1.5)  # keys and values are parts of one projection
            state |= {"k": qkv[:, heads:2 * heads], "v": qkv[:, 2 * heads:],
                      "k_cache": _normal(gen, (pages, page, heads, dim), store),
                      "v_cache": _normal(gen, (pages, page, heads, dim), store)}
            if store == torch.float8_e4m3fn:
                state |= {"k_scale": torch.rand(heads, generator=gen, device=DEVICE) * 0.05 + 0.01,
                          "v_scale": torch.rand(heads, generator=gen, device=DEVICE) * 0.05 + 0.01}
        else:
            state |= {"latent": _normal(gen, (tokens, dim), dtype), "rope": _normal(gen, (tokens, ROPE), dtype, 2.0),
                      "cache": _normal(gen, (pages, page, dim + ROPE), store)}
            if store == torch.float8_e4m3fn:
                state |= {"scale": torch.rand(1, generator=gen, device=DEVICE) * 0.05 + 0.01}
        return state
    ctx, new = _lengths(case)
    table, pages = _pages(case, ctx, gen)
    state |= {"table": table}
    if case["op"] == "layout":
        held = _i32([-(-(c - n) // case["page"]) for c, n in zip(ctx, new)])
        taken = sum(-(-c // case["page"]) - -(-(c - n) // case["page"]) for c, n in zip(ctx, new))
        width = table.shape[1]
        # Only the pages of earlier tokens are in the table yet; the free list holds others.
        table = torch.where(torch.arange(width, device=DEVICE) < held[:, None], table, -1).to(torch.int32)
        free = torch.randperm(taken + 7, generator=gen, device=DEVICE).to(torch.int32) + pages
        state |= {"table": table, "free": free[:taken // 2] if case["short"] else free, "lengths": _i32(ctx),
                  "new": _i32(new), "capacity": -(-sum(new) // 64) * 64}
        return state
    dtype, store = DTYPES[case["dtype"]], DTYPES[case["store"]]
    heads, dim, page = case["heads"], case["dim"], case["page"]
    e4m3 = store == torch.float8_e4m3fn
    if case["op"] == "prefill":
        starts = np.cumsum([0] + new)
        state |= {"lengths": _i32(ctx), "starts": _i32(starts), "context": sum(ctx), "most_new": max(new),
                  "most_context": max(ctx),
                  "q": _normal(gen, (int(starts[-1]), heads, NOPE + ROPE), dtype),
                  "w_k": _normal(gen, (heads, NOPE, dim), dtype, 1 / math.sqrt(dim)),
                  "w_v": _normal(gen, (heads, VALUE, dim), dtype, 1 / math.sqrt(dim)),
                  "cache": _normal(gen, (pages, page, dim + ROPE), store, 25.0 if e4m3 else 1.0),
                  "scale": torch.full((1,), 0.04, device=DEVICE) if e4m3 else None,
                  "softmax_scale": 1 / math.sqrt(NOPE + ROPE)}
        return state
    lengths = torch.as_tensor(_rows(case), device=DEVICE)
    rows = lengths.numel()
    state |= {"lengths": lengths, "most": int(lengths.max())}
    if case["top"]:
        # Distinct positions of each row's context, ascending, -1 past the last: what the top-K returns.
        width = max(case["max_len"], case["top"])
        n = lengths.reshape(-1, 1)
        x = torch.rand((rows, width), generator=gen, device=DEVICE)
        x.masked_fill_(torch.arange(width, device=DEVICE) >= n, -1.0)
        v, at = x.topk(case["top"], dim=1)
        at = torch.where(v >= 0, at, width).sort(dim=1).values
        state |= {"chosen": torch.where(at < n, at, -1).to(torch.int32).contiguous()}
    if case["op"] == "attention":
        kv = case["kv_heads"]
        state |= {"q": _normal(gen, (rows, heads, dim), dtype),
                  "k_cache": _normal(gen, (pages, page, kv, dim), store, 25.0 if e4m3 else 1.0),
                  "v_cache": _normal(gen, (pages, page, kv, dim), store, 25.0 if e4m3 else 1.0),
                  "k_scale": torch.rand(kv, generator=gen, device=DEVICE) * 0.02 + 0.03 if e4m3 else None,
                  "v_scale": torch.rand(kv, generator=gen, device=DEVICE) * 0.02 + 0.03 if e4m3 else None,
                  "softmax_scale": 1 / math.sqrt(dim)}
    else:
        state |= {"q": _normal(gen, (rows, heads, dim + ROPE), dtype),
                  "cache": _normal(gen, (pages, page, dim + ROPE), store, 25.0 if e4m3 else 1.0),
                  "scale": torch.full((1,), 0.04, device=DEVICE) if e4m3 else None,
                  "softmax_scale": 1 / math.sqrt(NOPE + ROPE)}
    return state


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    if own:
        return _own(state)
    return {"layout": _layout, "append": _append, "attention": _attention, "latent": _latent,
            "prefill": _prefill}[state["case"]["op"]](state)


def _own(state):
    import row_radix_top_amd as rrt

    op = state["case"]["op"]
    if op == "layout":
        out = rrt.paged_layout(state["lengths"], state["new"], state["free"], state["table"],
                               page_size=state["case"]["page"], capacity=state["capacity"])
        return {"table": state["table"], "slots": out.slots, "row_lengths": out.row_lengths, "row_seqs": out.row_seqs,
                "starts": out.starts, "pages": out.pages}
    if op == "append":
        if "latent" in state:
            rrt.latent_append(state["slots"], state["latent"], state["rope"], state["cache"], scale=state.get("scale"))
            return {"cache": state["cache"]}
        rrt.paged_append(state["slots"], state["k"], state["v"], state["k_cache"], state["v_cache"],
                         k_scale=state.get("k_scale"), v_scale=state.get("v_scale"))
        return {"k_cache": state["k_cache"], "v_cache": state["v_cache"]}
    if op == "attention":
        out, lse = rrt.paged_attention(state["q"], state["k_cache"], state["v_cache"], state["table"],
                                       state["lengths"], chosen=state.get("chosen"),
                                       softmax_scale=state["softmax_scale"], k_scale=state["k_scale"],
                                       v_scale=state["v_scale"])
    elif op == "latent":
        out, lse = rrt.latent_attention(state["q"], state["cache"], state["table"], state["lengths"],
                                        chosen=state.get("chosen"), softmax_scale=state["softmax_scale"],
                                        scale=state["scale"])
    else:
        out, lse = rrt.latent_prefill(state["q"], state["cache"], state["table"], state["starts"], state["lengths"],
                                      state["w_k"], state["w_v"], context_tokens=state["context"],
                                      softmax_scale=state["softmax_scale"], scale=state["scale"])
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _layout(s):
    page, capacity, table, free = s["case"]["page"], s["capacity"], s["table"], s["free"]
    length, new = s["lengths"].long(), s["new"].long()
    held, need = (length - new + page - 1) // page, (length + page - 1) // page
    first = (need - held).cumsum(0) - (need - held)
    j = torch.arange(table.shape[1], device=table.device)
    i = first[:, None] + j - held[:, None]
    fresh = torch.where(i < free.numel(), free[i.clamp(0, max(free.numel() - 1, 0))], -1) if free.numel() else torch.full_like(table, -1)
    table.copy_(torch.where((j >= held[:, None]) & (j < need[:, None]), fresh, table))
    starts = torch.cat([new.new_zeros(1), new.cumsum(0)])
    t = torch.arange(capacity, device=table.device)
    seq = (torch.searchsorted(starts, t, right=True) - 1).clamp(max=length.numel() - 1)
    inside = t < starts[-1]
    pos = length[seq] - new[seq] + t - starts[seq]
    pos = torch.where(inside, pos, 0)
    at = table[seq, pos // page].long()
    return {"table": table, "slots": torch.where(inside & (at >= 0), at * page + pos % page, -1).to(torch.int32),
            "row_lengths": torch.where(inside, pos + 1, 0).to(torch.int32),
            "row_seqs": torch.where(inside, seq, -1).to(torch.int32), "starts": starts.to(torch.int32),
            "pages": (need - held).sum().reshape(1).to(torch.int32)}


def _stored(x, scale, store):
    """The values that the cache holds for x: rounded once, the largest magnitudes of 8 bits kept."""
    if store == torch.float8_e4m3fn:
        x = (x / scale).clamp(-E4M3_MAX, E4M3_MAX)
    return x.to(store)


def _append(s):
    slots = s["slots"].long()
    at = slots[slots >= 0]
    if "latent" in s:
        x = torch.cat([s["latent"], s["rope"]], dim=-1).float()[slots >= 0]
        s["cache"].view(-1, x.shape[1])[at] = _stored(x, s.get("scale"), s["cache"].dtype)
        return {"cache": s["cache"]}
    k, v = s["k"].float()[slots >= 0], s["v"].float()[slots >= 0]
    by = (s["k_scale"][:, None], s["v_scale"][:, None]) if "k_scale" in s else (None, None)
    s["k_cache"].view(-1, *k.shape[1:])[at] = _stored(k, by[0], s["k_cache"].dtype)
    s["v_cache"].view(-1, *v.shape[1:])[at] = _stored(v, by[1], s["v_cache"].dtype)
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _positions(s):
    """[rows, width] positions of the cache that each row reads, whether it does, and their slots."""
    page, table = s["case"]["page"], s["table"].long()
    lengths = s["lengths"].reshape(-1, 1).long()
    if "chosen" in s:
        pos = s["chosen"].long()
        seen = (pos >= 0) & (pos < lengths)
    else:
        pos = torch.arange(max(s["most"], 1), device=table.device).expand(lengths.shape[0], -1)
        seen = pos < lengths
    pos = torch.where(seen, pos, 0)
    at = torch.repeat_interleave(table, s["case"]["next_n"], dim=0).gather(1, pos // page)
    seen = seen & (at >= 0)
    return seen, torch.where(seen, at * page + pos % page, 0)


def _softmax(x):
    """Probabilities and log-sum-exp over the last axis; zeros and -inf where nothing is left."""
    top = x.amax(-1, keepdim=True)
    p = (x - torch.where(top == -math.inf, 0.0, top)).exp()
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, 1.0, total), (top + total.log()).squeeze(-1)


def _attention(s):
    kv, dim = s["case"]["kv_heads"], s["case"]["dim"]
    seen, slots = _positions(s)
    rows, width = slots.shape
    k = s["k_cache"].view(-1, kv, dim)[slots].float()
    v = s["v_cache"].view(-1, kv, dim)[slots].float()
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"][:, None], v * s["v_scale"][:, None]
    v = torch.where(seen[..., None, None], v, 0.0)
    q = s["q"].float().view(rows, kv, -1, dim)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["softmax_scale"]
    p, lse = _softmax(torch.where(seen[:, None, None], scores, -math.inf))
    out = torch.matmul(p, v.transpose(1, 2))
    return {"out": out.reshape(rows, -1, dim).to(s["q"].dtype), "lse": lse.reshape(rows, -1)}


def _latent(s):
    dim = s["case"]["dim"]
    seen, slots = _positions(s)
    c = s["cache"].view(-1, dim + ROPE)[slots].float()
    if s["scale"] is not None:
        c = c * s["scale"]
    c = torch.where(seen[..., None], c, 0.0)
    scores = torch.matmul(s["q"].float(), c.transpose(1, 2)) * s["softmax_scale"]
    p, lse = _softmax(torch.where(seen[:, None], scores, -math.inf))
    return {"out": torch.matmul(p, c[..., :dim].contiguous()).to(s["q"].dtype), "lse": lse}


def _prefill(s):
    page, dim, heads = s["case"]["page"], s["case"]["dim"], s["case"]["heads"]
    lengths, starts = s["lengths"].long(), s["starts"].long()
    seqs, dev = lengths.numel(), lengths.device
    pos = torch.arange(s["most_context"], device=dev)
    at = s["table"].long()[:, pos // page]
    inside = (pos < lengths[:, None]) & (at >= 0)
    c = s["cache"].view(-1, dim + ROPE)[torch.where(inside, at * page + pos % page, 0)].float()
    if s["scale"] is not None:
        c = c * s["scale"]
    c = torch.where(inside[..., None], c, 0.0)
    k = torch.matmul(c[..., :dim].reshape(-1, dim), s["w_k"].float().view(-1, dim).t()).view(seqs, -1, heads, NOPE)
    v = torch.matmul(c[..., :dim].reshape(-1, dim), s["w_v"].float().view(-1, dim).t()).view(seqs, -1, heads, VALUE)
    k = torch.cat([k, c[:, :, None, dim:].expand(-1, -1, heads, -1)], dim=-1)
    new = starts[1:] - starts[:-1]
    j = torch.arange(s["most_new"], device=dev)
    q = s["q"].float()[(starts[:-1, None] + j).clamp(max=max(s["q"].shape[0] - 1, 0))]
    sees = inside[:, None] & (pos <= (lengths - new)[:, None, None] + j[:, None])
    scores = torch.matmul(q.transpose(1, 2), k.permute(0, 2, 3, 1)) * s["softmax_scale"]
    p, lse = _softmax(scores.masked_fill_(~sees[:, None], -math.inf))
    out = torch.matmul(p, v.transpose(1, 2)).transpose(1, 2)
    t = torch.arange(s["q"].shape[0], device=dev)
    seq = torch.searchsorted(starts, t, right=True) - 1
    return {"out": out[seq, t - starts[seq]].to(s["q"].dtype), "lse": lse.transpose(1, 2)[seq, t - starts[seq]]}


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    size = {"bf16": 2, "fp16": 2, "e4m3": 1}
    if case["op"] == "append":
        wide = 2 * case["heads"] * case["dim"] if case["kind"] == "kv" else case["dim"] + ROPE
        kept = case["tokens"] - case["tokens"] // 16
        return {"bytes": kept * wide * (size[case["dtype"]] + size[case["store"]]) + 4 * case["tokens"], "flops": 0}
    ctx, new = _lengths(case)
    if case["op"] == "layout":
        page = case["page"]
        fresh = sum(-(-c // page) - -(-(c - n) // page) for c, n in zip(ctx, new))
        capacity = -(-sum(new) // 64) * 64
        return {"bytes": 4 * (3 * len(ctx) + 1 + 2 * fresh + len(ctx) + 3 * capacity + 1), "flops": 0}
    item, held, heads, dim = size[case["dtype"]], size[case["store"]], case["heads"], case["dim"]
    if case["op"] == "prefill":
        pairs = sum(n * (c - n) + n * (n + 1) // 2 for c, n in zip(ctx, new))
        total, rows = sum(ctx), sum(new)
        return {"bytes": total * (dim + ROPE) * held + heads * (NOPE + VALUE) * dim * item
                + rows * heads * ((NOPE + ROPE + VALUE) * item + 4),
                "flops": 2 * total * dim * heads * (NOPE + VALUE) + 2 * pairs * heads * (NOPE + ROPE + VALUE)}
    seen = _rows(case)
    if case["top"]:
        seen = np.minimum(seen, case["top"])
    pairs = int(seen.sum())
    # Rows of one sequence share its cache: each position is read once, and no more than the sequence has.
    read = int(np.minimum(seen.sum(1), np.asarray(ctx)).sum()) if case["top"] else int(seen.max(1).sum())
    rows = seen.size
    k_dim = dim if case["op"] == "attention" else dim + ROPE
    token = 2 * case["kv_heads"] * dim if case["op"] == "attention" else dim + ROPE
    return {"bytes": read * token * held + rows * heads * ((k_dim + dim) * item + 4) + 4 * rows
            + 4 * read // case["page"] + (4 * rows * case["top"]), "flops": 2 * pairs * heads * (k_dim + dim)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _row_attention(q, k, v, scale):
    """One row's heads q [h, d] over its keys [n, d] and values [n, e], in 64 bits."""
    if k.shape[0] == 0:
        return q.new_zeros(q.shape[0], v.shape[1]), q.new_full((q.shape[0],), -math.inf)
    x = (q @ k.T) * scale
    lse = torch.logsumexp(x, dim=1)
    return torch.exp(x - lse[:, None]) @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "layout":
        return _exact_layout(s)
    if case["op"] == "append":
        return _exact_append(s)
    page, table, lengths = case["page"], s["table"].cpu().numpy(), s["lengths"].cpu().numpy()

    def slots_of(seq, positions):
        p = np.asarray(positions, dtype=np.int64)
        return torch.as_tensor(table[seq][p // page].astype(np.int64) * page + p % page, device=DEVICE)

    outs, lses = [], []
    if case["op"] == "prefill":
        by = 1.0 if s["scale"] is None else s["scale"].double()
        starts = s["starts"].cpu().numpy()
        for b, n in enumerate(lengths):
            c = s["cache"].reshape(-1, case["dim"] + ROPE)[slots_of(b, np.arange(n))].double() * by
            q = s["q"][starts[b]:starts[b + 1]].double()
            future = torch.arange(n, device=DEVICE) > torch.arange(n - q.shape[0], n, device=DEVICE)[:, None]
            out, lse = q.new_empty(q.shape[0], case["heads"], VALUE), q.new_empty(q.shape[0], case["heads"])
            for h in range(case["heads"]):
                k = torch.cat([c[:, :case["dim"]] @ s["w_k"][h].double().T, c[:, case["dim"]:]], dim=1)
                x = ((q[:, h] @ k.T) * s["softmax_scale"]).masked_fill_(future, -math.inf)
                lse[:, h] = torch.logsumexp(x, dim=1)
                out[:, h] = torch.exp(x - lse[:, h, None]) @ (c[:, :case["dim"]] @ s["w_v"][h].double().T)
            outs.append(out)
            lses.append(lse)
        return {"out": torch.cat(outs), "lse": torch.cat(lses)}
    flat = lengths.reshape(-1)
    chosen = s["chosen"].cpu().numpy() if "chosen" in s else None
    for r, n in enumerate(flat):
        p = np.arange(n) if chosen is None else chosen[r][chosen[r] >= 0]
        at = slots_of(r // case["next_n"], p)
        q = s["q"][r].double()
        if case["op"] == "latent":
            c = s["cache"].reshape(-1, case["dim"] + ROPE)[at].double() * (1.0 if s["scale"] is None else s["scale"].double())
            out, lse = _row_attention(q, c, c[:, :case["dim"]], s["softmax_scale"])
        else:
            group = case["heads"] // case["kv_heads"]
            k = s["k_cache"].reshape(-1, case["kv_heads"], case["dim"])[at].double()
            v = s["v_cache"].reshape(-1, case["kv_heads"], case["dim"])[at].double()
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"].double()[:, None], v * s["v_scale"].double()[:, None]
            parts = [_row_attention(q[h * group:(h + 1) * group], k[:, h], v[:, h], s["softmax_scale"])
                     for h in range(case["kv_heads"])]
            out, lse = torch.cat([o for o, _ in parts]), torch.cat([x for _, x in parts])
        outs.append(out)
        lses.append(lse)
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}


def _exact_layout(s):
    page, table, free = s["case"]["page"], s["table"].cpu().numpy().copy(), s["free"].cpu().numpy()
    slots, row_lengths, row_seqs, starts, taken = [], [], [], [0], 0
    for b, (n, new) in enumerate(zip(s["lengths"].tolist(), s["new"].tolist())):
        for j in range(-(-(n - new) // page), -(-n // page)):
            table[b, j] = free[taken] if taken < len(free) else -1
            taken += 1
        p = np.arange(n - new, n)
        at = table[b, p // page]
        slots.append(np.where(at >= 0, at * page + p % page, -1))
        row_lengths.append(p + 1)
        row_seqs.append(np.full(new, b))
        starts.append(starts[-1] + new)
    pad = s["capacity"] - starts[-1]
    ends = {"slots": (slots, -1), "row_lengths": (row_lengths, 0), "row_seqs": (row_seqs, -1)}
    full = {k: np.concatenate(v + [np.full(pad, f)]).astype(np.int32) for k, (v, f) in ends.items()}
    return {"table": table} | full | {"starts": np.asarray(starts, np.int32), "pages": np.asarray([taken], np.int32)}


def _exact_append(s):
    slots = s["slots"].long()
    rows = torch.nonzero(slots >= 0).squeeze(1)

    def into(cache, values, scale):
        flat = cache.double().reshape(-1, values[0].numel())
        x = values.double()
        if scale is not None:
            x = torch.minimum(torch.maximum(x / scale.double(), x.new_tensor(-E4M3_MAX)), x.new_tensor(E4M3_MAX))
        flat[slots[rows]] = x.reshape(x.shape[0], -1)[rows]
        return flat.reshape(cache.shape)

    if "latent" in s:
        return {"cache": into(s["cache"], torch.cat([s["latent"], s["rope"]], dim=1), s.get("scale"))}
    scales = (s["k_scale"][:, None], s["v_scale"][:, None]) if "k_scale" in s else (None, None)
    return {"k_cache": into(s["k_cache"], s["k"], scales[0]), "v_cache": into(s["v_cache"], s["v"], scales[1])}
