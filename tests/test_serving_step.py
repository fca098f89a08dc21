"""The operators together, as a sparse-attention server runs them: pages and
slots for a step's new tokens, their write into the caches, the prompt chunks'
causal attention, then single tokens: top-K of the indexer's scores and
attention over the chosen positions, eagerly and replayed from one graph."""

from __future__ import annotations

import numpy as np
import pytest

import row_radix_top_amd as rrt
from oracle import topk_ragged_oracle
from tests import paged_ref
from tests.gpu_util import note, require_gpu
from tests.test_latent_prefill import HEAD, ROPE
from tests.test_latent_prefill import Case as PrefillCase

pytestmark = pytest.mark.gpu

KV, HEADS, DIM, LATENT, PAGE, WIDTH, K, SEQS = 2, 10, 128, 256, 16, 12, 32, 5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


class Server:
    """Caches on the GPU and, in 64 bits, every sequence's tokens as stored."""

    def __init__(self, store):
        import torch
        self.rng = np.random.default_rng(7)
        torch.manual_seed(7)
        self.dt = torch.bfloat16
        self.st = self.dt if store == "same" else getattr(torch, store)
        self.pages = SEQS * WIDTH + 4

        def cache(*shape):  # NaN wherever no token is written
            x = torch.full((self.pages, PAGE) + shape, float("nan"), device="cuda").to(self.st)
            assert bool(x.float().isnan().all())
            return x

        self.kc, self.vc, self.c = cache(KV, DIM), cache(KV, DIM), cache(LATENT + ROPE)
        f8 = self.st != self.dt
        self.ks = torch.tensor([0.5, 0.75], device="cuda") if f8 else None
        self.vs = torch.tensor([1.25, 0.5], device="cuda") if f8 else None
        self.by = torch.tensor([0.5], device="cuda") if f8 else None
        self.table = torch.full((SEQS, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.free = self.rng.permutation(self.pages).astype(np.int32)
        self.lengths = np.zeros(SEQS, dtype=np.int64)
        self.past = [dict(k=[], v=[], c=[]) for _ in range(SEQS)]

    def stored(self, x, scale):
        """What the cache holds of x, read back, in 64 bits."""
        if scale is None:
            return x.double().cpu().numpy()
        y = (x.float() / scale).clamp(-448, 448).to(self.st)
        return y.double().cpu().numpy() * scale.double().cpu().numpy()

    def inputs(self, tokens):
        import torch
        r = lambda *s: torch.randn(*s, device="cuda").to(self.dt)  # noqa: E731
        return r(tokens, KV, DIM), r(tokens, KV, DIM), r(tokens, LATENT), r(tokens, ROPE)

    def write(self, lengths, new, free, capacity, x):
        """The step's layout and appends."""
        out = rrt.paged_layout(lengths, new, free, self.table, page_size=PAGE, capacity=capacity)
        k, v, latent, rope = x
        rrt.paged_append(out.slots, k, v, self.kc, self.vc, k_scale=self.ks, v_scale=self.vs)
        rrt.latent_append(out.slots, latent, rope, self.c, scale=self.by)
        return out

    def advance(self, new, x):
        """The same on the host; pages taken leave the free list."""
        import torch
        k, v, latent, rope = x
        ks, vs = (None, None) if self.ks is None else (self.ks[:, None], self.vs[:, None])
        k, v, c = self.stored(k, ks), self.stored(v, vs), self.stored(torch.cat([latent, rope], 1), self.by)
        at = 0
        for s, n in enumerate(new):
            for name, y in (("k", k), ("v", v), ("c", c)):
                self.past[s][name].extend(y[at:at + n])
            at += n
        held = -(-self.lengths // PAGE)
        self.lengths = self.lengths + new
        self.free = self.free[int((-(-self.lengths // PAGE) - held).sum()):]

    def expected(self, seqs, chosen, q, lq, scale, lscale):
        """Attention of each row over its chosen positions: of both caches."""
        u = paged_ref.half_step(self.dt)
        res = []
        for latent in (False, True):
            x = (lq if latent else q).double().cpu().numpy()
            width = LATENT if latent else DIM
            out, tol = (np.zeros((len(seqs), HEADS, width)) for _ in range(2))
            lse, tlog = (np.full((len(seqs), HEADS), f) for f in (-np.inf, 0.0))
            for r, s in enumerate(seqs):
                at = chosen[r][chosen[r] >= 0]
                if s < 0 or len(at) == 0:
                    continue
                for h in range(HEADS):
                    if latent:
                        keys = np.array(self.past[s]["c"])[at]
                        got = paged_ref.attend(x[r, h], keys, keys[:, :LATENT], lscale, u, False)
                    else:
                        g = h // (HEADS // KV)
                        got = paged_ref.attend(x[r, h], np.array(self.past[s]["k"])[at, g],
                                               np.array(self.past[s]["v"])[at, g], scale, u, False)
                    out[r, h], lse[r, h], tol[r, h], tlog[r, h] = got
            res.append((out, lse, tol, tlog))
        return res


@pytest.mark.parametrize("store", ["same", "float8_e4m3fn"])
def test_prompts_then_single_tokens(store):
    import torch
    s = Server(store)
    dev = lambda x: torch.as_tensor(np.asarray(x), device="cuda").to(torch.int32)  # noqa: E731

    # Prompts, in two chunks; sequence 2 starts with the second.
    for new in ([100, 37, 0, 64, 1], [20, 3, 70, 1, 0]):
        new = np.array(new)
        tokens, after = int(new.sum()), s.lengths + new
        note(f"serving step {store} prompt new={new.tolist()}")
        x = s.inputs(tokens)
        layout = s.write(dev(after), dev(new), dev(s.free), tokens, x)
        s.advance(new, x)
        p = PrefillCase.__new__(PrefillCase)
        p.lengths, p.new, p.starts, p.tokens = after, new, layout.starts.cpu().numpy(), tokens
        p.table, p.page_size, p.width, p.pages = s.table.cpu().numpy(), PAGE, WIDTH, s.pages
        p.heads, p.dim, p.dt, p.st, p.c, p.by, p.scale = 2, LATENT, s.dt, s.st, s.c, s.by, (HEAD + ROPE) ** -0.5
        p.q = torch.randn(tokens, p.heads, HEAD + ROPE, device="cuda").to(s.dt)
        p.wk, p.wv = ((torch.randn(p.heads, HEAD, LATENT, device="cuda") / 16).to(s.dt) for _ in range(2))
        for q in range(SEQS):  # the cache holds what was appended
            have = s.c.double().cpu().numpy().reshape(-1, LATENT + ROPE)[p.slots(q)]
            np.testing.assert_array_equal(have * (1.0 if s.by is None else float(s.by)),
                                          np.array(s.past[q]["c"]).reshape(-1, LATENT + ROPE))
        out, lse = rrt.latent_prefill(p.q, s.c, s.table, layout.starts, dev(after), p.wk, p.wv,
                                      context_tokens=int(after.sum()), softmax_scale=p.scale, scale=s.by)
        exp, elog, tol, tlog = p.expected()
        paged_ref.check(out.double().cpu().numpy(), exp, tol, "prompt out")
        paged_ref.check(lse.double().cpu().numpy(), elog, tlog, "prompt lse")

    # Single tokens: one graph over fixed buffers, every step against the host.
    rows, span = SEQS, WIDTH * PAGE
    lengths, new, free = dev(s.lengths), dev([0] * SEQS), dev(np.full(SEQS, -1))
    x = s.inputs(rows)
    q = torch.randn(rows, HEADS, DIM, device="cuda").to(s.dt)
    lq = torch.randn(rows, HEADS, LATENT + ROPE, device="cuda").to(s.dt)
    scores = torch.randn(rows, span, device="cuda")
    scale, lscale = DIM ** -0.5, (HEAD + ROPE) ** -0.5

    def step():
        layout = s.write(lengths, new, free, rows, x)
        chosen = rrt.topk_ragged(scores, layout.row_lengths, K)
        tables = s.table.index_select(0, layout.row_seqs.clamp(min=0))
        kv = rrt.paged_attention(q, s.kc, s.vc, tables, layout.row_lengths, chosen=chosen, k_scale=s.ks, v_scale=s.vs)
        latent = rrt.latent_attention(lq, s.c, tables, layout.row_lengths, chosen=chosen, softmax_scale=lscale,
                                      scale=s.by)
        return layout, chosen, kv, latent

    step()  # no new tokens: every row is padding
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layout, chosen, kv, latent = step()
    for i, fresh in enumerate(([1, 1, 1, 1, 1], [0, 1, 0, 1, 1], [1, 0, 0, 0, 0], [0, 0, 0, 0, 0], [1, 1, 1, 1, 1])):
        fresh = np.array(fresh)
        note(f"serving step {store} token {i} new={fresh.tolist()}")
        y = s.inputs(rows)
        for a, b in zip(x, y):
            a.copy_(b)
        q.normal_(), lq.normal_(), scores.normal_()
        lengths.copy_(dev(s.lengths + fresh)), new.copy_(dev(fresh)), free.copy_(dev(s.free[:SEQS]))
        kept = s.table.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (layout.slots, layout.row_lengths, layout.row_seqs, chosen, *kv, *latent)]
        n = int(fresh.sum())
        _, slots, row_lengths, row_seqs, starts, taken = paged_ref.layout(s.lengths + fresh, fresh, s.free,
                                                                          kept.cpu().numpy(), PAGE, rows)
        for have, exp in zip(got, (slots, row_lengths, row_seqs)):
            np.testing.assert_array_equal(have.cpu().numpy(), exp)
        assert layout.starts.tolist() == list(starts) and int(layout.pages) == taken
        s.advance(fresh, tuple(t[:n] for t in y))
        picked = topk_ragged_oracle(scores.cpu().numpy(), row_lengths.astype(np.int32), K)
        np.testing.assert_array_equal(got[3].cpu().numpy(), picked)
        for (out, lse, tol, tlog), a, b, what in zip(s.expected(row_seqs, picked, q, lq, scale, lscale), got[4::2],
                                                     got[5::2], ("kv", "latent")):
            paged_ref.check(a.double().cpu().numpy(), out, tol, f"{what} out")
            paged_ref.check(b.double().cpu().numpy(), lse, tlog, f"{what} lse")
        # Eagerly, with the step's pages given back: the same bits.
        s.table.copy_(kept)
        again = step()
        for a, b in zip(got, (again[0].slots, again[0].row_lengths, again[0].row_seqs, again[1], *again[2], *again[3])):
            assert torch.equal(a, b)
