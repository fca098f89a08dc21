"""The operators on shared pages, shared prefixes and chosen blocks as a server
runs them: prompts, forks, steps of single tokens over a cache that grows, rows
that end, pages that move; against each row's own history in 64 bits.  The same
as a captured graph, replayed."""

from __future__ import annotations

import numpy as np
import pytest

import row_radix_top_amd as rrt
from tests import paged_ref
from tests.gpu_util import note, require_gpu

pytestmark = pytest.mark.gpu

PAGE, KV, HEADS, DIM, PAGES, WIDTH = 16, 2, 8, 128, 96, 12


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def dev(x):
    import torch
    return torch.as_tensor(np.asarray(x), device="cuda").to(torch.int32)


class Server:
    """A cache, its pages' bounds, and the rows' histories beside them."""

    def __init__(self, seed=0):
        import torch
        torch.manual_seed(seed)
        new = lambda *shape, **kw: torch.zeros(shape, device="cuda", **kw)  # noqa: E731
        self.k, self.v = (new(PAGES, PAGE, KV, DIM, dtype=torch.bfloat16) for _ in range(2))
        self.bounds, self.scales = new(PAGES, KV, 2, DIM, dtype=torch.int8), new(PAGES, KV)
        self.past = []  # of each row: [tokens, 2, kv heads, dim]

    def free(self):
        return rrt.paged_free(self.table, self.lengths, page_size=PAGE, num_pages=PAGES).free

    def append(self, counts):
        """New tokens of each row, into the cache, the bounds and the histories."""
        import torch
        total = sum(counts)
        x = torch.randn(2, total, KV, DIM, device="cuda").bfloat16()
        free = self.free()
        self.lengths = self.lengths + dev(counts)
        layout = rrt.paged_layout(self.lengths, dev(counts), free, self.table, page_size=PAGE, capacity=total)
        rrt.paged_append(layout.slots, x[0], x[1], self.k, self.v)
        rrt.paged_bounds(self.k, self.table, layout.starts, self.lengths, self.bounds, self.scales, num_tokens=total)
        at = 0
        for r, n in enumerate(counts):
            self.past[r] = np.concatenate([self.past[r], x[:, at:at + n].double().cpu().numpy().swapaxes(0, 1)])
            at += n

    def attend(self, q, starts, shared, num_blocks=4):
        near = rrt.paged_prefix_attention(q, self.k, self.v, self.table, self.lengths, dev(starts), dev(shared))
        blocks = rrt.paged_block_select(q, self.bounds, self.scales, self.table, self.lengths, page_size=PAGE,
                                        num_blocks=num_blocks)
        return near, blocks, rrt.paged_block_attention(q, self.k, self.v, self.table, self.lengths, blocks)

    def check(self, what, starts, shared):
        import torch
        q = torch.randn(len(self.past), HEADS, DIM, device="cuda").bfloat16()
        (out, lse), blocks, (some, some_lse) = self.attend(q, starts, shared)
        note(f"{what}: {[len(x) for x in self.past]}")
        u, group, host = paged_ref.half_step(torch.bfloat16), HEADS // KV, q.double().cpu().numpy()
        for r, past in enumerate(self.past):
            have = -(-len(past) // PAGE)
            for h in range(HEADS):
                k, v = past[:, 0, h // group], past[:, 1, h // group]
                chosen = blocks[r, h // group].tolist()
                real = [b for b in chosen if b >= 0]
                assert real == sorted(set(real)) and chosen == real + [-1] * (4 - len(real))
                assert len(real) == min(4, have) and (have == 0 or {0, have - 1} <= set(real))
                tokens = [t for b in real for t in range(b * PAGE, min(len(past), (b + 1) * PAGE))]
                for o, l, at in ((out, lse, slice(None)), (some, some_lse, tokens)):
                    exp = paged_ref.attend(host[r, h], k[at], v[at], DIM ** -0.5, u, False)
                    paged_ref.check(o[r, h].double().cpu().numpy(), exp[0], exp[2], f"{what} row {r} head {h} out")
                    paged_ref.check(l[r, h].double().cpu().numpy(), np.asarray(exp[1]), np.asarray(exp[3]),
                                    f"{what} row {r} head {h} lse")

    def fork(self, parents, keep):
        fork = rrt.paged_fork(self.table, self.lengths, dev(parents), self.free(), page_size=PAGE, keep=dev(keep))
        rrt.paged_copy(fork.src, fork.dst, [self.k, self.v], tokens=fork.tokens)
        self.table, self.lengths = fork.table, fork.lengths
        self.past = [self.past[p][:n] for p, n in zip(parents, keep)]

    def prompts(self, lengths):
        import torch
        self.table = torch.full((len(lengths), WIDTH), -1, dtype=torch.int32, device="cuda")
        self.lengths = dev([0] * len(lengths))
        self.past = [np.zeros((0, 2, KV, DIM))] * len(lengths)
        self.append(lengths)


def test_samples_that_fork_grow_end_and_move():
    import torch
    s = Server()
    s.prompts([70, 45])
    s.check("prompts", [0, 2], [0])
    s.fork([0, 0, 0, 0, 1, 1], [70, 70, 70, 64, 45, 30])
    s.check("forked", [0, 4, 6], [64, 16])
    for step in range(18):  # past the ends of pages, and of the first block that is chosen away
        s.append([1] * 6)
        if step in (0, 1, 17):
            s.check(f"step {step}", [0, 4, 6], [64, 16])
    s.append([3, 0, 33, 1, 0, 20])
    s.check("several tokens", [0, 4, 6], [64, 16])
    # Beams: rows go on from one another, shortened or not.
    s.fork([2, 2, 0, 5, 5, 4], [121, 90, 91, 50, 68, 63])
    s.append([1] * 6)
    s.check("beams", [0, 2, 3, 6], [80, 64, 16])
    # Two rows end, and what is left moves together.
    s.lengths = s.lengths * dev([1, 0, 1, 1, 0, 1])
    s.past = [x if r not in (1, 4) else x[:0] for r, x in enumerate(s.past)]
    s.check("ended", [0, 1, 3, 6], [64, 64, 16])
    q = torch.randn(6, HEADS, DIM, device="cuda").bfloat16()
    before = s.attend(q, [0, 1, 3, 6], [64, 64, 16])
    c = rrt.paged_compact(s.table, s.lengths, page_size=PAGE, num_pages=PAGES)
    rrt.paged_copy(c.src, c.dst, [s.k, s.v, s.bounds, s.scales])
    live = int(c.live)
    assert int(c.moves) > 0 and live == sum(int(x) for x in rrt.paged_free(c.table, s.lengths, page_size=PAGE,
                                                                          num_pages=PAGES).refs[:live] > 0)
    for x in (s.k, s.v):  # nothing reads the pages behind
        x[live:] = float("nan")
    s.table = c.table
    after = s.attend(q, [0, 1, 3, 6], [64, 64, 16])
    assert torch.equal(before[1], after[1])
    for a, b in zip((*before[0], *before[2]), (*after[0], *after[2])):
        assert torch.equal(a, b)
    s.append([1, 0, 1, 1, 0, 1])
    s.check("moved", [0, 1, 3, 6], [64, 64, 16])


def test_a_step_as_a_graph():
    """Fork, copy, append, bounds, choice and both attentions, captured; replays over other data agree with eager calls."""
    import torch
    s = Server(1)
    s.prompts([100, 37, 64])
    table, lengths, k0, v0 = s.table.clone(), s.lengths.clone(), s.k.clone(), s.v.clone()
    b0, s0 = s.bounds.clone(), s.scales.clone()
    parents, keep, ones = dev([0, 0, 2, 1, 1]), dev([100, 90, 64, 37, 20]), dev([1] * 5)
    starts, shared = dev([0, 2, 3, 5]), dev([80, 64, 16])
    new, q = (torch.randn(2, 5, n, DIM, device="cuda").bfloat16() for n in (KV, HEADS))
    cache = [k0.clone(), v0.clone(), b0.clone(), s0.clone()]

    def step():
        k, v, bounds, scales = cache
        pool = rrt.paged_free(table, lengths, page_size=PAGE, num_pages=PAGES)
        fork = rrt.paged_fork(table, lengths, parents, pool.free, page_size=PAGE, keep=keep)
        rrt.paged_copy(fork.src, fork.dst, [k, v], tokens=fork.tokens)
        # What neither the parents nor their forks hold.
        both, all_lengths = torch.cat([table, fork.table]), torch.cat([lengths, fork.lengths])
        rest = rrt.paged_free(both, all_lengths, page_size=PAGE, num_pages=PAGES)
        total = fork.lengths + ones
        layout = rrt.paged_layout(total, ones, rest.free, fork.table, page_size=PAGE, capacity=5)
        rrt.paged_append(layout.slots, new[0], new[1], k, v)
        rrt.paged_bounds(k, fork.table, layout.starts, total, bounds, scales, num_tokens=5)
        near = rrt.paged_prefix_attention(q[0], k, v, fork.table, total, starts, shared)
        blocks = rrt.paged_block_select(q[1], bounds, scales, fork.table, total, page_size=PAGE, num_blocks=3)
        return [*near, blocks, *rrt.paged_block_attention(q[1], k, v, fork.table, total, blocks), *fork, *layout]

    def reset():
        for x, y in zip(cache, (k0, v0, b0, s0)):
            x.copy_(y)

    step()
    reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        keep.copy_(dev([100 - i, 90, 64 - 16 * (i % 2), 37, 20 + i]))
        shared.copy_(dev([80, 48, 16 * (i % 3 != 0)]))
        new.copy_(torch.randn(new.shape, device="cuda"))
        q.copy_(torch.randn(q.shape, device="cuda"))
        reset()
        graph.replay()
        torch.cuda.synchronize()
        got, held = [x.clone() for x in out], [x.clone() for x in cache]
        reset()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
        for a, b in zip(held, cache):
            assert torch.equal(a, b)
