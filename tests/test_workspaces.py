"""Workspaces of the three attentions: a size that holds for smaller batches
too, buffers of the caller's own that hold anything before, and refusals."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest

import row_radix_top_amd as rrt
from row_radix_top_amd import attention as pa
from row_radix_top_amd import binding
from tests.gpu_util import note, require_gpu
from tests.test_latent_attention import Case as LatentCase
from tests.test_latent_prefill import Case as PrefillCase
from tests.test_paged_attention import Case as PagedCase

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _size(entry, args):
    need = ctypes.c_size_t(0)
    rc = getattr(pa.load(), entry + "_workspace_size")(ctypes.byref(args), None, need)
    assert rc == 0, binding.last_error()
    return need.value


def _attention(entry, rows, **changes):
    """Shapes alone count; nothing is launched."""
    dim = 512 if entry == "latent_attention" else 128
    a = pa.AttentionArgs()
    for k, v in dict(dict(q=256, k=512, v=1024, block_table=256, lengths=256, out=256, lse=256, q_row_stride=8 * dim,
                          q_head_stride=dim, page_stride=64 * dim, token_stride=dim, head_stride=dim, table_stride=4,
                          num_rows=rows, next_n=1, num_heads=8, num_kv_heads=2, head_dim=dim, page_size=16, num_pages=4,
                          table_width=2048, softmax_scale=0.1), **changes).items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("entry", ["paged_attention", "latent_attention"])
@pytest.mark.parametrize("changes", [dict(), dict(num_heads=64, num_kv_heads=8), dict(num_heads=128, num_kv_heads=1),
                                     dict(next_n=2), dict(chosen=256, num_chosen=2048, chosen_stride=2048),
                                     dict(chosen=256, num_chosen=2048, chosen_stride=2048, num_heads=128, num_kv_heads=4),
                                     dict(table_width=16), dict(max_splits=3)],
                         ids=lambda c: " ".join(f"{k}={v}" for k, v in c.items()) or "plain")
def test_a_size_holds_for_fewer_rows_and_shorter_ones(entry, changes):
    n = changes.get("next_n", 1)
    most = 0
    for rows in [n * r for r in range(1, 700)] + [n * 5000, n * 200000]:
        need = _size(entry, _attention(entry, rows, **changes))
        assert need >= most, f"{rows} rows need {need} bytes, fewer rows {most}"
        most = need
    long = _attention(entry, 64 * n, **changes)
    for width in (1, 7, 64, 300, 2047):
        short = _attention(entry, 64 * n, **dict(changes, table_width=min(width, changes.get("table_width", width))))
        assert _size(entry, short) <= _size(entry, long)
    if "chosen" in changes:
        for k in (1, 300, 512, 1024, 2047):
            assert _size(entry, _attention(entry, 64 * n, **dict(changes, num_chosen=k))) <= _size(entry, long)


def _prefill(**changes):
    a = pa.PrefillArgs()
    for k, v in dict(dict(q=256, cache=512, w_k=256, w_v=256, block_table=256, starts=256, lengths=256, out=256, lse=256,
                          q_row_stride=8 * 192, q_head_stride=192, page_stride=16 * 576, token_stride=576,
                          table_stride=4, context_tokens=100000, num_tokens=8192, num_seqs=4, num_heads=8,
                          latent_dim=512, page_size=16, num_pages=4, table_width=8192, softmax_scale=0.1),
                     **changes).items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("heads", [1, 8, 32])
def test_a_prefill_size_holds_for_smaller_chunks(heads):
    for name, values in [("num_tokens", list(range(1, 400, 3)) + [128 * r for r in range(4, 200)]),
                         ("context_tokens", [1, 63, 64, 500, 511, 512, 1000, 4097, 100000]),
                         ("num_seqs", [1, 2, 5, 64, 1000, 8000]), ("table_width", [1, 31, 32, 33, 1000, 8192])]:
        most = 0
        for v in values:
            need = _size("latent_prefill", _prefill(**{"num_heads": heads, name: v}))
            assert need >= most, f"{name} {v} needs {need} bytes, a smaller one {most}"
            most = need


def test_a_long_context_reserves_second_parts_for_its_first_tokens_alone():
    """A head: keys and values of 512 bytes a token and a power of two, 256 more of the first 1024 tokens, a flag a
    tile, the one row's partial outputs of 128 values and two statistics in at most 16 parts.  All heads: rope parts
    and their powers, a mask and a flag a tile."""
    tokens, tiles, heads = 131072, 131072 // 64 + 1, 128
    need = _size("latent_prefill", _prefill(context_tokens=tokens, num_heads=heads, num_seqs=1, num_tokens=1))
    assert need <= heads * (tiles * 64 * 514 + 1024 * 256 + tiles * 4 + 16 * 520) + tiles * (64 * 130 + 12) + 32


def _cases():
    """Of each operator: a large batch and smaller ones that are split further."""
    rng = np.random.default_rng(1)
    many = rng.integers(1, 700, size=60)
    return {
        "paged_attention": [PagedCase(many, heads=8, kv=4, dim=64, seed=1, width=200),
                            PagedCase([3100, 5, 700], heads=8, kv=4, dim=64, seed=2, width=200),
                            PagedCase([3000], heads=8, kv=4, dim=64, store="float8_e4m3fn", seed=3, width=200)],
        "latent_attention": [LatentCase(rng.integers(1, 700, size=90), heads=70, dim=256, seed=1),
                             LatentCase([1300, 5, 580], heads=70, dim=256, seed=2),
                             LatentCase([890], heads=70, dim=256, store="float8_e4m3fn", seed=3)],
        "latent_prefill": [PrefillCase([600, 900], [600, 800], heads=4, seed=1),
                           PrefillCase([700, 90], [3, 90], heads=4, seed=2),
                           PrefillCase([1300], [2], heads=4, store="float8_e4m3fn", seed=3),
                           PrefillCase([2500, 40, 1700], [2, 5, 3], heads=3, seed=4)],
    }


@pytest.mark.parametrize("entry", ["paged_attention", "latent_attention", "latent_prefill"])
def test_one_buffer_for_calls_of_other_shapes(entry):
    """Anything may be in it: what an earlier call left, or NaN everywhere."""
    import torch
    cases = _cases()[entry]
    buffer = torch.full((1 << 26,), 0xff, dtype=torch.uint8, device="cuda")
    for again in range(2):
        for c in cases:
            note(f"{entry} in a shared buffer, run {again}")
            alone, shared = c.run(), c.run(workspace=buffer)
            assert torch.equal(alone[0], shared[0]) and torch.equal(alone[1], shared[1])
        buffer.fill_(0xff)


def _need(c):
    """The size that a call of this shape asks for."""
    pa._sizes.clear()
    c.run()
    (need,) = pa._sizes.values()
    return need


@pytest.mark.parametrize("entry,case", [("paged_attention", 1), ("latent_attention", 1), ("latent_prefill", 1),
                                        ("latent_prefill", 3)])
def test_sizes_of_a_workspace(entry, case):
    """Exactly the size that is asked for will do, all ones before the call; a byte less is refused."""
    import torch
    c = _cases()[entry][case]
    need = _need(c)
    assert need > 0
    exact = torch.full((need + 64,), 0xff, dtype=torch.uint8, device="cuda")
    out, lse = c.check("exact workspace", workspace=exact[:need])
    assert bool((exact[need:] == 0xff).all())
    assert bool(out.isfinite().all())
    with pytest.raises(ValueError, match="workspace"):
        c.run(workspace=exact[:need - 1])
    with pytest.raises(ValueError, match="workspace"):
        c.run(workspace=torch.empty(need, dtype=torch.uint8))
    with pytest.raises(binding.TopKError, match="aligned"):
        c.run(workspace=exact[8:8 + need])
    with pytest.raises(ValueError, match="workspace"):
        c.run(workspace=torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2])


def test_a_workspace_of_the_largest_batch_serves_smaller_ones():
    """What a server does: one buffer for its largest batch, every batch in it."""
    import torch
    dev = lambda x: torch.as_tensor(x, device="cuda")  # noqa: E731
    c = LatentCase(np.random.default_rng(2).integers(200, 3000, size=90), heads=20, dim=256, seed=4)
    table, lengths = dev(c.table), dev(c.lengths)
    buffer = torch.full((_need(c),), 0xff, dtype=torch.uint8, device="cuda")
    for rows in (90, 64, 33, 12, 5, 2, 1):
        args = (c.q[:rows], c.c, table[:rows], lengths[:rows])
        alone = rrt.latent_attention(*args, softmax_scale=c.scale)
        shared = rrt.latent_attention(*args, softmax_scale=c.scale, workspace=buffer)
        assert torch.equal(alone[0], shared[0]) and torch.equal(alone[1], shared[1])
