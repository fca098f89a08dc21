"""Arguments that the paged-cache entry points refuse, through the C ABI and
without a GPU: every check comes before anything touches a device."""

from __future__ import annotations

import ctypes
import os
import re

import pytest

from row_radix_top_amd import attention as pa
from row_radix_top_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL = -1


def _header() -> str:
    text = open(os.path.join(ROOT, "include", "paged_attention.h")).read()
    return re.sub(r"/\*.*?\*/", "", text, flags=re.S)


def test_library_exports_every_declared_symbol():
    names = set(re.findall(r"^(?:int|int64_t|void) (\w+)\(", _header(), flags=re.M))
    assert names == set(pa.EXPORTED)
    for n in names:
        assert hasattr(binding.load(), n), n


@pytest.mark.parametrize("struct,name", [(pa.Part, "paged_part"), (pa.AttentionArgs, "paged_attention_args"),
                                         (pa.PrefillArgs, "latent_prefill_args")])
def test_ctypes_mirrors_follow_the_header(struct, name):
    body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", _header()).group(1)
    fields = []
    for decl in filter(None, (d.strip() for d in body.split(";"))):
        kind, names = re.match(r"((?:const )?\w+\s*\*?)\s*(.*)", decl, flags=re.S).groups()
        for n in names.split(","):
            fields.append((n.strip().lstrip("*"), "*" in kind or n.strip().startswith("*"), kind))
    assert [f[0] for f in fields] == [f[0] for f in struct._fields_]
    for (n, pointer, kind), (_, ctype) in zip(fields, struct._fields_):
        size = 8 if pointer or "int64" in kind else 4
        assert ctypes.sizeof(ctype) == size, n


def _attention(latent=False, **changes):
    a = pa.AttentionArgs()
    dim = 512 if latent else 128
    for k, v in dict(q=256, k=512, v=1024, block_table=256, lengths=256, out=256, lse=256, q_row_stride=8 * dim,
                     q_head_stride=dim, page_stride=64 * dim, token_stride=dim, head_stride=dim, table_stride=4,
                     chosen_stride=8, num_rows=2, next_n=1, num_heads=8, num_kv_heads=2, head_dim=dim, page_size=16,
                     num_pages=4, table_width=4, num_chosen=0, softmax_scale=0.1, dtype=0, store=0,
                     max_splits=0).items():
        setattr(a, k, changes.pop(k, v))
    for k, v in changes.items():
        setattr(a, k, v)
    return a


ATTENTION = [
    (dict(dtype=2), "dtype"), (dict(dtype=-1), "dtype"), (dict(store=1), "store"), (dict(num_rows=-1), "num_rows"),
    (dict(next_n=0), "next_n"), (dict(num_rows=3, next_n=2), "next_n"), (dict(num_heads=0), "num_heads"),
    (dict(head_dim=96), "head_dim"), (dict(page_size=0), "page_size"), (dict(table_width=0), "table_width"),
    (dict(max_splits=129), "max_splits"), (dict(max_splits=-1), "max_splits"), (dict(chosen=256), "num_chosen"),
    (dict(chosen=256, num_chosen=(1 << 30) + 1), "num_chosen"),
    (dict(softmax_scale=float("nan")), "softmax_scale"), (dict(softmax_scale=float("inf")), "softmax_scale"), (dict(softmax_scale=3e38), "softmax_scale"),
    (dict(num_pages=0), "num_pages"), (dict(q=None), "null"), (dict(k=None), "null"), (dict(lengths=None), "null"),
    (dict(block_table=None), "null"), (dict(out=None), "null"), (dict(q=264), "16 bytes"),
    (dict(q_row_stride=1028), "16 bytes"), (dict(k=520), "16 bytes"), (dict(token_stride=129), "16 bytes"),
    (dict(page_stride=-128), "strides"), (dict(out=264), "16-byte"), (dict(lse=257), "4-byte"),
    (dict(k_scales=256), "e4m3"), (dict(num_rows=1 << 30, num_heads=8), "2^31"),
    (dict(store=2, token_stride=136), "16 bytes"),
]


@pytest.mark.parametrize("changes,text", ATTENTION, ids=[str(sorted(c.items())) for c, _ in ATTENTION])
@pytest.mark.parametrize("latent", [False, True], ids=["paged", "latent"])
def test_attention_refuses(latent, changes, text):
    a = _attention(latent, **changes)
    fn = pa.load().latent_attention if latent else pa.load().paged_attention
    assert fn(ctypes.byref(a), None, None) == EINVAL
    assert text in binding.last_error()


@pytest.mark.parametrize("changes,text", [(dict(v=None), "null v"), (dict(num_kv_heads=3), "num_kv_heads"),
                                          (dict(num_kv_heads=0), "num_kv_heads"), (dict(head_stride=100), "16 bytes"),
                                          (dict(v_scales=256), "e4m3"), (dict(v=1032), "16 bytes")])
def test_paged_attention_refuses(changes, text):
    assert pa.load().paged_attention(ctypes.byref(_attention(**changes)), None, None) == EINVAL
    assert text in binding.last_error()


def test_no_rows_is_no_work():
    for fn in (pa.load().paged_attention, pa.load().latent_attention):
        a = _attention(fn is pa.load().latent_attention, num_rows=0, q=None, k=None, out=None)
        assert fn(ctypes.byref(a), None, None) == 0


def _prefill(**changes):
    a = pa.PrefillArgs()
    for k, v in dict(q=256, cache=512, w_k=256, w_v=256, block_table=256, starts=256, lengths=256, out=256, lse=256,
                     q_row_stride=8 * 192, q_head_stride=192, page_stride=16 * 576, token_stride=576, table_stride=4,
                     context_tokens=100, num_tokens=10, num_seqs=2, num_heads=8, latent_dim=512, page_size=16,
                     num_pages=4, table_width=4, softmax_scale=0.1, dtype=0, store=0).items():
        setattr(a, k, changes.pop(k, v))
    for k, v in changes.items():
        setattr(a, k, v)
    return a


PREFILL = [
    (dict(dtype=2), "dtype"), (dict(store=1), "store"), (dict(num_tokens=-1), "num_tokens"),
    (dict(num_seqs=-1), "num_seqs"), (dict(num_heads=0), "num_heads"), (dict(latent_dim=128), "latent_dim"),
    (dict(page_size=0), "page_size"), (dict(table_width=0), "table_width"), (dict(context_tokens=-1), "context_tokens"),
    (dict(softmax_scale=float("nan")), "softmax_scale"), (dict(num_pages=0), "num_pages"), (dict(q=None), "null"),
    (dict(cache=None), "null"), (dict(w_k=None), "null"), (dict(w_v=None), "null"), (dict(starts=None), "null"),
    (dict(lengths=None), "null"), (dict(block_table=None), "null"), (dict(out=None), "null"), (dict(q=264), "16 bytes"),
    (dict(cache=520), "16 bytes"), (dict(w_k=264), "16 bytes"), (dict(token_stride=577), "16 bytes"),
    (dict(q_head_stride=193), "16 bytes"), (dict(out=264), "16-byte"), (dict(lse=257), "4-byte"),
    (dict(scale=256), "e4m3"), (dict(page_stride=-16), "strides"),
]


@pytest.mark.parametrize("changes,text", PREFILL, ids=[str(sorted(c.items())) for c, _ in PREFILL])
def test_prefill_refuses(changes, text):
    assert pa.load().latent_prefill(ctypes.byref(_prefill(**changes)), None, None) == EINVAL
    assert text in binding.last_error()


def test_prefill_needs_its_workspace():
    assert pa.load().latent_prefill(ctypes.byref(_prefill()), None, None) == -3
    assert "workspace" in binding.last_error()
    assert pa.load().latent_prefill(ctypes.byref(_prefill(num_tokens=0, q=None)), None, None) == 0


def _layout(**changes):
    names = ("lengths", "new_tokens", "num_seqs", "free_pages", "num_free", "block_table", "table_stride",
             "table_width", "page_size", "capacity", "starts", "slots", "row_lengths", "row_seqs", "pages", "stream")
    base = dict(lengths=256, new_tokens=256, num_seqs=2, free_pages=256, num_free=4, block_table=256, table_stride=4,
                table_width=4, page_size=16, capacity=8, starts=256, slots=256, row_lengths=256, row_seqs=256,
                pages=256, stream=None)
    base.update(changes)
    return pa.load().paged_layout(*(base[n] for n in names))


@pytest.mark.parametrize("changes,text", [
    (dict(num_seqs=-1), "num_seqs"), (dict(num_free=-1), "num_free"), (dict(capacity=-1), "capacity"),
    (dict(page_size=0), "page_size"), (dict(table_width=0), "table_width"), (dict(table_stride=3), "table_stride"),
    (dict(lengths=None), "null"), (dict(new_tokens=None), "null"), (dict(block_table=None), "null"),
    (dict(free_pages=None), "free_pages"), (dict(starts=None), "starts"), (dict(pages=None), "pages"),
    (dict(slots=None), "slots"), (dict(row_lengths=None), "row_lengths"), (dict(row_seqs=None), "row_seqs"),
    (dict(slots=258), "4-byte"),
])
def test_layout_refuses(changes, text):
    assert _layout(**changes) == EINVAL
    assert text in binding.last_error()


def _append(tokens=2, parts=1, page_size=16, pages=4, dtype=0, store=0, slots=256, **part):
    p = pa.Part(256, 512, None, 64, 1024, 64, 32, 64, 32)
    for k, v in part.items():
        setattr(p, k, v)
    return pa.load().paged_append(slots, tokens, (pa.Part * 2)(p, p), parts, page_size, pages, dtype, store, None)


@pytest.mark.parametrize("changes,text", [
    (dict(tokens=-1), "num_tokens"), (dict(parts=0), "num_parts"), (dict(parts=3), "num_parts"),
    (dict(page_size=0), "page_size"), (dict(pages=-1), "num_pages"), (dict(dtype=2), "dtype"), (dict(store=1), "store"),
    (dict(slots=None), "slots"), (dict(slots=257), "slots"), (dict(width=0), "head_width"),
    (dict(head_width=48), "head_width"), (dict(src_stride=-64), "strides"), (dict(dst_token_stride=-1), "strides"),
    (dict(scales=256), "e4m3"), (dict(src=None), "null"), (dict(dst=None), "null"), (dict(src=257), "aligned"),
])
def test_append_refuses(changes, text):
    assert _append(**changes) == EINVAL
    assert text in binding.last_error()


def test_append_of_nothing():
    assert _append(tokens=0, slots=None) == 0
    assert _append(pages=0) == 0


@pytest.mark.parametrize("page_size", [1, 5, 16, 64])
def test_places_of_positions(page_size):
    num_pages, page_stride, token_stride = 7, 1 << 33, 1000
    table = [3, -1, 6, 7, -2147483648, 2147483647, 0]
    row = (ctypes.c_int32 * len(table))(*table)
    for pos in range(len(table) * page_size):
        page = table[pos // page_size]
        exp = page * page_stride + pos % page_size * token_stride if 0 <= page < num_pages else -1
        assert pa.load().paged_debug_place(row, page_size, num_pages, page_stride, token_stride, pos) == exp
    assert pa.load().paged_debug_place(row, page_size, 0, page_stride, token_stride, 0) == -1


def test_splits_cover_the_row():
    out = (ctypes.c_int32 * 2)()
    for unit in (32, 64, 128):
        for least in (unit, 2 * unit, 1000):
            for most in (1, 2, 7, 128):
                for n in (0, 1, 31, 32, 127, 128, 129, 999, 1000, 1001, 8192, 65537, (1 << 30) - 1, 1 << 30):
                    pa.load().paged_debug_split(n, most, least, unit, out)
                    parts, chunk = out[0], out[1]
                    assert 1 <= parts <= most and chunk % unit == 0 and chunk >= unit, (n, most, least, unit)
                    assert parts == max(1, -(-n // chunk))
                    assert parts == 1 or chunk >= least
