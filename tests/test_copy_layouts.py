"""Which tensors paged_copy takes as caches: any whose elements lie apart."""

from __future__ import annotations

import pytest

from row_radix_top_amd import pages


def taken(x, tokens=False):
    return pages._pages_of(x, x.shape[0], tokens, -1)


@pytest.mark.parametrize("tokens", [False, True])
def test_caches_whose_elements_share_memory(tokens):
    import torch
    x = torch.zeros(6, 16, 2, 64)
    for bad in (x[:1].expand(6, 16, 2, 64), x[:, :1].expand(6, 16, 2, 64), x[:, :, :1].expand(6, 16, 2, 64),
                x[..., :1].expand(6, 16, 2, 64), x.view(-1).as_strided((6, 16, 2, 64), (1024, 128, 64, 1)),
                x.view(-1).as_strided((6, 16, 128), (2048, 64, 1)), x.view(-1).as_strided((6, 16, 2, 64), (2048, 32, 512, 1))):
        with pytest.raises(ValueError, match="share memory|contiguous"):
            taken(bad, tokens)


def test_caches_that_are_taken():
    import torch
    both = torch.zeros(6, 2, 4, 16, 64)
    for x, tokens in [(both[:, 0].transpose(1, 2), True), (both[:, 1], False), (both[:, :, 1], False), (both[::2], False),
                      (both.transpose(0, 1).contiguous().transpose(0, 1)[:, 0].transpose(1, 2), True),
                      (both[:, 0, :, ::2].transpose(1, 2), True), (both[:1, 0].expand(1, 4, 16, 64), False),
                      (torch.zeros(6, 16, 3, 128)[..., 32:64], True), (torch.zeros(16, 6, 2, 64).transpose(0, 1), True),
                      (torch.zeros(6, 16, 2, 64)[:, :1].expand(6, 1, 2, 64), True), (torch.zeros(9, 1), False)]:
        q = taken(x, tokens)
        n = x[0].numel() * x.element_size()
        assert q.outer * q.width * (q.tokens if tokens else 1) == n and q.data == x.data_ptr()
