"""The paged cache's operators have no gradients, and say so instead of
returning outputs without a graph."""

from __future__ import annotations

import pytest

import row_radix_top_amd as rrt
from tests.gpu_util import require_gpu


def _calls(device):
    """name -> (function of tensors, its floating tensors, its other arguments)."""
    import torch
    f = lambda *s: torch.randn(*s, device=device).bfloat16()  # noqa: E731
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=device)  # noqa: E731
    table = i(0, 1)[None, :]
    return {
        "paged_append": (lambda k, v, kc, vc: rrt.paged_append(i(3, 9), k, v, kc, vc),
                         [f(2, 1, 64), f(2, 1, 64), f(2, 16, 1, 64), f(2, 16, 1, 64)]),
        "latent_append": (lambda a, b, c: rrt.latent_append(i(3, 9), a, b, c), [f(2, 256), f(2, 64), f(2, 16, 320)]),
        "paged_attention": (lambda q, k, v, o: rrt.paged_attention(q, k, v, table, i(20), out=o),
                            [f(1, 2, 64), f(2, 16, 1, 64), f(2, 16, 1, 64), f(1, 2, 64)]),
        "latent_attention": (lambda q, c, o: rrt.latent_attention(q, c, table, i(20), softmax_scale=0.1, out=o),
                             [f(1, 2, 320), f(2, 16, 320), f(1, 2, 256)]),
        "latent_prefill": (lambda q, c, a, b, o: rrt.latent_prefill(q, c, table, i(0, 1), i(20), a, b, context_tokens=20,
                                                                  softmax_scale=0.1, out=o),
                           [f(1, 2, 192), f(2, 16, 320), f(2, 128, 256), f(2, 128, 256), f(1, 2, 128)]),
    }


NAMES = ["paged_append", "latent_append", "paged_attention", "latent_attention", "latent_prefill"]


@pytest.mark.parametrize("name", NAMES)
def test_tensors_that_require_gradients_are_refused(name):
    """Before anything else is looked at, so without a GPU too."""
    fn, tensors = _calls("cpu")[name]
    for i in range(len(tensors)):
        given = [t.clone().requires_grad_(i == j) for j, t in enumerate(tensors)]
        with pytest.raises(RuntimeError, match=f"{name} has no gradients"):
            fn(*given)


@pytest.mark.gpu
def test_scales_that_require_gradients_are_refused():
    import torch
    require_gpu()
    table, n = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), torch.tensor([20], dtype=torch.int32, device="cuda")
    cache = torch.ones(2, 16, 320, device="cuda").to(torch.float8_e4m3fn)
    q, by = torch.ones(1, 2, 320, device="cuda").bfloat16(), torch.ones(1, device="cuda", requires_grad=True)
    with pytest.raises(RuntimeError, match="no gradients"):
        rrt.latent_attention(q, cache, table, n, softmax_scale=0.1, scale=by)
    with torch.no_grad():
        rrt.latent_attention(q, cache, table, n, softmax_scale=0.1, scale=by)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_they_are_taken_where_autograd_is_off(name):
    import torch
    require_gpu()
    fn, tensors = _calls("cuda")[name]
    with pytest.raises(RuntimeError, match="no gradients"):
        fn(*(t.clone().requires_grad_() for t in tensors))
    plain = fn(*tensors)
    for off in (torch.no_grad(), torch.inference_mode()):
        with off:
            again = fn(*(torch.nn.Parameter(t.clone()) for t in tensors))
        if plain is not None:
            assert torch.equal(again[0], plain[0]) and torch.equal(again[1], plain[1])
            assert not again[1].requires_grad
