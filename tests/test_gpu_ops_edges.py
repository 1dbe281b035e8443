"""The operators around the step where their inputs hold what they must not look
at, or what few programs hand over."""
import pytest
import torch

import zero_sharded_mixed_reduce_amd as z
from tests.gpu_helpers import say
from tests.test_gpu_ops import T16, gen, normal, space, tokens

pytestmark = pytest.mark.gpu


def xent_both(x, w, labels, weights=None, accumulate=None, scale=None):
    """Forward and backward: loss, lse, summary, dx, dw."""
    n, (vocab, width) = len(labels), w.shape
    loss, lse, summary = (torch.full((k,), float("nan"), device="cuda") for k in (n, n, 3))
    ws, _ = space(z.zsmr_xent_workspace(n, vocab, width))
    z.zsmr_xent_forward(x, w, labels, loss, lse, summary, ws)
    dx = torch.full_like(x, 7.0)
    dw = torch.full((vocab, width), 7.0, device="cuda", dtype=w.dtype) if accumulate is None else accumulate.clone()
    z.zsmr_xent_backward(x, w, labels, lse, dx, dw, ws, grad=weights, scale=summary[1:2] if scale is None else scale, accumulate=accumulate is not None)
    return loss, lse, summary, dx, dw


def bits(x):
    return x.contiguous().view(torch.int16 if x.element_size() == 2 else torch.int32)


@pytest.mark.parametrize("value", [1e10, 1e30, -3e38, float("inf"), float("nan")])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_weights_of_tokens_that_do_not_count(dt, value):
    """A token without a label has no gradient, whatever its weight: the bits of
    a weight of zero there."""
    say("[weights of padding]", dt, value)
    g, t = gen(21), T16[dt]
    x, w = normal(g, (150, 72), 1.0, t), normal(g, (700, 72), 0.2, t)
    labels = tokens(g, 150, 700, "some")
    labels[3], labels[9], labels[149] = -1, 700, -(1 << 40)
    off = (labels < 0) | (labels >= 700)
    weights = torch.randn(150, generator=g, device="cuda")
    clean, dirty = torch.where(off, 0.0, weights), torch.where(off, value, weights)
    want, got = xent_both(x, w, labels, clean), xent_both(x, w, labels, dirty)
    for a, b in zip(want, got):
        assert torch.equal(bits(a), bits(b))
    assert bool((got[3][off] == 0).all()) and bool((got[4] != 0).any())
