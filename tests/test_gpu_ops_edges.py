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


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -65504.0])
@pytest.mark.parametrize("n,vocab,width,stride,dt", [(70, 300, 64, 0, "bf16"), (300, 1000, 136, 0, "fp16"), (90, 600, 65, 67, "bf16"), (1, 40, 8, 0, "fp16")])
def test_hidden_states_of_tokens_that_do_not_count(n, vocab, width, stride, dt, value):
    """Nor does it matter what a token without a label holds in x: the bits of
    zeros there, in every gradient, and a loss of zero."""
    say("[x of padding]", n, vocab, width, stride, dt, value)
    g, t = gen(22), T16[dt]
    x, w = normal(g, (n, width), 1.0, t, stride), normal(g, (vocab, width), 0.2, t, stride)
    labels = tokens(g, n, vocab, "some")
    labels[0] = -1
    off = (labels < 0) | (labels >= vocab)
    old = normal(g, (vocab, width), 0.1, t)
    for accumulate in (None, old):
        x[off] = 0
        want = xent_both(x, w, labels, accumulate=accumulate)
        x[off] = value
        before = x.clone()
        got = xent_both(x, w, labels, accumulate=accumulate)
        assert torch.equal(bits(x), bits(before)), "x was written"
        for a, b, name in zip(want, got, ("loss", "lse", "summary", "dx", "dw")):
            keep = ~off if name == "lse" else slice(None)
            assert torch.equal(bits(a[keep]), bits(b[keep])), name
        assert bool((got[0][off] == 0).all()) and bool((got[3][off] == 0).all())
