"""The cross entropy's gradients against differences of its loss, along the
direction in which they show: each element moves by one step in the sign of its
gradient, so the slope is the sum of the gradient's magnitudes, and a gradient that
is wrong in sign, size or place gives another one.

x lies on a grid of 2^-5 and w on one of 2^-7, small enough for bf16 to hold both
with a step added.  Between the two ends the loss differs from its slope by a third
of its third derivative, which for a token is the third cumulant of its logits'
moves: the label's move by 0.4 at most gives 0.5% of the slope.  G's and the
result's roundings add 2^-9 each.  The bound is 2%.
"""
import pytest
import torch

N, VOCAB, WIDTH = 24, 90, 64
STEP = {"x": 2.0 ** -5, "w": 2.0 ** -7}
BOUND = 0.02


def inputs(seed, device):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(N, WIDTH, generator=g) / STEP["x"]).round().mul(STEP["x"]).clamp(-3.9, 3.9)
    w = (torch.randn(VOCAB, WIDTH, generator=g) * 0.25 / STEP["w"]).round().mul(STEP["w"]).clamp(-0.98, 0.98)
    labels = torch.randint(VOCAB, (N,), generator=g)
    labels[::7] = -1
    return x.to(torch.bfloat16).to(device), w.to(torch.bfloat16).to(device), labels.to(device)


def fits(total, x, w, name, gradient, claimed=None):
    """Whether the loss `total` has the slope that `claimed` says along the signs
    of `gradient`."""
    var = x if name == "x" else w
    move = torch.sign(gradient.double()) * STEP[name]
    ends = [(var.double() + move).to(torch.bfloat16), (var.double() - move).to(torch.bfloat16)]
    assert torch.equal(ends[0].double() - ends[1].double(), 2 * move), "the steps are not exact"
    slope = total(*((ends[0], w) if name == "x" else (x, ends[0]))) - total(*((ends[1], w) if name == "x" else (x, ends[1])))
    want = float(((gradient if claimed is None else claimed).double() * 2 * move).sum())
    return abs(slope - want) <= BOUND * abs(slope)


def wrong(d):
    """Gradients that a mistake would give."""
    return {"negated": -d, "doubled": 2 * d, "halved": d / 2, "rows shifted": d.roll(1, 0), "columns shifted": d.roll(1, 1), "a tenth more": 1.1 * d,
            "a row of zeros in eight": d * (torch.arange(len(d), device=d.device) % 8 != 1)[:, None]}


def plain(labels):
    def total(x, w):
        return float(torch.nn.functional.cross_entropy(x.double() @ w.double().t(), labels, ignore_index=-1, reduction="sum"))
    return total


@pytest.mark.parametrize("seed", range(20))
def test_differences_tell_right_gradients_from_wrong_ones(seed):
    """The comparison itself, on the CPU with gradients in 64 bits."""
    x, w, labels = inputs(seed, "cpu")
    xd, wd = x.double().requires_grad_(), w.double().requires_grad_()
    loss = torch.nn.functional.cross_entropy(xd @ wd.t(), labels, ignore_index=-1, reduction="sum")
    for name, d in zip("xw", torch.autograd.grad(loss, (xd, wd))):
        assert fits(plain(labels), x, w, name, d), name
        for what, claimed in wrong(d).items():
            assert not fits(plain(labels), x, w, name, d, claimed), (name, what)


@pytest.mark.gpu
@pytest.mark.parametrize("seed", [100, 101, 102])
def test_xent_gradient_along_itself(seed):
    import zero_sharded_mixed_reduce_amd as z
    x, w, labels = inputs(seed, "cuda")
    loss, lse, summary = (torch.empty(k, device="cuda") for k in (N, N, 3))
    ws = torch.empty(z.zsmr_xent_workspace(N, VOCAB, WIDTH), device="cuda", dtype=torch.uint8)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    z.zsmr_xent_forward(x, w, labels, loss, lse, summary, ws)
    z.zsmr_xent_backward(x, w, labels, lse, dx, dw, ws)

    def total(x2, w2):
        z.zsmr_xent_forward(x2, w2, labels, loss, lse, summary, ws)
        return float(loss.double().sum())

    for name, d in (("x", dx), ("w", dw)):
        assert fits(total, x, w, name, d), name
        for what, claimed in wrong(d).items():
            assert not fits(total, x, w, name, d, claimed), (name, what)
