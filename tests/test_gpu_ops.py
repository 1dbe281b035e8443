"""The operators around the step against plain 64-bit implementations.

Tolerances: an output of type t may be off by half a step of t, eps(t)/2
relative (and half a subnormal step), for its one rounding; an fp32 sum of n
terms by n * 2^-24 of the sum of their magnitudes; a 16-bit operand of a sum by
half its step of that sum's magnitudes.  Where a result is a product of such
values, their relative errors add up.
"""
import math

import numpy as np
import pytest
import torch

import zero_sharded_mixed_reduce_amd as z
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

T16 = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -24                                  # fp32: half a step
SUB = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}


def half(t):
    return torch.finfo(t).eps / 2


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, shape, sigma, dtype, stride=None, shift=0):
    """A matrix of the given row stride whose data starts `shift` elements into
    an aligned allocation."""
    rows, width = shape
    stride = stride or width
    raw = torch.full((rows * stride + shift + 64,), float("nan"), device="cuda", dtype=dtype)
    x = raw[shift:shift + rows * stride].view(rows, stride)[:, :width] if rows else raw[:0].view(0, width)
    if rows:
        x.copy_(torch.randn(shape, generator=g, device="cuda") * sigma)
    return x


def space(n):
    """A workspace whose content is not zero, with a guard behind it."""
    raw = torch.full((n + 256,), 0xA5, device="cuda", dtype=torch.uint8)
    return raw[:n] if n else raw[:0], raw


def intact(raw, n):
    assert bool((raw[n:] == 0xA5).all()), "written past the workspace"


def close(got, want, tol, what):
    """Elementwise |got - want| <= tol, NaN where NaN."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    bad = (got - want).abs() > tol
    if bool(bad.any()):
        i = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {got[tuple(i)].item()} "
                             f"for {want[tuple(i)].item()}")


def tokens(g, n, vocab, kind, dtype=torch.int64):
    if kind == "same":
        ids = torch.full((n,), vocab - 1, device="cuda")
    elif kind == "none":
        ids = torch.full((n,), -1, device="cuda")
        ids[::2] = vocab
    elif kind == "distinct":
        ids = torch.randperm(max(vocab, n), generator=g, device="cuda")[:n] % vocab
    else:
        ids = (torch.rand(n, generator=g, device="cuda") ** 3 * vocab).long().clamp_(max=vocab - 1)
        ids[torch.rand(n, generator=g, device="cuda") < 0.1] = -1
    return ids.to(dtype)


# ----------------------------------------------------------------- lookup --
@pytest.mark.parametrize("n,vocab,width,stride,shift", [
    (1, 1, 1, 0, 0), (3, 5, 7, 9, 1), (64, 1000, 4096, 0, 0), (1000, 50257, 768, 0, 0), (257, 999, 769, 770, 3), (130, 77, 2050, 2056, 5),
    (4099, 100, 8, 0, 0)])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_lookup(n, vocab, width, stride, shift, dt):
    say("[lookup]", n, vocab, width, stride, shift, dt)
    g = gen(1)
    table = normal(g, (vocab, width), 1.0, T16[dt], stride, shift)
    ids = tokens(g, n, vocab, "some", torch.int32 if shift % 2 else torch.int64)
    out = normal(g, (n, width), 1.0, T16[dt], stride, shift)
    guard = out.as_strided((out.untyped_storage().nbytes() // 2,), (1,), 0).clone()
    z.zsmr_embed_lookup(table, ids, out, scale=1.7)
    want = torch.where((ids >= 0)[:, None], table[ids.clamp(min=0).long()].double() * float(np.float32(1.7)), 0.0)
    close(out, want, want.abs() * (half(T16[dt]) + U) * (1 + 1e-6) + SUB[T16[dt]], "out")
    # nothing between the rows or behind them is touched
    after = out.as_strided(guard.shape, (1,), 0).clone()
    mask = torch.ones_like(after, dtype=torch.bool)
    mask.as_strided(out.shape, out.stride(), out.storage_offset())[:] = False
    assert torch.equal(after[mask].view(torch.int16), guard[mask].view(torch.int16))
    z.zsmr_embed_lookup(table, ids, out)
    assert torch.equal(out, torch.where((ids >= 0)[:, None], table[ids.clamp(min=0).long()], torch.zeros((), device="cuda", dtype=T16[dt])))


# ---------------------------------------------------------- embedding grad --
def embed_grad_case(n, vocab, width, kind, dt, accumulate, stride=0, shift=0, id_dtype=torch.int64):
    say("[embed_grad]", n, vocab, width, kind, dt, accumulate, stride, shift)
    g, t = gen(2), T16[dt]
    dout = normal(g, (n, width), 1.0, t, stride, shift)
    table = normal(g, (vocab, width), 1.0, t, stride, shift)
    old = table.clone()
    ids = tokens(g, n, vocab, kind, id_dtype)
    size = z.zsmr_embed_grad_workspace(vocab, width, n)
    ws, raw = space(size)
    scale = 0.75
    z.zsmr_embed_grad(dout, ids, table, ws, scale=scale, accumulate=accumulate)
    intact(raw, size)
    keep = (ids >= 0) & (ids < vocab)
    at = ids[keep].long()
    want = torch.zeros(vocab, width, device="cuda", dtype=torch.float64).index_add_(0, at, dout[keep].double() * scale)
    mass = torch.zeros_like(want).index_add_(0, at, dout[keep].double().abs() * scale)
    count = torch.bincount(at, minlength=vocab)
    if accumulate:
        untouched = count == 0
        assert torch.equal(table[untouched].view(torch.int16), old[untouched].view(torch.int16))
        want += old.double()
        mass += old.double().abs()
    close(table, want, half(t) * want.abs() * (1 + 1e-6) + (count[:, None] + 3) * U * mass * 1.01 + SUB[t], "dtable")
    again = old.clone() if not stride else None
    if again is not None:
        ws.fill_(0x3C)
        z.zsmr_embed_grad(dout, ids, again, ws, scale=scale, accumulate=accumulate)
        assert torch.equal(again.view(torch.int16), table.view(torch.int16)), "not the same bits"


@pytest.mark.parametrize("n,vocab,width,kind", [
    (1, 1, 1, "same"), (1, 10, 64, "some"), (63, 7, 65, "some"), (64, 40, 768, "distinct"), (65, 100, 9, "same"), (130, 3, 520, "some"),
    (1000, 50257, 768, "some"), (2049, 511, 24, "some"), (2048, 512, 2056, "some"), (4097, 4096, 64, "distinct"), (5000, 300000, 16, "some"),
    (70000, 1000, 8, "some"), (16384, 70000, 16, "some"),
    (16385, 300000, 8, "some"), (16000, 900, 24, "same"), (3000, 50, 128, "same"), (100, 20, 64, "none")])
@pytest.mark.parametrize("dt,accumulate", [("bf16", False), ("fp16", True)])
def test_embed_grad(n, vocab, width, kind, dt, accumulate):
    embed_grad_case(n, vocab, width, kind, dt, accumulate)


@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad_strides_and_alignments(accumulate):
    embed_grad_case(300, 90, 77, "some", "bf16", accumulate, stride=81, shift=3, id_dtype=torch.int32)
    embed_grad_case(300, 90, 520, "some", "fp16", accumulate, stride=521, shift=1, id_dtype=torch.int32)


def test_embed_grad_without_tokens():
    t = torch.ones(5, 40, device="cuda", dtype=torch.bfloat16)
    none, ids = torch.empty(0, 40, device="cuda", dtype=torch.bfloat16), torch.empty(0, device="cuda", dtype=torch.int64)
    z.zsmr_embed_grad(none, ids, t, None, accumulate=True)
    assert bool((t == 1).all())
    z.zsmr_embed_grad(none, ids, t, None)
    assert bool((t == 0).all())
    z.zsmr_embed_lookup(t, ids, none)


def test_embedding_past_32_bits():
    """A table of 2.4e9 elements: rows lie beyond 2^31 elements and 2^32 bytes."""
    vocab, width, t = 600_000, 4096, torch.bfloat16
    table = torch.zeros(vocab, width, device="cuda", dtype=t)
    ids = torch.tensor([vocab - 1, 0, 530_000, vocab - 1], device="cuda")
    rows = torch.randn(4, width, generator=gen(3), device="cuda").to(t)
    ws, raw = space(z.zsmr_embed_grad_workspace(vocab, width, 4))
    table[77] = 1
    z.zsmr_embed_grad(rows, ids, table, ws)
    assert torch.equal(table[530_000], rows[2]) and torch.equal(table[0], rows[1])
    assert torch.equal(table[vocab - 1], (rows[0].float() + rows[3].float()).to(t))
    assert int((table != 0).any(1).sum()) == 3
    out = torch.empty(4, width, device="cuda", dtype=t)
    z.zsmr_embed_lookup(table, ids, out)
    assert torch.equal(out, table[ids])


# ----------------------------------------------------- softmax cross entropy --
def xent_case(n, vocab, width, dt, kind="some", stride=0, shift=0, grad=False, accumulate=False, sigma=2.0, id_dtype=torch.int64):
    say("[xent]", n, vocab, width, dt, kind, stride, shift, grad, accumulate)
    g, t = gen(4), T16[dt]
    x = normal(g, (n, width), 1.0, t, stride, shift)
    w = normal(g, (vocab, width), sigma / math.sqrt(width), t, stride, shift)
    labels = tokens(g, n, vocab, kind, id_dtype)
    loss, lse, summary = (torch.full((k,), float("nan"), device="cuda") for k in (n, n, 3))
    size = z.zsmr_xent_workspace(n, vocab, width)
    ws, raw = space(size)
    z.zsmr_xent_forward(x, w, labels, loss, lse, summary, ws)
    weights = torch.randn(n, generator=g, device="cuda") if grad else None
    dx, dw = normal(g, (n, width), 1.0, t, stride, shift), normal(g, (vocab, width), 0.1, t, stride, shift)
    old = dw.clone()
    z.zsmr_xent_backward(x, w, labels, lse, dx, dw, ws, grad=weights, scale=summary[1:2], accumulate=accumulate)
    intact(raw, size)

    xd, wd = x.double(), w.double()
    s = xd @ wd.t()
    # an fp32 logit's error, the row's largest
    es = U * width * (xd.abs() @ wd.abs().t()).max(1, keepdim=True).values
    want_lse = torch.logsumexp(s, 1, keepdim=True)
    keep = ((labels >= 0) & (labels < vocab))[:, None]
    at = torch.where(keep, labels.long()[:, None], 0)
    want_loss = torch.where(keep, want_lse - s.gather(1, at), 0.0)
    # exponentials of fp32 arguments (2^-20 of their value), and about vocab/256 joins
    tol = es + 2.0 ** -20 + U * vocab / 64 + 4 * U * want_lse.abs()
    close(lse[:, None], want_lse, tol, "lse")
    close(loss[:, None], want_loss, tol + es + U * want_loss.abs(), "loss")
    count = int(keep.sum())
    assert summary[2].item() == count
    mean = float(want_loss.sum()) / count if count else 0.0
    assert abs(summary[0].item() - mean) <= float((tol + es).max()) + 2 * U * abs(mean)
    assert summary[1].item() == np.float32(1 / count if count else 0.0)

    scale = summary[1].double() * torch.where(keep, weights.double()[:, None] if grad else 1.0, 0.0)
    G = torch.exp(s - want_lse)
    slack = (torch.exp(es + tol) - 1 + 2.0 ** -20) * G                   # the probabilities' error before rounding
    G.scatter_add_(1, at, torch.full_like(want_lse, -1.0))
    top = float(weights.abs().max()) if grad and n else 1.0
    h = half(t)
    # each G rounded to 16 bits; fp16's are held times a power of two: 2^-39 of the largest weight below its normal range
    slack = (slack + G.abs() * (h + 2 * U) + (2.0 ** -38 if dt == "fp16" else 2.0 ** -133) * top) * scale.abs()
    G = G * scale
    want, mass = G @ wd, G.abs() @ wd.abs()
    close(dx, want, h * want.abs() * 1.001 + slack @ wd.abs() * 1.01 + (vocab + 8) * U * mass * 1.01 + SUB[t], "dx")
    norm = float(want.norm())
    assert float((dx.double() - want).norm()) <= max(h, float((tol + es).max())) * norm + SUB[t] * math.sqrt(want.numel())
    want, mass = G.t() @ xd, G.abs().t() @ xd.abs()
    if accumulate:
        want, mass = want + old.double(), mass + old.double().abs()
    close(dw, want, h * want.abs() * 1.001 + slack.t() @ xd.abs() * 1.01 + (n + 8) * U * mass * 1.01 + SUB[t], "dw")
    norm = float(want.norm())
    assert float((dw.double() - want).norm()) <= max(h, float((tol + es).max())) * norm + SUB[t] * math.sqrt(want.numel())
    # each gradient alone, and the same bits again
    dx2, dw2 = torch.empty_like(dx), old.clone()
    z.zsmr_xent_backward(x, w, labels, lse, dx2, None, ws, grad=weights, scale=summary[1:2])
    z.zsmr_xent_backward(x, w, labels, lse, None, dw2, ws, grad=weights, scale=summary[1:2], accumulate=accumulate)
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


@pytest.mark.parametrize("n,vocab,width", [
    (1, 1, 8), (1, 257, 64), (5, 100, 72), (16, 1000, 512), (64, 256, 64), (65, 255, 128), (128, 513, 136), (129, 1025, 768), (256, 2048, 64),
    (257, 777, 200), (513, 3000, 1032), (1000, 5000, 320)])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_xent(n, vocab, width, dt):
    xent_case(n, vocab, width, dt)


@pytest.mark.parametrize("n,vocab,width,stride,shift", [
    (7, 50, 1, 0, 0), (33, 300, 65, 0, 0), (130, 600, 96, 104, 8), (40, 300, 64, 64, 1), (40, 300, 64, 67, 0), (300, 520, 129, 131, 5)])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_xent_strides_and_alignments(n, vocab, width, stride, shift, dt):
    xent_case(n, vocab, width, dt, stride=stride, shift=shift, id_dtype=torch.int32)


@pytest.mark.parametrize("kind", ["none", "same"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_xent_labels(kind, dt):
    xent_case(70, 300, 64, dt, kind=kind)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_xent_weighted_accumulated_and_sharp(dt):
    xent_case(200, 700, 128, dt, grad=True, accumulate=True)
    xent_case(200, 700, 128, dt, sigma=12.0, grad=True)


@pytest.mark.parametrize("n,vocab,width,stride", [(8192, 33500, 64, 0), (5000, 60000, 65, 0), (33, 70000, 130, 131), (70, 300, 2056, 0)])
def test_xent_in_pieces(n, vocab, width, stride):
    """More than 2^28 probabilities (several pieces of the vocabulary), also
    where each piece of the weights is packed; and a split k."""
    xent_case(n, vocab, width, "bf16", stride=stride)


def test_xent_past_32_bits():
    """Weights of 2.2e9 elements; the last tokens' labels lie beyond 2^31."""
    n, vocab, width, t = 4, 540_000, 4096, torch.bfloat16
    g = gen(5)
    x = normal(g, (n, width), 1.0, t)
    w = torch.randn(vocab, width, generator=g, device="cuda", dtype=t).mul_(1 / 64)
    labels = torch.tensor([0, vocab - 1, 530_000, vocab], device="cuda")
    loss, lse, summary = (torch.empty(k, device="cuda") for k in (n, n, 3))
    ws, raw = space(z.zsmr_xent_workspace(n, vocab, width))
    z.zsmr_xent_forward(x, w, labels, loss, lse, summary, ws)
    s = torch.cat([x.double() @ part.double().t() for part in w.split(60_000)], 1)
    want = torch.logsumexp(s, 1)
    # fp32 logits of 4,096 products of magnitude about 0.01 each, sums over 540,000
    assert float((lse.double() - want).abs().max()) < 1e-4
    assert float((loss[:3].double() - (want - s.gather(1, labels.clamp(max=vocab - 1)[:, None])[:, 0])[:3]).abs().max()) < 2e-4
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    z.zsmr_xent_backward(x, w, labels, lse, dx, dw, ws)
    G = torch.exp(s - want[:, None])
    G[torch.arange(3), labels[:3]] -= 1
    G[3] = 0
    want = torch.stack([sum(G[:, i:i + 60_000] @ w[i:i + 60_000].double() for i in range(0, vocab, 60_000))])[0]
    assert float((dx.double() - want).norm() / want.norm()) < half(t)
    for rows in (slice(0, 300), slice(vocab - 300, vocab), slice(529_900, 530_100)):
        part = G.t()[rows] @ x.double()
        assert float((dw[rows].double() - part).norm() / part.norm()) < half(t)
    intact(raw, len(raw) - 256)


def test_xent_without_tokens():
    w, x = torch.ones(300, 64, device="cuda", dtype=torch.bfloat16), torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    ids, none = torch.empty(0, device="cuda", dtype=torch.int64), torch.empty(0, device="cuda")
    summary, dw = torch.full((3,), 7.0, device="cuda"), torch.ones_like(w)
    ws, raw = space(z.zsmr_xent_workspace(0, 300, 64))
    z.zsmr_xent_forward(x, w, ids, none, none, summary, ws)
    assert summary.tolist() == [0, 0, 0]
    z.zsmr_xent_backward(x, w, ids, none, x, dw, ws, accumulate=True)
    assert bool((dw == 1).all())
    z.zsmr_xent_backward(x, w, ids, none, x, dw, ws)
    assert bool((dw == 0).all())


def test_xent_gradient_against_differences():
    """The loss itself, moved along a direction: its slope is the gradient's
    product with the direction.  Steps are exact in bf16."""
    g, t = gen(6), torch.bfloat16
    n, vocab, width = 24, 90, 64
    x, w = normal(g, (n, width), 1.0, t), normal(g, (vocab, width), 0.25, t)
    labels = tokens(g, n, vocab, "some")
    loss, lse, summary = (torch.empty(k, device="cuda") for k in (n, n, 3))
    ws, _ = space(z.zsmr_xent_workspace(n, vocab, width))
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    z.zsmr_xent_forward(x, w, labels, loss, lse, summary, ws)
    z.zsmr_xent_backward(x, w, labels, lse, dx, dw, ws)

    def total(x2, w2):
        z.zsmr_xent_forward(x2, w2, labels, loss, lse, summary, ws)
        return float(loss.double().sum())

    for var, d in ((x, dx), (w, dw)):
        for _ in range(4):
            step = torch.sign(torch.randn(var.shape, generator=g, device="cuda")) * 2.0 ** -4
            up, down = (var.float() + step).to(t), (var.float() - step).to(t)
            moved = up.double() - down.double()              # what the rounding left of the step
            pair = [(up, w), (down, w)] if var is x else [(x, up), (x, down)]
            slope = total(*pair[0]) - total(*pair[1])
            want = float((d.double() * moved).sum())
            # central differences: third-order term; steps of 1/16 in 64 coordinates of values about 1
            size = float(d.double().abs().mul(moved.abs()).sum())
            assert abs(slope - want) <= 0.05 * size, (slope, want, size)


# ------------------------------------------------------------ norm, clipping --
LISTS = [[], [0], [1], [7, 0, 16384, 16385], [5, 8, 13, 100_003, 64, 3], [1] * 400, [1_000_001, 33, 4_000_000]]


def tensor_list(sizes, dts, seed=7, shift=0):
    g = gen(seed)
    out = []
    for i, n in enumerate(sizes):
        dt = dts[i % len(dts)]
        raw = torch.full((n + 32,), float("nan"), device="cuda", dtype=dt)
        raw[shift:shift + n] = (torch.randn(n, generator=g, device="cuda") * 0.01).to(dt)
        out.append(raw[shift:shift + n])
    return out


@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}t")
@pytest.mark.parametrize("dts", [(torch.float32,), (torch.bfloat16,), (torch.float16,), (torch.float32, torch.float16, torch.bfloat16)],
                         ids=lambda d: "-".join(str(t)[6:] for t in d))
@pytest.mark.parametrize("shift", [0, 1])
def test_norm_clip_flatten(sizes, dts, shift):
    xs = tensor_list(sizes, dts, shift=shift)
    total = sum(sizes)
    size = z.zsmr_norm_workspace(total, len(xs))
    ws, raw = space(size)
    out = torch.full((2,), 7.0, device="cuda")
    max_norm = 0.5 * 0.01 * math.sqrt(max(total, 1))
    z.zsmr_grad_norm(xs, max_norm, out, ws)
    intact(raw, size)
    norm = math.sqrt(sum(float(x.double().square().sum()) for x in xs))
    coef = min(1.0, max_norm / (norm + 1e-6))
    assert abs(out[0].item() - norm) <= 2 * U * norm and abs(out[1].item() - coef) <= 2 * U * coef
    for ft in (torch.bfloat16, torch.float16):
        raw = torch.full((total + 40 + shift,), 7.0, device="cuda", dtype=ft)
        flat = raw[shift:shift + total + 29]
        z.zsmr_clip_flatten(xs, out[1:], flat)
        want = torch.cat([x.double() for x in xs] + [torch.zeros(29, device="cuda", dtype=torch.float64)]) * float(out[1])
        close(flat, want, want.abs() * (half(ft) + U) * 1.001 + SUB[ft], "flat")
        assert bool((raw[shift + total + 29:] == 7).all()) and bool((raw[:shift] == 7).all())
    z.zsmr_clip_flatten(xs, None, flat)
    assert torch.equal(flat[:total], torch.cat([x.to(ft) for x in xs]) if xs else flat[:0])
    before = [x.double() for x in xs]
    z.zsmr_clip_grads(xs, out[1:])
    for x, b in zip(xs, before):
        close(x, b * float(out[1]), (b * float(out[1])).abs() * half(x.dtype) * 1.001 + SUB[x.dtype], "in place")


def test_norm_of_extremes_and_of_what_is_not_finite():
    out, ws = torch.empty(2, device="cuda"), space(4096)[0]
    big = torch.tensor([3e38, -3e38], device="cuda")
    z.zsmr_grad_norm([big / 2], 1.0, out, ws)
    assert abs(out[0].item() / (1.5e38 * math.sqrt(2)) - 1) < 1e-6
    z.zsmr_grad_norm([torch.full((100,), 1e-40, device="cuda")], 1.0, out, ws, eps=0.0)
    assert abs(out[0].item() / float(np.float32(1e-40) * 10.0) - 1) < 1e-3 and out[1].item() == 1
    z.zsmr_grad_norm([torch.zeros(10, device="cuda"), big * float("inf")], 1.0, out, ws)
    assert math.isinf(out[0].item()) and out[1].item() == 0
    z.zsmr_grad_norm([torch.tensor([1.0, float("nan")], device="cuda")], 1.0, out, ws)
    assert math.isnan(out[0].item()) and math.isnan(out[1].item())
    z.zsmr_grad_norm([torch.ones(4, device="cuda")], 100.0, out, ws)
    assert out.tolist() == [2.0, 1.0]
    z.zsmr_grad_norm([torch.ones(4, device="cuda")], 0.0, out, ws)
    assert out.tolist() == [2.0, 0.0]
    # a coefficient of one leaves tensors as they are, a NaN reaches every element
    x = torch.tensor([1.0, float("inf"), 2.0], device="cuda")
    z.zsmr_clip_grads([x], torch.ones(1, device="cuda"))
    assert x.tolist() == [1.0, float("inf"), 2.0]
    z.zsmr_clip_grads([x], torch.full((1,), float("nan"), device="cuda"))
    assert bool(torch.isnan(x).all())


def test_norm_list_as_arrays_gives_the_same_bits():
    xs = tensor_list([100, 20_000, 3], (torch.float32, torch.bfloat16))
    arrays = (np.array([x.data_ptr() for x in xs], np.int64), np.array([x.numel() for x in xs], np.int64), np.array([3, 2, 3], np.int32))
    a, b, ws = torch.empty(2, device="cuda"), torch.empty(2, device="cuda"), space(z.zsmr_norm_workspace(20_103, 3))[0]
    z.zsmr_grad_norm(xs, 1.0, a, ws)
    z.zsmr_grad_norm(arrays, 1.0, b, ws)
    assert torch.equal(a, b)


# ------------------------------------------------------------- clipped step --
@pytest.mark.parametrize("numel,world,dt,pad,shift", [
    (1, 1, "bf16", False, 0), (7, 1, "fp16", False, 1), (4096, 2, "bf16", False, 0), (65536, 4, "fp16", False, 0), (100_003, 3, "bf16", True, 1),
    (5000, 9, "fp16", True, 3), (1_234_567, 16, "bf16", True, 0), (300_000, 64, "bf16", True, 5)])
def test_clipped_step_has_the_bits_of_the_plain_steps(numel, world, dt, pad, shift):
    """Reduce, sum of squares, join, clipped Adam and cast against the calls of
    the unclipped step, whose bits they share: on the reduced gradient, and on
    the clipped one."""
    say("[clipped]", numel, world, dt, pad, shift)
    g, t = gen(8), T16[dt]
    ctx = z.zero_init_shards(numel, world, z.ZSMR_ZERO2, dt, pad=pad)
    ref = z.zero_init_shards(numel, world, z.ZSMR_ZERO2, dt, pad=pad)
    P, S = ctx.info()["padded_numel"], ctx.info()["shard_numel"]
    grads = normal(g, (world, P), 0.02, t, P + shift, shift)
    flat = grads.as_strided((world * (P + shift),), (1,), grads.storage_offset())
    state = [normal(g, (1, P), s, torch.float32, None, shift)[0] for s in (0.02, 1e-3, 1.0)]
    state[2].square_().mul_(1e-6)
    p16 = torch.empty(P + shift, device="cuda", dtype=t)[shift:]
    mine, plain = [x.clone() for x in state], [x.clone() for x in state]
    p16_ref = torch.empty_like(p16)
    sums, out = torch.full((world,), float("nan"), device="cuda", dtype=torch.float64), torch.empty(2, device="cuda")
    red, red_ref = torch.empty(P + shift, device="cuda")[shift:], torch.empty(P, device="cuda")
    size = z.zsmr_norm_workspace(S, 1)
    ws, raw = space(size)
    for r in range(world):
        o = r * S
        z.zero_reduce_shard_sumsq(ctx, r, 0, flat, P + shift, o, True, red[o:], sums[r:], ws)
        z.zero_reduce_shard(ref, r, 0, flat, P + shift, o, True, red_ref[o:])
    intact(raw, size)
    assert torch.equal(red.view(torch.int32), red_ref.view(torch.int32)), "reduced gradient"
    want = red_ref.double().view(world, S).square().sum(1)
    assert float(((sums - want).abs() - 1e-12 * want).max()) <= 0
    norm = math.sqrt(float(want.sum()))
    for max_norm in (0.5 * norm, 2 * norm):
        z.zsmr_clip_coef(sums, world, max_norm, out)
        coef = min(1.0, max_norm / (norm + 1e-6))
        assert abs(out[0].item() - norm) <= 2 * U * norm and abs(out[1].item() - coef) <= 2 * U * coef
        for r in range(world):
            o = r * S
            z.zero_clipped_step(ctx, r, 0, red[o:], out[1:], *(x[o:] for x in mine), p16[o:], 3, 1e-3)
            z.zero_adam_step(*(x[o:] for x in plain), red_ref[o:o + S] * out[1], S, 3, 1e-3)
            z.zero_gather_cast(ref, r, 0, plain[0][o:], p16_ref[o:])
        for a, b in zip(mine + [p16], plain + [p16_ref]):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    z.zero_clipped_step(ctx, 0, 0, red, None, *mine, p16, 4, 1e-3)
    z.zero_adam_step(*plain, red_ref, S, 4, 1e-3)
    assert torch.equal(mine[0], plain[0])
    a, b = (z.zero_counters(c, world - 1) for c in (ctx, ref))
    assert a["rs_elems"] == b["rs_elems"]
    # the third step's cast went to rank 0's peers too
    assert a["ag_elems"] == b["ag_elems"] + (S if world > 1 else 0)


@pytest.mark.parametrize("world,extra,shift,dt", [(16, 0, 0, "bf16"), (32, 0, 0, "bf16"), (33, 511, 1, "fp16"), (47, 5, 3, "bf16")])
def test_windowed_reduce(world, extra, shift, dt):
    """One rank's large shard with many rows, whose results are stored in write
    windows: the bits of zero_reduce_shard and the sum of their squares."""
    n, t = 1024 * 18 * 512 + extra, T16[dt]         # windows from 2^28 elements in 32 rows on
    g = gen(10)
    ctx = z.zero_init_shards(n * world, world, z.ZSMR_ZERO2, dt)
    raw = torch.randn(world * (n + shift) + 8, generator=g, device="cuda", dtype=t).mul_(0.01)[shift:]
    red = torch.full((n + 16,), 7.0, device="cuda")
    want, sums = torch.empty(n, device="cuda"), torch.empty(1, device="cuda", dtype=torch.float64)
    size = z.zsmr_norm_workspace(n, 1)
    ws, guard = space(size)
    z.zero_reduce_shard(ctx, 1, 0, raw, n + shift, 0, True, want)
    for _ in range(2):
        z.zero_reduce_shard_sumsq(ctx, 1, 0, raw, n + shift, 0, True, red, sums, ws)
        assert torch.equal(red[:n].view(torch.int32), want.view(torch.int32))
        exact = float(want.double().square().sum())
        assert abs(float(sums) - exact) <= 1e-11 * exact
    assert bool((red[n:] == 7).all())
    intact(guard, size)


def test_reduce_of_very_many_rows_of_a_short_piece():
    """16,400 ranks of 20,000: as much to read as a windowed reduce has, but
    fewer tiles than it has waves."""
    n, world = 20_000, 16_400
    ctx = z.zero_init_shards(n * world, world, z.ZSMR_ZERO2, "bf16")
    raw = torch.randn(world * n, generator=gen(12), device="cuda", dtype=torch.bfloat16)
    red, want, sums = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty(1, device="cuda", dtype=torch.float64)
    size = z.zsmr_norm_workspace(n, 1)
    ws, guard = space(size)
    z.zero_reduce_shard(ctx, 3, 0, raw, n, 0, True, want)
    z.zero_reduce_shard_sumsq(ctx, 3, 0, raw, n, 0, True, red, sums, ws)
    intact(guard, size)
    assert torch.equal(red.view(torch.int32), want.view(torch.int32))
    exact = float(want.double().square().sum())
    assert abs(float(sums) - exact) <= 1e-12 * exact


@pytest.mark.parametrize("sizes", [[40_000_003, 5, 30_000_000], [1] + [9_000_000] * 8])
def test_norm_clip_flatten_of_long_lists(sizes):
    """More chunks than workgroups, and than what is kept in the caches."""
    xs = tensor_list(sizes, (torch.bfloat16,))
    total = sum(sizes)
    size = z.zsmr_norm_workspace(total, len(xs))
    ws, guard = space(size)
    out = torch.empty(2, device="cuda")
    z.zsmr_grad_norm(xs, 1.0, out, ws)
    intact(guard, size)
    norm = math.sqrt(sum(float(x.double().square().sum()) for x in xs))
    assert abs(out[0].item() - norm) <= 2 * U * norm
    flat = torch.empty(total + 20_001, device="cuda", dtype=torch.float16)
    z.zsmr_clip_flatten(xs, out[1:], flat)
    want = (torch.cat(xs).float() * out[1]).half()
    assert torch.equal(flat[:total], want) and not bool(flat[total:].any())
    z.zsmr_clip_grads(xs, out[1:])
    assert torch.equal(torch.cat(xs), (torch.cat(tensor_list(sizes, (torch.bfloat16,))).float() * out[1]).bfloat16())


def test_join_of_many_sums():
    sums = torch.rand(5000, device="cuda", dtype=torch.float64)
    out = torch.empty(2, device="cuda")
    z.zsmr_clip_coef(sums, 5000, 1.0, out, eps=0.0)
    norm = math.sqrt(float(sums.sum()))
    assert abs(out[0].item() - norm) <= 2 * U * norm
    z.zsmr_clip_coef(sums, 0, 1.0, out)
    assert out.tolist() == [0.0, 1.0]


# ------------------------------------------------------------ streams, graphs --
def chain(x, w, table, ids, labels, buf):
    """Every operator once, from lookup to clipped gradient, into buffers."""
    z.zsmr_embed_lookup(table, ids, buf["x"])
    z.zsmr_xent_forward(buf["x"], w, labels, buf["loss"], buf["lse"], buf["summary"], buf["ws"])
    z.zsmr_xent_backward(buf["x"], w, labels, buf["lse"], buf["dx"], buf["dw"], buf["ws"], scale=buf["summary"][1:2])
    z.zsmr_embed_grad(buf["dx"], ids, buf["dt"], buf["ws2"])
    z.zsmr_grad_norm([buf["dw"], buf["dt"]], 0.01, buf["nc"], buf["ws3"])
    z.zsmr_clip_flatten([buf["dt"], buf["dw"]], buf["nc"][1:], buf["flat"])
    z.zsmr_clip_grads([buf["dw"], buf["dt"]], buf["nc"][1:])


@pytest.mark.parametrize("n,vocab,width", [(70, 900, 128), (300, 1000, 264)])
def test_stream_and_graph(n, vocab, width):
    """The chain on a stream of its own, and captured and replayed several times
    between eager runs, has the eager run's bits."""
    g, t = gen(9), torch.bfloat16
    w, table = normal(g, (vocab, width), 0.1, t), normal(g, (vocab, width), 1.0, t)
    ids, labels = tokens(g, n, vocab, "some"), tokens(g, n, vocab, "some")

    def buffers():
        e = lambda *s, d=torch.float32: torch.zeros(*s, device="cuda", dtype=d)  # noqa: E731
        return {"x": e(n, width, d=t), "loss": e(n), "lse": e(n), "summary": e(3), "dx": e(n, width, d=t), "dw": e(vocab, width, d=t),
                "dt": e(vocab, width, d=t), "nc": e(2), "flat": e(2 * vocab * width + 5, d=t),
                "ws": e(z.zsmr_xent_workspace(n, vocab, width), d=torch.uint8),
                "ws2": e(z.zsmr_embed_grad_workspace(vocab, width, n), d=torch.uint8),
                "ws3": e(z.zsmr_norm_workspace(2 * vocab * width, 2), d=torch.uint8)}

    keys = ("x", "loss", "lse", "summary", "dx", "dw", "dt", "nc", "flat")
    eager, other, captured = buffers(), buffers(), buffers()
    chain(None, w, table, ids, labels, eager)
    torch.cuda.synchronize()
    want = {k: eager[k].clone() for k in keys}
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        chain(None, w, table, ids, labels, other)
    stream.synchronize()
    for k in keys:
        assert torch.equal(other[k], want[k]), k
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        chain(None, w, table, ids, labels, captured)
    for _ in range(4):
        for k in keys:
            captured[k].fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for k in keys:
            assert torch.equal(captured[k], want[k]), k
        chain(None, w, table, ids, labels, eager)
        torch.cuda.synchronize()


# ------------------------------------------------------------------- example --
def test_example_trains_and_matches_a_plain_step():
    """The example's first step against the same step in 64 bits, and its loss
    falls over the next ones."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "bigram.py")
    spec = importlib.util.spec_from_file_location("bigram", path)
    bigram = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(bigram)
    torch.manual_seed(1)
    vocab, width, n, world = 301, 40, 130, 3
    model = bigram.Bigram(vocab, width, n, world, 0.05, 1e-2)
    g = gen(11)
    successor = torch.randperm(vocab, generator=g, device="cuda")
    x, y = bigram.batch(successor, world, n, g)
    params = model.params[:2 * vocab * width].double().requires_grad_()
    master = model.master.double()
    e, w = params.view(2, vocab, width)
    rows = []
    for r in range(world):
        loss = torch.nn.functional.cross_entropy(e[x[r]] @ w.t(), y[r], ignore_index=-1)
        rows.append(torch.autograd.grad(loss, params, retain_graph=r + 1 < world)[0])
    grad = torch.stack(rows).mean(0)
    norm = float(grad.norm())
    loss, norm_coef = model.step(x, y)
    # three 16-bit roundings a gradient element (G, dx, the row): their sum in the norm
    assert abs(norm_coef[0].item() - norm) <= 3 * half(torch.bfloat16) * norm
    coef = 0.05 / (norm + 1e-6)
    assert abs(norm_coef[1].item() - coef) <= 3 * half(torch.bfloat16) * coef
    # the first Adam step moves by lr * g / (|g| + eps'): compare where g is not near zero
    big = grad.abs() * coef > 1e-5
    moved = (model.master[:grad.numel()].double() - master[:grad.numel()])[big]
    assert float((moved + 1e-2 * torch.sign(grad[big])).abs().max()) < 1e-4
    assert torch.equal(model.params, model.master.to(torch.bfloat16))
    losses, _ = bigram.train(vocab=500, width=64, tokens=1000, world=2, steps=40, say=lambda *_: None)
    assert losses[0] > 0.9 * math.log(500) and losses[-1] < 0.5 * losses[0]
