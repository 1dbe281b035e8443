"""Scores of logits with finite masks and of rows far from zero, and their gradient,
against 64 bits.

Tolerances.  A term 2^d, d = (x - x_ref) scale log2 e, has the roundings of the
constant, of d and of the power; terms of |z - z_ref| up to 40 count, so its relative
error is below 2^-24 (2 * 4 * 40 + 2 * 100), however far from zero the row lies.  A lane
adds vocab / 256 terms (vocab / 64 where two waves share a row) one by one, the joins
some 30 more.  That is `sums`, the error of log sum 2^d and of logprob; entropy is a
mean of log p with these weights: 1 + H times it.  lse has half a step of its size,
2^-24, for the constant, the reference, the sum, the product with ln 2, and a quarter for
ln 2 itself; logprob has as many of its own.
"""
import pytest
import torch

import zero_sharded_mixed_reduce_amd as z
from tests.test_gpu_scores import BF16, F16, F32, HALF_STEP, INF, best, gen, near, score

pytestmark = pytest.mark.gpu


def reference(x, ids, scale):
    """In 64 bits.  Log probabilities are differences from the row's largest value first:
    lse of a row at 1e30 holds no log of a sum, in 64 bits either."""
    v = x.double() * torch.tensor(scale, dtype=F32).double().item()
    v = torch.where(v < -2.3e38, -INF, v)
    top = v.amax(1, keepdim=True)
    none = top == -INF
    d = torch.where(none, -INF, v - torch.where(none, 0.0, top))
    log_sum = torch.where(none, 0.0, d.exp().sum(1, keepdim=True).log())
    logp = d - log_sum
    p = logp.exp()
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(1)
    ok = (ids >= 0) & (ids < x.shape[1])
    logprob = torch.where(ok, logp.gather(1, torch.where(ok, ids, 0)[:, None])[:, 0], 0.0)
    return {"lse": (top + log_sum)[:, 0], "logprob": logprob, "entropy": entropy, "logp": logp, "p": p}


def sums(n, v):
    lane = v / (64 if n > 256 and v < 8192 else 256)
    return 2.0 ** -24 * (lane + 2 * (4 * 40 + 100) + 30)


def size(t):
    return torch.where(torch.isfinite(t), t.abs(), 0.0)


def check(x, ids, top, scale):
    out, ref, tol = score(x, ids, top, scale), reference(x, ids, scale), sums(*x.shape)
    near(out["lse"], ref["lse"], tol + 5 * 2.0 ** -24 * size(ref["lse"]))
    near(out["entropy"], ref["entropy"], tol * (1 + ref["entropy"]))
    near(out["logprob"], ref["logprob"], tol + 6 * 2.0 ** -24 * size(ref["logprob"]))
    if top:
        at = best(x, top)
        assert torch.equal(out["top_ids"], at)
        want = torch.where(at >= 0, ref["logp"].gather(1, at.clamp(min=0)), -INF)
        near(out["top_logprobs"], want, tol + 6 * 2.0 ** -24 * size(want))
    return out, ref


def masked(dtype, v, many, mask):
    """Rows of which a mask takes a random half, the first blocks, most, all but one,
    whole lanes, all, the second half, nothing."""
    x = torch.randn(8, v, generator=gen(v), device="cuda").mul_(2.0)
    c = torch.arange(v, device="cuda")
    out = torch.stack([torch.rand(v, generator=gen(5), device="cuda") < 0.5, c < v * 7 // 10, c < v - 10, c != v // 3, c // 8 % 3 == 0, c >= 0,
                       c >= v // 2, c < 0])
    x = torch.where(out, mask, x).to(dtype)
    ids = torch.tensor([1, 0, v - 3, v // 3, 9, 2, v - 1, -1], device="cuda")
    return x.repeat(many, 1), ids.repeat(many)


MASKS = [(t, m) for t in (F16, BF16, F32) for m in (-1e4, -1e9, -1e10, -1e30, torch.finfo(t).min) if t is not F16 or m >= torch.finfo(F16).min]
# a workgroup of eight waves a row, of two, and rows in segments
SHAPES = [(6000, 1), (700, 40), (90000, 1)]


@pytest.mark.parametrize("v,many", SHAPES)
@pytest.mark.parametrize("dtype,mask", MASKS)
def test_finite_masks(dtype, mask, v, many):
    x, ids = masked(dtype, v, many, mask)
    for scale in (0.25, 0.5, 0.65, 1.0, 1.25):
        for top in (0, 7):
            check(x, ids, top, scale)


def far_rows(dtype, v, many, at):
    """Rows about `at`: equal logits, and some steps of the format apart."""
    g = gen(7)
    step = torch.finfo(dtype).eps * abs(at)
    x = at + torch.randint(-3, 4, (6, v), generator=g, device="cuda") * step
    x[0] = at
    x[1, ::5] = at / 2
    x[2, 100:] = -INF
    x[3, :v // 2] = 0.5
    ids = torch.tensor([0, 5, 3, v - 1, 8, 77], device="cuda")
    return x.to(dtype).repeat(many, 1), ids.repeat(many)


FAR = [(t, a) for t in (F16, BF16, F32) for a in (3e4, -3e4, 1e6, -1e6, 3e7, -3e7, -1e9, 1e10, -1e10, -3e10, -1e30, -1e31, 1e38) if t is not F16 or abs(a) < 65000]


@pytest.mark.parametrize("v,many", SHAPES)
@pytest.mark.parametrize("dtype,at", FAR)
def test_rows_far_from_zero(dtype, at, v, many):
    x, ids = far_rows(dtype, v, many, at)
    for scale in (0.3, 1.0, 1.25):
        check(x, ids, 5, scale)


def check_gradient(x, ids, scale, what="gh", into=None):
    """The gradient where lse and entropy are what the forward pass left.

    p has the relative error of log p: `sums`, half steps of 2^-24 of d and of its
    product, and of lse (as in `check`) up to the size from which a row is summed again.  log p and H have those errors themselves; four roundings of the terms, the
    results' own, and powers below 2^-126 are zero."""
    out, ref, (n, v) = score(x, ids, 0, scale), reference(x, ids, scale), x.shape
    g = torch.randn(n, generator=gen(11), device="cuda") if "g" in what else None
    h = torch.randn(n, generator=gen(12), device="cuda") if "h" in what else None
    raw = x.clone()
    d = torch.empty_like(x) if into is None else into
    z.zsmr_logprobs_grad(x, ids, out["lse"], out["entropy"], d, dlogprob=g, dentropy=h, scale=scale)
    ok = (ids >= 0) & (ids < v)
    gg = torch.where(ok, g.double(), 0.0)[:, None] if g is not None else torch.zeros(n, 1, device="cuda")
    hh = h.double()[:, None] if h is not None else torch.zeros(n, 1, device="cuda")
    hit = torch.zeros(n, v, device="cuda", dtype=torch.float64).scatter_(1, torch.where(ok, ids, 0)[:, None], 1.0)
    p, entropy = ref["p"], ref["entropy"][:, None]
    logp = torch.where(p > 0, ref["logp"], 0.0)
    want = scale * (gg * hit - p * (gg + hh * (logp + entropy)))
    want[ref["lse"] == -INF] = 0
    tol = sums(n, v)
    off = tol + 2.0 ** -24 * (5 * size(ref["lse"])[:, None].clamp(max={F32: 64, F16: 512, BF16: 4096}[x.dtype]) + 6 * logp.abs())
    terms = gg.abs() + hh.abs() * (logp.abs() + entropy)
    slack = scale * (p * (off * terms + hh.abs() * (off + tol * (1 + entropy))) + 2.0 ** -22 * (p * terms + gg.abs() * hit) + 2.0 ** -126 * (terms + 100 * hh.abs()))
    slack = slack + want.abs() * HALF_STEP[x.dtype] + (2.0 ** -25 if x.dtype is F16 else 0.0)
    bad = ~((d.double() - want).abs() <= slack)
    assert not bad.any(), (bad.any(1).nonzero()[:5, 0], d[bad][:5], want[bad][:5])
    return d, raw, out, g, h


@pytest.mark.parametrize("v,many", SHAPES)
@pytest.mark.parametrize("dtype,mask", MASKS)
def test_gradient_of_finite_masks(dtype, mask, v, many):
    x, ids = masked(dtype, v, many, mask)
    for scale in (0.25, 0.5, 0.65, 1.0, 1.25):
        check_gradient(x, ids, scale)


@pytest.mark.parametrize("v,many", SHAPES)
@pytest.mark.parametrize("dtype,at", FAR + [(t, a) for t in (F16, BF16, F32) for a in (40.0, -90.0, 300.0, -600.0, 1500.0, 6e3, -6e3)])
def test_gradient_of_rows_far_from_zero(dtype, at, v, many):
    x, ids = far_rows(dtype, v, many, at)
    for scale, what in ((0.3, "gh"), (1.0, "g"), (1.25, "h")):
        check_gradient(x, ids, scale, what)
    # in place, and through a view with rows apart
    d, raw, out, g, h = check_gradient(x, ids, 1.0)
    z.zsmr_logprobs_grad(x, ids, out["lse"], out["entropy"], x, dlogprob=g, dentropy=h)
    assert torch.equal(x, d)
    wide = torch.full((len(x), v + 9), 4.0, device="cuda", dtype=dtype)
    z.zsmr_logprobs_grad(raw, ids, out["lse"], out["entropy"], wide[:, 3:3 + v], dlogprob=g, dentropy=h)
    assert torch.equal(wide[:, 3:3 + v], d) and (wide[:, :3] == 4).all() and (wide[:, 3 + v:] == 4).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_the_smallest_and_largest_scales(dtype):
    """At 2^-100 all log probabilities are equal, at 2^100 the largest logits are all."""
    x = torch.randn(5, 6000, generator=gen(13), device="cuda").to(dtype)
    x[1] = x[1].clamp(max=0.5)          # a tie of many
    x[2] -= 50.0
    x[3, ::2] = -INF
    x[4] = torch.finfo(dtype).min
    ids = torch.tensor([0, int(x[1].argmax()), 7, 1, -1], device="cuda")
    for scale in (2.0 ** -100, 2.0 ** 100):
        check(x, ids, 9, scale)
        check_gradient(x, ids, scale)


def test_nan_and_infinity_in_far_rows():
    x = torch.full((6, 90000), -1e9, device="cuda")
    x[0, 77] = float("nan")
    x[1, 80000] = INF
    x[2] = 1e9
    x[2, 5] = float("nan")
    x[3, 40000:] = -INF
    x[4, 0] = float("nan")
    x[4, 1:] = INF
    out = score(x, torch.zeros(6, device="cuda", dtype=torch.int64), 3)
    assert torch.isnan(out["lse"][[0, 2, 4]]).all() and torch.isnan(out["entropy"][[0, 2, 4]]).all() and torch.isnan(out["logprob"][[0, 2, 4]]).all()
    assert out["lse"][1] == INF and torch.equal(out["top_ids"], best(x, 3))
    good = [3, 5]
    check(x[good], torch.tensor([5, 89999], device="cuda"), 3, 1.0)
    d = torch.empty_like(x)
    one = torch.ones(6, device="cuda")
    z.zsmr_logprobs_grad(x, torch.zeros(6, device="cuda", dtype=torch.int64), out["lse"], out["entropy"], d, one, one)
    assert torch.isnan(d[[0, 2, 4]]).all() and torch.isfinite(d[good]).all()


def test_far_rows_captured():
    """Rows move between ordinary, masked and far ones from replay to replay."""
    x, ids = masked(BF16, 90000, 1, -1e9)
    out = {k: torch.empty(8, device="cuda") for k in ("logprob", "lse", "entropy")}
    d, g = torch.empty_like(x), torch.ones(8, device="cuda")
    ws = torch.empty(z.zsmr_logprobs_workspace(8, 90000, 0), device="cuda", dtype=torch.uint8)

    def run():
        z.zsmr_logprobs(x, ids, out["logprob"], out["lse"], out["entropy"], ws)
        z.zsmr_logprobs_grad(x, ids, out["lse"], out["entropy"], d, dlogprob=g, dentropy=g)

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for mask in (-1e30, -INF, torch.finfo(BF16).min, -1e9, 1e10):
        x.copy_(masked(BF16, 90000, 1, mask)[0])
        ws.fill_(0xff)
        graph.replay()
        got = [t.clone() for t in (*out.values(), d)]
        torch.cuda.synchronize()
        run()
        assert all(torch.equal(a, b) for a, b in zip(got, (*out.values(), d)))
        check(x, ids, 4, 1.0)
        check_gradient(x, ids, 1.0)


@pytest.mark.parametrize("v,many", SHAPES)
def test_rows_about_the_last_near_reference(v, many):
    """Products with log2 e of 2^20 and some powers more or fewer, of either sign."""
    edge = 2.0 ** 20 / 1.4426950408889634
    k = torch.tensor([-300.0, -100.0, -89.0, -60.0, -45.0, -44.0, -20.0, 0.0, 3.0, 20.0, 44.0, 45.0, 60.0, 89.0, 100.0, 300.0], device="cuda")
    at = torch.cat([edge + k, -edge + k])
    x = (at[:, None] + torch.randn(32, v, generator=gen(14), device="cuda") * 3).repeat(many, 1)
    ids = (torch.arange(32 * many, device="cuda") * 37) % v
    check(x, ids, 3, 1.0)
    check_gradient(x, ids, 1.0)
