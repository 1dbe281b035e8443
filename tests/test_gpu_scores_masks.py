"""Scores of logits with finite masks and of rows far from zero, against
64 bits.

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

from tests.test_gpu_scores import BF16, F16, F32, INF, best, gen, near, score

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
