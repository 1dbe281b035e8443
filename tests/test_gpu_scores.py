"""Scores of logits on the GPU against 64 bits: log probabilities of given tokens,
entropy, top alternatives, and the gradient.

Tolerances.  A term e = exp(z - ref) has the roundings of scale * s, of the difference
and of its product with log2 e, each half a step of a value of at most |z| + |ref| or
40 (smaller terms do not count), and the power's own: its relative error is below
2^-24 (2 (|z| + |ref|) + 100).  A lane adds vocab / 256 of them one by one, half a step
each at worst, and the joins a dozen more.  lse, logprob and entropy are sums of a few
such numbers.
"""
import pytest
import torch

import zero_sharded_mixed_reduce_amd as z

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (F16, BF16, F32)}
INF = float("inf")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def reference(x, ids, scale):
    """In 64 bits: values, and the probabilities."""
    s = torch.tensor(scale, dtype=F32).double().item()
    v = x.double() * s
    v = torch.where(v < -2.3e38, -INF, v)
    top = v.amax(1, keepdim=True)
    none = top[:, 0] == -INF
    e = torch.where(none[:, None], 0.0, (v - top).exp())
    lse = torch.where(none, -INF, e.sum(1).log() + top[:, 0])
    logp = torch.where(none[:, None], -INF, v - lse[:, None])
    p = logp.exp()
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(1)
    logprob = torch.zeros_like(lse)
    if ids is not None:
        ok = (ids >= 0) & (ids < x.shape[1])
        got = logp.gather(1, torch.where(ok, ids, 0).long()[:, None])[:, 0]
        logprob = torch.where(ok, got, 0.0)
    return {"lse": lse, "logprob": logprob, "entropy": entropy, "logp": logp, "p": p}


def bound(x, scale):
    """Of lse, logprob and entropy of each row."""
    v = x.double() * scale
    top = torch.where(torch.isfinite(v) & (v > -2.3e38), v, 0.0).abs().amax(1)
    return 2.0 ** -24 * (x.shape[1] / 256 + 2 * (4 * top + 100) + 30)


def best(x, k):
    """Indices of the k largest, ties by the lowest index; -1 where there are no more."""
    v = torch.where(torch.isnan(x), -INF, x.double() + 0.0)
    v, at = torch.sort(v, dim=1, descending=True, stable=True)
    return torch.where(v > -INF, at, -1)[:, :k]


def near(got, want, tol):
    got = got.double()
    ok = torch.where(torch.isfinite(want), (got - want).abs() <= tol, (got == want) | (torch.isnan(got) & torch.isnan(want)))
    assert ok.all(), (got[~ok][:5], want[~ok][:5])


def score(x, ids, top=0, scale=1.0, id_type=torch.int64):
    n, v = x.shape
    size = z.zsmr_logprobs_workspace(n, v, top)
    ws = torch.full((size + 64,), 0x5a, device="cuda", dtype=torch.uint8)
    out = {k: torch.full((n,), 9.0, device="cuda") for k in ("logprob", "lse", "entropy")}
    if top:
        out["top_ids"] = torch.full((n, top), 77, device="cuda", dtype=id_type)
        out["top_logprobs"] = torch.full((n, top), 9.0, device="cuda")
    z.zsmr_logprobs(x, ids, out["logprob"] if ids is not None else None, out["lse"], out["entropy"], ws[:size], top_ids=out.get("top_ids"),
                    top_logprobs=out.get("top_logprobs"), scale=scale)
    assert (ws[size:] == 0x5a).all(), "written past the workspace"
    return out


def check(x, ids, top=0, scale=1.0, **kw):
    out, ref, tol = score(x, ids, top, scale, **kw), reference(x, ids, scale), bound(x, scale)
    near(out["lse"], ref["lse"], tol)
    near(out["entropy"], ref["entropy"], tol)
    if ids is not None:
        near(out["logprob"], ref["logprob"], tol)
    if top:
        at = best(x, top)
        assert torch.equal(out["top_ids"].long(), at)
        want = torch.where(at >= 0, ref["logp"].gather(1, at.clamp(min=0)), -INF)
        near(out["top_logprobs"], want, tol[:, None])
    return out, ref


def logits(seed, n, v, dtype, sigma=2.0):
    g = gen(seed)
    return torch.randn(n, v, generator=g, device="cuda").mul_(sigma).to(dtype), torch.randint(-1, v, (n,), generator=g, device="cuda")


SIZES = [(1, 1), (3, 2), (1, 5), (2, 63), (3, 64), (5, 65), (3, 511), (2, 512), (5, 513), (7, 2047), (4, 2049), (3, 4097), (1, 8193), (5, 50257), (1, 128256),
         (16, 128256), (1025, 700), (300, 5000)]


@pytest.mark.parametrize("n,v", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_sizes(n, v, dtype):
    x, ids = logits(n * 31 + v, n, v, dtype)
    for top in sorted({0, 1, min(v, 20), min(v, 64)}):
        check(x, ids, top)


@pytest.mark.parametrize("scale", [0.25, 1.25, 1.0 / 0.7, 30.0])
def test_scale_orders_nothing_anew(scale):
    for dtype in (BF16, F32):
        x, ids = logits(4, 9, 3001, dtype)
        check(x, ids, 20, scale)


def test_strides_and_id_formats():
    x, ids = logits(5, 12, 1007, BF16)
    wide = torch.full((12, 1500), INF, device="cuda", dtype=BF16)
    wide[:, 3:1010] = x
    for view in (wide[:, 3:1010], x.flip(0).contiguous().flip(0)):
        check(view, ids, 7)
        check(view, ids.int(), 7, id_type=torch.int32)
    check(x, None, 3)


def test_ties_and_signed_zeros():
    x = torch.zeros(4, 5000, device="cuda")
    x[1, ::3] = -0.0
    x[2] = (torch.arange(5000, device="cuda") % 7).float()
    x[3] = -x[2]
    for dtype in (F32, BF16):
        check(x.to(dtype), torch.zeros(4, device="cuda", dtype=torch.int64), 64)


def test_rising_and_falling_rows():
    """Every logit is a new best one, or none is."""
    up = torch.arange(20000, device="cuda").float() / 1000
    x = torch.stack([up, up.flip(0), torch.where(up > 19.9, 50.0, up)])
    check(x, torch.tensor([0, 19999, 5], device="cuda"), 64)
    many = x.repeat(400, 1)         # whole rows of a workgroup
    check(many, torch.arange(1200, device="cuda"), 33)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("many", [1, 300])
def test_masked_rows(dtype, many):
    """Masks of -infinity and of the lowest value, rows that keep one, few or none."""
    low = torch.finfo(dtype).min
    x, _ = logits(7, 8, 6000, dtype)
    x[0, 1:] = -INF
    x[1] = -INF
    x[2] = -INF
    x[2, [5, 4000, 5999]] = 1.5
    x[3, ::2] = -INF
    x[4, 100:] = low
    x[5, :5990] = -INF
    x[6, :4096] = -INF
    x = x.repeat(many, 1)
    ids = torch.tensor([0, 3, 4000, 1, 5, 5995, 0, -1], device="cuda").repeat(many)
    check(x, ids, 8)
    if dtype is not F16:            # the lowest value alone counts as masked too
        x[:8] = low
        out = score(x[:8], ids[:8], 2)
        assert (out["lse"] == -INF).all() and (out["entropy"] == 0).all() and (out["logprob"][:7] == -INF).all() and out["logprob"][7] == 0


@pytest.mark.parametrize("v", [700, 90000])
def test_alternatives_of_a_masked_row(v):
    """Lowest values are alternatives (they are above -infinity) of no probability."""
    x, _ = logits(17, 3, v, BF16)
    x[1] = torch.finfo(BF16).min
    x[2, 1:] = torch.finfo(BF16).min
    out = score(x, None, 6)
    assert torch.equal(out["top_ids"], best(x, 6))
    assert (out["top_logprobs"][1] == -INF).all() and (out["top_logprobs"][2, 1:] == -INF).all()
    # the reference is x log2 e rounded once, half a step of a number below 16
    assert x[2, 0].abs() < 11 and out["top_logprobs"][2, 0].abs() <= 2.0 ** -24 * 16


def test_rows_past_32_bits():
    """The last rows lie more than 2^32 elements from the first."""
    n, v, stride = 2060, 1000, 1 << 21
    try:
        big = torch.empty(n * stride, device="cuda", dtype=BF16)
    except torch.cuda.OutOfMemoryError:
        pytest.skip("needs 9 GB")
    x, ids = logits(19, n, v, BF16)
    far = big.view(n, stride)[:, :v]
    far.copy_(x)
    got, want = score(far, ids, 5), score(x, ids, 5)
    assert all(torch.equal(got[k], want[k]) for k in want)
    g = torch.randn(n, device="cuda", generator=gen(20))
    dx = torch.empty_like(x)
    z.zsmr_logprobs_grad(x, ids, want["lse"], want["entropy"], dx, g, -g)
    z.zsmr_logprobs_grad(far, ids, want["lse"], want["entropy"], far, g, -g)
    assert torch.equal(far, dx)


def test_calls_on_two_streams_at_once():
    x, ids = logits(18, 40, 128256, BF16)
    want = score(x, ids, 9)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    size = z.zsmr_logprobs_workspace(40, 128256, 9)
    for stream in streams:
        out = {k: torch.full_like(t, 5) for k, t in want.items()}
        got.append((out, torch.empty(size, device="cuda", dtype=torch.uint8)))
    torch.cuda.synchronize()
    for _ in range(5):
        for stream, (out, ws) in zip(streams, got):
            z.zsmr_logprobs(x, ids, out["logprob"], out["lse"], out["entropy"], ws, top_ids=out["top_ids"], top_logprobs=out["top_logprobs"],
                            stream=stream)
    torch.cuda.synchronize()
    for out, _ in got:
        assert all(torch.equal(out[k], want[k]) for k in want)


def test_nan_and_infinity():
    x, ids = logits(8, 6, 3000, F32)
    x[1, 2999] = float("nan")
    x[3, 7] = INF
    x[4] = float("nan")
    out = score(x, ids.clamp(min=0), 5)
    for k in ("lse", "entropy", "logprob"):
        assert torch.isnan(out[k][[1, 4]]).all()
    assert out["lse"][3] == INF and torch.isnan(out["entropy"][3])
    good = [0, 2, 5]
    check(x[good], ids[good], 5)
    assert torch.equal(out["top_ids"], best(x, 5))
    assert (out["top_ids"][4] == -1).all() and out["top_ids"][3, 0] == 7


def test_rows_that_shift_far():
    """Large logits, and the largest at the end."""
    x, ids = logits(9, 5, 9000, F32, sigma=50.0)
    x[1] += 1e4
    x[2] -= 1e4
    x[3, -1] = 3e5
    x[4, 4500] = 700.0
    check(x, ids, 10)


def test_ids_outside_are_padding():
    x, _ = logits(10, 4, 100, BF16)
    ids = torch.tensor([-1, 100, 1 << 40, 99], device="cuda")
    out, _ = check(x, ids)
    assert (out["logprob"][:3] == 0).all()


def gradient(x, ids, g, h, scale=1.0, out=None):
    s = score(x, ids, 0, scale)
    d = torch.empty_like(x) if out is None else out
    z.zsmr_logprobs_grad(x, ids, s["lse"], s["entropy"], d, dlogprob=g, dentropy=h, scale=scale)
    return d


def check_gradient(x, ids, g, h, scale=1.0, out=None):
    ref, n, v = reference(x, ids, scale), *x.shape
    tol, raw = bound(x, scale), x.clone()
    d = gradient(x, ids, g, h, scale, out)
    gg = torch.zeros(n, device="cuda", dtype=torch.float64) if g is None else g.double()
    hh = torch.zeros_like(gg) if h is None else h.double()
    hit = torch.zeros(n, v, device="cuda", dtype=torch.float64)
    if g is not None:
        ok = (ids >= 0) & (ids < v)
        gg = torch.where(ok, gg, 0.0)
        hit.scatter_(1, torch.where(ok, ids, 0).long()[:, None], 1.0)
    slope = ref["p"] * (gg[:, None] + hh[:, None] * (ref["logp"].clamp(min=-1e9) + ref["entropy"][:, None]))
    want = scale * (gg[:, None] * hit - slope)
    want[ref["lse"] == -INF] = 0
    # p is off by the error of lse, log p and H by theirs; four roundings of the sums; the result's own
    size = ref["p"] * (gg.abs()[:, None] + hh.abs()[:, None] * (1 + ref["logp"].clamp(min=-1e9).abs() + ref["entropy"][:, None])) + gg.abs()[:, None] * hit
    slack = scale * size * (4 * tol[:, None] + 2.0 ** -21) + want.abs() * HALF_STEP[x.dtype] + 2.0 ** -25 * (x.dtype is F16) + 1e-37
    bad = (d.double() - want).abs() > slack
    assert not bad.any(), (d[bad][:5], want[bad][:5])
    return d, raw


@pytest.mark.parametrize("n,v", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_gradient(n, v, dtype):
    x, ids = logits(n + v, n, v, dtype)
    g, h = torch.randn(n, generator=gen(1), device="cuda"), torch.randn(n, generator=gen(2), device="cuda")
    check_gradient(x, ids, g, h, 0.8)
    check_gradient(x, ids.int(), g, None)
    check_gradient(x, None, None, h)


def test_gradient_of_masked_rows_and_in_place():
    x, _ = logits(11, 5, 5000, F32)
    x[0, 1:] = -INF
    x[1] = -INF
    x[2, ::2] = -INF
    x[3, 1:] = torch.finfo(F32).min
    ids = torch.tensor([0, 7, 2, 9, -1], device="cuda")     # 2 and 9 are masked: p = 0, the one-hot term stays
    g, h = torch.randn(5, device="cuda"), torch.randn(5, device="cuda")
    d, raw = check_gradient(x, ids, g, h)
    assert (d[1] == 0).all()
    gradient(x, ids, g, h, out=x)
    assert torch.equal(x, d)
    wide = torch.full((5, 5100), 4.0, device="cuda")
    gradient(raw, ids, g, h, out=wide[:, 7:5007])
    assert torch.equal(wide[:, 7:5007], d) and (wide[:, :7] == 4).all() and (wide[:, 5007:] == 4).all()


def test_gradient_without_weights_is_zero_and_nan_stays_in_its_row():
    x, ids = logits(12, 4, 900, BF16)
    assert (gradient(x, ids, None, None) == 0).all()
    x[2, 5] = float("nan")
    d = gradient(x, ids, torch.ones(4, device="cuda"), torch.ones(4, device="cuda"))
    assert torch.isnan(d[2]).all() and torch.isfinite(d[[0, 1, 3]]).all()


def test_gradient_against_differences():
    """Each logit moves by 2^-6 in the sign of its gradient, from a grid that fp32 holds
    with the step added: the two ends differ by the slope, the sum of the magnitudes,
    up to the step's square times the third derivative, below 2^-12 of it for a
    function of probabilities and log probabilities up to 10."""
    n, v, step = 20, 300, 2.0 ** -6
    x = (torch.randn(n, v, generator=gen(3), device="cuda") * 64).round() / 64
    ids = torch.randint(v, (n,), generator=gen(4), device="cuda")
    for wg, wh in ((1.0, 0.0), (0.0, 1.0), (0.5, -2.0)):
        g, h = torch.full((n,), wg, device="cuda"), torch.full((n,), wh, device="cuda")
        d = gradient(x, ids, g, h)
        move = d.sign() * step

        def total(y):
            s = score(y, ids)
            return wg * s["logprob"].double() + wh * s["entropy"].double()

        slope, want = (total(x + move) - total(x - move)), (2 * step * d.double().abs()).sum(1)
        assert ((slope - want).abs() <= 0.02 * want + 1e-5).all()


def test_captured_and_on_another_stream():
    x, ids = logits(13, 40, 7001, BF16)
    g, h, d = torch.ones(40, device="cuda"), torch.ones(40, device="cuda"), torch.empty_like(x)
    lp, lse, ent = torch.empty(3, 40, device="cuda")
    at, val = torch.empty(40, 9, device="cuda", dtype=torch.int64), torch.empty(40, 9, device="cuda")
    ws = torch.empty(z.zsmr_logprobs_workspace(40, 7001, 9), device="cuda", dtype=torch.uint8)

    def run(stream=None):
        z.zsmr_logprobs(x, ids, lp, lse, ent, ws, top_ids=at, top_logprobs=val, stream=stream)
        z.zsmr_logprobs_grad(x, ids, lse, ent, d, dlogprob=g, dentropy=h, stream=stream)

    run()
    everything = (lp, lse, ent, at, val, d)
    first = [t.clone() for t in everything]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, everything))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in range(4):
        x.copy_(logits(50 + seed, 40, 7001, BF16)[0])
        ws.fill_(0xff)
        graph.replay()
        got = [t.clone() for t in everything]
        torch.cuda.synchronize()
        run()
        assert all(torch.equal(a, b) for a, b in zip(got, everything))


def test_positions_beyond_32_bits():
    """The last row of a large batch starts past 2^32 elements."""
    n, v = 2100, 1 << 21
    x = torch.zeros(n, v, device="cuda", dtype=F16)
    x[-1, 5] = 20.0
    x[-1, v - 1] = 21.0
    ids = torch.full((n,), v - 1, device="cuda")
    out = score(x, ids, 2)
    near(out["lse"][:-1], torch.full((n - 1,), float(torch.tensor(float(v)).double().log()), device="cuda", dtype=torch.float64), 1e-4)
    check(x[-1:], ids[-1:], 2)
    assert out["top_ids"][-1].tolist() == [v - 1, 5] and out["top_ids"][0].tolist() == [0, 1]
    d = torch.empty(1, v, device="cuda", dtype=F16)
    z.zsmr_logprobs_grad(x[-1:], ids[-1:], out["lse"][-1:], out["entropy"][-1:], d, dlogprob=torch.ones(1, device="cuda"))
    z.zsmr_logprobs_grad(x, ids, out["lse"], out["entropy"], x, dlogprob=torch.ones(n, device="cuda"))
    assert torch.equal(x[-1:], d)
