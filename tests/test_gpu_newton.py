"""The orthogonalised update and its shard step on the GPU, against the same
polynomial in 64 bits.

Tolerances.  The kernels hold every matrix in 22 bits (an error of at most 2^-22 of
each element, and of half of fp16's smallest step, 2^-25, over the power of two the
matrix is held times, 2^14 at least for these polynomials: 2^-39), leave out products
of 2^-22, and sum 3 k / 32 partial sums of a product in fp32.  ``polynomial`` with
``noise`` makes the 64-bit computation with errors of these sizes, drawn at
random, at every place where the kernels have one; the distance of that from the
exact result, the largest of eight drawings (a single drawing says little of a
matrix of few elements), four times, is what a result may be off in the 2-norm, and
ten times its share of an element (a normal error passes five of its deviations
once in two million) what an element may, besides half a step of the result's own
format.
"""
import math

import pytest
import torch

import zero_sharded_mixed_reduce_amd as z
from zero_sharded_mixed_reduce_amd.ops import NS_COEFS

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (F16, BF16, F32)}
TINY = {F16: 2.0 ** -25, BF16: 0.0, F32: 0.0}       # half of the smallest step of a format


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def polynomial(x, coefs=NS_COEFS, eps=1e-7, noise=None, groups=()):
    """In 64 bits; noise: a generator of rounding errors; groups: steps that share one
    X X^T, as the kernels' do for 16-bit results of matrices that are not square."""
    x = x.double()
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT.contiguous() if tall else x.contiguous()
    norm = x.square().sum((-2, -1), keepdim=True).sqrt() + eps
    x = torch.where(norm == 0, 0.0, x / norm)

    def held(m):
        if noise is None:
            return m
        u = torch.rand(m.shape, generator=noise, device="cuda", dtype=torch.float64) * 2 - 1
        return m + u * (m.abs() * 2.0 ** -21 + 2.0 ** -39)

    def product(p, q):
        r = p @ q
        if noise is None:
            return r
        size = 2.0 ** -24 * (3 * p.shape[-1] / 32 + 1) ** 0.5 + 2.0 ** -22
        return r + (p.abs() @ q.abs()) * size * (torch.rand(r.shape, generator=noise, device="cuda", dtype=torch.float64) * 2 - 1)

    coefs = list(coefs)
    groups = list(groups) or [1] * len(coefs)
    while coefs:
        x = held(x)
        gram, total, total_a = held(product(x, x.mT.contiguous())), None, 1.0
        now, coefs = coefs[:groups[0]], coefs[groups[0]:]
        groups = groups[1:] or [2]
        for j, (a, b, c) in enumerate(now):
            if noise is not None:       # the coefficients, and the last additions, in fp32
                a, b, c = (k * (1 + 2.0 ** -23 * (2 * float(torch.rand((), generator=noise, device="cuda")) - 1)) for k in (a, b, c))
            part = held(b * gram + c * product(gram, gram))
            # the product of a I + part over the steps is total_a I + total
            total = part if total is None else held(total_a * part + a * total + product(total, part))
            total_a *= a
            if j + 1 < len(now):
                half = held(a * gram + product(gram, part))
                gram = held(a * half + product(half, part))
        x = total_a * x + product(total, x)
    return x.mT if tall else x


def grouped(x, dtype, coefs):
    """The longest groups of steps a call may form."""
    n, m = max(x.shape[-2:]), min(x.shape[-2:])
    return (3, 2) if dtype is not F32 and 5 * n >= 6 * m and len(coefs) > 1 else ()


def allowed(x, dtype, coefs=NS_COEFS, eps=1e-7):
    """The exact result, and the errors a result of `dtype` may have: of each
    element, and in the 2-norm of each matrix."""
    exact = polynomial(x, coefs, eps)
    off = torch.stack([(polynomial(x, coefs, eps, gen(k), grouped(x, dtype, coefs)) - exact).square().sum((-2, -1), keepdim=True).sqrt() for k in range(8)]).amax(0)
    step = exact.abs() * HALF_STEP[dtype] + TINY[dtype]
    each = step + 10 * 4 * off / (x.shape[-1] * x.shape[-2]) ** 0.5
    return exact, each * 1.001 + 1e-30, 4 * off + step.square().sum((-2, -1), keepdim=True).sqrt() + 1e-30


def agrees(out, x, coefs=NS_COEFS, eps=1e-7):
    exact, each, whole = allowed(x, out.dtype, coefs, eps)
    d = (out.double() - exact).abs()
    assert torch.isfinite(out).all()
    assert (d <= each).all(), (float((d / each).max()), tuple(x.shape))
    assert (d.square().sum((-2, -1), keepdim=True).sqrt() <= whole).all()


def call(x, out, **kw):
    rows, cols = x.shape[-2:]
    size = z.zsmr_orthogonalize_workspace(rows, cols, x.shape[0] if x.dim() == 3 else 1)
    ws = torch.full((size + 256,), 0x5a, device="cuda", dtype=torch.uint8)
    z.zsmr_orthogonalize(x, out, ws[:size], **kw)
    assert (ws[size:] == 0x5a).all(), "written past the workspace"
    return out


def matrices(seed, *shape, dtype=F32, rank=None):
    g = gen(seed)
    x = torch.randn(*shape, generator=g, device="cuda")
    if rank:
        x = x * 0.01 + torch.randn(*shape[:-1], rank, generator=g, device="cuda") @ torch.randn(*shape[:-2], rank, shape[-1], generator=g, device="cuda")
    return x.to(dtype)


SIZES = [(1, 1), (1, 9), (7, 1), (2, 3), (16, 16), (31, 33), (33, 31), (64, 64), (65, 200), (127, 129), (128, 128), (129, 128), (200, 65),
         (256, 384), (384, 130), (64, 128), (96, 250), (250, 96), (64, 512), (33, 480), (128, 160), (1, 700), (700, 2), (1, 1024), (1, 1100), (1500, 3), (333, 1001), (1100, 260)]


@pytest.mark.parametrize("rows,cols", SIZES)
def test_sizes(rows, cols):
    x = matrices(rows * 10007 + cols, rows, cols)
    agrees(call(x, torch.empty_like(x)), x)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("out", [F16, BF16, F32])
def test_formats(dtype, out):
    for shape in ((70, 95), (95, 70)):
        x = matrices(3, *shape, dtype=dtype)
        agrees(call(x, torch.empty(shape, device="cuda", dtype=out)), x)


@pytest.mark.parametrize("count,rows,cols", [(1, 40, 50), (3, 64, 64), (5, 130, 70), (24, 64, 64), (300, 3, 5), (9, 128, 300), (17000, 2, 2)])
def test_stacks(count, rows, cols):
    x = matrices(count, count, rows, cols, dtype=BF16)
    agrees(call(x, torch.empty(count, rows, cols, device="cuda", dtype=F16)), x)


def test_more_matrices_than_a_group_holds():
    x = matrices(8, 70, 512, 1024, dtype=BF16)          # 64 of them are 2^25 elements
    agrees(call(x, torch.empty_like(x)), x)


@pytest.mark.parametrize("rows,cols,count", [(200, 240, 1), (130, 700, 3), (700, 130, 2), (513, 1100, 1), (1100, 513, 1), (1290, 1290, 1), (640, 640, 7),
                                             (2100, 300, 1), (65, 6000, 1), (130, 2100, 2), (2300, 200, 1), (513, 2050, 1), (1000, 513, 20),
                                             (1500, 6100, 1), (9000, 2048, 1), (333, 5001, 3)])
def test_steps_in_groups_and_split_products(rows, cols, count):
    for rank in (None, 20):
        x = matrices(rows + cols, count, rows, cols, rank=rank)
        for dtype in (F16, F32):
            agrees(call(x, torch.empty(x.shape, device="cuda", dtype=dtype)), x)


@pytest.mark.parametrize("coefs", [((2.0, -1.5, 0.5),) * 7, ((3.9, -5.9, 2.5), (3.4, -4.6, 1.9)), ((20.0, -30.0, 12.0), (0.15, 0.0, 0.0), (1.5, -0.5, 0.0)),
                                   ((3.4445, -4.7750, 2.0315),) * 4, ((1.0, 0.0, 0.0),) * 3, ((-2.0, 1.5, -0.5),) * 5])
def test_other_polynomials_in_groups(coefs):
    x = matrices(9, 140, 2000)
    agrees(call(x, torch.empty(140, 2000, device="cuda", dtype=F16), coefs=coefs), x, coefs)


@pytest.mark.parametrize("rows,cols", [(40, 72), (72, 40), (129, 131)])
def test_strides(rows, cols):
    """Rows apart, matrices interleaved or repeated, odd addresses; what lies between stays."""
    big = matrices(5, rows, 3, cols + 5)
    x = big.transpose(0, 1)[:, :, 3:3 + cols]
    room = torch.full((rows, 3, cols + 7), 7.0, device="cuda", dtype=BF16)
    out = room.transpose(0, 1)[:, :, 5:5 + cols]
    agrees(call(x, out), x)
    out.fill_(7.0)
    assert (room == 7.0).all()
    same = big[:, 0, 1:1 + cols].expand(3, rows, cols)
    many = torch.empty(3, rows, cols, device="cuda", dtype=F16)
    agrees(call(same, many), same)
    assert torch.equal(many[0], many[2])


def test_decaying_spectra():
    """Singular values down to nothing, which the first passes raise the most."""
    for rank in (1, 4, 40):
        x = matrices(rank, 96, 160, rank=rank)
        agrees(call(x, torch.empty_like(x)), x)
    x = torch.ones(50, 60, device="cuda")               # rank one exactly
    agrees(call(x, torch.empty_like(x)), x)


@pytest.mark.parametrize("size", [1e-30, 1e-6, 1.0, 1e30])
def test_magnitudes(size):
    x = matrices(6, 50, 80) * size
    agrees(call(x, torch.empty_like(x), eps=0.0), x, eps=0.0)
    agrees(call(x, torch.empty_like(x)), x)


def test_zeros_nan_and_infinity_stay_in_their_matrix():
    x = matrices(7, 6, 66, 40)
    x[1] = 0
    x[2, 5, 7] = float("nan")
    x[4, 65, 39] = float("inf")
    for eps in (0.0, 1e-7):
        out = call(x, torch.empty_like(x), eps=eps)
        good = [0, 3, 5]
        agrees(out[good], x[good], eps=eps)
        assert (out[1] == 0).all() and torch.isnan(out[2]).all() and torch.isnan(out[4]).all()


@pytest.mark.parametrize("coefs", [((1.5, -0.5, 0.0),), ((2.0, -1.5, 0.5),) * 12, ((4.0, -6.0, 2.6), (3.9, -5.9, 2.5), (3.4, -4.6, 1.9)),
                                   ((0.0, 0.0, 0.0), (3.0, -3.0, 1.0)), ((1.0, 0.0, 0.0),), ((100.0, 0.0, 0.0), (0.01, 0.0, 0.0)), ((1.875, -1.25, 0.375),) * 16])
def test_other_polynomials(coefs):
    x = matrices(8, 48, 60)
    agrees(call(x, torch.empty_like(x), coefs=coefs), x, coefs)


def test_the_same_bits_again_on_another_stream_and_captured():
    x, out = matrices(9, 3, 200, 333), torch.empty(3, 200, 333, device="cuda")
    ws = torch.empty(z.zsmr_orthogonalize_workspace(200, 333, 3), device="cuda", dtype=torch.uint8)
    z.zsmr_orthogonalize(x, out, ws)
    first = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    z.zsmr_orthogonalize(x, out, ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z.zsmr_orthogonalize(x, out, ws)
    for seed in range(4):
        x.copy_(matrices(20 + seed, 3, 200, 333))
        ws.fill_(0xff)
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        z.zsmr_orthogonalize(x, out, ws)
        assert torch.equal(got, out)
    agrees(out, x)


@pytest.mark.parametrize("count,rows,cols", [(30, 64, 48), (2, 100, 128), (3, 333, 200), (40, 1000, 1000)])
def test_in_place(count, rows, cols):
    x = matrices(11, count, rows, cols, dtype=BF16)
    want = call(x, torch.empty_like(x))
    call(x, x)
    assert torch.equal(x, want)


@pytest.mark.parametrize("rows,cols", [(40, 72), (130, 150)])
def test_matrices_past_32_bits(rows, cols):
    far = (1 << 32) + 24
    try:
        big = torch.empty(far + rows * cols, device="cuda", dtype=BF16)
    except torch.cuda.OutOfMemoryError:
        pytest.skip("needs 9 GB")
    x = matrices(13, 2, rows, cols, dtype=BF16)
    apart = big.as_strided((2, rows, cols), (far, cols, 1))
    apart.copy_(x)
    want = call(x, torch.empty_like(x))
    assert torch.equal(call(apart, torch.empty_like(x)), want)
    call(x, apart)
    assert torch.equal(apart, want)


def test_calls_at_once_and_graphs_that_share_a_workspace():
    x = [matrices(12 + k, 2, 150, 1700) for k in range(2)]
    want = [call(t, torch.empty_like(t)) for t in x]
    size = z.zsmr_orthogonalize_workspace(150, 1700, 2)
    out, ws = [torch.zeros_like(t) for t in x], [torch.empty(size, device="cuda", dtype=torch.uint8) for _ in x]
    streams = [torch.cuda.Stream() for _ in x]
    torch.cuda.synchronize()
    for _ in range(4):
        for k, stream in enumerate(streams):
            z.zsmr_orthogonalize(x[k], out[k], ws[k], stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(out, want))
    graphs = [torch.cuda.CUDAGraph() for _ in x]
    for k, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            z.zsmr_orthogonalize(x[k], out[k], ws[0])
    for turn in range(3):
        for o in out:
            o.zero_()
        for graph in graphs if turn % 2 else graphs[::-1]:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(out, want))


# ---------------------------------------------------------------- shard step --
def muon(ctx, rank, unit, begin, rows, cols, count, s, **kw):
    size = z.zsmr_orthogonalize_workspace(rows, cols, count)
    ws = torch.full((size + 256,), 0x5a, device="cuda", dtype=torch.uint8)
    z.zero_muon_step(ctx, rank, unit, begin, rows, cols, count, s["grads"], s["grads"].shape[1], s["base"], s["master"], s["momentum"],
                     s["p16"], ws[:size], **kw)
    assert (ws[size:] == 0x5a).all(), "written past the workspace"


def state(seed, world, length, dtype, base=0):
    g = gen(seed)
    return {"grads": torch.randn(world, length + base, generator=g, device="cuda").mul_(1e-3).to(dtype), "base": base,
            "master": torch.randn(length, generator=g, device="cuda") * 0.02, "momentum": torch.randn(length, generator=g, device="cuda") * 1e-3,
            "p16": torch.full((length,), 3.0, device="cuda", dtype=dtype)}


def check_step(ctx, rank, unit, begin, rows, cols, count, s, lr=0.02, beta=0.9, weight_decay=0.1, scale=1.5, nesterov=True):
    n = rows * cols * count
    part = slice(begin, begin + n)
    before = {k: s[k].clone() for k in ("master", "momentum", "p16")}
    muon(ctx, rank, unit, begin, rows, cols, count, s, lr=lr, beta=beta, weight_decay=weight_decay, scale=scale, nesterov=nesterov)
    # reduce and momentum have one fp32 rounding an operation
    world, at = s["grads"].shape[0], s["base"] + begin
    g = s["grads"][0, at:at + n].float()
    for r in range(1, world):
        g = g + s["grads"][r, at:at + n].float()
    g = g / torch.full_like(g, world)       # a division: by a number torch multiplies by its reciprocal
    b = torch.tensor(beta, device="cuda", dtype=F32)
    m = b * before["momentum"][part] + g
    assert torch.equal(s["momentum"][part], m)
    u = (g + b * m if nesterov else m).view(count, rows, cols)
    exact, each, _ = allowed(u, F16)        # steps in groups, as for a 16-bit result
    old = before["master"][part].double()
    want = old * (1 - lr * weight_decay) - lr * scale * exact.reshape(-1)
    # three roundings: of master times decay, of rate times update, of the difference; constants are within half a step
    tol = lr * scale * each.reshape(-1) + 2.0 ** -24 * (2 * old.abs() + 2 * lr * scale * exact.reshape(-1).abs() + want.abs()) + 1e-30
    assert ((s["master"][part].double() - want).abs() <= tol).all()
    assert torch.equal(s["p16"][part], s["master"][part].to(s["p16"].dtype))
    for k in before:        # what is not a matrix of the call stays
        before[k][part] = s[k][part]
        assert torch.equal(before[k], s[k]), k


@pytest.mark.parametrize("world,dtype,rows,cols,count", [(1, "bf16", 64, 64, 1), (3, "fp16", 37, 50, 2), (4, "fp16", 128, 128, 4), (8, "bf16", 130, 66, 3),
                                                         (9, "bf16", 200, 333, 1), (16, "bf16", 1, 40, 5), (2, "fp16", 40, 1, 2), (20, "bf16", 129, 260, 2)])
def test_owned_unit(world, dtype, rows, cols, count):
    """Stage 4: whole units, the matrices somewhere inside one, and the counting of
    the fused step on as many elements."""
    n = rows * cols * count
    units = [n + 11, 5, n + 40]
    ctx = z.zero_init_shards(sum(units), world, z.ZSMR_ZERO3_OWNER, dtype, units=units)
    z.zero_set_unit_owners(ctx, [world - 1, 0, world // 2])
    t = {"bf16": BF16, "fp16": F16}[dtype]
    for unit, begin, base in ((0, 11, 0), (2, 17, 13), (2, 0, 1)):
        s = state(unit + world, world, units[unit], t, base)
        z.zero_reset_counters(ctx)
        check_step(ctx, z.zero_unit_owner(ctx, unit), unit, begin, rows, cols, count, s)
        got = [z.zero_counters(ctx, r) for r in range(world)]
        z.zero_reset_counters(ctx)
        v = torch.zeros_like(s["master"])
        z.zero_fused_step_range(ctx, z.zero_unit_owner(ctx, unit), unit, begin, n, s["grads"], s["grads"].shape[1], base, s["master"],
                                s["momentum"], v, s["p16"], 1, 1e-3)
        assert got == [z.zero_counters(ctx, r) for r in range(world)]


@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("kw", [dict(beta=0.0), dict(weight_decay=0.0), dict(lr=0.0), dict(scale=0.0)])
def test_hyper_parameters(kw, nesterov):
    ctx = z.zero_init_shards(3 * 48 * 30, 3, z.ZSMR_ZERO2, "bf16")
    check_step(ctx, 1, 0, 0, 48, 30, 1, state(1, 3, 48 * 30, BF16), nesterov=nesterov, **kw)


def test_formats_of_gradients_and_working_copy():
    for grad, param in (("fp16", "bf16"), ("bf16", "fp16")):
        ctx = z.zero_init_shards(60 * 70, 1, z.ZSMR_DP, grad, param)
        s = state(2, 1, 60 * 70, {"bf16": BF16, "fp16": F16}[grad])
        s["p16"] = s["p16"].to({"bf16": BF16, "fp16": F16}[param])
        check_step(ctx, 0, 0, 0, 60, 70, 1, s)


def test_steps_captured_into_a_graph():
    """Replays update the state as eager calls do."""
    rows, cols, count, world = 96, 130, 2, 4
    n = rows * cols * count
    ctx = z.zero_init_shards(n, world, z.ZSMR_ZERO3_OWNER, "bf16", units=[n])
    rank = z.zero_unit_owner(ctx, 0)
    a, b = state(5, world, n, BF16), state(5, world, n, BF16)
    wa, wb = (torch.empty(z.zero_muon_workspace(rows, cols, count), device="cuda", dtype=torch.uint8) for _ in range(2))

    def step(s, ws):
        z.zero_muon_step(ctx, rank, 0, 0, rows, cols, count, s["grads"], n, 0, s["master"], s["momentum"], s["p16"], ws, 0.02)

    step(a, wa)
    step(b, wb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a, wa)
    for i in range(4):
        fresh = state(30 + i, world, n, BF16)["grads"]
        a["grads"].copy_(fresh)
        b["grads"].copy_(fresh)
        graph.replay()
        step(b, wb)
        torch.cuda.synchronize()
        for k in ("master", "momentum", "p16"):
            assert torch.equal(a[k], b[k]), (i, k)


# ------------------------------------------------------------- used together --
@pytest.mark.parametrize("vocab,width,tokens,world", [(301, 72, 130, 3), (700, 140, 65, 2)])
def test_policy_example(vocab, width, tokens, world):
    """Scores, their gradient and the two kinds of step as a policy uses them: against
    the formulas in 64 bits, each from the 16-bit values it was given."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "policy.py")
    spec = importlib.util.spec_from_file_location("policy", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    torch.manual_seed(3)
    policy = module.Policy(vocab, width, tokens, world, 3e-3, 0.02, 0.05)
    g, u = gen(4), torch.finfo(BF16).eps / 2
    x = torch.randint(vocab, (world, tokens), device="cuda", generator=g)
    for r in range(world):
        hidden, logits = policy.logits(x[r])
        actions = torch.randint(vocab, (tokens,), device="cuda", generator=g)
        advantage = torch.randn(tokens, device="cuda", generator=g)
        policy.backward(r, x[r], hidden, logits, actions, advantage)
        leaf = logits.double().requires_grad_()
        p = torch.log_softmax(leaf, 1)
        picked, entropy = p.gather(1, actions[:, None]).squeeze(1), -(p.exp() * p).sum(1)
        # lse, its difference and the sums of V terms in fp32
        near = 2.0 ** -20 * (8 + leaf.detach().abs().amax(1))
        assert ((policy.logprob - picked).abs() <= near).all() and ((policy.entropy - entropy).abs() <= 4 * near).all()
        best = p.detach().gather(1, policy.top_ids)
        assert ((policy.top_logprobs - best).abs() <= near[:, None]).all()
        assert torch.equal(logits.gather(1, policy.top_ids), logits.topk(4).values)
        loss = -(advantage.double() * picked).mean() - 0.05 * entropy.mean()
        exact, = torch.autograd.grad(loss, leaf)
        # one bf16 rounding, and p's relative error times the terms it is in
        terms = (advantage.abs().double()[:, None] + 0.05 * (p.abs() + entropy[:, None]).detach()) / tokens
        assert ((policy.dlogits.double() - exact).abs() <= u * exact.abs() + 8 * near[:, None] * terms * p.exp().detach() + 2.0 ** -22 * terms).all()
        # products of 16-bit values, of which each is rounded once: dhidden and dx on the way;
        # sums of up to 700 terms in fp32: 701 roundings of 2^-24 are below 2^-14
        d, h, e = policy.dlogits.double(), hidden.double(), policy.x.double()
        w, head = policy.weights[1].double(), policy.weights[2].double()
        dh = d @ head
        for got, want, off in ((policy.weight_grads[2][r], d.t() @ h, d.abs().t() @ h.abs() * 2.0 ** -14),
                               (policy.weight_grads[1][r], dh.t() @ e, (u * dh.abs() + d.abs() @ head.abs() * 2.0 ** -14).t() @ e.abs() * (1 + 2.0 ** -8))):
            assert ((got.double() - want).abs() <= u * want.abs() + off * (1 + u) + 1e-30).all()
        dx = dh @ w
        dx_off = (u * dh.abs() + d.abs() @ head.abs() * 2.0 ** -14) @ w.abs() * (1 + 2.0 ** -8) + u * dx.abs()
        add = lambda t: torch.zeros(vocab, width, device="cuda", dtype=torch.float64).index_add_(0, x[r], t)
        want, off = add(dx), add(dx_off + 2.0 ** -14 * dx.abs())
        assert ((policy.weight_grads[0][r].double() - want).abs() <= u * want.abs() + off * (1 + u) + 1e-30).all()
    o, n = policy.at[1], width * width
    rows, old = policy.grads[:, o:o + n], policy.master[o:o + n].double()
    mean = rows[0].float()
    for r in range(1, world):
        mean = mean + rows[r].float()
    mean = mean / torch.full_like(mean, world)
    b = torch.tensor(0.95, device="cuda")
    exact, each, _ = allowed((mean + b * mean).view(1, width, width), F16)
    adam = [policy.master[s].clone() for s in (slice(0, o), slice(o + n, None))]
    policy.update()
    want = old - 0.02 * exact.reshape(-1)
    tol = 0.02 * each.reshape(-1) + 2.0 ** -24 * (2 * old.abs() + 4 * exact.reshape(-1).abs() + want.abs()) + 1e-30
    assert ((policy.master[o:o + n].double() - want).abs() <= tol).all()
    assert torch.equal(policy.m[o:o + n], mean)
    assert torch.equal(policy.params, policy.master.to(BF16))
    # Adam's first step is lr or less an element
    for before, s in zip(adam, (slice(0, o), slice(o + n, None))):
        moved = (policy.master[s] - before).abs()
        assert moved.max() <= 3e-3 * (1 + 1e-5) + 2.0 ** -23 * before.abs().max() and (moved > 0).any()


def test_policy_example_runs():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "policy.py")
    spec = importlib.util.spec_from_file_location("policy", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    rewards = module.train(vocab=100, width=64, tokens=256, world=2, steps=5, say=lambda *_: None)
    assert len(rewards) == 5 and all(math.isfinite(r) and 0 <= r <= 1 for r in rewards)
