"""The operators around the step where their inputs hold what they must not look
at, or what few programs hand over."""
import pytest
import torch

import zero_sharded_mixed_reduce_amd as z
from tests.gpu_helpers import say
from tests.test_gpu_ops import T16, U, gen, half, intact, normal, space, tokens

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


def test_logits_near_the_ends_of_fp32():
    """Rows of the head that give the lowest logits fp32 has are as good as
    absent, also where a whole tile of the vocabulary is of them; logits of
    3e38 make the statistics infinite and are not passed over."""
    g, t = gen(23), torch.bfloat16
    n, vocab, width = 40, 900, 64
    x, w = normal(g, (n, width), 1.0, t), normal(g, (vocab, width), 0.2, t)
    x[:, 0] = 1
    labels = torch.randint(256, (n,), generator=g, device="cuda")
    low = w.clone()
    low[256:768] = 0
    low[256:768, 0] = torch.finfo(t).min
    loss, lse, summary, dx, dw = xent_both(x, low, labels)
    rest = torch.cat([w[:256], w[768:]])
    want = xent_both(x, rest, labels)
    # fp32 sums of the same exponentials in another order
    tol = 2.0 ** -20 + 600 * U
    assert float((lse - want[1]).abs().max()) <= tol and float((loss - want[0]).abs().max()) <= tol
    assert bool((dw[256:768] == 0).all())
    # G, held in 16 bits, and the result's rounding
    assert float((dx.double() - want[3].double()).norm()) <= 2 * half(t) * float(want[3].double().norm())
    high = w.clone()
    high[300] = 0
    high[300, 0] = 3e38
    loss, lse, *_ = xent_both(x, high, labels)
    assert bool(torch.isinf(lse).all()) and bool((lse > 0).all()) and bool(torch.isinf(loss).all())


def test_a_list_that_can_be_gone_through_once():
    """The gradients of a model's parameters, as a generator gives them: the bits
    of the same tensors in a list."""
    g = gen(25)
    xs = [torch.randn(k, generator=g, device="cuda") for k in (7, 5000, 1)]
    a, b = torch.empty(2, device="cuda"), torch.empty(2, device="cuda")
    ws, _ = space(z.zsmr_norm_workspace(5008, 3))
    z.zsmr_grad_norm(xs, 1.0, a, ws)
    z.zsmr_grad_norm((x for x in xs), 1.0, b, ws)
    assert torch.equal(a, b) and a[0].item() > 0
    rows = [torch.empty(5008, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    z.zsmr_clip_flatten(xs, a[1:], rows[0])
    z.zsmr_clip_flatten((x for x in xs), a[1:], rows[1])
    assert torch.equal(bits(rows[0]), bits(rows[1]))
    ys = [x.clone() for x in xs]
    z.zsmr_clip_grads(xs, a[1:])
    z.zsmr_clip_grads((y for y in ys), a[1:])
    for x, y in zip(xs, ys):
        assert torch.equal(bits(x), bits(y))


def test_embedding_gradient_of_more_rows_than_a_launch_zeroes():
    """2^28 + 5 rows of width 8: a workgroup for every 16 of them would be 2^32
    work items and more."""
    vocab, t = (1 << 28) + 5, torch.bfloat16
    table = torch.ones(vocab, 8, device="cuda", dtype=t)
    ids = torch.tensor([vocab - 1, 0, 1 << 28, -1], device="cuda")
    rows = torch.randn(4, 8, generator=gen(26), device="cuda").to(t)
    ws, _ = space(z.zsmr_embed_grad_workspace(vocab, 8, 4))
    z.zsmr_embed_grad(rows, ids, table, ws)
    assert torch.equal(table[ids[:3]], rows[:3])
    assert sum(int((part != 0).any(1).sum()) for part in table.split(1 << 26)) == 3
    del table
    torch.cuda.empty_cache()


def test_lookup_of_more_elements_than_a_launch_has_work_items():
    """2^24 tokens of width 2,056: 2^32 groups of eight elements and more, 69 GB of
    output."""
    n, width, t = 1 << 24, 2056, torch.bfloat16
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB of free device memory")
    g = gen(27)
    table = normal(g, (1000, width), 1.0, t)
    ids = torch.randint(-1, 1000, (n,), generator=g, device="cuda", dtype=torch.int32)
    out = torch.full((n, width), 7.0, device="cuda", dtype=t)
    z.zsmr_embed_lookup(table, ids, out)
    whole = torch.cat([table, torch.zeros(1, width, device="cuda", dtype=t)])       # -1 reads the last row
    for k in range(0, n, 1 << 20):
        assert torch.equal(out[k:k + (1 << 20)], whole[ids[k:k + (1 << 20)].long()]), k
    del out
    torch.cuda.empty_cache()


def test_scores_of_more_tiles_than_a_launch_holds():
    """2^20 tokens over 2^20 + 300 rows: 2^24 tiles, which would be 2^33 work
    items.  The statistics of some tokens against 64 bits."""
    n, vocab, width, t = 1 << 20, (1 << 20) + 300, 64, torch.bfloat16
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    g = gen(28)
    x, w = normal(g, (n, width), 1.0, t), normal(g, (vocab, width), 0.25, t)
    labels = torch.randint(vocab, (n,), generator=g, device="cuda")
    some = torch.cat([torch.arange(40, device="cuda"), torch.randint(n, (40,), generator=g, device="cuda"), torch.arange(n - 40, n, device="cuda")])
    labels[some[::3]] = torch.randint(vocab - 300, vocab, (40,), generator=g, device="cuda")
    loss, lse, summary = (torch.full((k,), float("nan"), device="cuda") for k in (n, n, 3))
    size = z.zsmr_xent_workspace(n, vocab, width, backward=False)
    ws, raw = space(size)
    z.zsmr_xent_forward(x, w, labels, loss, lse, summary, ws)
    intact(raw, size)
    s = x[some].double() @ w.double().t()
    want = torch.logsumexp(s, 1)
    # fp32 logits of 64 products, exponentials of fp32 arguments, sums over parts of 256 rows
    es = float(U * width * (x[some].double().abs() @ w.double().abs().t()).max())
    tol = es + 2.0 ** -20 + U * vocab / 64 + 4 * U * float(want.max())
    assert float((lse[some].double() - want).abs().max()) <= tol
    assert float((loss[some].double() - (want - s.gather(1, labels[some][:, None])[:, 0])).abs().max()) <= tol + es
    assert bool(torch.isfinite(loss).all()) and summary[2].item() == n
    assert abs(summary[0].item() - float(loss.double().mean())) <= 2 * U * summary[0].item()
    del ws, raw
    torch.cuda.empty_cache()


def test_raw_addresses():
    """Every buffer but a matrix may be a raw address, which the caller has
    checked: the same bits as with tensors."""
    g, t = gen(24), torch.bfloat16
    n, vocab, width = 33, 200, 64
    x, w, labels = normal(g, (n, width), 1.0, t), normal(g, (vocab, width), 0.2, t), tokens(g, n, vocab, "some")
    weights = torch.rand(n, generator=g, device="cuda")
    a, b = ([torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty(3, device="cuda"), torch.empty_like(x), torch.empty_like(w)]
            for _ in range(2))
    size = max(z.zsmr_xent_workspace(n, vocab, width), z.zsmr_embed_grad_workspace(vocab, width, n), z.zsmr_norm_workspace(vocab * width, 1))
    ws, _ = space(size)
    for (loss, lse, summary, dx, dw), f in ((a, lambda y: y), (b, lambda y: y.data_ptr())):
        z.zsmr_xent_forward(x, w, labels, f(loss), f(lse), f(summary), f(ws))
        z.zsmr_xent_backward(x, w, labels, f(lse), dx, dw, f(ws), grad=f(weights), scale=f(summary) + 4 if f(ws) is not ws else summary[1:2])
        z.zsmr_embed_grad(dx, labels, dw, f(ws), accumulate=True)
        out = torch.empty(2, device="cuda")
        z.zsmr_grad_norm([dw], 1e-3, f(out), f(ws))
        z.zsmr_clip_grads([dw], f(out) + 4 if f(ws) is not ws else out[1:])
    for p, q in zip(a, b):
        assert torch.equal(bits(p), bits(q))
