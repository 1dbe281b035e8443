"""The accuracy of the shard step's update, which goes into an fp32 master: in the
2-norm and of each element, with gradients of white noise and of decaying spectra.

Tolerances are those of ``test_gpu_newton``: the 64-bit computation with errors of the
kernels' sizes at every place where they have one, steps in groups where a call may
take them; four times its distance in the 2-norm and ten times its share of an element,
and no rounding of a result but fp32's.  The step moves the master by as much as it
holds, so that nothing of the update is lost in it."""
import pytest
import torch

import zero_sharded_mixed_reduce_amd as z
from tests.test_gpu_newton import BF16, F16, gen, matrices, muon, polynomial

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": BF16, "fp16": F16}


def spectrum(seed, count, rows, cols, kind):
    if kind == "noise":
        return matrices(seed, count, rows, cols)
    if kind == "rank 1":
        return matrices(seed, count, rows, cols, rank=1)
    k, exponent = min(rows, cols), {"1/k": -1.0, "1/k^3": -3.0}[kind]
    left, right = (torch.linalg.qr(matrices(seed + i, count, n, k).double())[0] for i, n in enumerate((rows, cols)))
    s = torch.arange(1, k + 1, device="cuda").double() ** exponent
    return ((left * s) @ right.mT.contiguous()).float()


def groups(rows, cols):
    m, n = sorted((rows, cols))
    stays = n <= 256 if m <= 64 else n <= 128       # in a CU's LDS, step by step
    return (3, 2) if not stays and 5 * n >= 6 * m else ()


@pytest.mark.parametrize("kind", ["noise", "rank 1", "1/k", "1/k^3"])
@pytest.mark.parametrize("world,dtype,rows,cols,count", [(1, "fp16", 64, 64, 3), (3, "bf16", 37, 250, 2), (4, "fp16", 128, 128, 4), (2, "bf16", 130, 130, 2),
                                                         (4, "bf16", 200, 333, 1), (3, "fp16", 140, 2000, 2), (2, "bf16", 2050, 513, 1), (1, "fp16", 1000, 1003, 1),
                                                         (2, "bf16", 1600, 4000, 1)])
def test_update(world, dtype, rows, cols, count, kind):
    n = rows * cols * count
    ctx = z.zero_init_shards(world * n, world, z.ZSMR_ZERO3_OWNER, dtype, units=[n] * world)
    rank, g = z.zero_unit_owner(ctx, 0), spectrum(rows + cols, count, rows, cols, kind)
    g = g / g.square().mean().sqrt()
    noise = torch.randn(world, n, generator=gen(2), device="cuda") * 2.0 ** -12
    s = {"grads": (g.reshape(1, -1) + noise).to(DTYPES[dtype]), "base": 0, "momentum": torch.zeros(n, device="cuda"),
         "master": torch.randn(n, generator=gen(3), device="cuda") / max(rows, cols) ** 0.5, "p16": torch.empty(n, device="cuda", dtype=DTYPES[dtype])}
    old = s["master"].double().view(count, rows, cols)
    muon(ctx, rank, 0, 0, rows, cols, count, s, lr=1.0, beta=0.5, weight_decay=0.5, scale=1.0, nesterov=True)
    u = s["momentum"]       # g, and u = 1.5 g: a factor of the norm alone
    mean = s["grads"][0].float()
    for r in range(1, world):
        mean = mean + s["grads"][r].float()
    assert torch.equal(u, mean / torch.full_like(mean, world))
    x = (u + 0.5 * u).view(count, rows, cols)
    exact = polynomial(x)
    off = torch.stack([(polynomial(x, noise=gen(k), groups=groups(rows, cols)) - exact).square().sum((-2, -1), keepdim=True).sqrt() for k in range(8)]).amax(0)
    want = 0.5 * old - exact
    # of master times decay, of rate times update, of the difference, and the update's own
    rounding = 2.0 ** -24 * (0.5 * old.abs() + 2 * exact.abs() + want.abs())
    d = (s["master"].view(count, rows, cols).double() - want).abs()
    assert (d.square().sum((-2, -1), keepdim=True).sqrt() <= 4 * off + rounding.square().sum((-2, -1), keepdim=True).sqrt()).all()
    assert (d <= 40 * off / (rows * cols) ** 0.5 + rounding).all()
    assert torch.equal(s["p16"], s["master"].to(s["p16"].dtype))
