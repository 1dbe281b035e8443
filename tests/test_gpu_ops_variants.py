"""Every form that the kernels of the operators are compiled in, at sizes that
select it.  That the cross entropy's sizes select all of them is checked on the CPU
(``tests/test_xent_plan.py``)."""
import pytest
import torch

import zero_sharded_mixed_reduce_amd as z
from tests.gpu_helpers import say
from tests.test_gpu_ops import T16, gen, intact, space, xent_case

pytestmark = pytest.mark.gpu

# tokens, vocabulary, width
XENT_SHAPES = [
    (4, 65600, 16), (1, 257, 8), (70, 33030, 64), (1900, 2101, 16), (2739, 2830, 24), (3810, 3210, 8),  # logits and G: tiles of 64, 128, 192, 256 tokens
    (129, 50257, 64), (100, 40000, 64),
    (2133, 700, 1816), (2945, 700, 2672), (4049, 700, 2888), (40, 600, 520),                            # dx: one piece, one split
    (4133, 2337, 8), (5431, 3584, 8), (6257, 4462, 8), (66, 8123, 5504), (2, 8667, 7344), (33, 3000, 72),     # several splits
    (10791, 24958, 16), (11998, 24790, 8), (14399, 18547, 8),                                           # several pieces and splits
    (10786, 42868, 624), (18842, 16145, 464), (18210, 15900, 528),                                      # several pieces, one split
    (300, 2504, 3128), (5000, 60000, 65), (257, 70000, 130),                                            # dw of 256 rows; packed pieces
]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("n,vocab,width", XENT_SHAPES)
def test_xent_variants(n, vocab, width, dt):
    xent_case(n, vocab, width, dt)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("n,vocab,width", [(2739, 2830, 24), (3810, 3210, 8), (70, 33030, 64)])
def test_xent_variants_weighted_and_accumulated(n, vocab, width, dt):
    xent_case(n, vocab, width, dt, grad=True, accumulate=True)


@pytest.mark.parametrize("world,n,shift,dt", [(16, (1 << 26) + 517, 0, "bf16"), (17, (1 << 26) + 3, 1, "fp16"), (31, (1 << 25) + (1 << 21), 0, "bf16")])
def test_windowed_reduce_of_few_rows(world, n, shift, dt):
    """16 to 31 rows, stored in write windows from 2^30 elements on: the bits of
    zero_reduce_shard and the sum of their squares."""
    say("[windows]", world, n, shift, dt)
    assert 16 <= world < 32 and world * n >= 1 << 30
    ctx = z.zero_init_shards(n * world, world, z.ZSMR_ZERO2, dt)
    raw = torch.randn(world * (n + shift) + 8, generator=gen(31), device="cuda", dtype=T16[dt]).mul_(0.01)[shift:]
    red, want = torch.full((n + 16,), 7.0, device="cuda"), torch.empty(n, device="cuda")
    sums = torch.empty(1, device="cuda", dtype=torch.float64)
    size = z.zsmr_norm_workspace(n, 1)
    ws, guard = space(size)
    z.zero_reduce_shard(ctx, 1, 0, raw, n + shift, 0, True, want)
    exact = float(want.double().square().sum())
    for _ in range(2):
        z.zero_reduce_shard_sumsq(ctx, 1, 0, raw, n + shift, 0, True, red, sums, ws)
        assert torch.equal(red[:n].view(torch.int32), want.view(torch.int32))
        assert abs(float(sums) - exact) <= 1e-11 * exact
    assert bool((red[n:] == 7).all())
    intact(guard, size)
