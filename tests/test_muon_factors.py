"""The shard step's factors in fp32, on a machine without a GPU.  Addresses are
placeholders that nothing reads."""
import pytest

import zero_sharded_mixed_reduce_amd as z
from zero_sharded_mixed_reduce_amd import ops

A, B, C, D, W = 1 << 20, 2 << 20, 3 << 20, 4 << 20, 5 << 20


@pytest.mark.parametrize("kw", [dict(lr=1e30, scale=1e30), dict(lr=1e200, scale=1e200), dict(lr=1e39), dict(scale=1e41), dict(lr=1e30, weight_decay=1e30, scale=0.0),
                                dict(lr=1e200, weight_decay=1e200, scale=0.0)])
def test_factors_past_fp32_are_refused(kw):
    """lr * scale and 1 - lr * weight_decay are fp32 in the kernels: an infinite one would
    make the master NaN wherever its other factor is zero."""
    ctx = z.zero_init_shards(200 * 300, 1, z.ZSMR_ZERO2, "bf16")
    hp = ops.zsmr_muon(**(dict(lr=0.02, beta=0.9, weight_decay=0.0, scale=1.0, nesterov=1, pad=0) | kw))
    ns = ops.zsmr_newton(1e-7, 1, 0)
    ns.coef[0][:] = (1.5, -0.5, 0.0)
    size = z.zero_muon_workspace(200, 300, 1)
    call = (ctx.handle, 0, 0, 0, 200, 300, 1, A, 200 * 300, 0, B, C, D, hp, ns, W, size - 1, None)
    # too small a workspace is the last check: nothing is launched either way
    assert ops._lib().zero_muon_step(*call) == z.ZSMR_ERR_ARG
    # misaligned memory is looked at later than the factors
    assert ops._lib().zero_muon_step(*call[:10], B + 1, *call[11:]) == z.ZSMR_ERR_ARG
    assert z.zero_counters(ctx, 0)["traffic_elems"] == 0
