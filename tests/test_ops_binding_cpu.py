"""The binding of the operators on a machine without a GPU: what it makes of the
forms its arguments may have.  Addresses are placeholders that nothing reads."""
import numpy as np
import pytest
import torch

import zero_sharded_mixed_reduce_amd as z
from zero_sharded_mixed_reduce_amd import ops


def test_a_list_of_tensors_may_be_any_iterable():
    """Tensors that can be gone through only once are a list like any other: the
    first of them is refused here because it lies in host memory."""
    xs, out = [torch.zeros(5), torch.zeros(3, dtype=torch.bfloat16)], torch.zeros(2)
    for tensors in (xs, tuple(xs), (x for x in xs), map(torch.Tensor.view_as, xs, xs), dict(enumerate(xs)).values()):
        with pytest.raises(ValueError, match="a cpu tensor"):
            ops._list(tensors)
    for call in (lambda t: z.zsmr_grad_norm(t, 1.0, out, None, stream=0), lambda t: z.zsmr_clip_grads(t, out, stream=0),
                 lambda t: z.zsmr_clip_flatten(t, out, xs[1], stream=0)):
        with pytest.raises(ValueError, match="a cpu tensor"):
            call(x for x in xs)
    with pytest.raises(ValueError, match="tensor 1 is not contiguous"):
        ops._list(x for x in (xs[0], torch.zeros(4, 4).t()))


def test_raw_addresses_are_the_callers_to_check():
    """A raw address reaches the library's own checks, a workspace's too, whose
    length is not known; the flat row has to be a tensor."""
    A, C, W = 1 << 20, 3 << 20, 5 << 20
    arrays = np.array([A]), np.array([20_000]), np.array([3], np.int32)
    for ws, code in ((None, z.ZSMR_ERR_ARG), (W + 8, z.ZSMR_ERR_ALIGN)):
        with pytest.raises(z.ZsmrError) as e:
            z.zsmr_grad_norm(arrays, 1.0, C, ws, stream=0)
        assert e.value.code == code
    ctx = z.zero_init_shards(20_000, 1, z.ZSMR_ZERO2, "bf16")
    with pytest.raises(z.ZsmrError) as e:
        z.zero_reduce_shard_sumsq(ctx, 0, 0, A, 20_000, 0, True, C, C, W + 8, stream=0)
    assert e.value.code == z.ZSMR_ERR_ALIGN
    for flat in (C, None):
        with pytest.raises(ValueError, match="flat: a tensor"):
            z.zsmr_clip_flatten(arrays, None, flat, stream=0)
