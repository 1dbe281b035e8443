"""The binding of the operators on a machine without a GPU: what it makes of the
forms its arguments may have.  Addresses are placeholders that nothing reads."""
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
