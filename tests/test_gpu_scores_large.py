"""Scores of more rows than one launch has workgroups for."""
import math

import pytest
import torch

import zero_sharded_mixed_reduce_amd as z
from tests.test_gpu_scores import BF16, gen, logits, score

pytestmark = pytest.mark.gpu


def test_more_rows_than_a_launch_holds():
    """2^23 + 5 rows of 8,192 logits, eight waves each: 2^32 work items and more, 137 GB.  The
    first and the last rows are as in a call of their own, the rows between are zeros."""
    n, v = (1 << 23) + 5, 8192
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GB of free device memory")
    x = torch.zeros(n, v, device="cuda", dtype=BF16)
    ids = torch.zeros(n, device="cuda", dtype=torch.int64)
    some = torch.cat([torch.arange(9), torch.arange(n - 9, n)]).cuda()
    x[some], ids[some] = logits(21, 18, v, BF16)
    got, want = score(x, ids, 3), score(x[some], ids[some], 3)
    assert all(torch.equal(got[k][some], want[k]) for k in want)
    # log 8,192 in fp32, from one power a logit
    lse = math.log(v)
    assert ((got["lse"][9:-9] - lse).abs() < 1e-5).all() and ((got["logprob"][9:-9] + lse).abs() < 1e-5).all()
    assert (got["top_ids"][9:-9] == torch.arange(3, device="cuda")).all()
    g = torch.randn(n, device="cuda", generator=gen(22))
    d = torch.empty(18, v, device="cuda", dtype=BF16)
    z.zsmr_logprobs_grad(x[some], ids[some], want["lse"], want["entropy"], d, g[some], -g[some])
    z.zsmr_logprobs_grad(x, ids, got["lse"], got["entropy"], x, g, -g)
    assert torch.equal(x[some], d)
    del x
    torch.cuda.empty_cache()
