"""GPU tests of attention whose scores all lie far below zero: a prefix of no rows, or
slopes of zero, change nothing there either.

Scores times log2(e) are between -2^31 and -2^32, where a product's rounding is up to
2^7: a row's largest weight is two to the power of that, which its sum takes out again.
Past 2^127 or below 2^-126 the row has no finite sum: a few rows in 128, which are left out."""
import math

import pytest
import torch

from test_gpu_attention import dev, make

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,Hq,Hkv,D", [(200, 4, 2, 64), (1040, 64, 16, 64), (900, 64, 64, 128)])
def test_changes_of_nothing_far_below_zero(N, Hq, Hkv, D, dtype):
    import sample_grad_norms_amd as dp
    q, k, v, _ = make(N, Hq, Hkv, D, dtype, 81)
    size = math.sqrt(2.0 ** 31.2 / math.log2(math.e) * math.sqrt(D))   # 2^31.2 .. 2^31.6
    g = torch.Generator().manual_seed(82)
    q[..., 0] = (-size * (1.0 + 0.3 * torch.rand(N, Hq, generator=g))).to(dtype)
    k[..., 0] = torch.tensor(size).to(dtype)
    q, k, v = (x.to(dev()) for x in (q, k, v))
    o, lse = dp.attention_forward(q, k, v, sequences=2)
    fine = o.isfinite().all(dim=-1) & lse.t().isfinite()   # (a sum may pass 2^128 where its weighted values do not)
    assert float(fine.float().mean()) > 0.9 and float((lse.t()[fine] * math.log2(math.e)).max()) < -2.0 ** 31
    for how in (dict(prefix=torch.zeros(2, dtype=torch.int32, device=dev())), dict(slopes=torch.zeros(Hq, device=dev())),
                dict(slopes=torch.zeros(Hq, device=dev()), prefix=torch.zeros(2, dtype=torch.int32, device=dev()))):
        o2, lse2 = dp.attention_forward(q, k, v, sequences=2, **how)
        assert torch.equal(o2[fine], o[fine]) and torch.equal(lse2.t()[fine], lse.t()[fine]), how
