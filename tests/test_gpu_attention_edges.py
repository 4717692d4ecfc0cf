"""Attention at the edges of its tiles: values that are not finite, and rows that
fill a tile's end, in every form that the kernels have (by rows and by tiles of 128
queries, keys and queries shared by work groups or not).

Rows compared with another call's are compared bit for bit: the two calls do the
same operations on them. Which form a shape takes is pinned by
test_attention_forms_host.py.
"""
import math

import pytest
import torch

from test_gpu_attention import dev, make

pytestmark = pytest.mark.gpu

FORMS = [   # N, Hq, Hkv, D, by way of
    (330, 2, 1, 64),       # shared keys and queries
    (320, 2, 1, 64),
    (700, 64, 64, 64),     # 32 keys a work group, four waves
    (704, 64, 64, 64),
    (1040, 64, 16, 64),    # eight waves for bfloat16
    (1056, 64, 16, 64),
    (330, 3, 1, 128),
    (704, 64, 64, 104),
    (707, 64, 64, 88),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,Hq,Hkv,D", FORMS)
def test_keys_without_weight_get_no_gradient(N, Hq, Hkv, D, dtype):
    """Keys whose score is -infinity for every query: dk and dv are 0, and every other
    key's are what they are with scores so low that exp gives 0 (below -400)."""
    import sample_grad_norms_amd as dp
    q, k, v, do = make(N, Hq, Hkv, D, dtype, 31)
    q = q.abs() + 0.125
    gone = torch.tensor([9, 10, 33, 64, N // 2, N - 33, N - 12, N - 1])
    low = k.clone()
    low[gone, :, 3] = -1e5     # 0.125 x 1e5 / sqrt(128) = 1104
    k[gone, :, 3] = -math.inf
    qd, kd, ld, vd, dod = (x.to(dev()) for x in (q, k, low, v, do))
    o, lse = dp.attention_forward(qd, ld, vd)
    _, dk, dv = dp.attention_backward(dod, qd, kd, vd, o, lse)
    _, dk2, dv2 = dp.attention_backward(dod, qd, ld, vd, o, lse)
    assert bool((dk[gone] == 0).all()) and bool((dv[gone] == 0).all())
    same = torch.equal(dk, dk2) and torch.equal(dv, dv2)
    assert same
