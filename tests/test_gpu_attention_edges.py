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

import attention_forms
from test_gpu_attention import dev, make, test_forward_and_backward as forward_and_backward

pytestmark = pytest.mark.gpu

EVERY = [(torch.bfloat16, *s) for s in attention_forms.BF16] + [(torch.float32, *s) for s in attention_forms.F32]
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


@pytest.mark.parametrize("dtype,N,Hq,Hkv,D", EVERY)
def test_every_form_against_its_definition(N, Hq, Hkv, D, dtype):
    forward_and_backward([N], Hq, Hkv, D, dtype)


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype,N,Hq,Hkv,D", EVERY)
def test_a_row_that_is_not_finite_leaves_the_others(N, Hq, Hkv, D, dtype, value):
    """Rows that do not see a row with an infinity or NaN get what they get without it, bit
    for bit, in the last rows of a step, of a wave and of a tile and in the middle of each."""
    import sample_grad_norms_amd as dp
    q, k, v, do = (x.to(dev()) for x in make(N, Hq, Hkv, D, dtype, 32))
    o, lse = dp.attention_forward(q, k, v)
    dq, dk, dv = dp.attention_backward(do, q, k, v, o, lse)
    for row in (5, 63, 64, N // 2, N - 33, N - 1):
        for name in ("k", "v"):
            args = {"q": q, "k": k.clone(), "v": v.clone()}
            args[name][row, :, 3] = value
            o2, lse2 = dp.attention_forward(**args)
            same = torch.equal(o2[:row], o[:row]) and torch.equal(lse2[:, :row], lse[:, :row])
            assert same, (name, row)
            if name == "v":   # every later query sees it, in its column alone
                later = o2[row:, :, 3].float()
                seen = bool((later.isnan() if math.isnan(value) else later == value).all())
                same = torch.equal(o2[:, :, :3], o[:, :, :3]) and torch.equal(o2[:, :, 4:], o[:, :, 4:]) and torch.equal(lse2, lse)
                assert seen and same, row
            dq2, _, _ = dp.attention_backward(do, args["q"], args["k"], args["v"], o, lse)
            same = torch.equal(dq2[:row], dq[:row])
            assert same, (name, row)
        for name in ("do", "q"):
            args = {"do": do.clone(), "q": q.clone()}
            args[name][row, :, 3] = value
            _, dk2, dv2 = dp.attention_backward(args["do"], args["q"], k, v, o, lse)
            same = torch.equal(dk2[row + 1:], dk[row + 1:]) and torch.equal(dv2[row + 1:], dv[row + 1:])
            assert same, (name, row)


@pytest.mark.parametrize("dtype,N,Hq,Hkv,D", EVERY)
def test_keys_of_minus_infinity_leave_the_forward_pass(N, Hq, Hkv, D, dtype):
    """Scores of -infinity, against scores so low that exp gives 0: the same output, bit for
    bit, also in the waves whose rows past the end meet those keys."""
    import sample_grad_norms_amd as dp
    q, k, v, _ = make(N, Hq, Hkv, D, dtype, 33)
    q = q.abs() + 0.125
    gone = torch.tensor([9, 10, 33, 64, N // 2, N - 33, N - 12, N - 1])
    low = k.clone()
    low[gone, :, 3] = -1e5
    k[gone, :, 3] = -math.inf
    qd, kd, ld, vd = (x.to(dev()) for x in (q, k, low, v))
    o, lse = dp.attention_forward(qd, kd, vd)
    o2, lse2 = dp.attention_forward(qd, ld, vd)
    same = torch.equal(o, o2) and torch.equal(lse, lse2)
    assert same and bool(o.isfinite().all())


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype,N,Hq,Hkv,D", EVERY)
def test_an_output_gradient_that_is_not_finite_reaches_dv_as_it_is(N, Hq, Hkv, D, dtype, value):
    """dv_u = sum_t p_tu dO_t with weights above zero: the keys that a row of dO with an
    infinity or NaN sees get that value in its column, wherever the row lies in its tile
    (weights of scores of a few units, far from where exp gives 0)."""
    import sample_grad_norms_amd as dp
    q, k, v, do = (x.to(dev()) for x in make(N, Hq, Hkv, D, dtype, 34))
    o, lse = dp.attention_forward(q, k, v)
    _, dk0, dv0 = dp.attention_backward(do, q, k, v, o, lse)
    for row in (5, 63, N // 2, N - 1):
        do2 = do.clone()
        do2[row, :, 3] = value
        _, dk, dv = dp.attention_backward(do2, q, k, v, o, lse)
        seen = dv[:row + 1, :, 3].float()
        right = bool((seen.isnan() if math.isnan(value) else seen == value).all())
        others = torch.cat([dv[:, :, :3], dv[:, :, 4:]], dim=2), torch.cat([dv0[:, :, :3], dv0[:, :, 4:]], dim=2)
        assert right and torch.equal(*others) and torch.equal(dv[row + 1:], dv0[row + 1:]), row
        assert not bool(dk[:row + 1].isfinite().any()) and torch.equal(dk[row + 1:], dk0[row + 1:]), row


@pytest.mark.parametrize("dtype,N,Hq,Hkv,D", EVERY)
def test_a_query_without_weights_gives_nan(N, Hq, Hkv, D, dtype):
    """A query all of whose scores are -infinity: exp(-inf - -inf) is NaN for every key
    that it sees, and so are those keys' gradients, in the query's own tile as elsewhere."""
    import sample_grad_norms_amd as dp
    q, k, v, do = make(N, Hq, Hkv, D, dtype, 35)
    k[:, :, 3] = k[:, :, 3].abs() + 0.125
    q, k, v, do = (x.to(dev()) for x in (q, k, v, do))
    o, lse = dp.attention_forward(q, k, v)
    _, dk0, dv0 = dp.attention_backward(do, q, k, v, o, lse)
    for row in (5, 63, N // 2, N - 1):
        q2 = q.clone()
        q2[row, :, 3] = -math.inf
        o, lse = dp.attention_forward(q2, k, v)
        assert bool(o[row].isnan().all()) and bool((lse[:, row] == -math.inf).all())
        dq, dk, dv = dp.attention_backward(do, q2, k, v, o, lse)
        gone = bool(dv[:row + 1].isnan().all()) and bool(dk[:row + 1].isnan().all()) and bool(dq[row].isnan().all())
        assert gone and torch.equal(dk[row + 1:], dk0[row + 1:]) and torch.equal(dv[row + 1:], dv0[row + 1:]), row
