"""GPU tests of attention biased by distance with negative slopes, which raise far keys:
up to their documented limit, |slope| (length - 1) = 2^14, against the definition in
float64, and past it, where a head's results of that sequence are NaN.

Tolerances are those of test_gpu_attention_scores.py. They count every rounding of a
score, its maximum and its log-sum-exp relative to the bias and to |lse|: at the limit
10 u 2^14 = 2^-10 * 10 for the weights of the gradients, 1 %, whose square, 1e-4, is
below the 2 % by which the bounds are raised for products of errors.
"""
import math

import pytest
import torch

from test_gpu_attention import dev, make, offsets
from test_gpu_attention_scores import Change, check

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
LIMIT = 2.0 ** 14


def steepest(length):
    """The limit's slope of a sequence, towards zero where float32 does not hold it."""
    s = torch.tensor(-LIMIT / (length - 1), dtype=torch.float64)
    f = s.float()
    return float(f if f.double() >= s else torch.nextafter(f, torch.zeros(())))


# by rows (shared keys and not) and by tiles, at sequences of a tile and less, with offsets inside one
SHAPES = [([17], 4, 2, 64), ([200, 1, 33], 4, 2, 64), ([500], 3, 1, 128), ([1025], 64, 16, 64), ([700, 321], 64, 64, 88)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kw", [{}, dict(cap=5.0), dict(prefix=0.4), dict(cap=5.0, prefix=0.4)])
@pytest.mark.parametrize("lengths,Hq,Hkv,D", SHAPES)
def test_slopes_up_to_the_limit(lengths, Hq, Hkv, D, kw, dtype):
    ch = Change(Hq, lengths, slopes=1.0, **kw)
    top = steepest(max(lengths))
    # the limit itself, a half and a thousandth of it, and a positive one
    ch.slopes = torch.tensor([(top, top / 2, top / 1000, 0.3)[h % 4] for h in range(Hq)], dtype=torch.float32)
    check(lengths, Hq, Hkv, D, dtype, ch)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kw", [{}, dict(cap=5.0), dict(prefix=True), dict(cap=5.0, prefix=True)])
@pytest.mark.parametrize("Hq,Hkv,D,lengths", [(4, 2, 64, [1, 37, 200, 18]), (4, 2, 128, [37, 1, 18, 200]), (64, 16, 64, [1040, 1, 700, 18])])
@pytest.mark.parametrize("slope", ["next", -2.0 ** 24, -2.0 ** 28, -2.0 ** 32, -math.inf])
def test_steeper_slopes_give_nan(slope, Hq, Hkv, D, lengths, kw, dtype):
    """Past the limit all of a head's results of the sequence are NaN, and so are the gradients
    of its key head; other heads, and sequences within the limit, keep their bits."""
    import sample_grad_norms_amd as dp
    steep = 1
    if slope == "next":
        slope = float(torch.nextafter(torch.tensor(steepest(max(lengths))), torch.tensor(-math.inf)))
        past = [n == max(lengths) for n in lengths]
    else:
        past = [n > 1 or slope == -math.inf for n in lengths]   # (a lone row is at distance 0, and 0 times infinity NaN)
    S, rep = len(lengths), Hq // Hkv
    q, k, v, do = (x.to(dev()) for x in make(sum(lengths), Hq, Hkv, D, dtype, 61))
    cu = offsets(lengths)
    how = dict(kw, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=dev()))
    if how.pop("prefix", False):
        how["prefix"] = torch.tensor([min(n, 40) for n in lengths], dtype=torch.int32, device=dev())
    slopes = torch.full((Hq,), 0.25, device=dev())
    o0, lse0 = dp.attention_forward(q, k, v, slopes=slopes, **how)
    grads0 = dp.attention_backward(do, q, k, v, o0, lse0, slopes=slopes, **how)
    slopes[steep] = slope
    o, lse = dp.attention_forward(q, k, v, slopes=slopes, **how)
    grads = dp.attention_backward(do, q, k, v, o, lse, slopes=slopes, **how)
    # (the limit holds in the gradients whatever statistics they are given)
    given = dp.attention_backward(do, q, k, v, o0, lse0, slopes=slopes, **how)
    others = [h for h in range(Hq) if h != steep]
    assert torch.equal(o[:, others], o0[:, others]) and torch.equal(lse[others], lse0[others])
    other_keys = [h for h in range(Hkv) if h != steep // rep]
    for got in (grads, given):
        assert torch.equal(got[0][:, others], grads0[0][:, others])
        assert all(torch.equal(a[:, other_keys], b[:, other_keys]) for a, b in zip(got[1:], grads0[1:]))
    for i in range(S):
        a, b = cu[i], cu[i + 1]
        parts = lambda g: [g[0][a:b, steep], *(t[a:b, steep // rep] for t in g[1:])]
        for t in [o[a:b, steep], lse[steep, a:b], *parts(grads)]:
            assert bool(t.isnan().all() if past[i] else t.isfinite().all()), (i, lengths[i])
        assert not past[i] or all(bool(t.isnan().all()) for t in parts(given)), (i, lengths[i])
