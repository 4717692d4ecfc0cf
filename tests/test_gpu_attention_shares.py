"""GPU parity of attention with a prefix where two or three work groups share the keys'
queries of dk and dv (attention_shares.py), at prefixes of a few rows to most of them,
against the definition in float64; and a row that is not finite there."""
import math

import pytest
import torch

from attention_shares import SHARES
from sample_grad_norms_amd import _lib
from test_gpu_attention_scores import BF16, F32, Change, check
from test_gpu_attention_scores import test_a_row_that_is_not_finite_leaves_the_others as one_row_that_is_not_finite

pytestmark = pytest.mark.gpu
DTYPES = {_lib.BF16: BF16, _lib.F32: F32}
SMALL = [(DTYPES[dt], list(lengths), hq, hkv, d) for dt, lengths, hq, hkv, d in SHARES if sum(lengths) <= 1100]


@pytest.mark.parametrize("change", [dict(prefix=0.4), dict(slopes=0.5, prefix=33), dict(cap=8.0, slopes=0.1, prefix=0.95)])
@pytest.mark.parametrize("dtype,lengths,Hq,Hkv,D", SMALL)
def test_shared_keys(dtype, lengths, Hq, Hkv, D, change):
    check(lengths, Hq, Hkv, D, dtype, Change(Hq, lengths, **change))


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("change", [dict(prefix=40), dict(cap=10.0, prefix=97)])
@pytest.mark.parametrize("dtype,lengths,Hq,Hkv,D", [s for s in SMALL if len(s[1]) == 1][:3])
def test_a_row_that_is_not_finite(dtype, lengths, Hq, Hkv, D, change, value):
    one_row_that_is_not_finite(lengths[0], Hq, Hkv, D, change, value, dtype)
