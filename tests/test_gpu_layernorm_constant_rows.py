"""GPU tests of layer norm's gradients on constant rows of large values, whose h = (x - mu) r
is 0 while mu r passes float32's range, against the definition in float64.

With h = 0, dx = r (g - mean(g)) for g = dy w, dw = 0 and db = sum dy. Tolerances as in
test_gpu_layernorm.py, from which h's share falls away: mean(g) is off by 66 u mean|g|,
the difference and the products by 3 u, and the result by half a step of the type.
"""
import pytest
import torch

from test_gpu_layernorm import BF16, F32, U, dev, half, inside

pytestmark = pytest.mark.gpu


def check(B, T, d, dtype, value, mean, rstd):
    import sample_grad_norms_amd as dp
    g = torch.Generator().manual_seed(71)
    G, w = torch.randn(B, T, d, generator=g).to(dtype), (1.0 + 0.3 * torch.randn(d, generator=g)).to(dtype)
    x = torch.full((B, T, d), value).to(dtype)
    x[:, 1::2] = torch.randn(x[:, 1::2].shape, generator=g).to(dtype)   # ordinary rows between them
    xd, Gd, wd = (t.to(dev()) for t in (x, G, w))
    y, m, r = dp.layernorm_forward(xd, wd, eps=rstd ** -2)
    if mean is None:
        assert bool((m[:, 0::2].double().cpu() == x[:, 0::2, 0].double()).all())
    else:
        m[:, 0::2], r[:, 0::2] = mean, rstd
    rows = slice(0, T, 2)
    assert bool((m[:, rows] * r[:, rows]).isinf().all())   # (what the padding must not meet)
    dx, dw, db = dp.layernorm_backward(Gd, xd, wd, m, r)
    assert all(bool(t.isfinite().all()) for t in (dx, dw, db))
    gw, rr = G[:, rows].double() * w.double(), r[:, rows].double().cpu()[..., None]
    want = rr * (gw - gw.mean(dim=-1, keepdim=True))
    bound = rr * (2 * U * gw.abs() + 69 * U * gw.abs().mean(dim=-1, keepdim=True) + 3 * U * gw.abs()) + 1.01 * half(dtype) * want.abs()
    inside(dx[:, rows], want, bound, "dx")


@pytest.mark.parametrize("dtype,d", [(BF16, 8), (BF16, 16), (BF16, 64), (F32, 4), (F32, 16), (F32, 64)])
@pytest.mark.parametrize("value,eps", [(2.0 ** 121, 2.0 ** -16), (-2.0 ** 121, 2.0 ** -16), (2.0 ** 110, 2.0 ** -40)])
def test_rows_as_the_forward_call_takes_them(value, eps, dtype, d):
    """Powers of two: every sum of such a row is exact, and its mean is its value."""
    check(2, 9, d, dtype, value, None, eps ** -0.5)


@pytest.mark.parametrize("dtype,d", [(BF16, 72), (BF16, 520), (BF16, 1032), (BF16, 2056), (BF16, 4104), (BF16, 8200), (BF16, 16392),
                                     (F32, 260), (F32, 516), (F32, 1000), (F32, 1028), (F32, 2052), (F32, 4100), (F32, 8196), (F32, 16388)])
def test_every_width_with_the_rows_own_statistics(dtype, d):
    """In every form of a row on its lanes, with the statistics that the definition gives."""
    check(2, 9, d, dtype, 2.0 ** 120, 2.0 ** 120, 2.0 ** 9)
