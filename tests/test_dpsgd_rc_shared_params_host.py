"""What the step wrapper does about one parameter in two places of a norm layer, and
that it noises and averages every parameter once, on the CPU."""
import pytest
import torch
from torch import nn

from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
from sample_grad_norms_amd.layers import LayerNorm, RMSNorm

D = 8


def model(*norms):
    return nn.Sequential(*norms, nn.Linear(D, D, bias=False))


@pytest.mark.parametrize("verify", [True, False])
@pytest.mark.parametrize("trained", [True, False])
def test_a_gain_that_is_its_own_bias_is_refused(verify, trained):
    """Its gradient is sum G (h + 1), whose norm is not that of the two sums G h and G: up to
    the square root of two times larger."""
    m = model(LayerNorm(D))
    m[0].bias = m[0].weight
    m[0].weight.requires_grad_(trained)
    if trained:
        with pytest.raises(ValueError, match="gain and bias"):
            RandomizedClipping(m, C=1.0, noise_multiplier=1.0, verify_coverage=verify)
    else:   # (nothing of it is clipped)
        assert len(RandomizedClipping(m, C=1.0, noise_multiplier=1.0, verify_coverage=verify).params) == 1


def test_every_parameter_counts_once():
    """Of layers that share gain and bias, or one of several kinds, each parameter is listed once,
    so that the noise and the division by the batch reach it once."""
    a, b, c = LayerNorm(D), LayerNorm(D), RMSNorm(D)
    b.weight, b.bias = a.weight, a.bias
    m = model(a, b, c, c)
    rc = RandomizedClipping(m, C=1.0, noise_multiplier=0.0)
    assert [id(p) for p in rc.params] == [id(m[-1].weight), id(a.weight), id(a.bias), id(c.weight)]
    for p in rc.params:
        p.grad = torch.full_like(p, 6.0)
    rc._batch = 3
    rc.add_noise()
    assert all(bool((p.grad == 2.0).all()) for p in rc.params)
