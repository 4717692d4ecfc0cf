"""The step wrapper's norm layers without a GPU: what it covers, refuses, records and
hands to the norm path, whose calls are replaced by their definitions in plain torch.

The models are small and in float64; sums of a few hundred terms carry roundings of
1e-13, and a gradient given to the wrong sample or weight changes a norm by far more.
"""
import pytest
import torch
from torch import nn

from workloads import llama_block as lb

B, T, D = 4, 6, 8


@pytest.fixture(autouse=True)
def plain_calls(monkeypatch):
    import sample_grad_norms_amd as dp
    from sample_grad_norms_amd import layers

    def parts(x, eps, rms):
        mean = None if rms else x.mean(-1)
        c = x if rms else x - mean[..., None]
        return mean, 1.0 / torch.sqrt((c * c).mean(-1) + eps), c

    def forward(x, weight, bias=None, eps=1e-5, rms=False, out=None):
        mean, rstd, c = parts(x, eps, rms)
        y = c * rstd[..., None] * weight
        return y if bias is None else y + bias, mean, rstd

    def backward(dy, x, weight, mean, rstd, bias=True, weights=None, need_dx=True, need_dw=True):
        h = (x if mean is None else x - mean[..., None]) * rstd[..., None]
        f = 1.0 if weights is None else weights.to(x.dtype).view(-1, *[1] * (x.dim() - 1))
        g = dy * weight
        dx = g - h * (g * h).mean(-1, keepdim=True)
        if mean is not None:
            dx = dx - g.mean(-1, keepdim=True)
        total = lambda t: (t * f).reshape(-1, x.shape[-1]).sum(0)
        return (dx * rstd[..., None] if need_dx else None, total(dy * h) if need_dw else None,
                total(dy) if bias and mean is not None else None)

    def norm(x, G, eps=1e-5, rms=False, gain=True, bias=True, out=None, accumulate=False):
        _, rstd, c = parts(x, eps, rms)
        n = torch.zeros(x.shape[0], dtype=x.dtype)
        if gain:
            n = n + (G * c * rstd[..., None]).sum(1).pow(2).sum(1)
        if bias and not rms:
            n = n + G.sum(1).pow(2).sum(1)
        return out.add_(n) if accumulate else out.copy_(n)

    def exact(A, G, out=None, accumulate=False):
        per = (A.transpose(1, 2) @ G).pow(2).sum((1, 2))
        return out.add_(per) if accumulate else out.copy_(per)

    monkeypatch.setattr(dp, "layernorm_forward", forward)
    monkeypatch.setattr(dp, "layernorm_backward", backward)
    monkeypatch.setattr(dp, "layernorm_norm", norm)
    monkeypatch.setattr(dp, "exact", exact)
    monkeypatch.setattr(dp, "clip_factors", lambda n, C: torch.clamp(C / n.sqrt(), max=1.0))
    assert layers.dp is dp


class _Model(nn.Module):
    """norms in a row with linear layers between, and what `use` makes of them."""

    def __init__(self, use=None, kinds=("layer", "rms", "layer")):
        super().__init__()
        from sample_grad_norms_amd.layers import LayerNorm, RMSNorm
        f64 = dict(dtype=torch.float64)
        self.norms = nn.ModuleList(LayerNorm(D, **f64) if k == "layer" else LayerNorm(D, bias=False, **f64) if k == "gain" else RMSNorm(D, **f64)
                                   for k in kinds)
        self.linears = nn.ModuleList(nn.Linear(D, D, bias=False, **f64) for _ in kinds)
        g = torch.Generator().manual_seed(1)
        for p in self.parameters():
            with torch.no_grad():
                p.add_(torch.randn(p.shape, generator=g, dtype=torch.float64) * 0.3)
        self.use = use

    def forward(self, x):
        if self.use is not None:
            return self.use(self, x)
        for n, l in zip(self.norms, self.linears):
            x = x + l(torch.tanh(n(x)))
        return x


def inputs(b=B, t=T, seed=2):
    return torch.randn(b, t, D, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def losses_of(model, x):
    w = torch.randn(x.shape, generator=torch.Generator().manual_seed(3), dtype=torch.float64)
    return (model(x) * w).sum((1, 2))


def step(model, x, C=1e9, **kw):
    from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
    rc = RandomizedClipping(model, C=C, noise_multiplier=0.0, estimator="exact", **kw)
    with rc.capture():
        losses = losses_of(model, x)
    n, c = rc.clip_factors(losses)
    rc.clipped_backward(losses, c)
    assert rc._norm_recs == []
    return n, c


def true_grads(model, x):
    params = [p for p in model.parameters() if p.requires_grad]
    return params, [[torch.zeros_like(p) if g is None else g for p, g in
                     zip(params, torch.autograd.grad(l, params, retain_graph=True, allow_unused=True))] for l in losses_of(model, x)]


def check(model, x, C, **kw):
    params, grads = true_grads(model, x)
    want = torch.stack([sum((g ** 2).sum() for g in gs) for gs in grads])
    n, c = step(model, x, C, **kw)
    assert torch.allclose(n.double(), want, rtol=1e-6)
    factors = torch.clamp(C / want.sqrt(), max=1.0)
    assert C > 1e8 or float(factors.min()) < 0.9
    for j, p in enumerate(params):
        # n and c are float32: n is off by half a step of 2^-23, its root by half of that, c by another half
        # step of its own, in all below 2^-22 relative, of each sample's share
        terms = [f * gs[j] for f, gs in zip(factors, grads)]
        got = torch.zeros_like(p) if p.grad is None else p.grad   # (a weight that is not used)
        assert bool(((got - sum(terms)).abs() <= 2.0 ** -22 * sum(t.abs() for t in terms) + 1e-12).all())


@pytest.mark.parametrize("kinds", [("layer",), ("rms",), ("gain",), ("layer", "rms", "layer")])
@pytest.mark.parametrize("C", [1e9, 5.0])
def test_norms_and_clipped_gradients(kinds, C):
    check(_Model(kinds=kinds), inputs(), C)


@pytest.mark.parametrize("frozen", [["norms.0.weight"], ["norms.0.bias"], ["norms.0.weight", "norms.0.bias"],
                                    ["linears.0.weight", "linears.1.weight", "linears.2.weight"]])
def test_frozen_weights_do_not_count(frozen):
    from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
    model = _Model()
    for name, p in model.named_parameters():
        p.requires_grad_(name not in frozen)
    assert len(RandomizedClipping(model, C=1.0, noise_multiplier=0.0).params) == 3 + 5 - len(frozen)
    check(model, inputs(), 4.0)


def test_a_norm_used_twice_and_norms_of_one_weight():
    """Their uses make one gradient; so do those of inputs of other shapes."""
    def twice(m, x):
        h = m.norms[0](x) + m.norms[0](x.flip(1) * 0.5 + 1.0)
        return m.linears[0](h) + m.norms[2](x.reshape(x.shape[0], 2, -1, D)).reshape(x.shape) * 2.0

    check(_Model(twice, ("layer", "rms", "layer")), inputs(), 3.0)
    model = _Model()
    model.norms[2].weight, model.norms[2].bias = model.norms[0].weight, model.norms[0].bias
    check(model, inputs(), 3.0)


def test_what_is_shared_in_part_is_refused():
    from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
    for change in ("weight", "bias", "eps", "kind", "linear"):
        model = _Model()
        if change in ("weight", "eps"):
            model.norms[2].weight = model.norms[0].weight
        if change in ("bias", "eps"):
            model.norms[2].bias = model.norms[0].bias
        if change == "eps":
            model.norms[2].eps = 1e-3
        if change == "kind":
            model.norms[1].weight = model.norms[0].weight
        if change == "linear":
            model.other = nn.Module()
            model.other.weight = model.norms[0].weight
        with pytest.raises(ValueError, match="share"):
            RandomizedClipping(model, C=1.0, noise_multiplier=0.0)


def test_a_use_outside_the_module_is_caught():
    def outside(m, x):
        return m.linears[0](m.norms[0](x) + x * m.norms[0].weight)
    with pytest.raises(RuntimeError, match="hooks do not see"):
        step(_Model(outside), inputs())


@pytest.mark.parametrize("verify", [True, False])
def test_rows_that_samples_share_are_refused(verify):
    """A norm of rows that are added to every sample: by shape, or by the first step's check."""
    def shared(m, x):
        return m.linears[0](x + m.norms[0](torch.linspace(-1, 1, T * D, dtype=torch.float64).view(T, D)))

    with pytest.raises(ValueError, match="sample"):
        step(_Model(shared), inputs(), verify_coverage=verify)
    with pytest.raises((ValueError, RuntimeError), match="sample"):   # as many rows as samples
        step(_Model(shared), inputs(b=T), verify_coverage=verify)


def test_torch_norms_are_refused():
    from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
    with pytest.raises(ValueError, match="unclipped"):
        RandomizedClipping(nn.Sequential(nn.LayerNorm(8), nn.Linear(8, 8, bias=False)), C=1.0, noise_multiplier=1.0)


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_the_stack_with_norms_that_train(norm):
    from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
    model = lb.build(5, layers=1, dim=32, heads=2, kv_heads=1, hidden=64, vocab=16, norm=norm, cap=5.0, distance=True)
    rc = RandomizedClipping(model, C=1.0, noise_multiplier=1.0)
    assert len(rc.params) == 8 + 3 * (2 if norm == "layer" else 1)
    plain = dict(lb.build(5, layers=1, dim=32, heads=2, kv_heads=1, hidden=64, vocab=16).named_parameters())
    assert all(torch.equal(p, plain[n]) for n, p in model.named_parameters() if n in plain)
    with pytest.raises(ValueError, match="norm"):
        lb.LlamaStack(layers=1, dim=32, heads=2, kv_heads=1, hidden=64, vocab=16, norm="other")


@pytest.mark.parametrize("C", [1e9, 1.0])
def test_a_bias_whose_gradient_cancels(C):
    """What a sample's rows have in common is taken off behind the norm (as a softmax takes it
    off its keys): the bias's gradient is zero up to rounding, which is no error."""
    def centred(m, x):
        h = m.norms[0](x)
        return m.linears[0](h - h.mean(1, keepdim=True))
    model, x = _Model(centred, ("layer",)), inputs()
    params, grads = true_grads(model, x)
    at = [j for j, p in enumerate(params) if p is model.norms[0].bias]
    assert all(float(gs[at[0]].abs().max()) < 1e-12 for gs in grads)
    n, c = step(model, x, C)
    assert torch.allclose(n.double(), torch.stack([sum((g ** 2).sum() for g in gs) for gs in grads]), rtol=1e-6)


def test_a_parameter_that_a_subclass_adds_is_refused():
    """Only gain and bias have a norm here; anything else a norm layer holds would go unclipped."""
    from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
    from sample_grad_norms_amd.layers import RMSNorm

    class Gated(RMSNorm):
        def __init__(self, dim, **kw):
            super().__init__(dim, **kw)
            self.gate = nn.Parameter(torch.ones(dim, dtype=torch.float64))

        def forward(self, x):
            return super().forward(x) * self.gate

    model = nn.Sequential(Gated(D, dtype=torch.float64))
    with pytest.raises(ValueError, match="gate"):
        RandomizedClipping(model, C=1.0, noise_multiplier=0.0)
    model[0].gate.requires_grad_(False)
    assert [p is model[0].weight for p in RandomizedClipping(model, C=1.0, noise_multiplier=0.0).params] == [True]
    for held in (0, 1):   # its own gain, or another layer's, in the added place
        model = nn.Sequential(Gated(D, dtype=torch.float64), RMSNorm(D, dtype=torch.float64))
        model[0].gate = model[held].weight
        with pytest.raises(ValueError, match="gate"):
            RandomizedClipping(model, C=1.0, noise_multiplier=0.0)


def test_an_input_changed_in_place_later_is_recorded_as_it_was():
    """A layer copies rows that it cannot read as they lie, so autograd lets them be changed
    behind it; the recording is of what the layer saw."""
    def use(m, x):
        h = (x * 1.0).transpose(0, 1).contiguous().transpose(0, 1)   # [B][T][D], not contiguous
        y = m.norms[0](h)
        h.add_(inputs(seed=9))
        return y

    model, x = _Model(use, kinds=("layer",)), inputs()
    params, per = true_grads(model, x)
    n, _ = step(model, x, verify_coverage=False)
    want = torch.stack([sum((g ** 2).sum() for g in gs) for gs in per])
    assert torch.allclose(n.double(), want, rtol=1e-6, atol=0)   # (n is kept in float32: a few halves of 2^-23)
