"""The norm layers and attention with changed scores as differentiable layers, and the
DP-SGD-RC step of a Llama-shaped stack that trains its norms and caps, biases and
prefixes its attention.

Ground truth is autograd in float64 on the CPU of the same model in plain torch
operations, per sample one at a time for the norms. The model runs in float32 on the
GPU: its losses and gradients carry float32 roundings through a few layers, 1e-4
relative being far above them and far below any mistake.
"""
import copy
import math

import numpy as np
import pytest
import torch
import torch.nn.functional as F

from workloads import llama_block as lb

pytestmark = pytest.mark.gpu
TINY = dict(layers=2, dim=32, heads=4, kv_heads=2, hidden=64, vocab=16, vocab_in=40, embed_scale=3.0)


def dev():
    return torch.device("cuda:0")


def rel(a, b):
    a, b = a.detach().double().cpu(), b.detach()
    return float((a - b).norm() / b.norm())


def plain_norm(x, m):
    """The layer m (its weights float64) of x."""
    c = x if m.rms else x - x.mean(-1, keepdim=True)
    y = c / torch.sqrt(c.pow(2).mean(-1, keepdim=True) + m.eps) * m.weight
    return y if m.bias is None else y + m.bias


def random_weights(model, seed):
    """Gains around 1 and biases around 0 in every norm of the model."""
    from sample_grad_norms_amd.layers import LayerNorm
    g = torch.Generator().manual_seed(seed)
    for m in model.modules():
        if isinstance(m, LayerNorm):
            for p in m.parameters(recurse=False):
                with torch.no_grad():
                    p.add_((torch.randn(p.shape, generator=g) * 0.3).to(p))
    return model


@pytest.mark.parametrize("kind", ["layer", "gain", "rms"])
@pytest.mark.parametrize("shape", [(3, 41, 72), (5, 2048), (2, 3, 4, 24), (64,)])
def test_norm_gradients_run_twice(shape, kind):
    from sample_grad_norms_amd.layers import LayerNorm, RMSNorm
    g = torch.Generator().manual_seed(61)
    d = shape[-1]
    m = RMSNorm(d, eps=1e-4, device=dev()) if kind == "rms" else LayerNorm(d, eps=1e-4, bias=kind == "layer", device=dev())
    random_weights(m, 62)
    ref = copy.deepcopy(m).double().cpu()
    x = torch.randn(*shape, generator=g)
    xc, xg = x.double().requires_grad_(True), x.to(dev()).requires_grad_(True)
    want, got = plain_norm(xc, ref), m(xg)
    assert got.shape == want.shape and rel(got, want) <= 1e-6
    ws = torch.randn(*shape, generator=g, dtype=torch.float64)
    for a, b in ((want.sum(), got.sum()), ((want * ws).sum(), (got * ws.to(dev()).float()).sum())):
        for i, j in zip(torch.autograd.grad(b, [xg, *m.parameters()], retain_graph=True),
                        torch.autograd.grad(a, [xc, *ref.parameters()], retain_graph=True)):
            # (the gradient of a sum of normalised rows nearly cancels: against the size of what is summed)
            assert float((i.double().cpu() - j).norm()) <= 1e-5 * float(j.norm()) + 1e-5 * math.sqrt(j.numel())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_views_and_frozen_weights(dtype):
    """Inputs and gradients that are not contiguous or off a 16-byte boundary give what copies
    give, bit for bit; what needs no gradient gets none."""
    from sample_grad_norms_amd.layers import LayerNorm
    g = torch.Generator().manual_seed(63)
    m = random_weights(LayerNorm(48, device=dev(), dtype=dtype), 64)
    x = torch.randn(7, 5, 48, generator=g).to(dtype).to(dev())
    w = torch.randn(7, 5, 48, generator=g).to(dtype).to(dev())

    def off(t):
        return torch.cat([torch.zeros(1, dtype=dtype, device=dev()), t.flatten()])[1:].view(t.shape)
    views = [x, off(x), x.transpose(0, 1).contiguous().transpose(0, 1), torch.cat([x, x], dim=2)[:, :, 48:]]
    base = None
    for v in views:
        for up in (w, off(w), w.transpose(0, 1).contiguous().transpose(0, 1)):
            v = v.detach().requires_grad_(True)
            y = m(v)
            got = (y, *torch.autograd.grad(y, [v, m.weight, m.bias], grad_outputs=up))
            base = base or got
            assert all(torch.equal(a, b) for a, b in zip(base, got))
    m.weight.requires_grad_(False)
    y = m(x)
    (db,) = torch.autograd.grad(y, [m.bias], grad_outputs=w)
    assert torch.equal(db, base[3])
    m.bias.requires_grad_(False)
    assert not m(x).requires_grad
    v = x.clone().requires_grad_(True)
    (dx,) = torch.autograd.grad(m(v), [v], grad_outputs=w)
    assert torch.equal(dx, base[1])


def test_a_write_to_the_input_before_the_backward_pass_is_an_error():
    from sample_grad_norms_amd.layers import RMSNorm
    m = RMSNorm(32, device=dev())
    x = torch.randn(4, 32, device=dev())
    y = m(x)
    x += 1
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.sum().backward()


def plain_attention(q, k, v, cap, slopes, p):
    """Attention of one sequence [T][H][D], float64."""
    rep, T = q.shape[1] // k.shape[1], q.shape[0]
    k, v = k.repeat_interleave(rep, dim=1), v.repeat_interleave(rep, dim=1)
    s = torch.einsum("thd,uhd->htu", q, k) / math.sqrt(q.shape[2])
    if cap:
        s = cap * torch.tanh(s / cap)
    at = torch.arange(T)
    if slopes is not None:
        s = s - slopes.double()[:, None, None] * (at[:, None] - at[None]).abs()
    s = s.masked_fill((at[None] > at[:, None]) & (at[None] >= p), -math.inf)
    return torch.einsum("htu,uhd->thd", torch.softmax(s, dim=-1), v)


@pytest.mark.parametrize("batched", [True, False])
@pytest.mark.parametrize("cap,biased,prefixed", [(2.0, False, False), (None, True, False), (None, False, True), (3.0, True, True)])
def test_attention_gradients_run_twice(batched, cap, biased, prefixed):
    from sample_grad_norms_amd.layers import attention
    g = torch.Generator().manual_seed(65)
    B, T, Hq, Hkv, D = 3, 41, 4, 2, 40
    cu = [0, 41, 82, 123] if batched else [0, 41, 41, 100, 123]
    x = [torch.randn(*((B, T) if batched else (B * T,)), h, D, generator=g) for h in (Hq, Hkv, Hkv)]
    slopes = torch.tensor([0.4, 0.1, -0.03, 0.0]) if biased else None
    prefix = [7, 60, 33] if batched else [7, 5, 33, 0]
    cpu = [t.double().requires_grad_(True) for t in x]
    gpu = [t.to(dev()).requires_grad_(True) for t in x]
    flat = [t.reshape(B * T, *t.shape[-2:]) for t in cpu]
    want = torch.cat([plain_attention(*(t[a:b] for t in flat), cap, slopes, p if prefixed else 0) for a, b, p in zip(cu[:-1], cu[1:], prefix)])
    got = attention(*gpu, cu_seqlens=None if batched else torch.tensor(cu, dtype=torch.int32, device=dev()), cap=cap,
                    slopes=None if slopes is None else slopes.to(dev()),
                    prefix=torch.tensor(prefix, dtype=torch.int32, device=dev()) if prefixed else None)
    want = want.view(got.shape)
    assert rel(got, want) <= 1e-5
    w = torch.randn(want.shape, generator=g, dtype=torch.float64)
    for a, b in ((want.sum(), got.sum()), ((want * w).sum(), (got * w.to(dev()).float()).sum())):
        for i, j in zip(torch.autograd.grad(b, gpu, retain_graph=True), torch.autograd.grad(a, cpu, retain_graph=True)):
            assert rel(i, j) <= 2e-5 or float(j.norm()) < 1e-6


def test_empty_batches():
    from sample_grad_norms_amd.layers import LayerNorm, attention
    q = torch.empty(0, 5, 2, 32, device=dev(), requires_grad=True)
    attention(q, q, q, cap=4.0, slopes=torch.ones(2, device=dev()), prefix=torch.empty(0, dtype=torch.int32, device=dev())).sum().backward()
    assert q.grad.shape == q.shape
    m = LayerNorm(16, device=dev())
    m(torch.empty(2, 0, 16, device=dev())).sum().backward()
    assert bool((m.weight.grad == 0).all()) and bool((m.bias.grad == 0).all())


def plain_stack(model, tok, prefix):
    """One sample [T] through the model (float64 on the CPU) in plain torch operations."""
    x = model.embed.scale * model.embed.weight[tok.clamp(min=0)] * (tok >= 0)[..., None]
    for layer in model.layers:
        T = x.shape[0]
        h = plain_norm(x, layer.attn_norm)
        y = plain_attention(layer.q(h).view(T, layer.heads, layer.hd), layer.k(h).view(T, layer.kv_heads, layer.hd),
                            layer.v(h).view(T, layer.kv_heads, layer.hd), layer.cap, layer.slopes, prefix)
        x = x + layer.o(y.reshape(T, -1))
        h = plain_norm(x, layer.mlp_norm)
        x = x + layer.down(F.silu(layer.gate(h)) * layer.up(h))
    return model.head(plain_norm(x, model.norm))


@pytest.mark.parametrize("norm,how", [("rms", dict(cap=1.5)), ("layer", dict(distance=True)), ("layer", dict(cap=1.5, distance=True))])
def test_step_norms_and_clipped_gradients_match_per_sample_gradients(norm, how):
    from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
    model = random_weights(lb.build(71, device=dev(), ops="library", norm=norm, **TINY, **how), 72)
    B, T = 4, 19
    tok, y = lb.token_batch(73, B, T, TINY["vocab_in"], TINY["vocab"])
    tok[0, T - 3:] = -1          # a padded sample
    prefix = torch.tensor([3, 0, 19, 8], dtype=torch.int32)
    rc = RandomizedClipping(model, C=0.7, noise_multiplier=0.0, estimator="exact")
    assert len(rc.params) == 2 * 7 + 2 + 5 * (2 if norm == "layer" else 1)
    with rc.capture():
        losses = lb.per_sample_loss(model(tok.to(dev()), prefix.to(dev())), y.to(dev()))
    n, c = rc.clip_factors(losses)
    rc.clipped_backward(losses, c)     # checks its coverage of the weights, the norms' among them
    ref = copy.deepcopy(model).double().cpu()
    params = dict(ref.named_parameters())
    grads = [torch.autograd.grad(F.cross_entropy(plain_stack(ref, tok[i], int(prefix[i])), y[i], reduction="sum"), list(params.values()))
             for i in range(B)]
    want = np.array([sum(float((g ** 2).sum()) for g in gs) for gs in grads])
    np.testing.assert_allclose(n.cpu().double().numpy(), want, rtol=1e-4)
    factors = np.minimum(0.7 / np.sqrt(want), 1.0)
    assert factors.min() < 0.9        # some sample is clipped
    for j, (name, p) in enumerate(model.named_parameters()):
        assert rel(p.grad, sum(f * gs[j] for f, gs in zip(factors, grads))) <= 1e-4, name


@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_step_trains_the_norms_in_bfloat16(norm):
    """A few whole steps with padded samples, noise and the Hutchinson estimator: everything
    stays finite and every weight moves."""
    from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
    shape = dict(TINY, dim=256, hidden=512)
    model = lb.build(74, device=dev(), dtype=torch.bfloat16, ops="library", norm=norm, cap=20.0, distance=True, **shape)
    before = {k: v.detach().clone() for k, v in model.named_parameters()}
    rc = RandomizedClipping(model, C=1.0, noise_multiplier=0.5, k=32, seed=1, noise_seed=2)
    opt = torch.optim.SGD(rc.params, lr=0.5)
    for step in range(3):
        tok, y = lb.token_batch(90 + step, 3, 130, shape["vocab_in"], shape["vocab"])
        tok[0, 127:] = -1
        with rc.capture():
            losses = lb.per_sample_loss(model(tok.to(dev()), torch.tensor([5, 0, 64], dtype=torch.int32, device=dev())), y.to(dev()))
        n, c = rc.step(losses, opt)
        assert bool(torch.isfinite(n).all()) and bool((n > 0).all()) and bool((c <= 1).all())
    for k, v in model.named_parameters():
        assert bool(torch.isfinite(v).all()) and not torch.equal(v, before[k]), k


def test_the_library_model_matches_the_torch_model():
    """Losses and gradients of the stack with the library's attention, its scores capped, biased
    and with a prefix, against the same stack with the float32 one."""
    shape = dict(TINY, norm="layer", cap=2.0, distance=True)
    models = [random_weights(lb.build(75, device=dev(), ops=ops, **shape), 76) for ops in ("library", "torch")]
    tok, y = lb.token_batch(77, 3, 50, TINY["vocab_in"], TINY["vocab"])
    prefix = torch.tensor([10, 0, 50], dtype=torch.int32, device=dev())
    res = []
    for m in models:
        loss = lb.per_sample_loss(m(tok.to(dev()), prefix), y.to(dev()))
        loss.sum().backward()
        res.append((loss.detach(), [p.grad for p in m.parameters()]))
    assert rel(res[0][0], res[1][0].cpu().double()) <= 1e-5
    for a, b in zip(res[0][1], res[1][1]):
        assert rel(a, b.cpu().double()) <= 1e-4


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_run_of_all_calls_captured_and_replayed(dtype):
    """Norm, attention, norm, their gradients and per-sample norms in one captured graph,
    replayed beside eager work, with two graphs that have workspaces of their own."""
    import sample_grad_norms_amd as dp
    B, T, H, D = 2, 90, 4, 64
    d = H * D
    g = torch.Generator().manual_seed(78)
    make = lambda *s: torch.randn(*s, generator=g).to(dtype).to(dev())
    w, b = make(d), make(d)
    how = dict(sequences=B, cap=5.0, slopes=torch.rand(H, generator=g).to(dev()),
               prefix=torch.tensor([20, 70], dtype=torch.int32, device=dev()))
    sets = [(make(B, T, d), make(B, T, d)) for _ in range(3)]

    def run(x, do):
        y, mean, rstd = dp.layernorm_forward(x, w, b)
        q = y.view(B * T, H, D)
        o, lse = dp.attention_forward(q, q, q, **how)
        z, _, r2 = dp.layernorm_forward(o.view(B, T, d), w, rms=True)
        dz, dw2, _ = dp.layernorm_backward(do, o.view(B, T, d), w, None, r2)
        dq, dk, dv = dp.attention_backward(dz.view(B * T, H, D), q, q, q, o, lse, **how)
        dy = (dq + dk + dv).view(B, T, d)
        n = dp.layernorm_norm(x, dy)
        dp.layernorm_norm(o.view(B, T, d), do, rms=True, out=n, accumulate=True)
        c = dp.clip_factors(n, 1.0)
        return (z, n, c, dw2, *dp.layernorm_backward(dy, x, w, mean, rstd, weights=c))
    want = [run(*s) for s in sets]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        held = [t.clone() for t in sets[0]]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run(*held)
        graphs.append((graph, held, out))
    for j in (1, 2, 0, 1):
        for i, (graph, held, _) in enumerate(graphs):
            for h, t in zip(held, sets[(j + i) % 3]):
                h.copy_(t)
            graph.replay()
        eager = run(*sets[j])
        torch.cuda.synchronize()
        for i, (_, _, out) in enumerate(graphs):
            assert all(torch.equal(p, q) for p, q in zip(out, want[(j + i) % 3])), (j, i)
        assert all(torch.equal(p, q) for p, q in zip(eager, want[j]))
