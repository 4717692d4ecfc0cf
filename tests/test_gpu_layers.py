"""The differentiable layers (embedding table, attention), and the DP-SGD-RC step
of a Llama-shaped stack that has both.

Ground truth is autograd in float64 on the CPU of the same model written in
plain torch operations, per sample one at a time for the norms. The model runs
in float32 on the GPU: its losses and gradients carry float32 roundings through
a few layers, 1e-4 relative being far above them and far below any mistake.
"""
import copy
import math

import numpy as np
import pytest
import torch
import torch.nn.functional as F
from torch import nn

from workloads import llama_block as lb

pytestmark = pytest.mark.gpu
TINY = dict(layers=2, dim=32, heads=4, kv_heads=2, hidden=64, vocab=16, vocab_in=40, embed_scale=3.0, ops="library")


def dev():
    return torch.device("cuda:0")


def plain_attention(q, k, v, scale=None):
    """Causal attention of one sequence [T][H][D], float64."""
    rep = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(rep, dim=1), v.repeat_interleave(rep, dim=1)
    s = torch.einsum("thd,uhd->htu", q, k) * (scale if scale is not None else 1 / math.sqrt(q.shape[2]))
    s = s.masked_fill(torch.ones(q.shape[0], q.shape[0], dtype=torch.bool).triu(1), -math.inf)
    return torch.einsum("htu,uhd->thd", torch.softmax(s, dim=-1), v)


def rel(a, b):
    a, b = a.detach().double().cpu(), b.detach()
    return float((a - b).norm() / b.norm())


@pytest.mark.parametrize("batched", [True, False])
def test_attention_gradients_run_twice(batched):
    """Two backward passes on one forward pass, of different output gradients,
    one of them repeated over rows as sum() makes it."""
    from sample_grad_norms_amd.layers import attention
    g = torch.Generator().manual_seed(3)
    B, T, Hq, Hkv, D = 3, 41, 4, 2, 40
    shape = (B, T) if batched else (B * T,)
    x = [torch.randn(*shape, h, D, generator=g) for h in (Hq, Hkv, Hkv)]
    cpu = [t.double().requires_grad_(True) for t in x]
    gpu = [t.to(dev()).requires_grad_(True) for t in x]
    cu = [0, 41, 41, 100, 123]
    if batched:
        want = torch.stack([plain_attention(*(t[i] for t in cpu), scale=0.3) for i in range(B)])
        got = attention(*gpu, scale=0.3)
    else:
        want = torch.cat([plain_attention(*(t[a:b] for t in cpu), scale=0.3) for a, b in zip(cu[:-1], cu[1:])])
        got = attention(*gpu, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=dev()), scale=0.3)
    assert got.shape == want.shape and rel(got, want.detach()) <= 1e-5
    w = torch.randn(want.shape, generator=g, dtype=torch.float64)
    for out_w, out_g in ((want.sum(), got.sum()), ((want * w).sum(), (got * w.to(dev()).float()).sum())):
        a = torch.autograd.grad(out_w, cpu, retain_graph=True)
        b = torch.autograd.grad(out_g, gpu, retain_graph=True)
        for i, j in zip(b, a):
            assert rel(i, j) <= 1e-5


def test_attention_of_views_of_one_projection():
    """q, k and v as slices of one projection's output: gradients reach it."""
    from sample_grad_norms_amd.layers import attention
    g = torch.Generator().manual_seed(4)
    B, T, D = 2, 70, 64
    x = torch.randn(B, T, 4 * D, generator=g)
    cpu, gpu = x.double().requires_grad_(True), x.to(dev()).requires_grad_(True)
    q, k, v = gpu.view(B, T, 4, D).split([2, 1, 1], dim=2)
    out = attention(q, k, v)
    qc, kc, vc = cpu.view(B, T, 4, D).split([2, 1, 1], dim=2)
    want = torch.stack([plain_attention(qc[i], kc[i], vc[i]) for i in range(B)])
    w = torch.randn(want.shape, generator=g, dtype=torch.float64)
    (out * w.to(dev()).float()).sum().backward()
    (want * w).sum().backward()
    assert rel(out.detach(), want.detach()) <= 1e-5 and rel(gpu.grad, cpu.grad) <= 1e-5


def test_empty_batches():
    from sample_grad_norms_amd.layers import Embedding, attention
    q = torch.empty(0, 5, 2, 32, device=dev(), requires_grad=True)
    attention(q, q, q).sum().backward()
    assert q.grad.shape == q.shape
    e = Embedding(6, 16, device=dev())
    e(torch.empty(2, 0, dtype=torch.int64, device=dev())).sum().backward()
    assert bool((e.weight.grad == 0).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_embedding_gradient(dtype):
    from sample_grad_norms_amd.layers import Embedding
    g = torch.Generator().manual_seed(5)
    e = Embedding(30, 48, scale=2.5, device=dev(), dtype=dtype)
    tok = torch.randint(-1, 31, (3, 4, 20), generator=g)
    w = torch.randn(3, 4, 20, 48, generator=g).to(dtype)
    out = e(tok.to(dev()))
    W = e.weight.detach().cpu().double().requires_grad_(True)
    ok = (tok >= 0) & (tok < 30)
    want = torch.where(ok[..., None], 2.5 * W[tok.clamp(0, 29)], torch.zeros(1, dtype=torch.float64))
    (out * w.to(dev())).sum().backward()
    (want * w.double()).sum().backward()
    tol = 1e-6 if dtype == torch.float32 else 2 ** -8
    assert rel(out.detach(), want.detach()) <= tol and rel(e.weight.grad, W.grad) <= tol


def plain_stack(model, tok):
    """The model in plain torch operations (float64 on the CPU)."""
    x = model.embed.scale * model.embed.weight[tok.clamp(min=0)] * (tok >= 0)[..., None]
    for layer in model.layers:
        layer.ops = "torch"
        B, T, _ = x.shape
        h = layer.attn_norm(x)
        y = torch.stack([plain_attention(layer.q(h[i]).view(T, layer.heads, layer.hd), layer.k(h[i]).view(T, layer.kv_heads, layer.hd),
                                         layer.v(h[i]).view(T, layer.kv_heads, layer.hd)) for i in range(B)])
        x = x + layer.o(y.reshape(B, T, -1))
        h = layer.mlp_norm(x)
        x = x + layer.down(F.silu(layer.gate(h)) * layer.up(h))
    return model.head(model.norm(x))


def double(model):
    ref = copy.deepcopy(model).double().cpu()
    for m in ref.modules():   # RMSNorm computes in float32 whatever its input is
        if isinstance(m, lb.RMSNorm):
            m.forward = (lambda m: lambda x: x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + m.eps) * m.weight)(m)
    return ref


def per_sample(ref, tok, y):
    weights = [p for p in ref.parameters() if p.requires_grad]
    grads = []
    for i in range(tok.shape[0]):
        logits = plain_stack(ref, tok[i:i + 1])
        loss = F.cross_entropy(logits[0], y[i], reduction="sum")
        grads.append(torch.autograd.grad(loss, weights))
    return weights, grads


def data(seed, B, T):
    tok, y = lb.token_batch(seed, B, T, TINY["vocab_in"], TINY["vocab"])
    tok[0, T - 3:] = -1          # a padded sample
    return tok, y


def test_step_norms_and_clipped_gradients_match_per_sample_gradients():
    from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
    model = lb.build(81, device=dev(), **TINY)
    tok, y = data(82, 4, 19)
    rc = RandomizedClipping(model, C=0.7, noise_multiplier=0.0, estimator="exact")
    assert len(rc.params) == 2 * 7 + 2 and rc.params[-1] is model.embed.weight
    with rc.capture():
        losses = lb.per_sample_loss(model(tok.to(dev())), y.to(dev()))
    n, c = rc.clip_factors(losses)
    rc.clipped_backward(losses, c)     # checks its coverage of the weights, the table among them
    weights, grads = per_sample(double(model), tok, y)
    want = np.array([sum(float((g ** 2).sum()) for g in gs) for gs in grads])
    np.testing.assert_allclose(n.cpu().double().numpy(), want, rtol=1e-4)
    names = {name: p for name, p in model.named_parameters()}
    factors = np.minimum(0.7 / np.sqrt(want), 1.0)
    assert factors.min() < 0.9        # some sample is clipped
    ref_names = [name for name, p in model.named_parameters() if p.requires_grad]
    for j, name in enumerate(ref_names):
        total = sum(f * gs[j] for f, gs in zip(factors, grads))
        assert rel(names[name].grad, total) <= 1e-4, name


def test_step_trains_the_table_in_bfloat16():
    """A few whole steps with padded samples, noise and the Hutchinson
    estimator: everything stays finite and every weight moves."""
    from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
    shape = dict(TINY, dim=256, hidden=512)
    model = lb.build(83, device=dev(), dtype=torch.bfloat16, **shape)
    before = {k: v.detach().clone() for k, v in model.named_parameters() if v.requires_grad}
    rc = RandomizedClipping(model, C=1.0, noise_multiplier=0.5, k=32, seed=1, noise_seed=2)
    opt = torch.optim.SGD(rc.params, lr=0.5)
    for step in range(3):
        tok, y = data(90 + step, 3, 130)
        with rc.capture():
            losses = lb.per_sample_loss(model(tok.to(dev())), y.to(dev()))
        n, c = rc.step(losses, opt)
        assert bool(torch.isfinite(n).all()) and bool((n > 0).all()) and bool((c <= 1).all())
    for k, v in model.named_parameters():
        if v.requires_grad:
            assert bool(torch.isfinite(v).all()) and not torch.equal(v, before[k]), k


def test_the_library_model_matches_the_torch_model():
    """Losses and gradients of the stack with the library's attention against
    the same stack with the float32 one."""
    from sample_grad_norms_amd.layers import Embedding  # noqa: F401  (the table of both)
    a = lb.build(84, device=dev(), **TINY)
    b = lb.build(84, device=dev(), **dict(TINY, ops="torch"))
    tok, y = data(85, 3, 50)
    res = []
    for m in (a, b):
        loss = lb.per_sample_loss(m(tok.to(dev())), y.to(dev()))
        loss.sum().backward()
        res.append((loss.detach(), [p.grad for p in m.parameters() if p.requires_grad]))
    assert rel(res[0][0], res[1][0].cpu().double()) <= 1e-5
    for x, z in zip(res[0][1], res[1][1]):
        assert rel(x, z.cpu().double()) <= 1e-4


class _ReusedTable(nn.Module):
    def __init__(self, device):
        super().__init__()
        from sample_grad_norms_amd.layers import Embedding
        self.emb = Embedding(12, 16, device=device)
        self.head = nn.Linear(16, 8, bias=False, device=device)

    def forward(self, tok):
        return self.head(self.emb(tok) + F.embedding(tok, self.emb.weight))


def test_a_use_of_the_table_outside_its_module_is_caught():
    from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
    model = _ReusedTable(dev())
    rc = RandomizedClipping(model, C=1.0, noise_multiplier=0.0, estimator="exact")
    tok, y = lb.token_batch(86, 3, 9, 12, 8, device=dev())
    with rc.capture():
        losses = lb.per_sample_loss(model(tok), y)
    _, c = rc.clip_factors(losses)
    with pytest.raises(RuntimeError, match="hooks do not see"):
        rc.clipped_backward(losses, c)


class _TwiceLookedUp(nn.Module):
    def __init__(self, device):
        super().__init__()
        from sample_grad_norms_amd.layers import Embedding
        self.emb = Embedding(12, 16, device=device)
        self.head = nn.Linear(16, 8, bias=False, device=device)

    def forward(self, tok):
        return self.head(self.emb(tok) * 0.5 + self.emb(tok.flip(1).contiguous()))


def test_a_table_looked_up_twice_is_one_gradient():
    from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
    torch.manual_seed(6)
    model = _TwiceLookedUp(dev())
    rc = RandomizedClipping(model, C=1.0, noise_multiplier=0.0, estimator="exact")
    tok, y = lb.token_batch(87, 3, 9, 12, 8, device=dev())
    with rc.capture():
        losses = lb.per_sample_loss(model(tok), y)
    n, c = rc.clip_factors(losses)
    rc.clipped_backward(losses, c)
    want = []
    for i in range(3):
        t = tok[i:i + 1]
        W, H = model.emb.weight.detach().double().requires_grad_(True), model.head.weight.detach().double().requires_grad_(True)
        loss = F.cross_entropy(((W[t] * 0.5 + W[t.flip(1)]) @ H.t())[0], y[i], reduction="sum")
        want.append(sum(float((g ** 2).sum()) for g in torch.autograd.grad(loss, [W, H])))
    np.testing.assert_allclose(n.cpu().double().numpy(), np.array(want), rtol=1e-4)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_lone_row_may_have_any_stride(dtype):
    """One token, or one head, of a wider buffer: its stride is never used."""
    import sample_grad_norms_amd as dp
    from sample_grad_norms_amd.layers import attention
    g = torch.Generator().manual_seed(23)
    for N, Hq, Hkv in ((1, 4, 2), (9, 1, 1), (1, 1, 1)):
        D = 64
        x = [torch.randn(N, h, D, generator=g).to(dtype).to(dev()) for h in (Hq, Hkv, Hkv)]
        want, lse = dp.attention_forward(*x)
        strides = [(3 if N == 1 else h * D, 5 if h == 1 else D) for h in (Hq, Hkv, Hkv)]
        odd = [t.as_strided(t.shape, (st, sh, 1)) for t, (st, sh) in zip(x, strides)]
        far = [t.as_strided(t.shape, (1 << 40 if N == 1 else t.stride(0), 1 << 50 if t.shape[1] == 1 else t.stride(1), 1)) for t in x]
        for y in (odd, far):
            o, lse2 = dp.attention_forward(*y)
            assert torch.equal(o, want) and torch.equal(lse, lse2)
            grads = dp.attention_backward(o, *y, o, lse)
            assert all(torch.equal(i, j) for i, j in zip(grads, dp.attention_backward(want, *x, want, lse)))
            assert torch.equal(attention(*y), want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_inputs_and_gradients_off_a_boundary(dtype):
    """q, k, v and the output's gradient as contiguous views that start one element into a
    buffer: the results and gradients of the same values on a boundary, bit for bit."""
    from sample_grad_norms_amd.layers import Embedding, attention
    g = torch.Generator().manual_seed(21)
    N, Hq, Hkv, D = 37, 4, 2, 64

    def off(t):
        return torch.cat([torch.zeros(1, dtype=dtype, device=dev()), t.flatten()])[1:].view(t.shape)

    x = [torch.randn(N, h, D, generator=g).to(dtype).to(dev()).requires_grad_(True) for h in (Hq, Hkv, Hkv)]
    w = torch.randn(N, Hq, D, generator=g).to(dtype).to(dev())
    a = attention(*x)
    want = torch.autograd.grad(a, x, grad_outputs=w)
    b = attention(*(off(t) for t in x))
    got = torch.autograd.grad(b, x, grad_outputs=off(w))
    assert torch.equal(a, b) and all(torch.equal(i, j) for i, j in zip(want, got))
    e = Embedding(30, 48, device=dev(), dtype=dtype)
    tok = torch.randint(0, 30, (3, 20), generator=g).to(dev())
    w = torch.randn(3, 20, 48, generator=g).to(dtype).to(dev())
    (want,) = torch.autograd.grad(e(tok), [e.weight], grad_outputs=w)
    (got,) = torch.autograd.grad(e(tok), [e.weight], grad_outputs=off(w))
    assert torch.equal(want, got)


def test_ids_need_not_be_contiguous():
    from sample_grad_norms_amd.layers import Embedding
    e = Embedding(30, 48, device=dev())
    tok = torch.randint(0, 30, (4, 21), generator=torch.Generator().manual_seed(22)).to(dev())
    for ids in (tok[:, :-1], tok[:, 1:], tok.t(), tok[0].expand(4, 21), tok[::2, ::3]):
        out = e(ids)
        assert torch.equal(out, e(ids.contiguous())) and torch.equal(out, e.weight[ids])
        (got,) = torch.autograd.grad(out.sum(), [e.weight])
        assert torch.equal(got, torch.bincount(ids.flatten(), minlength=30)[:, None].expand(30, 48).float())


def test_a_write_to_the_ids_before_the_backward_pass_is_an_error():
    """Contiguous or not: the gradient would be that of other rows."""
    from sample_grad_norms_amd.layers import Embedding
    e = Embedding(30, 48, device=dev())
    for cut in (slice(None), slice(0, 20), slice(3, 4)):
        tok = torch.randint(0, 30, (4, 21), generator=torch.Generator().manual_seed(24)).to(dev())
        ids = tok[:, cut]
        out = e(ids)
        (got,) = torch.autograd.grad(out.sum(), [e.weight], retain_graph=True)
        assert torch.equal(got, torch.bincount(ids.flatten(), minlength=30)[:, None].expand(30, 48).float())
        tok += 1
        with pytest.raises(RuntimeError, match="modified by an inplace"):
            out.sum().backward()
