"""Which rows belong to which sample in the step wrapper, without a GPU: the
norm path's calls are replaced by their definitions in plain torch, so what is
tested is what the wrapper records and hands to them.

The models are small and in float64; sums of a few hundred terms carry roundings
of 1e-13, and a row given to the wrong sample changes a norm by far more.
"""
import pytest
import torch
from torch import nn

B, T, V, D = 4, 32, 32, 8


@pytest.fixture(autouse=True)
def plain_calls(monkeypatch):
    import sample_grad_norms_amd as dp

    def lookup(tokens, W, scale=1.0):
        ok = ((tokens >= 0) & (tokens < W.shape[0]))[..., None]
        return torch.where(ok, scale * W[tokens.clamp(0, W.shape[0] - 1)], torch.zeros((), dtype=W.dtype))

    def grad(order, G, V=None, scale=1.0, weights=None):
        tok, V = order if isinstance(order, tuple) else (order, V)
        w = torch.ones(G.shape[0], dtype=G.dtype) if weights is None else weights.to(G.dtype)
        rows = (G * w.view(-1, 1, 1)).reshape(-1, G.shape[2])
        return scale * torch.zeros(V, G.shape[2], dtype=G.dtype).index_add_(0, tok.reshape(-1).long(), rows)

    def norm(order, G, scale=1.0, out=None, accumulate=False):
        tok, V = order
        per = torch.stack([(grad((tok[i:i + 1], V), G[i:i + 1], scale=scale) ** 2).sum() for i in range(G.shape[0])])
        return out.add_(per) if accumulate else out.copy_(per)

    def exact(A, G, out=None, accumulate=False):
        per = (A.transpose(1, 2) @ G).pow(2).sum((1, 2))
        return out.add_(per) if accumulate else out.copy_(per)

    monkeypatch.setattr(dp, "embed_lookup", lookup)
    monkeypatch.setattr(dp, "embed_order", lambda tok, V: (tok.clone(), V))
    monkeypatch.setattr(dp, "embed_norm", norm)
    monkeypatch.setattr(dp, "embed_grad", grad)
    monkeypatch.setattr(dp, "exact", exact)
    monkeypatch.setattr(dp, "clip_factors", lambda n, C: torch.clamp(C / n.sqrt(), max=1.0))


class _Positions(nn.Module):
    """A token table and a learned position table, whose ids the caller makes."""

    def __init__(self, ids):
        super().__init__()
        from sample_grad_norms_amd.layers import Embedding
        self.emb, self.pos = Embedding(V, D, dtype=torch.float64), Embedding(T, D, dtype=torch.float64)
        self.head = nn.Linear(D, 5, bias=False, dtype=torch.float64)
        self.ids = ids

    def forward(self, tok):
        return self.head(torch.tanh(self.emb(tok) + self.pos(self.ids(tok))))


def losses_of(model, tok, seed=3):
    w = torch.randn(tok.shape[0], tok.shape[1], 5, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
    return (model(tok) * w).sum((1, 2))


def step(model, tok, C=1e9, **kw):
    """One step in which nothing is clipped (unless C says so): (n, c)."""
    from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
    rc = RandomizedClipping(model, C=C, noise_multiplier=0.0, estimator="exact", **kw)
    with rc.capture():
        losses = losses_of(model, tok)
    n, c = rc.clip_factors(losses)
    rc.clipped_backward(losses, c)
    return n, c


def true_norms(model, tok):
    losses = losses_of(model, tok)
    params = list(model.parameters())
    return torch.stack([sum((g ** 2).sum() for g in torch.autograd.grad(x, params, retain_graph=True)) for x in losses])


def tokens(b=B, t=T):
    return torch.randint(0, V, (b, t), generator=torch.Generator().manual_seed(5))


@pytest.mark.parametrize("ids", [lambda tok: torch.arange(T), lambda tok: torch.arange(T)[None]])
@pytest.mark.parametrize("verify", [True, False])
def test_a_table_looked_up_once_for_the_batch_is_refused(ids, verify):
    torch.manual_seed(1)
    with pytest.raises(ValueError, match="sample"):
        step(_Positions(ids), tokens(), verify_coverage=verify)


@pytest.mark.parametrize("verify", [True, False])
def test_as_many_positions_as_samples_are_refused(verify):
    """pos(arange(T)) with T == B has the shape of one id a sample."""
    torch.manual_seed(2)
    with pytest.raises((ValueError, RuntimeError), match="sample"):
        step(_Positions(lambda tok: torch.arange(4)), tokens(4, 4), verify_coverage=verify)


class _SequenceFirst(nn.Module):
    def __init__(self):
        super().__init__()
        from sample_grad_norms_amd.layers import Embedding
        self.emb = Embedding(V, D, dtype=torch.float64)
        self.head = nn.Linear(D, 5, bias=False, dtype=torch.float64)

    def forward(self, tok):
        return self.head(torch.tanh(self.emb(tok.t().contiguous()))).transpose(0, 1)


@pytest.mark.parametrize("t", [B, 2 * B, 7])
def test_ids_with_the_positions_first_are_refused(t):
    torch.manual_seed(3)
    with pytest.raises((ValueError, RuntimeError), match="sample"):
        step(_SequenceFirst(), tokens(B, t))


class _SharedInput(nn.Module):
    """A linear layer applied once to rows that every sample then uses."""

    def __init__(self, lead):
        super().__init__()
        self.mix, self.head = nn.Linear(D, D, bias=False, dtype=torch.float64), nn.Linear(D, 5, bias=False, dtype=torch.float64)
        g = torch.Generator().manual_seed(7)
        self.rows = torch.randn(*lead, D, generator=g, dtype=torch.float64)
        self.table = torch.randn(V, D, generator=g, dtype=torch.float64)

    def forward(self, tok):
        return self.head(torch.tanh(self.table[tok] + self.mix(self.rows)))


@pytest.mark.parametrize("lead", [(T,), (1, T)])
def test_a_linear_layer_shared_over_the_batch_is_refused(lead):
    torch.manual_seed(4)
    with pytest.raises((ValueError, RuntimeError), match="sample"):
        step(_SharedInput(lead), tokens())


class _Flattened(nn.Module):
    """Rows of all samples in one dimension, samples in order; one id a sample too."""

    def __init__(self, column=False):
        super().__init__()
        from sample_grad_norms_amd.layers import Embedding
        self.emb, self.kind = Embedding(V, D, scale=0.5, dtype=torch.float64), Embedding(3, D, dtype=torch.float64)
        self.mix, self.head = nn.Linear(D, D, bias=False, dtype=torch.float64), nn.Linear(D, 5, bias=False, dtype=torch.float64)
        self.column = column

    def forward(self, tok):
        kinds = (tok[:, :1] if self.column else tok[:, 0]) % 3
        x = self.emb(tok) + self.kind(kinds.contiguous()).view(-1, 1, D)
        x = self.mix(x.reshape(-1, D)).view_as(x)
        return self.head(torch.tanh(x).reshape(1, -1, D)).view(*tok.shape, 5)


@pytest.mark.parametrize("C", [1e9, 0.5])
@pytest.mark.parametrize("column,verify", [(False, True), (True, True), (True, False)])
def test_one_id_a_sample_and_flattened_rows_keep_their_norms(C, column, verify):
    torch.manual_seed(6)
    model = _Flattened(column)
    for b in (B, 1, 11):
        tok = tokens(b)
        n, c = step(model, tok, C=C, verify_coverage=verify)
        want = true_norms(model, tok)
        torch.testing.assert_close(n.double(), want, rtol=1e-6, atol=0)    # n is float32: 2^-24 for each of its four sums
        got = [p.grad.clone() for p in model.parameters()]
        model.zero_grad()
        (c.double() * losses_of(model, tok)).sum().backward()
        for p, g in zip(model.parameters(), got):
            torch.testing.assert_close(g, p.grad, rtol=1e-12, atol=1e-12)
        model.zero_grad()


def test_the_first_step_has_the_gradients_of_the_others():
    """The first step's check leaves the recordings bit for bit as they are without it."""
    from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
    torch.manual_seed(8)
    model = _Flattened(True).float()
    tok = tokens(11)
    res = []
    for verify in (True, False):
        rc = RandomizedClipping(model, C=1.0, noise_multiplier=0.0, estimator="exact", verify_coverage=verify, keep_layers=True)
        state = torch.get_rng_state()
        with rc.capture():
            losses = (model(tok) * 0.5).sum((1, 2))
        n, _ = rc.clip_factors(losses)
        assert torch.equal(state, torch.get_rng_state())
        res.append((n, [G for _, G, _ in rc.last_layers]))
    assert torch.equal(res[0][0], res[1][0])
    assert all(torch.equal(x, y) for x, y in zip(res[0][1], res[1][1]))


class _Transposed(nn.Module):
    """Two layers that read one square tensor, as it is and transposed."""

    def __init__(self):
        super().__init__()
        self.a, self.b = (nn.Linear(6, 6, bias=False) for _ in range(2))

    def forward(self, x):
        return self.a(x) + self.b(x.transpose(1, 2))


def test_a_tensor_and_its_transpose_are_recorded_apart():
    from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
    x = torch.randn(3, 6, 6, generator=torch.Generator().manual_seed(9))
    model = _Transposed()
    rc = RandomizedClipping(model, C=1.0, noise_multiplier=0.0)
    with rc.capture():
        losses = model(x).sum((1, 2))
    (A, _), (A2, _) = rc._collect(losses)
    assert torch.equal(A, x) and torch.equal(A2, x.transpose(1, 2))


class _HeadsApart(nn.Module):
    """Layers whose inputs lie transposed, so that a recording copies them before it casts them."""

    def __init__(self):
        super().__init__()
        self.layers = nn.ModuleList(nn.Linear(64, 64, bias=False) for _ in range(6))

    def forward(self, x):
        return sum(layer((x * (i + 1)).transpose(1, 2)) for i, layer in enumerate(self.layers))


def test_casts_of_copies_are_recorded_apart():
    from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
    x = torch.randn(3, 64, 50, 64, generator=torch.Generator().manual_seed(10)).bfloat16()
    model = _HeadsApart().bfloat16()
    rc = RandomizedClipping(model, C=1.0, noise_multiplier=0.0, norm_dtype=torch.float32)
    with rc.capture():
        losses = model(x).float().sum((1, 2, 3))
    for i, (A, _) in enumerate(rc._collect(losses)):
        assert torch.equal(A, (x * (i + 1)).transpose(1, 2).reshape(3, -1, 64).float()), i


def test_layers_that_read_one_tensor_share_its_copy():
    from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
    x = torch.randn(3, 5, 6, generator=torch.Generator().manual_seed(11)).bfloat16()
    model = nn.ModuleList(nn.Linear(6, 6, bias=False) for _ in range(2)).bfloat16()
    rc = RandomizedClipping(model, C=1.0, noise_multiplier=0.0, norm_dtype=torch.float32)
    with rc.capture():
        losses = (model[0](x) + model[1](x)).float().sum((1, 2))
    (A, _), (A2, _) = rc._collect(losses)
    assert A.data_ptr() == A2.data_ptr()


def test_a_tables_gradients_are_let_go_after_the_norm(monkeypatch):
    """Only the step that is checked keeps the order and output gradients of a table for
    the second backward pass."""
    import gc
    import weakref

    import sample_grad_norms_amd as dp
    from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
    plain, held = dp.embed_norm, []

    def norm(order, G, **kw):
        held.append(weakref.ref(G))
        return plain(order, G, **kw)

    monkeypatch.setattr(dp, "embed_norm", norm)
    torch.manual_seed(12)
    model = _Flattened(True)
    rc = RandomizedClipping(model, C=1.0, noise_multiplier=0.0, estimator="exact")
    for j in range(3):
        held.clear()
        with rc.capture():
            losses = losses_of(model, tokens())
        _, c = rc.clip_factors(losses)
        gc.collect()
        assert len(held) == 2 and all((g() is not None) == (j == 0) for g in held)
        rc.clipped_backward(losses, c)
        gc.collect()
        assert all(g() is None for g in held)
