"""GPU parity of the embedding calls (lookup, per-sample norm, gradient of the
table) against their definitions in float64 on the CPU.

Tolerances. A lookup is one product rounded once: half a step of the type,
plus for bfloat16 the float32 rounding of the product before it. A row of the
table's gradient is a float32 sum of m products rounded once: half a step of
the type of the result plus (m + 2) 2^-24 sum |terms|. A norm is a sum of
squares of such rows: each row's sum is off by at most (m + 1) 2^-24 of the
sum of its terms' magnitudes, its square and the sum over at most d columns in
float32 by (d / 64 + 10) 2^-24 more, and the rest is float64.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def dev():
    return torch.device("cuda:0")


def ids(B, T, V, seed, kind, dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    if kind == "uniform":
        t = torch.randint(0, V, (B, T), generator=g)
    elif kind == "zipf":
        t = (torch.exp(torch.rand(B, T, generator=g, dtype=torch.float64) * math.log(V + 1.0)) - 1).long().clamp(0, V - 1)
    elif kind == "same":
        t = torch.full((B, T), V - 1, dtype=torch.int64)
    elif kind == "two":   # long runs whose ends fall inside chunks
        t = (torch.rand(B, T, generator=g) < 0.5).long() * (V - 1)
    elif kind == "none":
        t = torch.full((B, T), -1, dtype=torch.int64)
    elif kind == "padded":   # ids outside the table at the ends of the samples and among them
        t = torch.randint(-2, V + 2, (B, T), generator=g)
        t[:, T - T // 3:] = -1
        if B > 1:
            t[1] = V
    return t.to(dtype)


def rows(shape, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * torch.exp(torch.randn(shape[0], *([1] * (len(shape) - 1)), generator=g))).to(dtype)


def eps(dtype):
    return torch.finfo(dtype).eps / 2


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape,V,d", [((1, 1), 1, 8), ((3, 37), 100, 264), ((2, 5), 1000, 2056), ((7,), 33, 4096),
                                       ((2, 3, 4), 17, 512)])
@pytest.mark.parametrize("idx", [torch.int32, torch.int64])
def test_lookup(dtype, shape, V, d, idx):
    import sample_grad_norms_amd as dp
    g = torch.Generator().manual_seed(5)
    tok = torch.randint(-1, V + 1, shape, generator=g).to(idx)
    W = rows((V, d), 6, dtype)
    scale = 1.7
    out = dp.embed_lookup(tok.to(dev()), W.to(dev()), scale=scale)
    assert out.dtype == dtype and tuple(out.shape) == shape + (d,)
    ok = (tok >= 0) & (tok < V)
    f = float(torch.tensor(scale, dtype=torch.float32))
    want = torch.where(ok[..., None], W.double()[tok.long().clamp(0, V - 1)] * f, torch.zeros(1, dtype=torch.float64))
    err = (out.cpu().double() - want).abs()
    # the product rounds to float32 and then to the type
    assert bool((err <= want.abs() * (eps(dtype) * (1 + 2 ** -23) + (2 ** -24 if dtype == torch.bfloat16 else 0))).all())
    assert bool((out.cpu()[~ok] == 0).all())


CASES = [   # B, T, V, d, kind
    (1, 1, 1, 8, "uniform"),
    (2, 3, 5, 8, "none"),
    (1, 130, 1, 16, "same"),
    (3, 61, 40, 256, "padded"),
    (2, 700, 3, 520, "two"),
    (5, 333, 1000, 264, "zipf"),
    (4, 2048, 50257, 64, "zipf"),
    (1, 24576, 262144, 8, "zipf"),      # the largest order made in one launch
    (1, 24577, 5000, 8, "zipf"),        # one position more: radix passes
    (3, 3001, 262145, 72, "zipf"),      # one table row more: radix passes
    (1, 20000, 128, 8, "padded"),       # fewer ids than buckets
    (2, 66000, 2, 8, "uniform"),        # more positions of a wave than stay in registers
    (2, 5000, 700, 40, "padded"),
    (1, 9001, 9, 48, "same"),
    (70, 150, 11, 24, "uniform"),
    (1, 40000, 65536, 8, "zipf"),
    (2, 37, 20, 2056, "two"),
    (3, 256, 300, 256, "zipf"),         # the largest samples of a norm in one launch
    (1, 256, 5, 1032, "padded"),        # and the largest batch of a gradient
    (300, 2, 50, 16, "uniform"),
    (4, 64, 4, 8, "none"),
]


def norm_reference(tok, G, V, scale):
    n, bound = [], []
    f = float(torch.tensor(scale, dtype=torch.float32))
    d = G.shape[2]
    for t, g in zip(tok.long(), G.double()):
        s = torch.zeros(V + 1, d, dtype=torch.float64)
        a = torch.zeros(V + 1, d, dtype=torch.float64)
        m = torch.zeros(V + 1, 1, dtype=torch.float64)
        at = torch.where((t >= 0) & (t < V), t, torch.full_like(t, V))
        s.index_add_(0, at, g)
        a.index_add_(0, at, g.abs())
        m.index_add_(0, at, torch.ones(len(t), 1, dtype=torch.float64))
        s, a, m = s[:V], a[:V], m[:V]
        e = (m + 1) * 2 ** -24 * a
        n.append(float((s * s).sum()) * f * f)
        bound.append(float((2 * s.abs() * e + e * e + s * s * (d / 64 + 10) * 2 ** -24).sum()) * f * f + n[-1] * 2 ** -22)
    return torch.tensor(n, dtype=torch.float64), torch.tensor(bound, dtype=torch.float64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,V,d,kind", CASES)
def test_norm(B, T, V, d, kind, dtype):
    import sample_grad_norms_amd as dp
    tok, G = ids(B, T, V, 11, kind), rows((B, T, d), 12, dtype)
    want, bound = norm_reference(tok, G, V, 0.75)
    t, g = tok.to(dev()), G.to(dev())
    n = dp.embed_norm(t, g, V, scale=0.75)
    again = dp.embed_norm(dp.embed_order(t.int(), V), g, scale=0.75)
    # (a call with an order may add a run's rows in other groups)
    assert torch.equal(again, dp.embed_norm(dp.embed_order(t, V), g, scale=0.75)) and torch.equal(n, dp.embed_norm(t, g, V, scale=0.75))
    assert bool(((again.cpu().double() - want).abs() <= bound).all())
    err = (n.cpu().double() - want).abs()
    print(f"max err / bound {float((err / bound.clamp(min=1e-300)).max()):.3f}", flush=True)
    assert bool((err <= bound).all())
    base = torch.linspace(1.0, 2.0, B, device=dev())
    total = dp.embed_norm(t, g, V, scale=0.75, out=base.clone(), accumulate=True)
    assert bool(((total.cpu().double() - (base.cpu().double() + want)).abs() <= bound + (base.cpu() + want) * 2 ** -23).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,V,d,kind", CASES)
def test_grad(B, T, V, d, kind, dtype):
    import sample_grad_norms_amd as dp
    tok, G = ids(B, T, V, 21, kind), rows((B, T, d), 22, dtype)
    c = torch.linspace(0.1, 1.0, B)
    f = float(torch.tensor(1.25, dtype=torch.float32))
    at = torch.where((tok >= 0) & (tok < V), tok, torch.full_like(tok, V)).reshape(-1)
    terms = (G.double() * (c.double() * f)[:, None, None]).reshape(-1, d)
    want = torch.zeros(V + 1, d, dtype=torch.float64).index_add_(0, at, terms)[:V]
    mag = torch.zeros(V + 1, d, dtype=torch.float64).index_add_(0, at, terms.abs())[:V]
    m = torch.zeros(V + 1, 1, dtype=torch.float64).index_add_(0, at, torch.ones(len(at), 1, dtype=torch.float64))[:V]
    bound = want.abs() * eps(dtype) + (m + 2) * 2 ** -24 * mag * (1 + eps(dtype))
    t, g, w = tok.to(dev()), G.to(dev()), c.to(dev())
    out = torch.full((V, d), float("nan"), dtype=dtype, device=dev())
    dW = dp.embed_grad(t, g, V, scale=1.25, weights=w, out=out)
    assert dW is out
    err = (dW.cpu().double() - want).abs()
    print(f"max err / bound {float((err / bound.clamp(min=1e-300)).max()):.3f}", flush=True)
    assert bool((err <= bound).all())
    assert torch.equal(dW, dp.embed_grad(t, g, V, scale=1.25, weights=w))
    ordered = dp.embed_grad(dp.embed_order(t, V), g, scale=1.25, weights=w)
    assert bool(((ordered.cpu().double() - want).abs() <= bound).all())
    # added to the rows that occur; the others keep their bits
    old = rows((V, d), 23, dtype)
    acc = dp.embed_grad(t, g, V, scale=1.25, weights=w, out=old.to(dev()), accumulate=True).cpu()
    absent = (m == 0).reshape(-1)
    assert torch.equal(acc[absent], old[absent])
    total = want + old.double()
    assert bool(((acc.double() - total).abs() <= total.abs() * eps(dtype) + (m + 3) * 2 ** -24 * (mag + old.double().abs()) * (1 + eps(dtype))).all())


def test_grad_without_weights_is_weights_of_one():
    import sample_grad_norms_amd as dp
    tok, G = ids(3, 100, 50, 31, "zipf").to(dev()), rows((3, 100, 64), 32, torch.float32).to(dev())
    assert torch.equal(dp.embed_grad(tok, G, 50), dp.embed_grad(tok, G, 50, weights=torch.ones(3, device=dev())))


def test_not_a_number_stays_with_its_sample_and_row():
    """A NaN or infinity in G reaches its sample's norm and its id's row only,
    and one at a padded position reaches nothing."""
    import sample_grad_norms_amd as dp
    tok, G = ids(4, 90, 30, 41, "uniform"), rows((4, 90, 40), 42, torch.float32)
    tok[3, 80:] = -1
    clean_n = dp.embed_norm(tok.to(dev()), G.to(dev()), 30).cpu()
    clean_g = dp.embed_grad(tok.to(dev()), G.to(dev()), 30).cpu()
    G[3, 85] = float("nan")
    assert torch.equal(dp.embed_norm(tok.to(dev()), G.to(dev()), 30).cpu(), clean_n)
    assert torch.equal(dp.embed_grad(tok.to(dev()), G.to(dev()), 30).cpu(), clean_g)
    G[1, 7, 3] = float("nan")
    n, dW = dp.embed_norm(tok.to(dev()), G.to(dev()), 30).cpu(), dp.embed_grad(tok.to(dev()), G.to(dev()), 30).cpu()
    assert bool(n[1].isnan()) and torch.equal(n[[0, 2, 3]], clean_n[[0, 2, 3]])
    bad = torch.zeros(30, 40, dtype=torch.bool)
    bad[tok[1, 7], 3] = True
    assert torch.equal(dW.isnan(), bad) and torch.equal(dW[~bad], clean_g[~bad])


def test_empty_batches():
    import sample_grad_norms_amd as dp
    tok = torch.empty(2, 0, dtype=torch.int64, device=dev())
    G = torch.empty(2, 0, 16, device=dev())
    assert tuple(dp.embed_lookup(tok, torch.ones(4, 16, device=dev())).shape) == (2, 0, 16)
    assert dp.embed_norm(tok, G, 4).tolist() == [0.0, 0.0]
    assert bool((dp.embed_grad(tok, G, 4) == 0).all())


def test_replayed_graph_matches_eager():
    """Lookup, order, norm and gradient captured together, replayed on new
    contents of the same buffers with eager work between the replays."""
    import sample_grad_norms_amd as dp
    B, T, V, d = 3, 3500, 2000, 136
    tok, G = ids(B, T, V, 51, "zipf").to(dev()), rows((B, T, d), 52, torch.bfloat16).to(dev())
    W, c = rows((V, d), 53, torch.bfloat16).to(dev()), torch.rand(B, device=dev())

    def step():
        order = dp.embed_order(tok, V)
        return dp.embed_lookup(tok, W, scale=3.0), dp.embed_norm(order, G), dp.embed_grad(order, G, weights=c)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    for r in range(4):
        tok.copy_(ids(B, T, V, 60 + r, "zipf" if r % 2 else "padded"))
        G.copy_(rows((B, T, d), 70 + r, torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in res]
        for x, y in zip(got, step()):
            assert torch.equal(x, y)


def test_refusals():
    import sample_grad_norms_amd as dp
    tok = torch.zeros(2, 5, dtype=torch.int64, device=dev())
    G, W = torch.zeros(2, 5, 16, device=dev()), torch.zeros(9, 16, device=dev())
    for call in (lambda: dp.embed_lookup(tok, W[:, :6].contiguous()),          # width
                 lambda: dp.embed_lookup(tok, W, scale=float("inf")),
                 lambda: dp.embed_norm(tok, G, 0),
                 lambda: dp.embed_grad(tok, G, 9, scale=float("nan"))):
        with pytest.raises(dp.DpnormError):
            call()
    order = dp.embed_order(tok, 9)
    for call in (lambda: dp.embed_lookup(tok, W.t()),
                 lambda: dp.embed_lookup(tok[:, ::2], W),
                 lambda: dp.embed_lookup(tok, W, out=torch.zeros(2, 4, 16, device=dev())),
                 lambda: dp.embed_order(tok.reshape(-1), 9),
                 lambda: dp.embed_norm(tok, G),
                 lambda: dp.embed_norm(order, G, 8),
                 lambda: dp.embed_norm(order, G[:, :4].contiguous()),
                 lambda: dp.embed_norm(order, G, accumulate=True),
                 lambda: dp.embed_grad(order, G, weights=torch.ones(3, device=dev())),
                 lambda: dp.embed_grad(order, G, out=torch.zeros(8, 16, device=dev())),
                 lambda: dp.embed_grad(order, G, workspace=torch.zeros(8, dtype=torch.uint8, device=dev()))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: dp.embed_lookup(tok.float(), W), lambda: dp.embed_lookup(tok, W.half()),
                 lambda: dp.embed_grad(order, G, weights=torch.ones(2, dtype=torch.float64, device=dev()))):
        with pytest.raises(TypeError):
            call()


def test_more_blocks_than_one_grid_dimension_holds():
    """Calls whose blocks have 2^32 threads and more along one dimension: a block a
    sample (2^22 of 1024 threads), and a block for every 16 of 2^28 and more rows."""
    import sample_grad_norms_amd as dp
    B, d = 2 ** 22 + 3, 8
    tok = torch.zeros(B, 1, dtype=torch.int32, device=dev())
    tok[::5] = -1
    G = (torch.arange(B, device=dev()) % 251).to(torch.bfloat16).view(B, 1, 1).expand(B, 1, d).contiguous()
    n = dp.embed_norm(tok, G, V=1)
    want = d * (torch.arange(B, device=dev()) % 251).double() ** 2     # whole numbers below 2^24
    want[::5] = 0
    same = bool((n.double() == want).all())
    assert same
    V, d = 2 ** 28 + 5, 4
    rows = torch.tensor([[0, 17, 2 ** 28 - 1, 2 ** 28, V - 1, 17]], device=dev())
    dW = dp.embed_grad(rows, torch.ones(1, 6, d, device=dev()), V)
    touched = dW[rows[0, :5]]
    assert bool((touched == torch.tensor([1, 2, 1, 1, 1], device=dev())[:, None]).all())
    assert float(dW.double().sum()) == 6 * d and int(torch.count_nonzero(dW)) == 5 * d
    out = dp.embed_lookup(rows, dW, scale=2.0)
    assert bool((out[0] == 2 * dW[rows[0]]).all())


def test_more_chunks_than_one_grid_dimension_holds():
    """2^24 chunks of 16 positions for the join of cut runs, and 2^30 rows to clear."""
    import sample_grad_norms_amd as dp
    T, d = 2 ** 27 + 40, 8
    tok = torch.arange(2 * T, device=dev(), dtype=torch.int32).view(2, T) // 40     # runs of 40: cut at most chunk ends
    tok = tok.remainder_(1 << 20)
    G = torch.ones(2, T, d, dtype=torch.bfloat16, device=dev())
    n = dp.embed_norm(tok, G, V=1 << 20)
    for i in range(2):
        c = torch.bincount(tok[i].long(), minlength=1 << 20).double()
        assert float(n[i]) == pytest.approx(d * float((c * c).sum()), rel=2.0 ** -24)
    del tok, G
    V, d = 1 << 30, 4
    tok = torch.arange(0, 600, device=dev()).view(1, 600) * 1789569
    dW = dp.embed_grad(tok, torch.ones(1, 600, d, device=dev()), V)
    assert bool((dW[tok[0]] == 1).all()) and int(torch.count_nonzero(dW.view(torch.int32))) == 600 * d
