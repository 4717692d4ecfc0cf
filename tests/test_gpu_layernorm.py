"""GPU parity of layer norm and RMS norm (forward, gradients, per-sample norms)
against their definitions in float64 on the CPU.

Tolerances (u = 2^-24, s = half a step of the type, 2^-8 for bfloat16):
  * a row's sums pass through at most 32 additions in a lane, 6 over the lanes, 16 over
    the waves and a few roundings of their terms: 64 u of the sum of magnitudes. The
    mean is then off by m = 64 u mean|x|, the variance by (64 + 4) u of itself and m^2,
    so r by e = (36 + 4) u + (m r)^2 relative, and h = (x - mu) r by m r + (e + 2 u) |h|;
  * a column's sum over N rows passes through at most 16 rows a wave (N / 4096 where
    there are more) and 40 additions over waves and work groups: K = 64 + N / 512
    times u of the sum of magnitudes;
  * results are rounded once, s relative.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def dev():
    return torch.device("cuda:0")


def half(dtype):
    return torch.finfo(dtype).eps / 2


def make(B, T, d, dtype, seed, size=1.0, offset=0.3):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(B, T, d, generator=g) * torch.exp(0.5 * torch.randn(d, generator=g)) + offset * torch.randn(d, generator=g)) * size
    G = torch.randn(B, T, d, generator=g)
    w, b = 1.0 + 0.3 * torch.randn(d, generator=g), 0.5 * torch.randn(d, generator=g)
    return x.to(dtype), G.to(dtype), w.to(dtype), b.to(dtype), torch.rand(B, generator=g) + 0.1


def normal(x, eps, rms):
    """mu, r, h in float64 and the bounds of mu, r (relative) and h."""
    x = x.double()
    mu = torch.zeros_like(x[..., :1]) if rms else x.mean(dim=-1, keepdim=True)
    r = 1.0 / torch.sqrt(((x - mu) ** 2).mean(dim=-1, keepdim=True) + eps)
    h = (x - mu) * r
    m = 0.0 * r if rms else 64 * U * x.abs().mean(dim=-1, keepdim=True)
    e = 40 * U + (m * r) ** 2
    return mu, r, h, m, e, m * r + (e + 2 * U) * h.abs()


def inside(got, want, bound, what):
    assert tuple(got.shape) == tuple(want.shape), what
    err = (got.cpu().double() - want).abs()
    ratio = float((err / bound.clamp(min=1e-300)).max()) if err.numel() else 0.0
    print(f"{what}: max err / bound {ratio:.3f}", flush=True)
    assert ratio <= 1.0, what


WIDTHS = {BF16: [8, 72, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384, 16392, 32768],
          F32: [4, 12, 256, 260, 512, 516, 1000, 1028, 2048, 2052, 4096, 4100, 8192, 8196, 16384, 16388, 32768]}
CASES = [(dt, 2, 19, d) for dt, ds in WIDTHS.items() for d in ds] + [
    (dt, *s) for dt in (BF16, F32) for s in ((1, 1, 64), (1, 1, 2048), (3, 1, 128), (1, 2, 8), (5, 61, 256), (2, 700, 512), (33, 40, 1024),
                                             (1, 4099, 104), (700, 3, 64), (3, 333, 2304), (2, 130, 5120))]


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype,B,T,d", CASES)
def test_against_the_definition(dtype, B, T, d, rms):
    import sample_grad_norms_amd as dp
    x, G, w, b, c = make(B, T, d, dtype, 11)
    eps, s = 1e-5, half(dtype)
    xd, Gd, wd, bd, cd = (t.to(dev()) for t in (x, G, w, b, c))
    mu, r, h, m, e, eh = normal(x, float(torch.tensor(eps)), rms)
    wf, bf, Gf, cf = w.double(), 0.0 if rms else b.double(), G.double(), c.double()[:, None, None]

    y, mean, rstd = dp.layernorm_forward(xd, wd, None if rms else bd, eps=eps, rms=rms)
    want = h * wf + bf
    inside(y, want, wf.abs() * eh + 2 * U * ((h * wf).abs() + abs(bf)) + s * 1.01 * want.abs(), "y")
    inside(rstd, r[..., 0], (e * r)[..., 0] * 1.01, "rstd")
    if rms:
        assert mean is None
    else:
        inside(mean, mu[..., 0], m[..., 0] + U * mu[..., 0].abs(), "mean")

    # the gradients read the statistics that they are given
    mean_in, rstd_in = mu[..., 0].float(), r[..., 0].float()
    hg = (x.double() - mean_in.double()[..., None]) * rstd_in.double()[..., None]
    g = Gf * wf
    m1, m2 = (0.0 if rms else g.mean(dim=-1, keepdim=True)), (g * hg).mean(dim=-1, keepdim=True)
    rg = rstd_in.double()[..., None]
    dx = rg * (g - hg * m2 - m1)
    bx = rg * (2 * U * g.abs() + hg.abs() * (70 * U * (g * hg).abs().mean(dim=-1, keepdim=True) + 4 * U * m2.abs())
               + 66 * U * g.abs().mean(dim=-1, keepdim=True) + 3 * U * (g.abs() + (hg * m2).abs() + abs(m1))) + 1.01 * s * dx.abs()
    K = (64 + B * T / 512) * U
    dw, aw = (cf * Gf * hg).sum(dim=(0, 1)), (cf * Gf * hg).abs().sum(dim=(0, 1))
    db, ab = (cf * Gf).sum(dim=(0, 1)), (cf * Gf).abs().sum(dim=(0, 1))
    args = (Gd, xd, wd, None if rms else mean_in.to(dev()), rstd_in.to(dev()))
    got = dp.layernorm_backward(*args, weights=cd)
    inside(got[0], dx, bx, "dx")
    inside(got[1], dw, (K + 4 * U) * aw + 1.01 * s * dw.abs(), "dw")
    if rms:
        assert got[2] is None
    else:
        inside(got[2], db, (K + 2 * U) * ab + 1.01 * s * db.abs(), "db")
    again = dp.layernorm_backward(*args, weights=cd)
    assert all(p is q or torch.equal(p, q) for p, q in zip(got, again))

    n = dp.layernorm_norm(xd, Gd, eps=eps, rms=rms)
    K = (64 + T / 512) * U
    sw, bw = (Gf * h).sum(dim=1), (Gf.abs() * eh).sum(dim=1) + (K + 2 * U) * (Gf * h).abs().sum(dim=1)
    sb, bb = Gf.sum(dim=1), K * Gf.abs().sum(dim=1)
    both = [(sw, bw)] if rms else [(sw, bw), (sb, bb)]
    want = sum((v ** 2).sum(dim=1) for v, _ in both)
    bound = sum((2 * v.abs() * t + t * t).sum(dim=1) for v, t in both) + 2 * U * want
    inside(n, want, bound, "n")
    assert torch.equal(n, dp.layernorm_norm(xd, Gd, eps=eps, rms=rms))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,d", [(3, 50, 64), (2, 900, 256), (4, 300, 3000), (2, 40, 9000)])
def test_parts_weights_and_accumulation(B, T, d, dtype):
    """Each output alone is what it is beside the others, bit for bit; a norm's parts add up."""
    import sample_grad_norms_amd as dp
    x, G, w, b, c = (t.to(dev()) for t in make(B, T, d, dtype, 12))
    y, mean, rstd = dp.layernorm_forward(x, w, b)
    no_bias = dp.layernorm_forward(x, w, torch.zeros_like(b))[0]
    assert torch.equal(dp.layernorm_forward(x, w)[0], no_bias)
    dx, dw, db = dp.layernorm_backward(G, x, w, mean, rstd, weights=c)
    plain = dp.layernorm_backward(G, x, w, mean, rstd)
    assert torch.equal(plain[0], dx) and not torch.equal(plain[1], dw)
    ones = dp.layernorm_backward(G, x, w, mean, rstd, weights=torch.ones_like(c))
    # (samples' factors of 1 sum the same rows in the same order)
    assert torch.equal(ones[1], plain[1]) and torch.equal(ones[2], plain[2])
    for kw, keep in ((dict(bias=False, need_dw=False), (0,)), (dict(need_dx=False, bias=False), (1,)),
                     (dict(need_dx=False, need_dw=False), (2,)), (dict(need_dx=False), (1, 2)), (dict(bias=False), (0, 1))):
        got = dp.layernorm_backward(G, x, w, mean, rstd, weights=c, **kw)
        for j, (p, q) in enumerate(zip(got, (dx, dw, db))):
            same = torch.equal(p, q) if j in keep else p is None
            assert same, (kw, j)
    n, gain = dp.layernorm_norm(x, G), dp.layernorm_norm(x, G, bias=False)
    bias = dp.layernorm_norm(x, G, gain=False)
    want = gain.double() + bias.double()
    inside(n, want.cpu(), 4 * U * want.cpu(), "parts of a norm")
    acc = torch.full((B,), 3.0, device=dev())
    res = dp.layernorm_norm(x, G, out=acc, accumulate=True)
    assert res is acc
    inside(acc, n.cpu().double() + 3.0, 3 * U * (n.cpu().double() + 3.0), "accumulated")


def test_differences():
    """The gradients against differences of the definition in 64 bits along random directions."""
    import sample_grad_norms_amd as dp
    for rms in (False, True):
        x, G, w, b, _ = make(2, 9, 96, F32, 13)
        y, mean, rstd = dp.layernorm_forward(x.to(dev()), w.to(dev()), None if rms else b.to(dev()), rms=rms)
        dx, dw, db = dp.layernorm_backward(G.to(dev()), x.to(dev()), w.to(dev()), mean, rstd)
        g = torch.Generator().manual_seed(14)

        def loss(x, w, b):
            h = normal(x, 1e-5, rms)[2]
            return float(((h * w + (0.0 if rms else b)) * G.double()).sum())
        at = [t.double() for t in (x, w, b)]
        for j, got in enumerate((dx, dw, db)):
            if got is None:
                continue
            v = torch.randn(at[j].shape, generator=g, dtype=torch.float64)
            ends = [loss(*[t + f * 1e-5 * v if i == j else t for i, t in enumerate(at)]) for f in (1.0, -1.0)]
            want = (ends[0] - ends[1]) / 2e-5
            have = float((got.cpu().double() * v).sum())
            # float32 gradients of 1728 terms of size about 1; the differences' own error is 1e-10 of the third derivative
            assert abs(have - want) <= 1e-4 * (1.0 + float((got.cpu().double() * v).abs().sum()) * 0.01), (rms, j, have, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("d", [64, 1024, 2048, 4096, 12288])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_rows_that_are_not_finite_stay_alone(d, dtype, rms, value):
    """Such a row of x or dy changes no bit of the other rows of y and dx, and no other sample's norm."""
    import sample_grad_norms_amd as dp
    x, G, w, b, _ = (t.to(dev()) for t in make(3, 37, d, dtype, 15))
    b = None if rms else b
    y, mean, rstd = dp.layernorm_forward(x, w, b, rms=rms)
    dx = dp.layernorm_backward(G, x, w, mean, rstd)[0]
    n = dp.layernorm_norm(x, G, rms=rms)
    for row in (0, 5, 36):
        x2, G2 = x.clone(), G.clone()
        x2[1, row, 7] = value
        G2[1, row, 7] = value
        keep = torch.ones(3, 37, dtype=torch.bool, device=dev())
        keep[1, row] = False
        y2, mean2, rstd2 = dp.layernorm_forward(x2, w, b, rms=rms)
        assert torch.equal(y2[keep], y[keep]) and torch.equal(rstd2[keep], rstd[keep])
        assert bool(y2[1, row].isnan().any())
        dx2 = dp.layernorm_backward(G2, x, w, mean, rstd)[0]
        assert torch.equal(dx2[keep], dx[keep]) and not bool(dx2[1, row].isfinite().any())
        n2, n3 = dp.layernorm_norm(x2, G, rms=rms), dp.layernorm_norm(x, G2, rms=rms)
        assert torch.equal(n2[::2], n[::2]) and torch.equal(n3[::2], n[::2])
        assert not bool(n2[1].isfinite()) and not bool(n3[1].isfinite())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_and_constant_rows(dtype):
    """A mean far larger than the deviation: squares are taken after the mean; rows of one value; zero rows."""
    import sample_grad_norms_amd as dp
    x, _, w, b, _ = make(1, 40, 512, dtype, 16)
    x[0, 10:20] += 300.0
    x[0, 20] = 7.0
    x[0, 21] = 0.0
    x[0, 22] = 1e-20
    x[0, 23] *= 1e-12
    mu, r, h, m, e, eh = normal(x, float(torch.tensor(1e-5)), False)
    y, mean, rstd = dp.layernorm_forward(x.to(dev()), w.to(dev()), b.to(dev()))
    want = h * w.double() + b.double()
    inside(y, want, w.double().abs() * eh + 2 * U * ((h * w.double()).abs() + b.double().abs()) + 1.01 * half(dtype) * want.abs() + 1e-30, "y")
    # a row of one value has a variance of at most m^2, against eps
    inside(rstd, r[..., 0], ((e + (m * r) ** 2) * r)[..., 0] * 1.01, "rstd")


def test_shapes_without_rows():
    import sample_grad_norms_amd as dp
    w = torch.ones(64, device=dev())
    x = torch.zeros(0, 5, 64, device=dev())
    y, mean, rstd = dp.layernorm_forward(x, w, w)
    assert y.shape == x.shape and mean.shape == rstd.shape == (0, 5)
    dx, dw, db = dp.layernorm_backward(x, x, w, mean, rstd)
    assert dx.shape == x.shape and bool((dw == 0).all()) and bool((db == 0).all())
    x = torch.zeros(4, 0, 64, device=dev())
    n = dp.layernorm_norm(x, x)
    assert n.shape == (4,) and bool((n == 0).all())
    one = torch.randn(64, device=dev())
    y, mean, rstd = dp.layernorm_forward(one, w)
    assert y.shape == (64,) and mean.shape == ()
    assert dp.layernorm_backward(one, one, w, mean, rstd)[0].shape == (64,)
    assert torch.equal(y, dp.layernorm_forward(one[None], w)[0][0])


def test_offsets_past_32_bits():
    """Rows behind 2^31 elements are what a call on them alone gives, bit for bit."""
    import sample_grad_norms_amd as dp
    N, d = 70000, 32768
    g = torch.Generator(device=dev()).manual_seed(17)
    x = torch.randn(N, d, generator=g, device=dev(), dtype=BF16)
    w = torch.randn(d, generator=g, device=dev(), dtype=BF16)
    y, _, rstd = dp.layernorm_forward(x, w, rms=True)
    y2, _, rstd2 = dp.layernorm_forward(x[-50:].clone(), w, rms=True)
    assert torch.equal(y[-50:], y2) and torch.equal(rstd[-50:], rstd2)
    del y
    dx = dp.layernorm_backward(x, x, w, None, rstd, need_dw=False)[0]
    assert torch.equal(dx[-50:], dp.layernorm_backward(x[-50:].clone(), x[-50:].clone(), w, None, rstd2, need_dw=False)[0])
    del dx
    n = dp.layernorm_norm(x.view(2, N // 2, d), x.view(2, N // 2, d), rms=True)
    assert torch.equal(n[1:], dp.layernorm_norm(x[N // 2:].clone()[None], x[N // 2:].clone()[None], rms=True)) or \
        abs(float(n[1]) / float(dp.layernorm_norm(x[N // 2:][None], x[N // 2:][None], rms=True)) - 1.0) < 1e-4


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_streams_and_graphs(dtype):
    """Calls on another stream, two at once, and a captured run replayed beside eager work."""
    import sample_grad_norms_amd as dp
    B, T, d = 3, 900, 384
    sets = [tuple(t.to(dev()) for t in make(B, T, d, dtype, 18 + j)) for j in range(3)]

    def calls(x, G, w, b, c):
        y, mean, rstd = dp.layernorm_forward(x, w, b)
        return (y, mean, rstd, *dp.layernorm_backward(G, x, w, mean, rstd, weights=c), dp.layernorm_norm(x, G))
    want = [calls(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s, data in zip(streams, sets):
        with torch.cuda.stream(s):
            got.append([calls(*data) for _ in range(5)][-1])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    held = [t.clone() for t in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls(*held)
    for j in (1, 2, 0, 1):
        for h, t in zip(held, sets[j]):
            h.copy_(t)
        graph.replay()
        eager = calls(*sets[(j + 1) % 3])
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want[j])), j
        assert all(torch.equal(p, q) for p, q in zip(eager, want[(j + 1) % 3])), j


def test_refusals():
    import sample_grad_norms_amd as dp
    x = torch.zeros(2, 5, 64, device=dev(), dtype=BF16)
    w = torch.ones(64, device=dev(), dtype=BF16)
    y, mean, rstd = dp.layernorm_forward(x, w, w)
    with pytest.raises(TypeError):
        dp.layernorm_forward(x, w.float())
    with pytest.raises(TypeError):
        dp.layernorm_forward(x.half(), w.half())
    with pytest.raises(ValueError):
        dp.layernorm_forward(x.transpose(0, 1), w)
    with pytest.raises(ValueError):
        dp.layernorm_forward(x, w[:32])
    with pytest.raises(ValueError):
        dp.layernorm_forward(x, w, w, rms=True)
    with pytest.raises(ValueError):
        dp.layernorm_forward(x, w, out=torch.empty(2, 5, 32, device=dev(), dtype=BF16))
    with pytest.raises(ValueError):
        dp.layernorm_forward(x, w.cpu())
    for bad in (dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(out=x)):
        with pytest.raises(dp.DpnormError):
            dp.layernorm_forward(x, w, **bad)
    with pytest.raises(dp.DpnormError):   # not on a 16-byte boundary
        dp.layernorm_forward(torch.zeros(2 * 5 * 64 + 4, device=dev(), dtype=BF16)[4:].view(2, 5, 64), w)
    with pytest.raises(dp.DpnormError):
        dp.layernorm_forward(torch.zeros(2, 12, device=dev(), dtype=BF16), torch.ones(12, device=dev(), dtype=BF16))
    with pytest.raises(dp.DpnormError):
        dp.layernorm_forward(torch.zeros(1, 32776, device=dev(), dtype=BF16), torch.ones(32776, device=dev(), dtype=BF16))
    with pytest.raises(ValueError):
        dp.layernorm_backward(x[:1], x, w, mean, rstd)
    with pytest.raises(ValueError):
        dp.layernorm_backward(x, x, w, mean[:1], rstd)
    with pytest.raises(ValueError):
        dp.layernorm_backward(x, x, w, mean, rstd, weights=torch.ones(3, device=dev()))
    with pytest.raises(TypeError):
        dp.layernorm_backward(x, x, w, mean, rstd, weights=torch.ones(2, device=dev(), dtype=BF16))
    with pytest.raises(ValueError):
        dp.layernorm_backward(x, x, w, mean, rstd, need_dx=False, need_dw=False, bias=False)
    with pytest.raises(ValueError):
        dp.layernorm_norm(x[0], x[0])
    with pytest.raises(ValueError):
        dp.layernorm_norm(x, x, rms=True, gain=False)
    with pytest.raises(ValueError):
        dp.layernorm_norm(x, x, accumulate=True)


def test_a_missing_weight_is_refused():
    import sample_grad_norms_amd as dp
    x = torch.zeros(2, 5, 64, device=dev(), dtype=BF16)
    rstd = torch.ones(2, 5, device=dev())
    with pytest.raises(TypeError, match="weight"):
        dp.layernorm_forward(x, None)
    with pytest.raises(TypeError, match="weight"):
        dp.layernorm_backward(x, x, None, None, rstd)
