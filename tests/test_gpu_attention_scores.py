"""GPU parity of attention whose scores are changed before the softmax (capped by a
tanh, biased by distance, a prefix that every row sees) and of its gradients, against
their definitions in float64 on the CPU, in every form that the kernels have.

Tolerances as in test_gpu_attention.py (u = 2^-24), and for a changed score s':
  * the cap is C tanh(z) with tanh = 1 - 2 / (1 + exp(2 z)): exp's argument and value are
    off by (2 |z| + 2) u relative, 1 / (1 + E) by r (1 - r) times that, at most 0.9 u, and 2 u more
    for the sum and the reciprocal, so the tanh by 8 u with its last rounding, the capped
    score by 8 u C; for float32 below |z| = 0.3 the series is off by 8 u relative. An
    error of z passes with the tanh's derivative, at most 1;
  * the bias is off by 4 u relative (slope, unit, product, sum);
  * the derivative 1 - tanh^2 by 24 u, and by 0.77 times z's error;
  * numbers below 2^-126, the least normal one of float32 and bfloat16, may become 0:
    exp(-600) is 2^-865 and its float32 is 0. That is an error of up to 2^-126 in a weight
    and in a result, whatever their relative bounds.
"""
import math

import pytest
import torch

import attention_forms
from test_gpu_attention import CASES, U, dev, half, inside, make, offsets, sequences

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
TINY = 2.0 ** -126


class Change:
    def __init__(self, Hq, lengths, cap=None, slopes=None, prefix=None):
        self.cap = cap
        self.slopes = None if slopes is None else torch.tensor([slopes * 2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)])
        self.prefix = None if prefix is None else torch.tensor([int(prefix * n) if prefix <= 1 else int(prefix) for n in lengths],
                                                               dtype=torch.int32)

    def gpu(self):
        on = lambda t: t if t is None else t.to(dev())
        return dict(cap=self.cap, slopes=on(self.slopes), prefix=on(self.prefix))

    def scores(self, Q, K, scale, j, i):
        """(s', its bound, the derivative 1 - tanh^2, its bound, visible) for head j of sequence i."""
        n, D = Q.shape
        s = (Q @ K.t()) * scale
        e = (D + 8) * U * ((Q.abs() @ K.abs().t()) * scale).amax(dim=1, keepdim=True).expand(n, n)
        f, ef = torch.ones_like(s), torch.zeros_like(s)
        if self.cap:
            z = s / self.cap
            t = torch.tanh(z)
            f, ef = 1.0 / torch.cosh(z) ** 2, 24 * U + 0.77 * e / self.cap
            s = self.cap * t
            e = e + 8 * U * (torch.where(z.abs() < 0.29, s.abs(), torch.full_like(s, self.cap)) if self.relative else self.cap)
        at = torch.arange(n)
        if self.slopes is not None:
            bias = self.slopes[j].double() * (at[:, None] - at[None]).abs()
            s = s - bias
            e = e + 4 * U * bias.abs()
        p = 0 if self.prefix is None else min(max(int(self.prefix[i]), 0), n)
        seen = (at[None] <= at[:, None]) | (at[None] < p)
        return s.masked_fill(~seen, -math.inf), e + 2 * U * s.abs(), f, ef, seen


def forward_reference(ch, q, k, v, cu, scale):
    N, Hq, D = q.shape
    rep, h = Hq // k.shape[1], half(q.dtype)
    hw = h if q.dtype == BF16 else 0.0
    ch.relative = q.dtype == F32
    o, lse = torch.full((N, Hq, D), math.nan, dtype=torch.float64), torch.full((Hq, N), math.nan, dtype=torch.float64)
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    for i, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        if a == b:
            continue
        n = b - a
        for j in range(Hq):
            Q, K, V = q[a:b, j].double(), k[a:b, j // rep].double(), v[a:b, j // rep].double()
            s, e, _, _, seen = ch.scores(Q, K, scale, j, i)
            z = torch.logsumexp(s, dim=1)
            P = torch.exp(s - z[:, None])
            lse[j, a:b], o[a:b, j] = z, P @ V
            # a weight's own error, and its share of the sum's
            x = (P * e.masked_fill(~seen, 0.0)).sum(dim=1, keepdim=True)
            We = P * (hw + e.masked_fill(~seen, 0.0) + x + 8 * U) + TINY
            bo[a:b, j] = We @ V.abs() + (2 * n + 64) * U * (P @ V.abs()) + h * o[a:b, j].abs() + TINY
            bl[j, a:b] = x[:, 0] + (n + 64) * U + 2 * U * z.abs()
    return o, lse, bo * 1.02, bl * 1.02


def backward_reference(ch, do, q, k, v, o, lse, cu, scale):
    N, Hq, D = q.shape
    Hkv = k.shape[1]
    rep, h = Hq // Hkv, half(q.dtype)
    hw = h if q.dtype == BF16 else 0.0
    ch.relative = q.dtype == F32
    res = [torch.zeros(N, H, D, dtype=torch.float64) for H in (Hq, Hkv, Hkv)]
    bnd = [torch.zeros(N, H, D, dtype=torch.float64) for H in (Hq, Hkv, Hkv)]
    for i, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        n = b - a
        for j in range(Hq if n else 0):
            c = j // rep
            Q, K, V = q[a:b, j].double(), k[a:b, c].double(), v[a:b, c].double()
            dO, O = do[a:b, j].double(), o[a:b, j].double()
            s, e, f, ef, seen = ch.scores(Q, K, scale, j, i)
            z = lse[j, a:b].double()
            P = torch.exp(s - z[:, None])
            dp, delta = dO @ V.t(), (dO * O).sum(dim=1, keepdim=True)
            d0 = P * (dp - delta)
            ds = d0 * f
            res[0][a:b, j] = ds @ K * scale
            res[1][a:b, c] += ds.t() @ Q * scale
            res[2][a:b, c] += P.t() @ dO
            rel = hw + e.masked_fill(~seen, 0.0) + (4 * U * z.abs() + (2 * n * rep + 64) * U)[:, None]
            eds = f * (rel * d0.abs() + P * (D + 4) * U * (dO.abs() @ V.abs().t() + (dO.abs() * O.abs()).sum(dim=1, keepdim=True))) + ef * d0.abs() \
                + TINY * (1.0 + dp.abs() + delta.abs())
            bnd[0][a:b, j] = eds @ K.abs() * scale
            bnd[1][a:b, c] += eds.t() @ Q.abs() * scale
            bnd[2][a:b, c] += (rel * P + TINY).t() @ dO.abs()
    return res, [(e + h * r.abs() + TINY) * 1.02 for e, r in zip(bnd, res)]


def check(lengths, Hq, Hkv, D, dtype, ch, seed=41, big=3.0):
    import sample_grad_norms_amd as dp
    cu = offsets(lengths)
    N, scale = cu[-1], float(torch.tensor(1.0 / math.sqrt(D), dtype=torch.float32))
    q, k, v, do = make(N, Hq, Hkv, D, dtype, seed, big)
    how = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=dev()), scale=scale, **ch.gpu())
    qd, kd, vd, dod = (x.to(dev()) for x in (q, k, v, do))
    o, lse = dp.attention_forward(qd, kd, vd, **how)
    wo, wl, bo, bl = forward_reference(ch, q, k, v, cu, scale)
    inside(o, wo, bo, "o")
    inside(lse, wl, bl, "lse")
    o2, lse2 = dp.attention_forward(qd, kd, vd, **how)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o_in, lse_in = wo.to(dtype), wl.float()
    args = (dod, qd, kd, vd, o_in.to(dev()), lse_in.to(dev()))
    grads = dp.attention_backward(*args, **how)
    want, bound = backward_reference(ch, do, q, k, v, o_in, lse_in, cu, scale)
    for name, x, w, b in zip(("dq", "dk", "dv"), grads, want, bound):
        inside(x, w, b, name)
    assert all(torch.equal(x, y) for x, y in zip(grads, dp.attention_backward(*args, **how)))


CHANGES = [dict(cap=5.0), dict(slopes=1.0), dict(prefix=0.5), dict(cap=30.0, slopes=0.5), dict(slopes=-0.02, prefix=0.3),
           dict(cap=2.0, slopes=0.3, prefix=0.7)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("change", CHANGES)
@pytest.mark.parametrize("lengths,Hq,Hkv,D", CASES)
def test_ragged_sequences(lengths, Hq, Hkv, D, change, dtype):
    check(lengths, Hq, Hkv, D, dtype, Change(Hq, lengths, **change))


EVERY = [(BF16, *s) for s in attention_forms.BF16] + [(F32, *s) for s in attention_forms.F32]


@pytest.mark.parametrize("change", [dict(cap=20.0), dict(slopes=0.5, prefix=0.4), dict(cap=8.0, slopes=0.1, prefix=100)])
@pytest.mark.parametrize("dtype,N,Hq,Hkv,D", EVERY)
def test_every_form(N, Hq, Hkv, D, change, dtype):
    check([N], Hq, Hkv, D, dtype, Change(Hq, [N], **change))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("prefix", [1, 2, 31, 32, 33, 63, 64, 65, 95, 96, 127, 128, 129, 159, 160, 199, 200])
def test_prefixes_at_the_edges_of_tiles(prefix, dtype):
    check([200], 2, 1, 64, dtype, Change(2, [200], prefix=prefix if prefix > 1 else 1.0 / 200 + 1e-9))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cap,big", [(0.001, 1.0), (0.5, 10.0), (50.0, 1e-3), (50.0, 100.0), (1000.0, 1.0), (1024.0, 300.0)])
def test_small_and_large_caps(cap, big, dtype):
    check([130, 40], 2, 1, 64, dtype, Change(2, [130, 40], cap=cap), big=big)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,Hq,Hkv,D", [(200, 4, 2, 64), (1040, 64, 16, 64), (900, 64, 64, 128)])
def test_changes_of_nothing(N, Hq, Hkv, D, dtype):
    """Prefixes of no row or of less, and no cap: plain causal attention, bit for bit."""
    import sample_grad_norms_amd as dp
    q, k, v, do = (x.to(dev()) for x in make(N, Hq, Hkv, D, dtype, 42))
    o, lse = dp.attention_forward(q, k, v, sequences=2)
    grads = dp.attention_backward(do, q, k, v, o, lse, sequences=2)
    for how in (dict(cap=0.0), dict(prefix=torch.zeros(2, dtype=torch.int32, device=dev())),
                dict(prefix=torch.tensor([-5, -2 ** 31], dtype=torch.int32, device=dev())), dict(slopes=torch.zeros(Hq, device=dev()))):
        o2, lse2 = dp.attention_forward(q, k, v, sequences=2, **how)
        assert torch.equal(o, o2) and torch.equal(lse, lse2), how
        assert all(torch.equal(a, b) for a, b in zip(grads, dp.attention_backward(do, q, k, v, o, lse, sequences=2, **how))), how
    # a prefix of the whole sequence, and of more
    whole = [dp.attention_forward(q, k, v, sequences=2, prefix=torch.full((2,), p, dtype=torch.int32, device=dev()))
             for p in (N // 2, N, 2 ** 31 - 1)]
    assert all(torch.equal(whole[0][0], w[0]) and torch.equal(whole[0][1], w[1]) for w in whole)


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("change", [dict(cap=10.0), dict(slopes=0.002, prefix=40), dict(prefix=0.5), dict(cap=10.0, prefix=97)])
@pytest.mark.parametrize("dtype,N,Hq,Hkv,D", EVERY)
def test_a_row_that_is_not_finite_leaves_the_others(N, Hq, Hkv, D, change, value, dtype):
    """Rows that do not see a row with an infinity or NaN get what they get without it, bit for
    bit; those that do get it (values) or are not finite."""
    import sample_grad_norms_amd as dp
    ch = Change(Hq, [N], **change)
    how, p = ch.gpu(), 0 if ch.prefix is None else min(int(ch.prefix[0]), N)
    q, k, v, do = (x.to(dev()) for x in make(N, Hq, Hkv, D, dtype, 43))
    o, lse = dp.attention_forward(q, k, v, **how)
    dq, dk, dv = dp.attention_backward(do, q, k, v, o, lse, **how)
    at = torch.arange(N, device=dev())
    for row in (5, 39, 64, 98, N // 2, N - 33, N - 1):
        sees, seen_by = (at >= row) | (row < p), (at <= row) | (at < p)   # queries that see key `row`, keys that query `row` sees
        for name in ("k", "v"):
            args = {"q": q, "k": k.clone(), "v": v.clone()}
            args[name][row, :, 3] = value
            o2, lse2 = dp.attention_forward(**args, **how)
            assert torch.equal(o2[~sees], o[~sees]) and torch.equal(lse2[:, ~sees], lse[:, ~sees]), (name, row)
            if name == "v":
                got = o2[sees][:, :, 3].float()
                assert bool((got.isnan() if math.isnan(value) else got == value).all()), row
                assert torch.equal(o2[:, :, :3], o[:, :, :3]) and torch.equal(o2[:, :, 4:], o[:, :, 4:]) and torch.equal(lse2, lse)
            dq2, _, _ = dp.attention_backward(do, args["q"], args["k"], args["v"], o, lse, **how)
            assert torch.equal(dq2[~sees], dq[~sees]), (name, row)
            assert not bool(dq2[sees][:, :, 3].isfinite().any()) if name == "k" else True, row
        for name in ("do", "q"):
            args = {"do": do.clone(), "q": q.clone()}
            args[name][row, :, 3] = value
            _, dk2, dv2 = dp.attention_backward(args["do"], args["q"], k, v, o, lse, **how)
            assert torch.equal(dk2[~seen_by], dk[~seen_by]) and torch.equal(dv2[~seen_by], dv[~seen_by]), (name, row)
            if name == "do":
                got = dv2[seen_by][:, :, 3].float()
                assert bool((got.isnan() if math.isnan(value) else got == value).all()), row
            else:
                assert not bool(dk2[seen_by][:, :, 3].isfinite().any()), row


@pytest.mark.parametrize("dtype,N,Hq,Hkv,D", EVERY)
def test_infinite_products_are_capped(N, Hq, Hkv, D, dtype):
    """Scores of +-infinity are +-C: a query with an infinity gives what one with 1e30 there
    gives, and its keys get those weights."""
    import sample_grad_norms_amd as dp
    q, k, v, do = make(N, Hq, Hkv, D, dtype, 44)
    k[:, :, 3] = torch.where(k[:, :, 3] < 0, k[:, :, 3] - 0.125, k[:, :, 3] + 0.125)
    q, k, v, do = (x.to(dev()) for x in (q, k, v, do))
    rows = torch.tensor([7, 40, 64, N // 2, N - 1], device=dev())
    big, inf = q.clone(), q.clone()
    big[rows, :, 3] = 1e30
    inf[rows, :, 3] = math.inf
    for how in (dict(cap=4.0), dict(cap=4.0, prefix=torch.tensor([50], dtype=torch.int32, device=dev()))):
        o, lse = dp.attention_forward(big, k, v, **how)
        o2, lse2 = dp.attention_forward(inf, k, v, **how)
        assert bool(o2.isfinite().all()) and torch.equal(o, o2) and torch.equal(lse, lse2)
        dv = dp.attention_backward(do, big, k, v, o, lse, **how)[2]
        _, dk2, dv2 = dp.attention_backward(do, inf, k, v, o, lse, **how)
        assert torch.equal(dv, dv2)
        # 0 (the derivative) times infinity: NaN in that column, for the keys that such a row sees
        assert bool(dk2[:, :, 3].isnan().all()) and bool(dk2[:, :, :3].isfinite().all()) and bool(dk2[:, :, 4:].isfinite().all())


def test_differences():
    """The gradients along random directions against differences of the definition in 64 bits."""
    import sample_grad_norms_amd as dp
    lengths, Hq, Hkv, D = [40, 25], 4, 2, 32
    ch = Change(Hq, lengths, cap=3.0, slopes=0.3, prefix=0.4)
    q, k, v, do = make(65, Hq, Hkv, D, F32, 45, 2.0)
    cu, scale = offsets(lengths), float(torch.tensor(1.0 / math.sqrt(D)))
    how = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=dev()), scale=scale, **ch.gpu())
    qd, kd, vd, dod = (t.to(dev()) for t in (q, k, v, do))
    o, lse = dp.attention_forward(qd, kd, vd, **how)
    grads = dp.attention_backward(dod, qd, kd, vd, o, lse, **how)
    ch.relative = True

    def loss(q, k, v):
        total = 0.0
        for i, (a, b) in enumerate(sequences(cu)):
            for j in range(Hq):
                s = ch.scores(q[a:b, j], k[a:b, j // 2], scale, j, i)[0]
                total += float((torch.softmax(s, dim=1) @ v[a:b, j // 2] * do[a:b, j].double()).sum())
        return total
    g = torch.Generator().manual_seed(46)
    at = [t.double() for t in (q, k, v)]
    for j, got in enumerate(grads):
        d = torch.randn(at[j].shape, generator=g, dtype=torch.float64)
        ends = [loss(*[t + f * 1e-5 * d if i == j else t for i, t in enumerate(at)]) for f in (1.0, -1.0)]
        want, terms = (ends[0] - ends[1]) / 2e-5, got.cpu().double() * d
        # float32 gradients (1e-5 of the terms' size, as they add), and 1e-10 of the third derivative
        assert abs(float(terms.sum()) - want) <= 1e-5 * float(terms.abs().sum()) + 1e-6, (j, float(terms.sum()), want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_streams_and_graphs(dtype):
    """Strided heads, two streams at once, and a captured run replayed beside eager work."""
    import sample_grad_norms_amd as dp
    N, Hq, Hkv, D = 190, 4, 2, 72
    ch = Change(Hq, [100, 90], cap=6.0, slopes=0.2, prefix=0.3)
    how = dict(cu_seqlens=torch.tensor([0, 100, 190], dtype=torch.int32, device=dev()), **ch.gpu())
    sets = [tuple(x.to(dev()) for x in make(N, Hq, Hkv, D, dtype, 47 + j)) for j in range(3)]

    def calls(q, k, v, do):
        o, lse = dp.attention_forward(q, k, v, **how)
        return (o, lse, *dp.attention_backward(do, q, k, v, o, lse, **how))
    want = [calls(*s) for s in sets]
    strided = calls(*(x.transpose(0, 1).contiguous().transpose(0, 1) for x in sets[0]))
    assert all(torch.equal(a, b) for a, b in zip(strided, want[0]))
    torch.cuda.synchronize()
    got = []
    for s, data in zip([torch.cuda.Stream() for _ in range(2)], sets):
        with torch.cuda.stream(s):
            got.append([calls(*data) for _ in range(5)][-1])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))
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
        assert all(torch.equal(a, b) for a, b in zip(out, want[j])) and all(torch.equal(a, b) for a, b in zip(eager, want[(j + 1) % 3]))


def test_rows_of_no_sequence_and_hostile_offsets():
    import sample_grad_norms_amd as dp
    q, k, v, do = (x.to(dev()) for x in make(100, 4, 2, 64, BF16, 48))
    ch = Change(4, [30, 40], cap=6.0, slopes=0.2, prefix=20)
    cu = torch.tensor([10, 40, 80], dtype=torch.int32, device=dev())
    o, lse = dp.attention_forward(q, k, v, cu_seqlens=cu, **ch.gpu())
    inner = torch.tensor([0, 30, 70], dtype=torch.int32, device=dev())
    o2, lse2 = dp.attention_forward(q[10:80], k[10:80], v[10:80], cu_seqlens=inner, **ch.gpu())
    assert torch.equal(o[10:80], o2) and torch.equal(lse[:, 10:80], lse2)
    assert not bool(o[:10].any()) and not bool(o[80:].any()) and not bool(lse[:, :10].any())
    held = torch.full_like(q, 3.0), torch.full_like(lse, 4.0)
    dp.attention_forward(q, k, v, cu_seqlens=cu, out=held[0], lse=held[1], **ch.gpu())
    assert torch.equal(held[0][10:80], o2) and bool((held[0][:10] == 3.0).all()) and bool((held[1][:, 80:] == 4.0).all())
    for bad in ([0, 2 ** 30, 50], [-9, 50, 20], [90, 10, 1000]):
        cu = torch.tensor(bad, dtype=torch.int32, device=dev())
        a = dp.attention_forward(q, k, v, cu_seqlens=cu, **ch.gpu())
        dp.attention_backward(do, q, k, v, *a, cu_seqlens=cu, **ch.gpu())
    torch.cuda.synchronize()


def test_refusals():
    import sample_grad_norms_amd as dp
    q, k, v, do = (x.to(dev()) for x in make(20, 4, 2, 64, BF16, 49))
    slopes, prefix = torch.ones(4, device=dev()), torch.ones(1, dtype=torch.int32, device=dev())
    o, lse = dp.attention_forward(q, k, v)
    for bad in (dict(cap=-1.0), dict(cap=math.nan), dict(cap=math.inf), dict(cap=2000.0), dict(cap=1e-4), dict(slopes=slopes, scale=1e-30)):
        with pytest.raises(dp.DpnormError):
            dp.attention_forward(q, k, v, **bad)
        with pytest.raises(dp.DpnormError):
            dp.attention_backward(do, q, k, v, o, lse, **bad)
    for bad in (dict(slopes=slopes[:2]), dict(slopes=slopes.cpu()), dict(prefix=prefix.repeat(2)), dict(prefix=prefix.cpu()),
                dict(slopes=slopes.repeat(2)[::2])):
        with pytest.raises(ValueError):
            dp.attention_forward(q, k, v, **bad)
    for bad in (dict(slopes=slopes.double()), dict(prefix=prefix.long())):
        with pytest.raises(TypeError):
            dp.attention_backward(do, q, k, v, o, lse, **bad)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kw", [{}, dict(cap=5.0), dict(prefix=True), dict(cap=5.0, prefix=True)])
@pytest.mark.parametrize("Hq,lengths", [(4, [1, 70, 33]), (64, [1, 1500, 1333])])   # by rows, by tiles
def test_the_steepest_slopes(dtype, kw, Hq, lengths):
    """Slopes of 2^32: every row has itself alone, since the next weight is exp(-2^32) = 0. So
    o = v, and lse is the row's own score; dp - delta is 0 but for roundings.

    Bounds (h the type's half step): in the forward pass the weight is exp(s - m) of one s, off by
    4 (|s| + 2) u, and o by 2 h more (the weight's rounding, the result's). The backward pass's
    weight exp(s - lse) is off by what its s and the forward pass's are off besides: each by
    (D + 8) u of sum |q k| scale and by 8 u of the cap, |s| and 1. dp and delta are
    sums of D products of the same numbers but for o's rounding error, so their difference
    is at most (2 D + 8) u + 4 (20 + 2) u + 2 h (1 + h) of sum |do v|, of which 2 h is there only
    where the forward pass did not return v bit for bit, as is asserted for bfloat16; that times
    scale, |k| and 1.1 (roundings of ds and of the result) bounds dq, and likewise dk. |lse| < 20:
    scores are cap at most, or 64 products of normals over 8.
    """
    import sample_grad_norms_amd as dp
    Hkv, D = 2, 64
    q, k, v, do = make(sum(lengths), Hq, Hkv, D, dtype, 51)
    kw = dict(kw)
    if kw.pop("prefix", False):
        kw["prefix"] = torch.tensor([1, 40, 0], dtype=torch.int32, device=dev())
    kw.update(slopes=torch.full((Hq,), 2.0 ** 32, device=dev()), cu_seqlens=torch.tensor(offsets(lengths), dtype=torch.int32, device=dev()))
    on = [x.to(dev()) for x in (q, k, v, do)]
    o, lse = dp.attention_forward(*on[:3], **kw)
    got = [x.double().cpu() for x in dp.attention_backward(on[3], *on[:3], o, lse, **kw)]
    q, k, v, do = (x.double() for x in (q, k, v, do))
    kr, vr = (x.repeat_interleave(Hq // Hkv, dim=1) for x in (k, v))
    h, scale = half(dtype), D ** -0.5
    s = (q * kr).sum(-1) * scale
    size = (q * kr).abs().sum(-1) * scale
    if "cap" in kw:
        s = kw["cap"] * torch.tanh(s / kw["cap"])
    assert float(s.abs().max()) < 20
    err = (lse.double().cpu().t() - s).abs()
    assert bool((err <= (D + 8) * U * size + 8 * U * (kw.get("cap", 0.0) + s.abs() + 1)).all())
    if dtype == BF16:
        assert torch.equal(o.double().cpu(), vr)
    loose = 4 * 22 * U + (0 if dtype == BF16 else 2 * h)
    assert bool(((o.double().cpu() - vr).abs() <= (4 * 22 * U + 2 * h) * vr.abs()).all())
    ds = ((2 * D + 8) * U + loose) * (do * vr).abs().sum(-1, keepdim=True) * scale * 1.1
    group = lambda x: x.view(x.shape[0], Hkv, Hq // Hkv, D).sum(2)
    assert all(bool(torch.isfinite(x).all()) for x in got)
    assert bool((got[0].abs() <= ds * kr.abs()).all())
    assert bool((got[1].abs() <= group(ds * q.abs())).all())
    again = 2 * U * ((D + 8) * float(size.max()) + 8 * (kw.get("cap", 0.0) + 20 + 1))
    assert bool(((got[2] - group(do)).abs() <= (4 * 22 * U + again + 2 * h) * group(do.abs())).all())
