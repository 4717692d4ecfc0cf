"""GPU parity of causal attention of packed sequences with grouped heads, and
of its gradients, against their definitions in float64 on the CPU.

Tolerances (u = 2^-24, h = half a step of the type, 2^-8 for bfloat16):
  * a score is a float32 sum of D products times the scale, and the exponent
    adds roundings relative to the score and the largest score: an error of at
    most x = 2 (D + 8) u A, A the largest scale sum_d |q_d k_d| of the row, so a
    weight is off by at most 2 x relative (numerator and normalisation);
  * bfloat16 weights are rounded (h relative) before they multiply rows, and
    sums over n keys in tiles add (2 n + 64) u relative to the sum of magnitudes;
  * the result is rounded once, h relative. For float32 h counts once, as u.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def dev():
    return torch.device("cuda:0")


def half(dtype):
    return torch.finfo(dtype).eps / 2


def make(N, Hq, Hkv, D, dtype, seed, big=1.0):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(N, Hq, D, generator=g) * big).to(dtype)
    k, v = torch.randn(N, Hkv, D, generator=g).to(dtype), torch.randn(N, Hkv, D, generator=g).to(dtype)
    do = torch.randn(N, Hq, D, generator=g).to(dtype)
    return q, k, v, do


def offsets(lengths, first=0):
    cu = [first]
    for n in lengths:
        cu.append(cu[-1] + n)
    return cu


def sequences(cu):
    return [(a, b) for a, b in zip(cu[:-1], cu[1:]) if b > a]


def masked_scores(q, k, scale):
    n = q.shape[0]
    s = (q @ k.t()) * scale
    return s.masked_fill(torch.ones(n, n, dtype=torch.bool).triu(1), -math.inf)


def forward_reference(q, k, v, cu, scale):
    """o, lse and their bounds, float64; rows of no sequence are NaN."""
    N, Hq, D = q.shape
    rep, h = Hq // k.shape[1], half(q.dtype)
    hw = h if q.dtype == torch.bfloat16 else 0.0
    o = torch.full((N, Hq, D), math.nan, dtype=torch.float64)
    lse = torch.full((Hq, N), math.nan, dtype=torch.float64)
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    for a, b in sequences(cu):
        n = b - a
        for j in range(Hq):
            Q, K, V = q[a:b, j].double(), k[a:b, j // rep].double(), v[a:b, j // rep].double()
            s = masked_scores(Q, K, scale)
            lse[j, a:b] = torch.logsumexp(s, dim=1)
            P = torch.exp(s - lse[j, a:b, None])
            o[a:b, j] = P @ V
            A = torch.where(s == -math.inf, torch.zeros_like(s), (Q.abs() @ K.abs().t()) * scale).amax(dim=1)
            x = 2 * (D + 8) * U * A + 8 * U
            bo[a:b, j] = (hw + 2 * x + (2 * n + 64) * U)[:, None] * (P @ V.abs()) + h * o[a:b, j].abs()
            bl[j, a:b] = x + (n + 64) * U + 2 * U * lse[j, a:b].abs()
    return o, lse, bo * 1.01, bl * 1.01


def backward_reference(do, q, k, v, o, lse, cu, scale):
    N, Hq, D = q.shape
    Hkv = k.shape[1]
    rep, h = Hq // Hkv, half(q.dtype)
    hw = h if q.dtype == torch.bfloat16 else 0.0
    res = [torch.zeros(N, H, D, dtype=torch.float64) for H in (Hq, Hkv, Hkv)]
    bnd = [torch.zeros(N, H, D, dtype=torch.float64) for H in (Hq, Hkv, Hkv)]
    for a, b in sequences(cu):
        n = b - a
        for j in range(Hq):
            c = j // rep
            Q, K, V = q[a:b, j].double(), k[a:b, c].double(), v[a:b, c].double()
            dO, O = do[a:b, j].double(), o[a:b, j].double()
            s = masked_scores(Q, K, scale)
            z = lse[j, a:b].double()
            P = torch.exp(s - z[:, None])
            A = torch.where(s == -math.inf, torch.zeros_like(s), (Q.abs() @ K.abs().t()) * scale).amax(dim=1)
            dp, delta = dO @ V.t(), (dO * O).sum(dim=1, keepdim=True)
            ds = P * (dp - delta)
            res[0][a:b, j] = ds @ K * scale
            res[1][a:b, c] += ds.t() @ Q * scale
            res[2][a:b, c] += P.t() @ dO
            rel = (hw + 2 * (D + 8) * U * A + 4 * U * z.abs() + (2 * n * rep + 64) * U)[:, None]
            eds = rel * ds.abs() + P * (D + 4) * U * (dO.abs() @ V.abs().t() + (dO.abs() * O.abs()).sum(dim=1, keepdim=True))
            bnd[0][a:b, j] = eds @ K.abs() * scale
            bnd[1][a:b, c] += eds.t() @ Q.abs() * scale
            bnd[2][a:b, c] += (rel * P).t() @ dO.abs()
    return res, [(e + h * r.abs()) * 1.01 for e, r in zip(bnd, res)]


def inside(got, want, bound, what):
    err = (got.cpu().double() - want).abs()
    rows = want.isfinite()
    ratio = float((err[rows] / bound[rows].clamp(min=1e-300)).max()) if bool(rows.any()) else 0.0
    print(f"{what}: max err / bound {ratio:.3f}", flush=True)
    assert ratio <= 1.0, what


CASES = [   # lengths, Hq, Hkv, D
    ([1], 1, 1, 8),
    ([5], 2, 1, 64),
    ([64], 4, 2, 64),
    ([65, 1, 127], 4, 4, 32),
    ([128, 128], 2, 1, 128),
    ([0, 33, 0, 0, 129, 0], 6, 3, 80),
    ([257, 31], 3, 1, 64),
    ([1] * 70 + [40], 2, 2, 40),        # more sequences than the lanes of a wave
    ([500, 1, 2, 3], 8, 2, 96),
    ([1030], 2, 1, 128),
    ([1029], 2, 2, 64),
    ([400, 1, 299], 64, 32, 64),        # many heads: work groups of 128 queries, and of four waves for dk and dv
    ([333, 370], 64, 32, 104),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lengths,Hq,Hkv,D", CASES)
def test_forward_and_backward(lengths, Hq, Hkv, D, dtype):
    import sample_grad_norms_amd as dp
    cu = offsets(lengths)
    N, scale = cu[-1], 1.0 / math.sqrt(D)
    q, k, v, do = make(N, Hq, Hkv, D, dtype, 7)
    cud = torch.tensor(cu, dtype=torch.int32, device=dev())
    qd, kd, vd, dod = (x.to(dev()) for x in (q, k, v, do))
    o, lse = dp.attention_forward(qd, kd, vd, cu_seqlens=cud)
    wo, wl, bo, bl = forward_reference(q, k, v, cu, scale)
    inside(o, wo, bo, "o")
    inside(lse, wl, bl, "lse")
    o2, lse2 = dp.attention_forward(qd, kd, vd, cu_seqlens=cud)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o_in, lse_in = wo.to(dtype), wl.float()
    grads = dp.attention_backward(dod, qd, kd, vd, o_in.to(dev()), lse_in.to(dev()), cu_seqlens=cud)
    want, bound = backward_reference(do, q, k, v, o_in, lse_in, cu, scale)
    for name, x, w, b in zip(("dq", "dk", "dv"), grads, want, bound):
        inside(x, w, b, name)
    again = dp.attention_backward(dod, qd, kd, vd, o_in.to(dev()), lse_in.to(dev()), cu_seqlens=cud)
    assert all(torch.equal(x, y) for x, y in zip(grads, again))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_equal_lengths_need_no_offsets(dtype):
    import sample_grad_norms_amd as dp
    q, k, v, do = (x.to(dev()) for x in make(3 * 150, 4, 2, 64, dtype, 8))
    cu = torch.tensor([0, 150, 300, 450], dtype=torch.int32, device=dev())
    a, b = dp.attention_forward(q, k, v, sequences=3), dp.attention_forward(q, k, v, cu_seqlens=cu)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x = dp.attention_backward(do, q, k, v, *a, sequences=3)
    y = dp.attention_backward(do, q, k, v, *b, cu_seqlens=cu)
    assert all(torch.equal(i, j) for i, j in zip(x, y))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("big,scale", [(30.0, 0.125), (1.0, 3.0), (1e-3, 1e-4)])
def test_large_and_small_scores(big, scale, dtype):
    """Softmaxes that are nearly one-hot, and nearly uniform."""
    import sample_grad_norms_amd as dp
    q, k, v, _ = make(200, 2, 1, 64, dtype, 9, big)
    o, lse = dp.attention_forward(q.to(dev()), k.to(dev()), v.to(dev()), scale=scale)
    f = float(torch.tensor(scale, dtype=torch.float32))
    wo, wl, bo, bl = forward_reference(q, k, v, [0, 200], f)
    inside(o, wo, bo, "o")
    inside(lse, wl, bl, "lse")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_and_repeated_rows(dtype):
    """q, k and v as views of one buffer, as [H][N][D] tensors, and a key head
    repeated over the heads with a stride of 0."""
    import sample_grad_norms_amd as dp
    N, Hq, Hkv, D = 190, 4, 2, 72
    q, k, v, do = (x.to(dev()) for x in make(N, Hq, Hkv, D, dtype, 10))
    cu = torch.tensor([0, 100, 190], dtype=torch.int32, device=dev())
    o, lse = dp.attention_forward(q, k, v, cu_seqlens=cu)
    g = dp.attention_backward(do, q, k, v, o, lse, cu_seqlens=cu)
    fused = torch.cat([q, k, v], dim=1)
    views = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    hnd = tuple(x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v))
    for a, b, c in (views, hnd):
        out = torch.empty(Hq, N, D, dtype=dtype, device=dev()).transpose(0, 1)
        o2, lse2 = dp.attention_forward(a, b, c, cu_seqlens=cu, out=out, lse=torch.empty_like(lse))
        assert o2 is out and torch.equal(o2, o) and torch.equal(lse2, lse)
        grads = tuple(torch.empty(x.shape[1], N, D, dtype=dtype, device=dev()).transpose(0, 1) for x in (a, b, c))
        g2 = dp.attention_backward(do.transpose(0, 1).contiguous().transpose(0, 1), a, b, c, o2, lse2, cu_seqlens=cu, out=grads)
        assert all(torch.equal(x, y) for x, y in zip(g, g2))
    k1, v1 = k[:, :1], v[:, :1]
    a = dp.attention_forward(q, k1.expand(N, 2, D), v1.expand(N, 2, D), cu_seqlens=cu)
    b = dp.attention_forward(q, k1.contiguous(), v1.contiguous(), cu_seqlens=cu)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_no_sequence(dtype):
    """Rows before the first and behind the last sequence: not read (they hold
    NaN), and left as they were; nothing of a neighbour sequence is read."""
    import sample_grad_norms_amd as dp
    N, Hq, Hkv, D = 220, 4, 2, 64
    q, k, v, do = make(N, Hq, Hkv, D, dtype, 11)
    cu = [3, 70, 70, 201]
    for x in (q, k, v, do):
        x[:3] = math.nan
        x[201:] = math.nan
    cud = torch.tensor(cu, dtype=torch.int32, device=dev())
    args = [x.to(dev()) for x in (q, k, v)]
    out, lse = torch.full((N, Hq, D), 7.0, dtype=dtype, device=dev()), torch.full((Hq, N), 7.0, device=dev())
    dp.attention_forward(*args, cu_seqlens=cud, out=out, lse=lse)
    wo, wl, bo, bl = forward_reference(q, k, v, cu, 1 / 8)
    inside(out, wo, bo, "o")
    inside(lse, wl, bl, "lse")
    free = torch.ones(N, dtype=torch.bool)
    free[3:201] = False
    assert bool((out.cpu()[free] == 7).all()) and bool((lse.cpu()[:, free] == 7).all())
    grads = tuple(torch.full_like(x, 7.0) for x in args)
    dp.attention_backward(do.to(dev()), *args, out, lse, cu_seqlens=cud, out=grads)
    want, bound = backward_reference(do, q, k, v, out.cpu(), lse.cpu(), cu, 1 / 8)
    for name, x, w, b in zip(("dq", "dk", "dv"), grads, want, bound):
        assert bool((x.cpu()[free] == 7).all())
        inside(x[3:201], w[3:201], b[3:201], name)
    # made by the call, such rows are zero
    dirty = [torch.full_like(x, 9.0) for x in (out, lse, *args)]   # the allocator hands these out again
    del dirty
    o2, lse2 = dp.attention_forward(*args, cu_seqlens=cud)
    assert bool((o2.cpu()[free] == 0).all()) and bool((lse2.cpu()[:, free] == 0).all())
    for x, y in zip(dp.attention_backward(do.to(dev()), *args, out, lse, cu_seqlens=cud), grads):
        assert bool((x.cpu()[free] == 0).all()) and torch.equal(x[3:201], y[3:201])
    # a NaN in one sequence leaves the other as it was
    for x in args:
        x[3:70] = math.nan
    o3, _ = dp.attention_forward(*args, cu_seqlens=cud)
    assert torch.equal(o3[70:201], o2[70:201]) and bool(o3[3:70].isnan().all())


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hq,Hkv", [(2, 1), (64, 64)])
def test_a_row_that_is_not_finite_leaves_the_rows_before_it(Hq, Hkv, dtype, value):
    """Causality holds for infinities and NaN: rows before the row that holds one
    get what they get without it, forward and backward, bit for bit."""
    import sample_grad_norms_amd as dp
    N, D = 700 if Hq == 64 else 180, 64
    q, k, v, do = (x.to(dev()) for x in make(N, Hq, Hkv, D, dtype, 18))
    o, lse = dp.attention_forward(q, k, v)
    grads = dp.attention_backward(do, q, k, v, o, lse)
    for row in (N - 100, N - 1):
        for name in ("k", "v"):
            args = {"q": q, "k": k.clone(), "v": v.clone()}
            args[name][row, :, 5] = value
            o2, lse2 = dp.attention_forward(**args)
            assert torch.equal(o2[:row], o[:row]) and torch.equal(lse2[:, :row], lse[:, :row]), (name, row)
            # every later query sees it: in v as what it is, in k as NaN or as weights of 0 or 1
            if name == "v":
                later = o2[row:, :, 5].float()
                assert bool((later.isnan() if math.isnan(value) else later == value).all())
                assert bool(o2[row:, :, :5].isfinite().all())
            # dq of the rows before sees neither (its own do and o are as before)
            dq, _, _ = dp.attention_backward(do, args["q"], args["k"], args["v"], o, lse)
            assert torch.equal(dq[:row], grads[0][:row]), (name, row)
    # dk and dv of later keys see no earlier query
    for row in (0, 77):
        for name in ("do", "q"):
            args = {"do": do.clone(), "q": q.clone()}
            args[name][row, :, 5] = value
            _, dk, dv = dp.attention_backward(args["do"], args["q"], k, v, o, lse)
            assert torch.equal(dk[row + 1:], grads[1][row + 1:]) and torch.equal(dv[row + 1:], grads[2][row + 1:]), (name, row)
            if name == "do":
                assert not bool(dv[:row + 1, :, 5].isfinite().any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 96), (64, 64, 88), (3, 1, 128), (64, 64, 120)])
def test_wider_rows_that_are_not_finite_leave_the_others(Hq, Hkv, D, dtype):
    import sample_grad_norms_amd as dp
    N = 700 if Hq == 64 else 330
    q, k, v, do = (x.to(dev()) for x in make(N, Hq, Hkv, D, dtype, 19))
    o, lse = dp.attention_forward(q, k, v)
    dq, dk, dv = dp.attention_backward(do, q, k, v, o, lse)
    at, val = N - 75, torch.tensor([math.nan, math.inf, -math.inf], device=dev()).to(dtype)
    for name in ("k", "v"):
        args = {"q": q, "k": k.clone(), "v": v.clone()}
        args[name][at, :, :3] = val
        o2, _ = dp.attention_forward(**args)
        assert torch.equal(o2[:at], o[:at]), name
        dq2, _, _ = dp.attention_backward(do, args["q"], args["k"], args["v"], o, lse)
        assert torch.equal(dq2[:at], dq[:at]), name
    for name in ("do", "q"):
        args = {"do": do.clone(), "q": q.clone()}
        args[name][at, :, :3] = val
        _, dk2, dv2 = dp.attention_backward(args["do"], args["q"], k, v, o, lse)
        assert torch.equal(dk2[at + 1:], dk[at + 1:]) and torch.equal(dv2[at + 1:], dv[at + 1:]), name


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lengths", [[400, 397], [31, 1, 0, 801]])
def test_many_heads_of_88_columns(lengths, dtype):
    """Work groups of 128 queries, and one for each 32 keys, for rows of 65 to 96 columns."""
    test_forward_and_backward(lengths, 64, 32, 88, dtype)


@pytest.mark.parametrize("D", [40, 64])
def test_long_chains_of_few_keys(D):
    """Groups of 32 keys about as many as the places on the CUs, long chains of queries."""
    test_forward_and_backward([1040], 64, 16, D, torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 1, 64), (64, 64, 64), (64, 64, 104)])
def test_scores_of_minus_infinity_have_no_weight(Hq, Hkv, D, dtype):
    """Keys whose scores are -infinity, for a query's first steps and all through:
    the later rows are the attention of the other keys, the first have none."""
    import sample_grad_norms_amd as dp
    N, first = 700 if Hq == 64 else 330, 190
    q, k, v, _ = make(N, Hq, Hkv, D, dtype, 21)
    q = q.abs() + 0.125
    k[:first, :, 3] = -math.inf
    o, lse = dp.attention_forward(*(x.to(dev()) for x in (q, k, v)))
    wo, wl, bo, bl = forward_reference(q[first:], k[first:], v[first:], [0, N - first], 1.0 / math.sqrt(D))
    inside(o[first:], wo, bo, "o")
    inside(lse[:, first:], wl, bl, "lse")
    assert bool(o[:first].isnan().all()) and bool((lse[:, :first] == -math.inf).all())


@pytest.mark.parametrize("cu", [[0, 0, 0], [130, 130], [0, 64, 128], [100, 101, 133]])
def test_rows_of_no_sequence_are_cleared(cu):
    """No sequence at all, tiles that fill every slot, one row among many."""
    import sample_grad_norms_amd as dp
    for Hq, Hkv in ((2, 1), (64, 64)):
        N = 133 if Hq == 2 else 900
        q, k, v, do = (x.to(dev()) for x in make(N, Hq, Hkv, 64, torch.bfloat16, 17))
        cud = torch.tensor(cu, dtype=torch.int32, device=dev())
        dirty = [torch.full_like(x, 9.0) for x in (q, q, k, v)]
        del dirty
        o, lse = dp.attention_forward(q, k, v, cu_seqlens=cud)
        grads = dp.attention_backward(do, q, k, v, o, lse, cu_seqlens=cud)
        free = torch.ones(N, dtype=torch.bool)
        free[cu[0]:cu[-1]] = False
        for x in (o, lse.t(), *grads):
            assert bool((x.cpu()[free] == 0).all()) and bool(x.isfinite().all())


def test_offsets_outside_the_rows_are_clamped():
    import sample_grad_norms_amd as dp
    q, k, v, _ = (x.to(dev()) for x in make(70, 2, 1, 64, torch.bfloat16, 12))
    want, _ = dp.attention_forward(q, k, v)
    for cu in ([-5, 1000000], [0, 70, 90, 2000000000], [-2000000000, -3, 70]):
        o, _ = dp.attention_forward(q, k, v, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=dev()))
        assert torch.equal(o, want)


def test_byte_offsets_past_32_bits():
    import sample_grad_norms_amd as dp
    N, D, stride = 700, 64, 4_000_000
    q, k, v, do = make(N, 1, 1, D, torch.bfloat16, 13)
    buf = torch.empty(N * stride + D, dtype=torch.bfloat16, device=dev())
    wide = buf.as_strided((N, 1, D), (stride, D, 1))
    assert N * stride * 2 > 2 ** 32
    small = [x.to(dev()) for x in (q, k, v, do)]
    o, lse = dp.attention_forward(*small[:3])
    g = dp.attention_backward(small[3], *small[:3], o, lse)
    for j in range(3):
        wide.copy_(small[j])
        args = list(small)
        args[j] = wide
        o2, lse2 = dp.attention_forward(*args[:3])
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        assert all(torch.equal(x, y) for x, y in zip(g, dp.attention_backward(args[3], *args[:3], o, lse)))
    dp.attention_forward(*small[:3], out=wide, lse=lse2)
    assert torch.equal(wide, o)


def test_gradients_against_differences():
    """<dq, x> + <dk, y> + <dv, z> against the central difference of
    sum(do * o) in float64 along (x, y, z)."""
    import sample_grad_norms_amd as dp
    N, Hq, Hkv, D, cu = 90, 4, 2, 32, [0, 37, 90]
    q, k, v, do = make(N, Hq, Hkv, D, torch.float32, 14)
    cud = torch.tensor(cu, dtype=torch.int32, device=dev())
    args = [x.to(dev()) for x in (q, k, v)]
    o, lse = dp.attention_forward(*args, cu_seqlens=cud)
    grads = dp.attention_backward(do.to(dev()), *args, o, lse, cu_seqlens=cud)
    g = torch.Generator().manual_seed(15)
    scale, e = 1 / math.sqrt(D), 1e-4

    def value(a, b, c):
        return float((forward_reference(a, b, c, cu, scale)[0] * do.double()).sum())

    for _ in range(3):
        d = [torch.randn(x.shape, generator=g, dtype=torch.float64) for x in (q, k, v)]
        up = [x.double() + e * y for x, y in zip((q, k, v), d)]
        dn = [x.double() - e * y for x, y in zip((q, k, v), d)]
        diff = (value(*up) - value(*dn)) / (2 * e)
        dot = sum(float((x.cpu().double() * y).sum()) for x, y in zip(grads, d))
        size = sum(float((x.cpu().double() * y).abs().sum()) for x, y in zip(grads, d))
        # the difference is off by O(e^2) of third derivatives (order one here), the gradients by float32 roundings
        assert abs(dot - diff) <= 1e-6 * size + 100 * e * e * size


def test_replayed_graph_and_other_stream_match_eager():
    import sample_grad_norms_amd as dp
    q, k, v, do = (x.to(dev()) for x in make(400, 4, 2, 64, torch.bfloat16, 16))
    cu = torch.tensor([0, 130, 131, 400], dtype=torch.int32, device=dev())

    def step():
        o, lse = dp.attention_forward(q, k, v, cu_seqlens=cu)
        return (o, lse) + dp.attention_backward(do, q, k, v, o, lse, cu_seqlens=cu)

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    for r, new in enumerate(([0, 130, 131, 400], [0, 400, 400, 400], [5, 9, 9, 300])):
        cu.copy_(torch.tensor(new, dtype=torch.int32))
        q.copy_(make(400, 4, 2, 64, torch.bfloat16, 20 + r)[0])
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in res]
        assert all(torch.equal(x, y) for x, y in zip(got, step()))


def test_no_rows():
    import sample_grad_norms_amd as dp
    q = torch.empty(0, 4, 64, device=dev())
    o, lse = dp.attention_forward(q, q[:, :2], q[:, :2])
    assert tuple(o.shape) == (0, 4, 64) and tuple(lse.shape) == (4, 0)
    q = torch.ones(3, 2, 64, device=dev())
    o, lse = dp.attention_forward(q, q, q, cu_seqlens=torch.zeros(1, dtype=torch.int32, device=dev()))
    assert bool((o == 0).all()) and bool((lse == 0).all())


def test_refusals():
    import sample_grad_norms_amd as dp
    q, k = torch.zeros(12, 4, 64, device=dev()), torch.zeros(12, 2, 64, device=dev())
    cu = torch.zeros(2, dtype=torch.int32, device=dev())
    lse = torch.zeros(4, 12, device=dev())
    wide, odd = torch.zeros(12, 4, 132, device=dev()), torch.zeros(12, 4, 6, device=dev())
    buf = torch.zeros(12 * 4 * 64 + 8, device=dev())
    for call in (lambda: dp.attention_forward(wide, wide, wide), lambda: dp.attention_forward(odd, odd, odd),
                 lambda: dp.attention_forward(q, k, k, scale=0.0), lambda: dp.attention_forward(q, k, k, scale=float("nan")),
                 lambda: dp.attention_forward(q, k, k, out=q, lse=lse),                                        # an output over an input
                 lambda: dp.attention_forward(q, k, k, out=torch.zeros(1, 4, 64, device=dev()).expand(12, 4, 64), lse=lse),
                 lambda: dp.attention_forward(buf[1:1 + q.numel()].view(q.shape), k, k),              # not 16-byte aligned
                 lambda: dp.attention_backward(q.clone(), q, k, k, q.clone(), lse, out=(q.clone(), k, k.clone()))):
        with pytest.raises(dp.DpnormError):
            call()
    for call in (lambda: dp.attention_forward(q, k, k[:, :1]), lambda: dp.attention_forward(q[:, :3], k, k),
                 lambda: dp.attention_forward(q, k[:11], k[:11]), lambda: dp.attention_forward(q, k, k, sequences=5),
                 lambda: dp.attention_forward(q, k, k, sequences=1, cu_seqlens=cu),
                 lambda: dp.attention_forward(q.transpose(1, 2), k, k), lambda: dp.attention_forward(q.cpu(), k, k),
                 lambda: dp.attention_forward(q, k, k, out=q[:11], lse=lse), lambda: dp.attention_forward(q, k, k, lse=lse),
                 lambda: dp.attention_forward(q, k, k, out=q.clone(), lse=lse.t()),
                 lambda: dp.attention_backward(q[:11], q, k, k, q, lse),
                 lambda: dp.attention_backward(q, q, k, k, q, lse, workspace=torch.zeros(8, device=dev()))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: dp.attention_forward(q.half(), k.half(), k.half()), lambda: dp.attention_forward(q, k.bfloat16(), k),
                 lambda: dp.attention_forward(q, k, k, cu_seqlens=cu.long())):
        with pytest.raises(TypeError):
            call()
