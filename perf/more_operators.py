"""Cases of the normalisation layers and of attention with changed scores: inputs,
plain forms, calls.

The operators are those of a DP-SGD-RC training step whose normalisation layers
train too, and whose attention is not plain causal attention:
  ln            y = (x - mu) r w + b, with each row's mu = mean(x) and
                r = (mean((x - mu)^2) + eps)^-1/2; RMS norm: mu = 0 and no b
  ln_grad       its gradients dx, dw, db, the weights' with the samples' clip
                factors c: dw = sum_t c_i(t) dy_t h_t, db = sum_t c_i(t) dy_t,
                h = (x - mu) r
  ln_norm       n_i = || sum_t G_t h_t ||^2 + || sum_t G_t ||^2, the exact squared
                gradient norm of sample i's gain and bias (RMS norm: gain alone)
  attention     softmax attention of packed sequences with grouped heads over
                s_tu = cap tanh(a q_t . k_u / cap) - m_h |t - u|, where row t sees
                u <= t and the sequence's first rows u < prefix; and the log-sum-exp
  attention_grad its gradients dq, dk, dv from do, o and the log-sum-exp
"""
import math

import torch

own = False

_DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
_EPS = 1e-5


def listed():
    return [
        # a few tokens of a small model, all of a short sample: latency
        {"name": "ln_short", "op": "ln", "dtype": "fp32", "kind": "layer", "B": 1, "T": 37, "d": 1000},
        # the input of the measured training stack (B = 4, T = 4096, width 2048), RMS norm as there
        {"name": "ln_batch", "op": "ln", "dtype": "bf16", "kind": "rms", "B": 4, "T": 4096, "d": 2048},
        # gradients of a small batch of short samples
        {"name": "ln_grad_short", "op": "ln_grad", "dtype": "fp32", "kind": "layer", "B": 3, "T": 61, "d": 256, "pad": 0.3},
        # gradients of the measured stack's norms, clipped per sample
        {"name": "ln_grad_batch", "op": "ln_grad", "dtype": "bf16", "kind": "layer", "B": 4, "T": 4096, "d": 2048, "pad": 0.0},
        # per-sample norms of many padded samples of ordinary length
        {"name": "ln_norm_padded", "op": "ln_norm", "dtype": "bf16", "kind": "rms", "B": 33, "T": 1000, "d": 1024, "pad": 0.4},
        # per-sample norms of the measured stack's layers
        {"name": "ln_norm_batch", "op": "ln_norm", "dtype": "bf16", "kind": "layer", "B": 4, "T": 4096, "d": 2048, "pad": 0.0},
        # short samples packed one after another, the heads of the small test model, capped scores
        {"name": "attention_capped_short", "op": "attention", "dtype": "bf16", "lengths": "1,37,64,5", "Hq": 4, "Hkv": 2, "D": 64,
         "cap": 50.0, "slopes": False, "prefix": 0.0},
        # the attention of the measured DP-SGD-RC step (B = 4, T = 2048, 32 heads over 8) with capped scores
        {"name": "attention_capped_batch", "op": "attention", "dtype": "bf16", "lengths": "2048,2048,2048,2048", "Hq": 32, "Hkv": 8,
         "D": 64, "cap": 50.0, "slopes": False, "prefix": 0.0},
        # long documents packed with short ones, wide heads, a bias by distance in place of position embeddings
        {"name": "attention_biased_long", "op": "attention", "dtype": "bf16", "lengths": "10007,1,777,4100", "Hq": 16, "Hkv": 2,
         "D": 128, "cap": 0.0, "slopes": True, "prefix": 0.0},
        # gradients of the measured step's attention with capped scores
        {"name": "attention_grad_capped_batch", "op": "attention_grad", "dtype": "bf16", "lengths": "2048,2048,2048,2048", "Hq": 32,
         "Hkv": 8, "D": 64, "cap": 50.0, "slopes": False, "prefix": 0.0},
        # gradients of prompts that are seen whole and answers after them, biased by distance
        {"name": "attention_grad_prefix", "op": "attention_grad", "dtype": "bf16", "lengths": "1501,900,33,1200", "Hq": 16, "Hkv": 4,
         "D": 128, "cap": 0.0, "slopes": True, "prefix": 0.4},
        # gradients in float32, ragged lengths, a head width that is no power of two, all three at once
        {"name": "attention_grad_float", "op": "attention_grad", "dtype": "fp32", "lengths": "515,130,1,61", "Hq": 6, "Hkv": 3, "D": 80,
         "cap": 30.0, "slopes": True, "prefix": 0.3},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln", "ln_grad", "ln_norm", "attention", "attention", "attention_grad", "attention_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op.startswith("ln"):
        step = 8 if dtype == "bf16" else 4
        d = step * _log(rng, 4, 8192 // step)
        B = _log(rng, 1, 40)
        T = _log(rng, 1, max(1, (16384 * 2048) // (B * d * (2 if dtype == "fp32" else 1))))
        case = {"op": op, "dtype": dtype, "kind": rng.choice(["layer", "rms"]), "B": B, "T": min(T, 40000), "d": d}
        if op != "ln":
            case["pad"] = rng.choice([0.0, 0.0, 0.35])
        return case
    D = rng.choice([32, 64, 64, 72, 80, 96, 128, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    cap, slopes, prefix = rng.choice([(50.0, False, 0.0), (20.0, False, 0.0), (0.0, True, 0.0), (0.0, False, 0.5), (0.0, True, 0.3),
                                      (30.0, True, 0.0), (30.0, False, 0.7)])
    # pairs (row, key) times heads times width, at most a twentieth of the largest listed case in float32 or for gradients
    most = _pairs([10007], 0.0) * 16 * 128 // (20 if dtype == "fp32" or op == "attention_grad" else 2)
    lengths = []
    for j in range(rng.randint(1, 6)):
        room = most / (Hq * D) - _pairs(lengths, prefix)
        top = int(math.sqrt(max(2.0 * room / (1.0 + prefix), 1.0)))
        # (the gradients of q and k of a row alone are zero up to rounding: one sequence at least is longer)
        lengths.append(_log(rng, 16 if j == 0 else 1, max(16 if j == 0 else 1, min(top, 9000))))
    rng.shuffle(lengths)
    return {"op": op, "dtype": dtype, "lengths": ",".join(str(n) for n in lengths), "Hq": Hq, "Hkv": Hkv, "D": D, "cap": cap,
            "slopes": slopes, "prefix": prefix}


def _lengths(case):
    return [int(n) for n in case["lengths"].split(",")]


def _prefixes(lengths, share):
    return [int(n * share) for n in lengths]


def _pairs(lengths, share):
    """Pairs (row, key) that are seen: u <= t, and u < p for the rows before p."""
    return sum(n * (n + 1) // 2 + max(0, p * (p - 1) // 2) for n, p in zip(lengths, _prefixes(lengths, share)))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _DTYPE[case["dtype"]]
    st = dict(case)
    if case["op"].startswith("ln"):
        B, T, d = case["B"], case["T"], case["d"]
        # channels of different sizes and some offset, as the residual stream of a trained model has
        size = torch.exp(0.5 * torch.randn(d, generator=g, device=dev))
        off = 0.2 * torch.randn(d, generator=g, device=dev)
        st["x"] = (torch.randn(B, T, d, generator=g, device=dev) * size + off).to(dt)
        if case["op"] != "ln_norm":
            st["w"] = (1.0 + 0.2 * torch.randn(d, generator=g, device=dev)).to(dt)
            st["b"] = (0.1 * torch.randn(d, generator=g, device=dev)).to(dt) if case["kind"] == "layer" else None
        if case["op"] != "ln":
            G = torch.randn(B, T, d, generator=g, device=dev) * 0.01
            if case["pad"] > 0:  # samples shorter than T end in positions without a gradient
                keep = (T * (1.0 - case["pad"] * torch.rand(B, 1, 1, generator=g, device=dev))).ceil()
                G = torch.where(torch.arange(T, device=dev)[None, :, None] < keep, G, torch.zeros_like(G))
            st["G"] = G.to(dt)
            st["c"] = torch.rand(B, generator=g, device=dev) * 0.9 + 0.1
        if case["op"] == "ln_grad":
            st["mean"], st["rstd"] = _statistics(st)
        return st
    L, Hq, Hkv, D = _lengths(case), case["Hq"], case["Hkv"], case["D"]
    N = sum(L)
    st["L"] = L
    st["cu"] = torch.tensor([sum(L[:j]) for j in range(len(L) + 1)], dtype=torch.int32, device=dev)
    st["P"] = _prefixes(L, case["prefix"])
    st["prefix"] = torch.tensor(st["P"], dtype=torch.int32, device=dev) if case["prefix"] > 0 else None
    # slopes 2^(-8 j / Hq), j = 1 .. Hq
    st["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=dev) / Hq).float() if case["slopes"] else None
    # queries large enough for scores that a cap changes
    st["q"] = (torch.randn(N, Hq, D, generator=g, device=dev) * (4.0 if case["cap"] else 1.0)).to(dt)
    st["k"] = torch.randn(N, Hkv, D, generator=g, device=dev).to(dt)
    st["v"] = torch.randn(N, Hkv, D, generator=g, device=dev).to(dt)
    if case["op"] == "attention_grad":
        st["do"] = torch.randn(N, Hq, D, generator=g, device=dev).to(dt)
        st["o"], st["lse"] = _attention(st)
    return st


# ---- plain forms (float32, rounded once) ----

def _statistics(st):
    x = st["x"].float()
    mean = x.mean(dim=-1) if st["kind"] == "layer" else None
    if mean is not None:
        x = x - mean[..., None]
    return mean, 1.0 / torch.sqrt((x * x).mean(dim=-1) + _EPS)


def _normal(st, mean, rstd):
    x = st["x"].float()
    return (x if mean is None else x - mean[..., None]) * rstd[..., None]


def _ln(st):
    mean, rstd = _statistics(st)
    y = _normal(st, mean, rstd) * st["w"].float()
    if st["b"] is not None:
        y = y + st["b"].float()
    return (y.to(st["x"].dtype), rstd) if mean is None else (y.to(st["x"].dtype), mean, rstd)


def _ln_grad(st):
    dt, mean, rstd = st["x"].dtype, st["mean"], st["rstd"]
    h, dy, c = _normal(st, mean, rstd), st["G"].float(), st["c"][:, None, None]
    g = dy * st["w"].float()
    dx = g - h * (g * h).mean(dim=-1, keepdim=True)
    if mean is not None:
        dx = dx - g.mean(dim=-1, keepdim=True)
    dx = (dx * rstd[..., None]).to(dt)
    dw = (dy * h * c).sum(dim=(0, 1)).to(dt)
    return (dx, dw) if mean is None else (dx, dw, (dy * c).sum(dim=(0, 1)).to(dt))


def _ln_norm(st):
    h, G = _normal(st, *_statistics(st)), st["G"].float()
    n = ((G * h).sum(dim=1).double() ** 2).sum(dim=1)
    if st["kind"] == "layer":
        n = n + (G.sum(dim=1).double() ** 2).sum(dim=1)
    return n.float()


def _scores(st, q, k, p):
    """Scores [H, n, n] of one sequence's heads (q, k [n, H, D] float32) with a prefix of p rows, and tanh where they are capped."""
    n, cap, t = q.shape[0], st["cap"], None
    s = torch.matmul(q.transpose(0, 1), k.permute(1, 2, 0).contiguous()) * (1.0 / math.sqrt(st["D"]))
    if cap:
        t = torch.tanh(s / cap)
        s = t * cap
    at = torch.arange(n, device=q.device)
    if st["slopes"] is not None:
        s = s - st["slopes"][:, None, None] * (at[:, None] - at[None]).abs().float()
    return s.masked_fill_((at[None] > at[:, None]) & (at[None] >= p), float("-inf")), t


def _attention(st):
    rep = st["Hq"] // st["Hkv"]
    outs, lses = [], []
    for q, k, v, p in zip(*(st[x].split(st["L"]) for x in ("q", "k", "v")), st["P"]):
        s, _ = _scores(st, q.float(), k.float().repeat_interleave(rep, dim=1), p)
        m = s.amax(dim=-1, keepdim=True)
        p = torch.exp(s - m)
        del s
        l = p.sum(dim=-1, keepdim=True)
        o = torch.matmul(p, v.float().repeat_interleave(rep, dim=1).transpose(0, 1).contiguous()) / l
        outs.append(o.transpose(0, 1))
        lses.append((m + torch.log(l))[..., 0])
    return torch.cat(outs).to(st["q"].dtype), torch.cat(lses, dim=1).contiguous()


def _attention_grad(st):
    rep, D = st["Hq"] // st["Hkv"], st["D"]
    scale = 1.0 / math.sqrt(D)
    dqs, dks, dvs = [], [], []
    for q, k, v, o, do, lse, pre in zip(*(st[x].split(st["L"]) for x in ("q", "k", "v", "o", "do")), st["lse"].split(st["L"], dim=1), st["P"]):
        n = q.shape[0]
        q, do = q.float().transpose(0, 1), do.float().transpose(0, 1).contiguous()
        k, v = k.float().repeat_interleave(rep, dim=1), v.float().repeat_interleave(rep, dim=1)
        s, t = _scores(st, q.transpose(0, 1), k, pre)
        p = torch.exp(s - lse[..., None])
        del s
        dv = torch.matmul(p.transpose(1, 2).contiguous(), do)
        delta = (do * o.float().transpose(0, 1)).sum(dim=-1, keepdim=True)
        ds = torch.matmul(do, v.permute(1, 2, 0).contiguous()).sub_(delta).mul_(p)
        del p
        if t is not None:
            ds = ds * (1.0 - t * t)
        dq = torch.matmul(ds, k.transpose(0, 1).contiguous()) * scale
        dk = torch.matmul(ds.transpose(1, 2).contiguous(), q.contiguous()) * scale
        dqs.append(dq.transpose(0, 1))
        dks.append(dk.reshape(-1, rep, n, D).sum(dim=1).transpose(0, 1))
        dvs.append(dv.reshape(-1, rep, n, D).sum(dim=1).transpose(0, 1))
    return tuple(torch.cat(x).to(st["q"].dtype) for x in (dqs, dks, dvs))


def run(st):
    op = st["op"]
    if own:
        import sample_grad_norms_amd as dp
        if op.startswith("ln"):
            rms = st["kind"] == "rms"
            if op == "ln":
                y, mean, rstd = dp.layernorm_forward(st["x"], st["w"], st["b"], eps=_EPS, rms=rms)
                return (y, rstd) if rms else (y, mean, rstd)
            if op == "ln_norm":
                return dp.layernorm_norm(st["x"], st["G"], eps=_EPS, rms=rms, bias=not rms)
            dx, dw, db = dp.layernorm_backward(st["G"], st["x"], st["w"], st["mean"], st["rstd"], bias=not rms, weights=st["c"])
            return (dx, dw) if rms else (dx, dw, db)
        how = dict(cu_seqlens=st["cu"], cap=st["cap"] or None, slopes=st["slopes"], prefix=st["prefix"])
        if op == "attention":
            return dp.attention_forward(st["q"], st["k"], st["v"], **how)
        return dp.attention_backward(st["do"], st["q"], st["k"], st["v"], st["o"], st["lse"], **how)
    return {"ln": _ln, "ln_grad": _ln_grad, "ln_norm": _ln_norm, "attention": _attention, "attention_grad": _attention_grad}[op](st)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("ln"):
        N, d, two = case["B"] * case["T"], case["d"], 2 if case["kind"] == "layer" else 1
        if case["op"] == "ln":
            return {"bytes": 2 * N * d * e + two * d * e + two * 4 * N, "flops": (5 + 2 * two) * N * d}
        if case["op"] == "ln_norm":
            return {"bytes": 2 * N * d * e + 4 * case["B"], "flops": (5 + 2 * two) * N * d}
        return {"bytes": 3 * N * d * e + two * 4 * N + (1 + two) * d * e + 4 * case["B"], "flops": (10 + 2 * two) * N * d}
    L, Hq, Hkv, D = _lengths(case), case["Hq"], case["Hkv"], case["D"]
    N, pairs = sum(L), _pairs(_lengths(case), case["prefix"])
    if case["op"] == "attention":
        return {"bytes": N * D * e * (2 * Hq + 2 * Hkv) + 4 * N * Hq, "flops": 4 * D * Hq * pairs}
    return {"bytes": N * D * e * (4 * Hq + 4 * Hkv) + 4 * N * Hq, "flops": 10 * D * Hq * pairs}


# ---- the definitions in 64 bits ----

def _exact_ln(case, st):
    layer, res = case["kind"] == "layer", {"y": [], "mean": [], "rstd": [], "dx": [], "n": []}
    d = case["d"]
    dw = torch.zeros(d, dtype=torch.float64, device=st["x"].device)
    db = torch.zeros_like(dw)
    for i in range(case["B"]):
        x = st["x"][i].double()
        mu = x.sum(dim=1, keepdim=True) / d if layer else torch.zeros(x.shape[0], 1, dtype=torch.float64, device=x.device)
        r = torch.rsqrt(((x - mu) ** 2).sum(dim=1, keepdim=True) / d + _EPS)
        h = (x - mu) * r
        if case["op"] == "ln":
            y = h * st["w"].double()
            res["y"].append(y + st["b"].double() if layer else y)
            res["mean"].append(mu[:, 0])
            res["rstd"].append(r[:, 0])
            continue
        G = st["G"][i].double()
        sw, sb = torch.einsum("tj,tj->j", G, h), G.sum(dim=0)
        if case["op"] == "ln_norm":
            res["n"].append(sw.dot(sw) + (sb.dot(sb) if layer else 0.0))
            continue
        dw += sw * st["c"][i].double()
        db += sb * st["c"][i].double()
        g = G * st["w"].double()
        along = (g * h).sum(dim=1, keepdim=True) / d
        res["dx"].append(r * (g - along * h - (g.sum(dim=1, keepdim=True) / d if layer else 0.0)))
    if case["op"] == "ln_norm":
        return torch.stack(res["n"])
    if case["op"] == "ln":
        out = [torch.stack(res["y"]), torch.stack(res["rstd"])]
        return (out[0], torch.stack(res["mean"]), out[1]) if layer else tuple(out)
    dx = torch.stack(res["dx"])
    return (dx, dw, db) if layer else (dx, dw)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("ln"):
        return _exact_ln(case, st)
    op, Hq, Hkv, D, cap = case["op"], case["Hq"], case["Hkv"], case["D"], case["cap"]
    a = 1.0 / math.sqrt(D)
    N = st["q"].shape[0]
    f64 = dict(dtype=torch.float64, device=st["q"].device)
    o, lse = torch.zeros(N, Hq, D, **f64), torch.zeros(Hq, N, **f64)
    dq, dk, dv = torch.zeros(N, Hq, D, **f64), torch.zeros(N, Hkv, D, **f64), torch.zeros(N, Hkv, D, **f64)
    start = 0
    for n, pre in zip(st["L"], st["P"]):
        rows = slice(start, start + n)
        start += n
        for h in range(Hq):
            kv = h * Hkv // Hq
            Q, K, V = st["q"][rows, h].double(), st["k"][rows, kv].double(), st["v"][rows, kv].double()
            step = max(1, (1 << 27) // n)
            for r in range(0, n, step):
                e = min(n, r + step)
                m = max(e, pre)   # keys that some row of the step sees
                at = slice(rows.start + r, rows.start + e)
                t, u = torch.arange(r, e, device=K.device)[:, None], torch.arange(m, device=K.device)[None]
                S = (Q[r:e] @ K[:m].t()) * a
                slope = torch.ones_like(S)
                if cap:
                    slope = 1.0 / torch.cosh(S / cap) ** 2
                    S = cap * torch.tanh(S / cap)
                if st["slopes"] is not None:
                    S = S - st["slopes"][h].double() * (t - u).abs()
                S = torch.where((u > t) & (u >= pre), torch.full_like(S, float("-inf")), S)
                z = torch.logsumexp(S, dim=1)
                P = torch.exp(S - z[:, None])
                if op == "attention":
                    lse[h, at] = z
                    o[at, h] = P @ V[:m]
                else:
                    keys = slice(rows.start, rows.start + m)
                    dO = st["do"][at, h].double()
                    dv[keys, kv] += P.t() @ dO
                    dS = P * (dO @ V[:m].t() - (dO * st["o"][at, h].double()).sum(dim=1)[:, None]) * slope
                    dq[at, h] = dS @ K[:m] * a
                    dk[keys, kv] += dS.t() @ Q[r:e] * a
    return (o, lse) if op == "attention" else (dq, dk, dv)
