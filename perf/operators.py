"""Cases of the embedding and attention operators: inputs, plain forms, calls.

The operators are those of a DP-SGD-RC training step around its linear layers:
  lookup    out[i, t] = s W[tok[i, t]]
  norm      n_i = s^2 sum_v || sum_{t: tok[i, t] = v} G[i, t] ||^2
  grad      dW[v] = s sum_i c_i sum_{t: tok[i, t] = v} G[i, t]
  attention causal softmax attention of packed sequences with grouped heads:
            o_t = sum_{u <= t} softmax_u(a q_t . k_u) v_u, and the log-sum-exp
  attention_grad its gradients dq, dk, dv from do, o and the log-sum-exp
An id outside [0, V) (a padded position) has no row: it looks up zeros and adds
nothing to a norm or a gradient.
"""
import math

import torch

own = False

_DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # the first tokens of a prompt on a mid-sized table: latency
        {"name": "lookup_short", "op": "lookup", "dtype": "fp32", "B": 1, "T": 37, "V": 50257, "d": 1000, "pad": 0.0},
        # the input of the measured training stack (B = 4, T = 4096, width 2048) from a large vocabulary
        {"name": "lookup_batch", "op": "lookup", "dtype": "bf16", "B": 4, "T": 4096, "V": 131072, "d": 2048, "pad": 0.0},
        # a small padded batch of a small model, all of one training step's samples short
        {"name": "norm_short", "op": "norm", "dtype": "fp32", "B": 3, "T": 61, "V": 2048, "d": 256, "pad": 0.3},
        # per-sample norms of the table of the measured training stack
        {"name": "norm_batch", "op": "norm", "dtype": "bf16", "B": 4, "T": 4096, "V": 131072, "d": 2048, "pad": 0.0},
        # many padded samples of ordinary length
        {"name": "norm_padded", "op": "norm", "dtype": "bf16", "B": 33, "T": 1000, "V": 50257, "d": 1024, "pad": 0.4},
        # clipped gradient of a small table in float32
        {"name": "grad_short", "op": "grad", "dtype": "fp32", "B": 3, "T": 61, "V": 2048, "d": 256, "pad": 0.3},
        # clipped gradient of the measured stack's table, written whole
        {"name": "grad_batch", "op": "grad", "dtype": "bf16", "B": 4, "T": 4096, "V": 131072, "d": 2048, "pad": 0.0},
        # short samples packed one after another, the heads of the small test model
        {"name": "attention_short", "op": "attention", "dtype": "bf16", "lengths": "1,37,64,5", "Hq": 4, "Hkv": 2, "D": 64},
        # the attention of the measured DP-SGD-RC step: B = 4, T = 2048, 32 heads over 8
        {"name": "attention_batch", "op": "attention", "dtype": "bf16", "lengths": "2048,2048,2048,2048", "Hq": 32, "Hkv": 8, "D": 64},
        # long documents packed with short ones, wide heads
        {"name": "attention_long", "op": "attention", "dtype": "bf16", "lengths": "12289,1,777,4100", "Hq": 16, "Hkv": 2, "D": 128},
        # its gradients for the measured step
        {"name": "attention_grad_batch", "op": "attention_grad", "dtype": "bf16", "lengths": "2048,2048,2048,2048", "Hq": 32, "Hkv": 8, "D": 64},
        # gradients in float32, ragged lengths, a head width that is no power of two
        {"name": "attention_grad_float", "op": "attention_grad", "dtype": "fp32", "lengths": "515,130,1,61", "Hq": 6, "Hkv": 3, "D": 80},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lookup", "norm", "grad", "attention", "attention", "attention_grad", "attention_grad"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("lookup", "norm", "grad"):
        d = (8 if dtype == "bf16" else 4) * _log(rng, 8, 256)
        B = _log(rng, 1, 40)
        T = _log(rng, 1, max(1, (16384 * 2048) // (B * d * (2 if dtype == "fp32" else 1))))
        return {"op": op, "dtype": dtype, "B": B, "T": min(T, 40000), "V": _log(rng, 100, 131072 * 1024 // max(d, 1024)), "d": d,
                "pad": rng.choice([0.0, 0.0, 0.35])}
    D = rng.choice([32, 64, 64, 72, 80, 96, 128, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    # pairs (row, key) times heads times width, at most a twentieth of the largest listed case in float32 or for gradients
    most = 12289 * 12289 // 2 * 16 * 128 // (20 if dtype == "fp32" or op == "attention_grad" else 2)
    lengths = []
    for j in range(rng.randint(1, 6)):
        room = most - sum(n * n // 2 * Hq * D for n in lengths)
        top = int(math.sqrt(max(2.0 * room / (Hq * D), 1.0)))
        # (the gradients of q and k of a row alone are zero up to rounding: one sequence at least is longer)
        lengths.append(_log(rng, 16 if j == 0 else 1, max(16 if j == 0 else 1, min(top, 9000))))
    rng.shuffle(lengths)
    return {"op": op, "dtype": dtype, "lengths": ",".join(str(n) for n in lengths), "Hq": Hq, "Hkv": Hkv, "D": D}


def _lengths(case):
    return [int(n) for n in case["lengths"].split(",")]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _DTYPE[case["dtype"]]
    st = dict(case)
    if case["op"] in ("lookup", "norm", "grad"):
        B, T, V, d = case["B"], case["T"], case["V"], case["d"]
        # ids with P(id) ~ 1 / (id + 1), as the words of a text
        u = torch.rand(B, T, generator=g, device=dev, dtype=torch.float64)
        tok = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)
        if case["pad"] > 0:  # samples shorter than T end in padded positions
            keep = (T * (1.0 - case["pad"] * torch.rand(B, 1, generator=g, device=dev))).ceil()
            tok = torch.where(torch.arange(T, device=dev)[None] < keep, tok, torch.full_like(tok, -1))
        st.update(tok=tok, scale=math.sqrt(d))
        if case["op"] == "lookup":
            st["W"] = (torch.randn(V, d, generator=g, device=dev) * 0.02).to(dt)
        else:
            st["G"] = (torch.randn(B, T, d, generator=g, device=dev) * 0.01).to(dt)
            st["c"] = torch.rand(B, generator=g, device=dev) * 0.9 + 0.1
        return st
    L, Hq, Hkv, D = _lengths(case), case["Hq"], case["Hkv"], case["D"]
    N = sum(L)
    st["L"] = L
    st["cu"] = torch.tensor([sum(L[:j]) for j in range(len(L) + 1)], dtype=torch.int32, device=dev)
    st["q"] = torch.randn(N, Hq, D, generator=g, device=dev).to(dt)
    st["k"] = torch.randn(N, Hkv, D, generator=g, device=dev).to(dt)
    st["v"] = torch.randn(N, Hkv, D, generator=g, device=dev).to(dt)
    if case["op"] == "attention_grad":
        st["do"] = torch.randn(N, Hq, D, generator=g, device=dev).to(dt)
        st["o"], st["lse"] = _attention(st)
    return st


# ---- plain forms (float32, rounded once) ----

def _runs(keys):
    """A stable order of `keys` and, per sorted position, the index of its run of equal keys."""
    s, order = torch.sort(keys, stable=True)
    run = torch.zeros_like(s)
    run[1:] = (s[1:] != s[:-1]).long().cumsum(0)
    return order, run, s


def _lookup(st):
    tok, W = st["tok"], st["W"]
    valid = (tok >= 0) & (tok < st["V"])
    rows = W[tok.clamp(0, st["V"] - 1)].float() * st["scale"]
    return torch.where(valid[..., None], rows, torch.zeros_like(rows)).to(W.dtype)


def _norm(st):
    tok, B, T, V, d = st["tok"], st["B"], st["T"], st["V"], st["d"]
    valid = ((tok >= 0) & (tok < V)).reshape(-1)
    key = (torch.arange(B, device=tok.device)[:, None] * (V + 1) + torch.where((tok >= 0) & (tok < V), tok, torch.full_like(tok, V))).reshape(-1)
    order, run, s = _runs(key)
    rows = st["G"].reshape(B * T, d)[order].float() * valid[order][:, None]
    sums = torch.zeros(B * T, d, device=tok.device).index_add_(0, run, rows)
    sq = (sums * sums).sum(dim=1).double()[run]              # the run's squared norm at each of its positions
    first = torch.ones_like(s, dtype=torch.bool)
    first[1:] = s[1:] != s[:-1]
    n = torch.zeros(B, dtype=torch.float64, device=tok.device).index_add_(0, s // (V + 1), sq * first)
    return (n * st["scale"] ** 2).float()


def _grad(st):
    tok, G, V, d = st["tok"].reshape(-1), st["G"], st["V"], st["d"]
    valid = (tok >= 0) & (tok < V)
    rows = (G.float() * (st["c"] * st["scale"])[:, None, None]).reshape(-1, d)
    dW = torch.zeros(V + 1, d, device=G.device).index_add_(0, torch.where(valid, tok, torch.full_like(tok, V)), rows)
    return dW[:V].to(G.dtype)


def _scores(q, k, scale):
    """Masked scaled scores [H, n, n] of one sequence's heads (q, k [n, H, D] float32)."""
    s = torch.matmul(q.transpose(0, 1), k.permute(1, 2, 0).contiguous()) * scale
    n = q.shape[0]
    return s.masked_fill_(torch.ones(n, n, dtype=torch.bool, device=q.device).triu(1), float("-inf"))


def _attention(st):
    rep, scale = st["Hq"] // st["Hkv"], 1.0 / math.sqrt(st["D"])
    outs, lses = [], []
    for q, k, v in zip(*(st[x].split(st["L"]) for x in ("q", "k", "v"))):
        s = _scores(q.float(), k.float().repeat_interleave(rep, dim=1), scale)
        m = s.amax(dim=-1, keepdim=True)
        p = torch.exp(s - m)
        del s
        l = p.sum(dim=-1, keepdim=True)
        o = torch.matmul(p, v.float().repeat_interleave(rep, dim=1).transpose(0, 1).contiguous()) / l
        outs.append(o.transpose(0, 1))
        lses.append((m + torch.log(l))[..., 0])
    return torch.cat(outs).to(st["q"].dtype), torch.cat(lses, dim=1).contiguous()


def _attention_grad(st):
    rep, scale, D = st["Hq"] // st["Hkv"], 1.0 / math.sqrt(st["D"]), st["D"]
    dqs, dks, dvs = [], [], []
    for q, k, v, o, do, lse in zip(*(st[x].split(st["L"]) for x in ("q", "k", "v", "o", "do")), st["lse"].split(st["L"], dim=1)):
        n = q.shape[0]
        q, do = q.float().transpose(0, 1), do.float().transpose(0, 1).contiguous()
        k, v = k.float().repeat_interleave(rep, dim=1), v.float().repeat_interleave(rep, dim=1)
        p = torch.exp(_scores(q.transpose(0, 1), k, scale) - lse[..., None])
        dv = torch.matmul(p.transpose(1, 2).contiguous(), do)
        delta = (do * o.float().transpose(0, 1)).sum(dim=-1, keepdim=True)
        ds = torch.matmul(do, v.permute(1, 2, 0).contiguous()).sub_(delta).mul_(p)
        del p
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
        if op == "lookup":
            return dp.embed_lookup(st["tok"], st["W"], scale=st["scale"])
        if op == "norm":
            return dp.embed_norm(st["tok"], st["G"], st["V"], scale=st["scale"])
        if op == "grad":
            return dp.embed_grad(st["tok"], st["G"], st["V"], scale=st["scale"], weights=st["c"])
        if op == "attention":
            return dp.attention_forward(st["q"], st["k"], st["v"], cu_seqlens=st["cu"])
        return dp.attention_backward(st["do"], st["q"], st["k"], st["v"], st["o"], st["lse"], cu_seqlens=st["cu"])
    return {"lookup": _lookup, "norm": _norm, "grad": _grad, "attention": _attention, "attention_grad": _attention_grad}[op](st)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("lookup", "norm", "grad"):
        B, T, V, d = case["B"], case["T"], case["V"], case["d"]
        N = B * T
        if case["op"] == "lookup":
            # distinct ids expected under the law that they are drawn from
            z = math.log(V + 1.0)
            distinct = sum(1.0 - math.exp(-N * math.log1p(1.0 / r) / z) for r in range(1, V + 1)) if V <= 4096 else \
                _distinct(N, V, z)
            return {"bytes": 8 * N + (distinct + N) * d * e, "flops": N * d}
        if case["op"] == "norm":
            return {"bytes": 8 * N + N * d * e + 4 * B, "flops": 3 * N * d}
        return {"bytes": 8 * N + N * d * e + V * d * e + 4 * B, "flops": 2 * N * d}
    L, Hq, Hkv, D = _lengths(case), case["Hq"], case["Hkv"], case["D"]
    N, pairs = sum(L), sum(n * (n + 1) // 2 for n in L)
    if case["op"] == "attention":
        return {"bytes": N * D * e * (2 * Hq + 2 * Hkv) + 4 * N * Hq, "flops": 4 * D * Hq * pairs}
    return {"bytes": N * D * e * (4 * Hq + 4 * Hkv) + 4 * N * Hq, "flops": 10 * D * Hq * pairs}


def _distinct(N, V, z):
    """The same sum over V, taken at points spread over the logarithm of the rank."""
    total, lo = 0.0, 1
    while lo <= V:
        hi = max(lo + 1, int(lo * 1.02))
        mid = (lo + min(hi, V + 1) - 1) / 2.0
        total += (min(hi, V + 1) - lo) * (1.0 - math.exp(-N * math.log1p(1.0 / mid) / z))
        lo = hi
    return total


# ---- the definitions in 64 bits ----

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "lookup":
        tok, W = st["tok"], st["W"]
        table = torch.cat([W.double() * st["scale"], torch.zeros(1, W.shape[1], dtype=torch.float64, device=W.device)])
        ids = torch.where((tok < 0) | (tok >= st["V"]), torch.full_like(tok, st["V"]), tok)
        return table[ids]
    if op == "norm":
        res = []
        for ids, G in zip(st["tok"], st["G"]):
            ok = (ids >= 0) & (ids < st["V"])
            _, inv = torch.unique(ids[ok], return_inverse=True)
            per_id = torch.zeros(case["T"], case["d"], dtype=torch.float64, device=ids.device)
            per_id.index_add_(0, inv, G[ok].double())
            res.append((per_id ** 2).sum() * st["scale"] ** 2)
        return torch.stack(res)
    if op == "grad":
        dW = torch.zeros(case["V"], case["d"], dtype=torch.float64, device=st["G"].device)
        for ids, G, c in zip(st["tok"], st["G"], st["c"].double()):
            ok = (ids >= 0) & (ids < st["V"])
            dW.index_add_(0, ids[ok], G[ok].double() * (c * st["scale"]))
        return dW
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    a = 1.0 / math.sqrt(D)
    N = st["q"].shape[0]
    f64 = dict(dtype=torch.float64, device=st["q"].device)
    o, lse = torch.zeros(N, Hq, D, **f64), torch.zeros(Hq, N, **f64)
    dq, dk, dv = torch.zeros(N, Hq, D, **f64), torch.zeros(N, Hkv, D, **f64), torch.zeros(N, Hkv, D, **f64)
    start = 0
    for n in st["L"]:
        rows = slice(start, start + n)
        start += n
        for h in range(Hq):
            kv = h * Hkv // Hq
            Q, K, V = st["q"][rows, h].double(), st["k"][rows, kv].double(), st["v"][rows, kv].double()
            step = max(1, (1 << 27) // n)
            for r in range(0, n, step):
                e = min(n, r + step)
                at = slice(rows.start + r, rows.start + e)
                S = (Q[r:e] @ K[:e].t()) * a
                S = torch.where(torch.arange(e, device=S.device)[None] > torch.arange(r, e, device=S.device)[:, None],
                                torch.full_like(S, float("-inf")), S)
                if op == "attention":
                    z = torch.logsumexp(S, dim=1)
                    lse[h, at] = z
                    o[at, h] = torch.exp(S - z[:, None]) @ V[:e]
                else:
                    keys = slice(rows.start, rows.start + e)
                    P = torch.exp(S - torch.logsumexp(S, dim=1)[:, None])
                    dO = st["do"][at, h].double()
                    dv[keys, kv] += P.t() @ dO
                    dS = P * (dO @ V[:e].t() - (dO * st["o"][at, h].double()).sum(dim=1)[:, None])
                    dq[at, h] = dS @ K[:e] * a
                    dk[keys, kv] += dS.t() @ Q[r:e] * a
    return (o, lse) if op == "attention" else (dq, dk, dv)
