"""The C ABI of the embedding and attention calls without a GPU: sizes of
orders and workspaces, and every host-side check returning its documented
status before anything is enqueued (every call here fails a check). The file
also runs against the host layer built with sanitizers."""
import ctypes as C
import os
import subprocess
import sys

import pytest

from sample_grad_norms_amd import _lib

HERE = os.path.dirname(os.path.abspath(__file__))
TOK, W, OUT, ORDER, G, N, CW, WS = (0x10000000 * j for j in range(1, 9))   # aligned addresses, never read
BIG = 1 << 40


def order_sizes(lib, B=3, T=100, V=50):
    ob, wb = C.c_size_t(0), C.c_size_t(0)
    return lib.dpnorm_embed_order_sizes(B, T, V, C.byref(ob), C.byref(wb)), ob.value, wb.value


def test_order_sizes(lib):
    st, ob, wb = order_sizes(lib)
    assert st == _lib.OK and ob >= 3 * 100 * 8 and ob % 256 == 0 and wb == 0
    st, ob, wb = order_sizes(lib, 4, 16385, 131072)   # not in one launch: scratch of its own
    assert st == _lib.OK and ob >= 4 * 16385 * 8 and wb >= 4 * 16385 * 8
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 2 ** 30 + 1), (2 ** 16, 2 ** 15, 1), (2 ** 62, 2 ** 62, 1), (-1, 5, 5)):
        assert order_sizes(lib, *bad)[0] == _lib.ERR_SIZE
    assert lib.dpnorm_embed_order_sizes(1, 1, 1, None, None) == _lib.ERR_NULL


def test_lookup_checks(lib):
    def call(tok=TOK, it=_lib.I64, w=W, dt=_lib.BF16, n=300, v=50, d=64, scale=1.0, out=OUT):
        return lib.dpnorm_embed_lookup(tok, it, w, dt, n, v, d, scale, out, None)
    assert call(tok=None) == call(w=None) == call(out=None) == _lib.ERR_NULL
    assert call(dt=2) == call(it=2) == call(it=-1) == _lib.ERR_DTYPE
    assert call(n=0) == call(v=0) == call(d=0) == call(d=12) == call(d=2 ** 25) == call(n=2 ** 30 + 1) == _lib.ERR_SIZE
    assert call(dt=_lib.F32, d=6) == _lib.ERR_SIZE
    assert call(tok=TOK + 4) == call(w=W + 8) == call(out=OUT + 2) == _lib.ERR_ALIGN
    assert call(scale=float("nan")) == call(scale=float("-inf")) == _lib.ERR_VALUE
    assert call(out=W) == call(out=TOK) == call(out=W + 50 * 64 * 2 - 16) == _lib.ERR_VALUE


def test_order_checks(lib):
    _, ob, _ = order_sizes(lib)
    _, ob2, wb2 = order_sizes(lib, 4, 16385, 1000)

    def call(tok=TOK, it=_lib.I32, B=3, T=100, V=50, order=ORDER, size=ob, ws=None, ws_size=0):
        return lib.dpnorm_embed_order(tok, it, B, T, V, order, size, ws, ws_size, None)
    assert call(tok=None) == call(order=None) == _lib.ERR_NULL
    assert call(it=5) == _lib.ERR_DTYPE
    assert call(B=0) == call(V=-1) == _lib.ERR_SIZE
    assert call(tok=TOK + 2) == call(order=ORDER + 16) == _lib.ERR_ALIGN
    assert call(it=_lib.I64, tok=TOK + 4) == _lib.ERR_ALIGN
    assert call(size=ob - 1) == _lib.ERR_WORKSPACE
    assert call(order=TOK) == _lib.ERR_VALUE
    big = dict(B=4, T=16385, V=1000, size=ob2, ws=WS, ws_size=wb2)
    assert call(**{**big, "ws": None}) == _lib.ERR_NULL
    assert call(**{**big, "ws_size": wb2 - 1}) == _lib.ERR_WORKSPACE
    assert call(**{**big, "ws": WS + 64}) == _lib.ERR_ALIGN
    assert call(**{**big, "ws": ORDER}) == call(**{**big, "ws": TOK}) == _lib.ERR_VALUE


@pytest.mark.parametrize("which", ["norm", "grad"])
def test_norm_and_grad_checks(lib, which):
    query = getattr(lib, f"dpnorm_embed_{which}_workspace")
    sizes = []
    for ordered in (0, 1):
        nb = C.c_size_t(0)
        assert query(_lib.BF16, 3, 100, 50, 64, ordered, C.byref(nb)) == _lib.OK and nb.value % 256 == 0
        sizes.append(nb.value)
    # 100 ids a sample and 300 in all: the norm needs no order and no workspace, the gradient both
    assert sizes[0] == 0 < sizes[1] if which == "norm" else sizes[0] >= sizes[1] + order_sizes(lib)[1] > 0
    assert query(_lib.BF16, 3, 100, 50, 64, 0, None) == _lib.ERR_NULL
    assert query(_lib.BF16, 3, 100, 50, 64, 2, C.byref(nb)) == _lib.ERR_VALUE
    assert query(7, 3, 100, 50, 64, 0, C.byref(nb)) == _lib.ERR_DTYPE
    for bad in ((0, 100, 50, 64), (3, 100, 0, 64), (3, 100, 50, 60), (2 ** 20, 2 ** 11, 5, 8), (1, 2 ** 30, 1, 2 ** 24)):
        assert query(_lib.BF16, *bad, 0, C.byref(nb)) == _lib.ERR_SIZE

    def call(tok=None, it=_lib.I64, order=ORDER, g=G, dt=_lib.BF16, B=3, T=100, V=50, d=64, scale=1.0, out=OUT, c=CW, acc=0,
             ws=WS, ws_size=BIG):
        if which == "norm":
            return lib.dpnorm_embed_norm(tok, it, order, g, dt, B, T, V, d, scale, out, acc, ws, ws_size, None)
        return lib.dpnorm_embed_grad(tok, it, order, g, dt, B, T, V, d, scale, c, out, acc, ws, ws_size, None)
    assert call(order=None) == call(g=None) == call(out=None) == call(ws=None) == _lib.ERR_NULL
    assert call(dt=-3) == call(order=None, tok=TOK, it=3) == _lib.ERR_DTYPE
    assert call(T=0) == call(d=4) == _lib.ERR_SIZE
    assert call(order=ORDER + 4) == call(g=G + 8) == call(out=OUT + 2) == call(ws=WS + 16) == _lib.ERR_ALIGN
    assert call(order=None, tok=TOK + 4) == _lib.ERR_ALIGN
    assert call(scale=float("inf")) == call(acc=2) == call(acc=-1) == _lib.ERR_VALUE
    assert call(ws_size=sizes[1] - 1) == call(order=None, tok=TOK, T=300, ws_size=255) == _lib.ERR_WORKSPACE
    assert call(out=G) == call(out=ORDER) == call(out=WS) == call(ws=G) == call(ws=ORDER) == _lib.ERR_VALUE
    assert call(order=None, tok=TOK, out=TOK) == call(order=None, tok=TOK, T=300, ws=TOK) == _lib.ERR_VALUE
    if which == "grad":
        assert call(c=CW + 2) == _lib.ERR_ALIGN
        assert call(c=OUT) == call(c=WS) == _lib.ERR_VALUE


Q, K, V_, O, LSE, DO, DQ, DK, DV, CU = (0x100000000 * j for j in range(1, 11))


def shape(dtype=_lib.BF16, n=200, s=2, hq=4, hkv=2, d=64, cu=CU, scale=0.125, clear=0):
    return _lib.AttnShape(dtype, n, s, hq, hkv, d, cu, scale, clear)


def tensor(p, h, d=64, st=None, sh=None):
    return _lib.AttnTensor(p, h * d if st is None else st, d if sh is None else sh)


def forward(lib, sh=None, q=None, k=None, v=None, o=None, lse=LSE):
    args = [q or tensor(Q, 4), k or tensor(K, 2), v or tensor(V_, 2), o or tensor(O, 4)]
    return lib.dpnorm_attention_forward(C.byref(sh or shape()), *(C.byref(t) for t in args), lse, None)


def test_attention_forward_checks(lib):
    assert lib.dpnorm_attention_forward(None, None, None, None, None, None, None) == _lib.ERR_NULL
    assert lib.dpnorm_attention_forward(C.byref(shape()), None, None, None, None, LSE, None) == _lib.ERR_NULL
    assert forward(lib, lse=None) == forward(lib, q=tensor(None, 4)) == forward(lib, o=tensor(None, 4)) == _lib.ERR_NULL
    assert forward(lib, shape(dtype=2)) == _lib.ERR_DTYPE
    for bad in (dict(n=0), dict(s=0), dict(hq=0), dict(hkv=0), dict(hkv=3), dict(d=0), dict(d=136), dict(d=12),
                dict(n=2 ** 31), dict(s=2 ** 31), dict(hq=2 ** 17, hkv=1), dict(n=201, cu=None)):
        assert forward(lib, shape(**bad)) == _lib.ERR_SIZE, bad
    assert forward(lib, shape(cu=CU + 2)) == _lib.ERR_ALIGN
    assert forward(lib, shape(clear=2)) == forward(lib, shape(clear=-1)) == _lib.ERR_VALUE
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert forward(lib, shape(scale=scale)) == _lib.ERR_VALUE
    assert forward(lib, q=tensor(Q + 8, 4)) == forward(lib, lse=LSE + 2) == _lib.ERR_ALIGN
    assert forward(lib, k=tensor(K, 2, st=129)) == forward(lib, k=tensor(K, 2, sh=68)) == _lib.ERR_ALIGN
    assert forward(lib, v=tensor(V_, 2, st=-128)) == forward(lib, v=tensor(V_, 2, st=2 ** 23)) == _lib.ERR_SIZE
    # outputs that repeat rows, or lie on inputs or on each other
    assert forward(lib, o=tensor(O, 4, st=0)) == forward(lib, o=tensor(O, 4, sh=0)) == _lib.ERR_VALUE
    assert forward(lib, o=tensor(O, 4, st=64, sh=64)) == forward(lib, o=tensor(O, 4, st=192)) == _lib.ERR_VALUE
    assert forward(lib, o=tensor(Q, 4)) == forward(lib, o=tensor(V_, 4)) == forward(lib, o=tensor(CU, 4)) == _lib.ERR_VALUE
    assert forward(lib, lse=O) == forward(lib, lse=K) == forward(lib, o=tensor(Q + (200 * 256 - 64) * 2, 4)) == _lib.ERR_VALUE


def test_attention_backward_checks(lib):
    nb = C.c_size_t(0)
    assert lib.dpnorm_attention_backward_workspace(C.byref(shape()), C.byref(nb)) == _lib.OK
    assert nb.value >= 200 * 4 * 4 and nb.value % 256 == 0
    assert lib.dpnorm_attention_backward_workspace(C.byref(shape()), None) == _lib.ERR_NULL
    assert lib.dpnorm_attention_backward_workspace(None, C.byref(nb)) == _lib.ERR_NULL
    assert lib.dpnorm_attention_backward_workspace(C.byref(shape(d=7)), C.byref(nb)) == _lib.ERR_SIZE

    base = dict(do=tensor(DO, 4), q=tensor(Q, 4), k=tensor(K, 2), v=tensor(V_, 2), o=tensor(O, 4), dq=tensor(DQ, 4),
                dk=tensor(DK, 2), dv=tensor(DV, 2))

    def call(lse=LSE, ws=WS, size=BIG, sh=None, **kw):
        a = {**base, **kw}
        return lib.dpnorm_attention_backward(C.byref(sh or shape()), C.byref(a["do"]), C.byref(a["q"]), C.byref(a["k"]),
                                             C.byref(a["v"]), C.byref(a["o"]), lse, C.byref(a["dq"]), C.byref(a["dk"]),
                                             C.byref(a["dv"]), ws, size, None)
    assert call(lse=None) == call(ws=None) == call(do=tensor(None, 4)) == call(dv=tensor(None, 2)) == _lib.ERR_NULL
    assert call(ws=WS + 8) == call(lse=LSE + 1) == call(dk=tensor(DK + 8, 2)) == call(do=tensor(DO, 4, st=257)) == _lib.ERR_ALIGN
    assert call(size=nb.value - 1) == _lib.ERR_WORKSPACE
    assert call(o=tensor(O, 4, st=-8)) == call(sh=shape(d=200)) == _lib.ERR_SIZE
    assert call(dq=tensor(DQ, 4, st=0)) == call(dk=tensor(DK, 2, sh=0)) == _lib.ERR_VALUE
    for name in ("q", "k", "v", "o", "do"):
        assert call(dq=tensor(base[name].data, 4)) == _lib.ERR_VALUE
        assert call(ws=base[name].data) == _lib.ERR_VALUE
    assert call(dv=tensor(DK, 2)) == call(dk=tensor(LSE, 2)) == call(ws=DQ) == _lib.ERR_VALUE


@pytest.mark.skipif("DPNORM_TEST_LIB" in os.environ, reason="already the sanitized library")
def test_under_sanitizers(tmp_path):
    """This file and valid calls of every entry point against the host layer
    built with AddressSanitizer and UndefinedBehaviorSanitizer."""
    sys.path.insert(0, os.path.join(HERE, "hostcheck"))
    import build as hostcheck_build
    built = hostcheck_build.build(str(tmp_path))
    env = dict(os.environ, LD_PRELOAD=built["asan_runtime"], ASAN_OPTIONS="detect_leaks=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1", DPNORM_TEST_LIB=built["lib"])
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", os.path.abspath(__file__)],
                         capture_output=True, text=True, timeout=600, env=env, cwd=os.path.dirname(HERE))
    assert res.returncode == 0, res.stdout[-4000:] + res.stderr[-4000:]


@pytest.mark.skipif("DPNORM_TEST_LIB" not in os.environ, reason="launches are only counted by the sanitized library's stand-in")
@pytest.mark.parametrize("seed", range(40))
def test_valid_calls_launch_valid_grids(lib, seed):
    """Random valid sizes up to the limits: the call succeeds with the queried
    workspace (a launch that the stand-in refuses fails the call)."""
    import random
    rng = random.Random(seed)

    def log(lo, hi):
        return int(lo * (hi / lo) ** rng.random())
    dt = rng.choice([_lib.BF16, _lib.F32])
    B, V, d = log(1, 300), log(1, 2 ** 30), 8 * log(1, 1000)
    T = log(1, 2 ** 24 // B)
    st, ob, wb = order_sizes(lib, B, T, V)
    assert st == _lib.OK
    far = 1 << 44
    p = [far * (j + 1) for j in range(12)]
    assert lib.dpnorm_embed_order(p[0], _lib.I64, B, T, V, p[1], ob, p[2], wb, None) == _lib.OK
    nb = C.c_size_t(0)
    for ordered in (0, 1):
        ids = (None, 0, p[1]) if ordered else (p[0], _lib.I64, None)
        st = lib.dpnorm_embed_norm_workspace(dt, B, T, V, d, ordered, C.byref(nb))
        assert st in (_lib.OK, _lib.ERR_SIZE)
        assert lib.dpnorm_embed_norm(*ids, p[3], dt, B, T, V, d, 2.0, p[4], 0, p[5], nb.value, None) == st
        assert lib.dpnorm_embed_grad_workspace(dt, B, T, V, d, ordered, C.byref(nb)) == st
        assert lib.dpnorm_embed_grad(*ids, p[3], dt, B, T, V, d, 2.0, p[6], p[7], seed % 2, p[5], nb.value, None) == st
    assert lib.dpnorm_embed_lookup(p[0], _lib.I32, p[7], dt, B * T, V, d, 1.0, p[8], None) == _lib.OK
    hkv = rng.choice([1, 2, 3, 8])
    hq, D, S = hkv * rng.randint(1, 8), 8 * rng.randint(1, 16), log(1, 5000)
    n = log(1, 2 ** 22)
    sh = shape(dt, n, S, hq, hkv, D, p[9], clear=seed % 2)
    ten = [tensor(x, h, D) for x, h in ((p[0], hq), (p[1], hkv), (p[2], hkv), (p[3], hq), (p[4], hq), (p[5], hq), (p[6], hkv),
                                        (p[7], hkv))]
    q, k, v, o, do, dq, dk, dv = (C.byref(t) for t in ten)
    assert lib.dpnorm_attention_forward(C.byref(sh), q, k, v, o, p[8], None) == _lib.OK
    assert lib.dpnorm_attention_backward_workspace(C.byref(sh), C.byref(nb)) == _lib.OK
    assert lib.dpnorm_attention_backward(C.byref(sh), do, q, k, v, o, p[8], dq, dk, dv, p[10], nb.value, None) == _lib.OK


FAR = [(1 << 56) + (j << 50) for j in range(8)]


@pytest.mark.skipif("DPNORM_TEST_LIB" not in os.environ, reason="launches are only checked by the sanitized library's stand-in")
@pytest.mark.parametrize("dt", [_lib.BF16, _lib.F32])
@pytest.mark.parametrize("B,T,V,d", [
    (2 ** 22 - 1, 1, 50, 8), (2 ** 22, 1, 50, 8), (2 ** 24, 1, 50, 8), (2 ** 30, 1, 50, 8), (2 ** 22, 256, 50, 8),   # a block a sample
    (1, 1, 2 ** 28 - 16, 8), (1, 256, 2 ** 28, 8), (256, 1, 2 ** 30, 8),             # few positions, many rows
    (1, 257, 2 ** 30, 8), (1, 2 ** 24, 2 ** 30, 8), (2 ** 15, 2 ** 15, 2 ** 30, 8),  # many rows to clear
    (1, 2 ** 28 - 16, 50, 8), (1, 2 ** 28, 50, 8), (1, 2 ** 30, 50, 8), (2 ** 20, 2 ** 10, 7, 8),
    (1, 2 ** 24, 50, 4096), (3, 2 ** 20, 50, 2 ** 17), (1, 300, 2 ** 20, 2 ** 24), (1, 2 ** 20, 50, 2 ** 24), (5, 2 ** 26, 11, 2 ** 13)])
def test_largest_calls_launch_valid_grids(lib, B, T, V, d, dt):
    """Sizes around and far past 2^32 threads: every call either fails its query, and
    then launches nothing, or succeeds, with fewer than 2^32 threads along each dimension."""
    tok, order, g, out, ws, w, n, c = FAR
    launches = C.c_longlong.in_dll(lib, "dpnorm_fake_launches")
    wide = C.c_longlong.in_dll(lib, "dpnorm_fake_wide_launches")
    before = wide.value
    nb = C.c_size_t(0)
    for ordered in (0, 1):
        ids = (None, 0, order) if ordered else (tok, _lib.I32, None)
        for which in ("norm", "grad"):
            st = getattr(lib, f"dpnorm_embed_{which}_workspace")(dt, B, T, V, d, ordered, C.byref(nb))
            assert st in (_lib.OK, _lib.ERR_SIZE)
            at = launches.value
            if which == "norm":
                got = lib.dpnorm_embed_norm(*ids, g, dt, B, T, V, d, 1.0, n, 0, ws, nb.value, None)
                assert got == st
            else:
                for acc in (0, 1):
                    got = lib.dpnorm_embed_grad(*ids, g, dt, B, T, V, d, 1.0, c, out, acc, ws, nb.value, None)
                    assert got == st
            assert (launches.value > at) == (st == _lib.OK)
    at = launches.value
    got = lib.dpnorm_embed_lookup(tok, _lib.I64, w, dt, B * T, V, d, 1.0, out, None)
    assert got in (_lib.OK, _lib.ERR_SIZE) and (launches.value > at) == (got == _lib.OK)
    assert got == _lib.OK or B * T * d > 2 ** 38
    assert wide.value == before


@pytest.mark.skipif("DPNORM_TEST_LIB" not in os.environ, reason="valid calls launch: only on the sanitized library's stand-in")
def test_strides_of_a_lone_row_are_not_read(lib):
    one = shape(n=1, s=1, hq=1, hkv=1, cu=None)
    for st, sh in ((3, 5), (-7, -64), (1 << 60, 1 << 61), (0, 0)):
        ts = [C.byref(tensor(p, 1, st=st, sh=sh)) for p in (Q, K, V_, O)]
        assert lib.dpnorm_attention_forward(C.byref(one), *ts, LSE, None) == _lib.OK
        nb = C.c_size_t(0)
        assert lib.dpnorm_attention_backward_workspace(C.byref(one), C.byref(nb)) == _lib.OK
        ts = [C.byref(tensor(p, 1, st=st, sh=sh)) for p in (DO, Q, K, V_, O)]
        outs = [C.byref(tensor(p, 1, st=st, sh=sh)) for p in (DQ, DK, DV)]
        assert lib.dpnorm_attention_backward(C.byref(one), *ts, LSE, *outs, WS, nb.value, None) == _lib.OK
    # the last token stride that 31 bits of a step's rows reach
    assert forward(lib, k=tensor(K, 2, st=(1 << 22) - 8)) == _lib.OK and forward(lib, k=tensor(K, 2, st=1 << 22)) == _lib.ERR_SIZE
