"""The C ABI of attention with changed scores without a GPU: its host-side checks (every
call here fails one, but for those on the stand-in), and which kernels a change takes.
The file also runs against the host layer built with sanitizers."""
import ctypes as C
import os
import re
import subprocess
import sys

import pytest

import attention_forms
from sample_grad_norms_amd import _lib

HERE = os.path.dirname(os.path.abspath(__file__))
Q, K, V_, O, LSE, DO, DQ, DK, DV, CU, SL, PRE, WS = (0x100000000 * j for j in range(1, 14))
NAN, INF = float("nan"), float("inf")


def shape(dtype=_lib.BF16, n=200, s=2, hq=4, hkv=2, d=64, cu=CU, scale=0.125, clear=0):
    return _lib.AttnShape(dtype, n, s, hq, hkv, d, cu, scale, clear)


def tensor(p, h, d=64):
    return C.byref(_lib.AttnTensor(p, h * d, d))


def scores(cap=5.0, slopes=SL, prefix=PRE):
    return _lib.AttnScores(cap, slopes, prefix)


def forward(lib, sc, sh=None, o=O, lse=LSE, q=Q):
    return lib.dpnorm_attention_scores_forward(C.byref(sh or shape()), C.byref(sc) if sc else None, tensor(q, 4), tensor(K, 2),
                                               tensor(V_, 2), tensor(o, 4), lse, None)


def backward(lib, sc, sh=None, ws=WS, size=1 << 50, dq=DQ):
    return lib.dpnorm_attention_scores_backward(C.byref(sh or shape()), C.byref(sc) if sc else None, tensor(DO, 4), tensor(Q, 4),
                                                tensor(K, 2), tensor(V_, 2), tensor(O, 4), LSE, tensor(dq, 4), tensor(DK, 2),
                                                tensor(DV, 2), ws, size, None)


@pytest.mark.parametrize("call", [forward, backward])
def test_checks(lib, call):
    for cap in (-1.0, -0.0001, NAN, INF, -INF, 1e-4, 1025.0, 1e30):
        assert call(lib, scores(cap=cap)) == _lib.ERR_VALUE, cap
    assert call(lib, scores(slopes=SL + 2)) == call(lib, scores(prefix=PRE + 1)) == _lib.ERR_ALIGN
    assert call(lib, scores(), shape(scale=1e-30)) == call(lib, scores(slopes=None), shape(scale=1e30)) == _lib.ERR_VALUE
    for bad in (dict(n=0), dict(d=136), dict(hkv=3), dict(s=0)):
        assert call(lib, scores(), shape(**bad)) == _lib.ERR_SIZE
    assert call(lib, scores(), shape(dtype=3)) == _lib.ERR_DTYPE
    assert call(lib, scores(), shape(scale=-1.0)) == _lib.ERR_VALUE


def test_workspace(lib):
    nb, plain = C.c_size_t(0), C.c_size_t(0)
    query = lib.dpnorm_attention_scores_backward_workspace
    for sh in (shape(), shape(n=4096, s=2, hq=16, hkv=4), shape(dtype=_lib.F32, d=80)):
        assert lib.dpnorm_attention_backward_workspace(C.byref(sh), C.byref(plain)) == _lib.OK
        for sc in (None, scores(), scores(cap=0.0, slopes=None, prefix=None)):
            assert query(C.byref(sh), C.byref(sc) if sc else None, C.byref(nb)) == _lib.OK and nb.value >= plain.value
            assert nb.value % 256 == 0 and (nb.value == plain.value or sc.prefix)
    assert query(C.byref(shape()), C.byref(scores()), None) == query(None, None, C.byref(nb)) == _lib.ERR_NULL
    assert query(C.byref(shape()), C.byref(scores(cap=-1.0)), C.byref(nb)) == _lib.ERR_VALUE


def test_outputs_on_slopes_or_prefixes(lib):
    assert forward(lib, scores(), o=SL) == forward(lib, scores(), o=PRE) == forward(lib, scores(), lse=SL) == _lib.ERR_VALUE
    assert forward(lib, scores(), lse=PRE + 4) == forward(lib, scores(), lse=Q) == _lib.ERR_VALUE
    assert backward(lib, scores(), dq=SL) == backward(lib, scores(), ws=PRE) == backward(lib, scores(), ws=SL) == _lib.ERR_VALUE
    assert forward(lib, scores(), lse=None) == backward(lib, scores(), ws=None) == _lib.ERR_NULL
    assert backward(lib, scores(), size=100) == _lib.ERR_WORKSPACE
    assert lib.dpnorm_attention_scores_forward(None, None, None, None, None, None, None, None) == _lib.ERR_NULL


@pytest.mark.skipif("DPNORM_TEST_LIB" in os.environ, reason="already the sanitized library")
def test_under_sanitizers(tmp_path):
    sys.path.insert(0, os.path.join(HERE, "hostcheck"))
    import build as hostcheck_build
    built = hostcheck_build.build(str(tmp_path))
    env = dict(os.environ, LD_PRELOAD=built["asan_runtime"], ASAN_OPTIONS="detect_leaks=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1", DPNORM_TEST_LIB=built["lib"])
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", os.path.abspath(__file__)],
                         capture_output=True, text=True, timeout=600, env=env, cwd=os.path.dirname(HERE))
    assert res.returncode == 0, res.stdout[-4000:] + res.stderr[-4000:]


standin = pytest.mark.skipif("DPNORM_TEST_LIB" not in os.environ, reason="launches are only named by the sanitized library's stand-in")
SETS = [(None, 0), ((0.0, None, None), 0), ((0.0, SL, None), 1), ((0.0, None, PRE), 1), ((0.0, SL, PRE), 1), ((5.0, None, None), 2),
        ((5.0, None, PRE), 2), ((5.0, SL, None), 3), ((1024.0, SL, PRE), 3), ((1.0 / 1024, None, None), 2)]


@standin
@pytest.mark.parametrize("change,kernels", SETS)
def test_the_kernels_of_a_change(lib, change, kernels):
    """The set of kernels goes by the change; the forms are those of plain attention, but that
    with a prefix three work groups share keys with long chains."""
    names = lib.dpnorm_fake_launched
    names.restype = C.c_char_p
    sc = None if change is None else _lib.AttnScores(*change)
    for dt, table in ((_lib.BF16, attention_forms.BF16), (_lib.F32, attention_forms.F32)):
        for n, hq, hkv, d in table:
            sh = C.byref(_lib.AttnShape(dt, n, 1, hq, hkv, d, None, 0.1, 0))
            q, k, v, o, do, dq, dk, dv = (C.byref(_lib.AttnTensor((j + 1) << 44, h * d, d))
                                          for j, h in enumerate((hq, hkv, hkv, hq, hq, hq, hkv, hkv)))
            lse, ws, nb = 10 << 44, 11 << 44, C.c_size_t(0)
            rec = C.byref(sc) if sc else None
            assert lib.dpnorm_attention_scores_backward_workspace(sh, rec, C.byref(nb)) == _lib.OK
            plain_bytes = C.c_size_t(0)
            assert lib.dpnorm_attention_backward_workspace(sh, C.byref(plain_bytes)) == _lib.OK
            groups, steps = (n // 32 + 1) * hkv, n // 32 * (hq // hkv)
            shared = bool(sc and sc.prefix) and groups <= 1100 and steps > 104
            launched = []
            for plain in (True, False):
                names()
                if plain:
                    assert lib.dpnorm_attention_forward(sh, q, k, v, o, lse, None) == _lib.OK
                    assert lib.dpnorm_attention_backward(sh, do, q, k, v, o, lse, dq, dk, dv, ws, nb.value, None) == _lib.OK
                else:
                    assert lib.dpnorm_attention_scores_forward(sh, rec, q, k, v, o, lse, None) == _lib.OK
                    assert lib.dpnorm_attention_scores_backward(sh, rec, do, q, k, v, o, lse, dq, dk, dv, ws, nb.value, None) == _lib.OK
                launched.append([re.match(r"(.*)Li(\d)(EEEvNS0_4ArgsE)$", x).groups() for x in names().decode().split()])
            assert all(m == "0" for _, m, _ in launched[0]) and all(m == str(kernels) for _, m, _ in launched[1])
            forms = [[a for a, _, _ in x] for x in launched]
            if shared and "Lb1E" not in forms[0][2][-5:]:
                assert forms[0][:2] == forms[1][:2] and forms[1][2].endswith("Li4ELb1E") and nb.value > plain_bytes.value
            else:
                assert forms[0] == forms[1] and nb.value == plain_bytes.value


@standin
def test_scales_that_slopes_allow(lib):
    assert forward(lib, scores(cap=0.0, slopes=None), shape(scale=1e-30)) == _lib.OK
    assert forward(lib, scores(), shape(scale=2.0 ** -64)) == _lib.OK
