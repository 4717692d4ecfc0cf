"""How many work groups share the keys' queries of dk and dv, without and with a prefix
(which makes chains longer), from the workspace that a call asks for and the kernels
that it launches, on the CPU: the shapes of attention_shares.py."""
import ctypes as C
import os
import subprocess
import sys

import pytest

from attention_shares import SHARES
from sample_grad_norms_amd import _lib
from test_attention_forms_host import form

HERE = os.path.dirname(os.path.abspath(__file__))
CU, PRE, WS, LSE = (j << 46 for j in range(1, 5))


def up(n):
    return (n + 255) // 256 * 256


def shape(dt, lengths, hq, hkv, d):
    return _lib.AttnShape(dt, sum(lengths), len(lengths), hq, hkv, d, CU, 0.1, 0)


def wanted_bytes(lengths, hq, hkv, d, shares):
    """lse and delta of every query, a counter for each 32 keys, and the work groups' sums."""
    N, S = sum(lengths), len(lengths)
    slots = N // 32 + S + 1
    tile = 32 * 4 * (64 if d <= 64 else 96 if d <= 96 else 128)
    return up(N * hq * 8) + (up(slots * hkv * 4) + up(slots * hkv * shares * 2 * tile) if shares > 1 else 0)


@pytest.mark.parametrize("case,shares", SHARES.items())
def test_workspaces(lib, case, shares):
    dt, lengths, hq, hkv, d = case
    nb, query = C.c_size_t(0), lib.dpnorm_attention_scores_backward_workspace
    for sc, n in ((None, shares[0]), (_lib.AttnScores(5.0, PRE, None), shares[0]), (_lib.AttnScores(0.0, None, PRE), shares[1]),
                  (_lib.AttnScores(5.0, PRE, PRE), shares[1])):
        assert query(C.byref(shape(*case)), C.byref(sc) if sc else None, C.byref(nb)) == _lib.OK
        assert nb.value == wanted_bytes(lengths, hq, hkv, d, n), (case, n)


@pytest.mark.skipif("DPNORM_TEST_LIB" not in os.environ, reason="launches are only named by the sanitized library's stand-in")
@pytest.mark.parametrize("case,shares", SHARES.items())
def test_launches(lib, case, shares):
    dt, lengths, hq, hkv, d = case
    names = lib.dpnorm_fake_launched
    names.restype = C.c_char_p
    sh, nb = C.byref(shape(*case)), C.c_size_t(0)
    t = [C.byref(_lib.AttnTensor((j + 1) << 42, h * d, d)) for j, h in enumerate((hq, hq, hkv, hkv, hq))]
    g = [C.byref(_lib.AttnTensor((j + 6) << 42, h * d, d)) for j, h in enumerate((hq, hkv, hkv))]
    columns = 64 if d <= 64 else 96 if d <= 96 else 128
    for sc, n in ((_lib.AttnScores(0.0, PRE, None), shares[0]), (_lib.AttnScores(0.0, PRE, PRE + 4096), shares[1]),
                  (_lib.AttnScores(3.0, None, PRE), shares[1])):
        assert lib.dpnorm_attention_scores_backward_workspace(sh, C.byref(sc), C.byref(nb)) == _lib.OK
        names()
        assert lib.dpnorm_attention_scores_backward(sh, C.byref(sc), *t, LSE, *g, WS, nb.value, None) == _lib.OK
        got = [form(x.replace("Li1EEEv", "EEv").replace("Li2EEEv", "EEv").replace("Li3EEEv", "EEv"), dt) for x in names().decode().split()]
        assert len(got) == 2 and got[1].startswith(f"kv {columns} ") and got[1].endswith(" s") == (n > 1), (case, got)


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
