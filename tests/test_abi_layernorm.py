"""The C ABI of the layer-norm calls without a GPU: workspace sizes, and every
host-side check returning its documented status before anything is enqueued
(every call here fails a check, but for those on the stand-in). The file also
runs against the host layer built with sanitizers."""
import ctypes as C
import os
import subprocess
import sys

import pytest

from sample_grad_norms_amd import _lib

HERE = os.path.dirname(os.path.abspath(__file__))
X, Y, W, B_, DY, DX, DW, DB, MEAN, RSTD, N_, CW, WS = (0x100000000 * j for j in range(1, 14))   # aligned, never read
BIG = 1 << 50
NAN, INF = float("nan"), float("inf")
BAD = [dict(d=0), dict(d=-8), dict(d=12), dict(d=32776), dict(d=2 ** 40)]


def test_forward_checks(lib):
    def call(x=X, w=W, b=B_, dt=_lib.BF16, kind=_lib.LN_LAYER, n=300, d=64, eps=1e-5, y=Y, mean=MEAN, rstd=RSTD):
        return lib.dpnorm_layernorm_forward(x, w, b, dt, kind, n, d, eps, y, mean, rstd, None)
    assert call(x=None) == call(w=None) == call(y=None) == _lib.ERR_NULL
    assert call(dt=2) == call(dt=-1) == call(kind=2) == call(kind=-5) == _lib.ERR_DTYPE
    for bad in BAD + [dict(n=0), dict(n=-1), dict(n=2 ** 30 + 1), dict(dt=_lib.F32, d=6)]:
        assert call(**bad) == _lib.ERR_SIZE, bad
    assert call(x=X + 8) == call(w=W + 4) == call(b=B_ + 2) == call(y=Y + 8) == call(mean=MEAN + 2) == call(rstd=RSTD + 1) == _lib.ERR_ALIGN
    for eps in (-1e-6, NAN, INF):
        assert call(eps=eps) == _lib.ERR_VALUE
    assert call(kind=_lib.LN_RMS) == call(kind=_lib.LN_RMS, b=None) == call(kind=_lib.LN_RMS, mean=None) == _lib.ERR_VALUE
    assert call(y=X) == call(y=W) == call(y=B_) == call(mean=Y) == call(rstd=MEAN) == call(rstd=X) == _lib.ERR_VALUE
    assert call(y=X + 300 * 64 * 2 - 16) == call(mean=RSTD + 4) == _lib.ERR_VALUE


def sizes(lib, which, dt=_lib.BF16, kind=_lib.LN_LAYER, B=3, T=1000, d=64):
    nb = C.c_size_t(0)
    return getattr(lib, f"dpnorm_layernorm_{which}_workspace")(dt, kind, B, T, d, C.byref(nb)), nb.value


@pytest.mark.parametrize("which", ["backward", "norm"])
def test_workspaces(lib, which):
    st, nb = sizes(lib, which)
    assert st == _lib.OK and nb > 0 and nb % 256 == 0
    st, nb = sizes(lib, which, T=20)          # one work group (a sample) has it all
    assert st == _lib.OK and nb == 0
    assert getattr(lib, f"dpnorm_layernorm_{which}_workspace")(_lib.BF16, 0, 3, 100, 64, None) == _lib.ERR_NULL
    for bad in BAD + [dict(B=0), dict(T=0), dict(B=2 ** 20, T=2 ** 11), dict(B=2 ** 62, T=2 ** 62)]:
        assert sizes(lib, which, **bad)[0] == _lib.ERR_SIZE, bad
    assert sizes(lib, which, dt=9)[0] == sizes(lib, which, kind=9)[0] == _lib.ERR_DTYPE


def test_backward_checks(lib):
    need = sizes(lib, "backward")[1]

    def call(dy=DY, x=X, w=W, mean=MEAN, rstd=RSTD, dt=_lib.BF16, kind=_lib.LN_LAYER, B=3, T=1000, d=64, c=CW, dx=DX, dw=DW, db=DB, ws=WS,
             size=BIG):
        return lib.dpnorm_layernorm_backward(dy, x, w, mean, rstd, dt, kind, B, T, d, c, dx, dw, db, ws, size, None)
    assert call(dy=None) == call(x=None) == call(w=None) == call(mean=None) == call(rstd=None) == call(ws=None) == _lib.ERR_NULL
    assert call(dx=None, dw=None, db=None) == _lib.ERR_NULL
    assert call(dt=5) == call(kind=-1) == _lib.ERR_DTYPE
    for bad in BAD + [dict(B=0), dict(T=-1), dict(B=2 ** 29, T=3)]:
        assert call(**bad) == _lib.ERR_SIZE, bad
    assert call(dy=DY + 8) == call(x=X + 2) == call(w=W + 8) == call(dx=DX + 8) == call(dw=DW + 4) == call(db=DB + 8) == _lib.ERR_ALIGN
    assert call(mean=MEAN + 1) == call(rstd=RSTD + 2) == call(c=CW + 2) == call(ws=WS + 128) == _lib.ERR_ALIGN
    assert call(size=need - 1) == _lib.ERR_WORKSPACE
    rms = dict(kind=_lib.LN_RMS)
    assert call(**rms) == call(**rms, mean=None) == call(**rms, db=None) == _lib.ERR_VALUE
    for p in (DY, X, W, MEAN, RSTD, CW):
        assert call(dx=p) == call(dw=p) == call(db=p) == call(ws=p) == _lib.ERR_VALUE
    assert call(dw=DX) == call(db=DW) == call(ws=DX) == call(ws=DB) == _lib.ERR_VALUE


def test_norm_checks(lib):
    need = sizes(lib, "norm")[1]

    def call(x=X, g=DY, dt=_lib.BF16, kind=_lib.LN_LAYER, B=3, T=1000, d=64, eps=1e-5, parts=3, n=N_, acc=0, ws=WS, size=BIG):
        return lib.dpnorm_layernorm_norm(x, g, dt, kind, B, T, d, eps, parts, n, acc, ws, size, None)
    assert call(x=None) == call(g=None) == call(n=None) == call(ws=None) == _lib.ERR_NULL
    assert call(dt=5) == call(kind=2) == _lib.ERR_DTYPE
    for bad in BAD + [dict(B=0), dict(T=-1), dict(B=2 ** 29, T=3)]:
        assert call(**bad) == _lib.ERR_SIZE, bad
    assert call(x=X + 8) == call(g=DY + 2) == call(n=N_ + 2) == call(ws=WS + 16) == _lib.ERR_ALIGN
    assert call(parts=0) == call(parts=4) == call(parts=-1) == call(acc=2) == call(acc=-1) == call(eps=-1.0) == call(eps=NAN) == _lib.ERR_VALUE
    assert call(kind=_lib.LN_RMS) == call(kind=_lib.LN_RMS, parts=2) == _lib.ERR_VALUE
    assert call(size=need - 1) == _lib.ERR_WORKSPACE
    assert call(n=X) == call(n=DY) == call(n=WS) == call(ws=X) == call(ws=DY) == _lib.ERR_VALUE


@pytest.mark.skipif("DPNORM_TEST_LIB" in os.environ, reason="already the sanitized library")
def test_under_sanitizers(tmp_path):
    """This file and valid calls against the host layer built with AddressSanitizer and
    UndefinedBehaviorSanitizer."""
    sys.path.insert(0, os.path.join(HERE, "hostcheck"))
    import build as hostcheck_build
    built = hostcheck_build.build(str(tmp_path))
    env = dict(os.environ, LD_PRELOAD=built["asan_runtime"], ASAN_OPTIONS="detect_leaks=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1", DPNORM_TEST_LIB=built["lib"])
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", os.path.abspath(__file__)],
                         capture_output=True, text=True, timeout=600, env=env, cwd=os.path.dirname(HERE))
    assert res.returncode == 0, res.stdout[-4000:] + res.stderr[-4000:]


@pytest.mark.skipif("DPNORM_TEST_LIB" not in os.environ, reason="launches are only checked by the sanitized library's stand-in")
@pytest.mark.parametrize("seed", range(60))
def test_valid_calls_launch_valid_grids(lib, seed):
    """Valid sizes up to the limits succeed with the queried workspace, with fewer than
    2^32 threads along each dimension of every launch."""
    import random
    rng = random.Random(seed)

    def log(lo, hi):
        return int(lo * (hi / lo) ** rng.random())
    dt, kind = rng.choice([_lib.BF16, _lib.F32]), rng.choice([_lib.LN_LAYER, _lib.LN_RMS])
    B = rng.choice([1, log(1, 300), log(1, 2 ** 30), 2 ** 30])
    T, d = max(1, log(1, 2 ** 30) // B), 8 * rng.choice([log(1, 4096), 1, 4096])
    layer = kind == _lib.LN_LAYER
    far = [(1 << 56) + (j << 50) for j in range(12)]
    wide, launches = (C.c_longlong.in_dll(lib, f"dpnorm_fake_{n}") for n in ("wide_launches", "launches"))
    before, at = wide.value, launches.value
    assert lib.dpnorm_layernorm_forward(far[0], far[1], far[2] if layer else None, dt, kind, B * T, d, 0.0, far[3], far[4] if layer else None,
                                        far[5], None) == _lib.OK
    assert lib.dpnorm_layernorm_forward(far[0], far[1], None, dt, kind, B * T, d, 1e-6, far[3], None, None, None) == _lib.OK
    nb = C.c_size_t(0)
    assert lib.dpnorm_layernorm_backward_workspace(dt, kind, B, T, d, C.byref(nb)) == _lib.OK
    mean = far[4] if layer else None
    for dx, dw, db in ((1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1)):
        if not (dx or dw or (db and layer)):
            continue
        assert lib.dpnorm_layernorm_backward(far[0], far[1], far[2], mean, far[5], dt, kind, B, T, d, far[6], far[7] if dx else None,
                                             far[8] if dw else None, far[9] if db and layer else None, far[10], nb.value, None) == _lib.OK
    assert lib.dpnorm_layernorm_norm_workspace(dt, kind, B, T, d, C.byref(nb)) == _lib.OK
    for parts in (3, 1, 2) if layer else (1,):
        assert lib.dpnorm_layernorm_norm(far[0], far[1], dt, kind, B, T, d, 1e-5, parts, far[2], seed % 2, far[3], nb.value, None) == _lib.OK
    assert wide.value == before and launches.value > at
