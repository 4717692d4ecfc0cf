"""Which kernels a shape's attention takes, from the host layer's launches on a CPU
build with a stand-in for the HIP runtime: the shapes of attention_forms.py reach
the forms that they are listed for."""
import ctypes as C
import os
import re
import subprocess
import sys

import pytest

import attention_forms
from sample_grad_norms_amd import _lib

HERE = os.path.dirname(os.path.abspath(__file__))
CASES = [(dt, shape, forms) for dt, table in ((_lib.BF16, attention_forms.BF16), (_lib.F32, attention_forms.F32))
         for shape, forms in table.items()]


def form(name, dt):
    """A kernel's mangled name as its form."""
    m = re.match(r"_ZN3dpn4attn\d+k_(forward_rows|forward|backward_q_rows|backward_q|backward_kv)I(.*)EEvNS0_4ArgsE$", name)
    kind, args = m.group(1), [int(x) for x in re.findall(r"L[bi](\d+)E", m.group(2) + "E")]
    assert args[0] == (dt == _lib.BF16)
    if kind.startswith("forward"):
        return f"{'rows' if 'rows' in kind else 'tiles'} {args[1]}"
    if kind.startswith("backward_q"):
        return f"{'rows' if 'rows' in kind else 'tiles'} {args[1]}" + (" s" if len(args) > 3 and args[3] else "")
    return f"kv {args[1]} {args[2]}" + (" s" if args[3] else "")


@pytest.mark.skipif("DPNORM_TEST_LIB" not in os.environ, reason="launches are only named by the sanitized library's stand-in")
@pytest.mark.parametrize("dt,shape,forms", CASES)
def test_forms(lib, dt, shape, forms):
    N, Hq, Hkv, D = shape
    names = lib.dpnorm_fake_launched
    names.restype = C.c_char_p
    sh = _lib.AttnShape(dt, N, 1, Hq, Hkv, D, None, 0.1, 0)
    t = [_lib.AttnTensor((j + 1) << 44, h * D, D) for j, h in enumerate((Hq, Hkv, Hkv, Hq, Hq, Hq, Hkv, Hkv))]
    q, k, v, o, do, dq, dk, dv = (C.byref(x) for x in t)
    lse, ws, nb = 10 << 44, 11 << 44, C.c_size_t(0)
    names()
    assert lib.dpnorm_attention_forward(C.byref(sh), q, k, v, o, lse, None) == _lib.OK
    assert lib.dpnorm_attention_backward_workspace(C.byref(sh), C.byref(nb)) == _lib.OK
    assert lib.dpnorm_attention_backward(C.byref(sh), do, q, k, v, o, lse, dq, dk, dv, ws, nb.value, None) == _lib.OK
    assert tuple(form(x, dt) for x in names().decode().split()) == forms


@pytest.mark.skipif("DPNORM_TEST_LIB" in os.environ, reason="already the sanitized library")
def test_under_sanitizers(tmp_path):
    sys.path.insert(0, os.path.join(HERE, "hostcheck"))
    import build as hostcheck_build
    built = hostcheck_build.build(str(tmp_path))
    env = dict(os.environ, LD_PRELOAD=built["asan_runtime"], ASAN_OPTIONS="detect_leaks=0", DPNORM_TEST_LIB=built["lib"])
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", os.path.abspath(__file__)],
                         capture_output=True, text=True, timeout=600, env=env, cwd=os.path.dirname(HERE))
    assert res.returncode == 0, res.stdout[-4000:] + res.stderr[-4000:]
