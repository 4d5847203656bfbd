"""Outputs over inputs or over each other are refused, before any HIP call; the rule itself is exact."""
import ctypes
import os
import shutil
import subprocess

import pytest

from gc_testlib import ROOT
from test_train_capi import NULL, VP, Z, lib  # noqa: F401  (the library's fixture)

BASE = 1 << 40      # made-up addresses, never dereferenced: every call here is refused


def area(k):
    """Area k of a call: 2^30 bytes of its own, aligned to 256."""
    return VP(BASE + (k << 30))


def refused(lib, f, args, names):  # noqa: F811
    assert f(*args) == 1
    text = lib.gc_last_error().decode()
    assert "overlap" in text and all(n in text for n in names), text


def test_the_rule_against_sets_of_bytes(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("g++ is not available")
    exe = str(tmp_path / "overlap_brute")
    subprocess.run([gxx, "-std=c++17", "-O1", f"-I{os.path.join(ROOT, 'gradient_compression_ddp_amd', 'csrc')}",
                    os.path.join(ROOT, "tests", "pins", "overlap_brute.cpp"), "-o", exe], check=True)
    res = subprocess.run([exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout
    yes, no = map(int, res.stdout.split())
    assert yes > 50000 and no > 50000


def at(p, more):
    return VP(p.value + more)


def test_ckpt(lib):  # noqa: F811
    x, codes, exps = area(0), area(1), area(2)
    refused(lib, lib.gc_ckpt_pack, (2, x, 64, 8, 64, x, exps, NULL), ("x", "codes"))
    refused(lib, lib.gc_ckpt_pack, (2, x, 64, 8, 64, codes, at(x, 8 * 64 * 2 - 1), NULL), ("x", "exponents"))
    refused(lib, lib.gc_ckpt_pack, (2, x, 64, 8, 64, codes, at(codes, 511), NULL), ("codes", "exponents"))
    refused(lib, lib.gc_ckpt_unpack, (2, codes, exps, 8, 64, at(codes, 256), 64, NULL), ("codes", "out"))


def test_act(lib):  # noqa: F811
    x, y, codes, exps = (area(k) for k in range(4))
    refused(lib, lib.gc_act_forward, (2, 0, x, 64, 8, 64, x, 64, NULL, NULL, NULL, NULL, NULL), ("x", "y"))
    refused(lib, lib.gc_act_forward, (2, 0, x, 100, 8, 64, at(x, 2 * 63), 100, NULL, NULL, NULL, NULL, NULL), ("x", "y"))
    refused(lib, lib.gc_act_forward, (2, 0, x, 64, 8, 64, y, 64, codes, exps, codes, area(5), NULL), ("x's codes", "y's codes"))
    refused(lib, lib.gc_act_backward, (2, 0, x, 64, y, 64, NULL, NULL, 8, 64, x, 64, NULL), ("dy", "dx"))
    refused(lib, lib.gc_act_backward, (2, 0, x, 64, y, 64, NULL, NULL, 8, 64, at(y, 2), 70, NULL), ("dx", "x"))
    refused(lib, lib.gc_act_backward, (2, 0, x, 64, NULL, 0, codes, exps, 8, 64, at(exps, -1022), 64, NULL), ("dx", "exponents"))


def test_layernorm(lib):  # noqa: F811
    p = [area(k) for k in range(10)]
    good = [2, p[0], 64, 8, 64, 0, p[1], p[2], 1e-5, p[3], 64, p[4], p[5], p[6], p[7], p[8], p[9], NULL]

    def over(i, v, *names):
        a = list(good)
        a[i] = v
        refused(lib, lib.gc_layernorm_forward, a, names)
    over(9, p[0], "x", "y")
    over(11, p[5], "mean", "rstd")
    over(12, at(p[1], 252), "weight", "rstd")
    over(13, p[3], "y", "x's codes")
    need = Z(0)
    assert lib.gc_layernorm_backward_workspace(1000, 4096, ctypes.byref(need)) == 0
    good = [2, p[0], 4096, p[1], 4096, NULL, NULL, 1000, 4096, 0, p[2], p[3], p[4], p[5], 4096, p[6], p[7], 0, p[8], need.value, NULL]

    def over(i, v, *names):
        a = list(good)
        a[i] = v
        refused(lib, lib.gc_layernorm_backward, a, names)
    over(13, p[0], "dy", "dx")
    over(13, p[1], "dx", "x")
    over(15, p[7], "dw", "db")
    over(15, at(p[3], 3996), "mean", "dw")
    over(18, at(p[5], 1000 * 4096 * 2 - 256), "dx", "workspace")
    over(18, at(p[7], -256 * (need.value // 256 - 1)), "db", "workspace")


def test_linear_wgrad(lib):  # noqa: F811
    p = [area(k) for k in range(6)]
    need = Z(0)
    assert lib.gc_linear_wgrad_workspace(2, 8192, 256, 256, ctypes.byref(need)) == 0
    good = [2, p[0], 256, p[1], p[2], 8192, 256, 256, p[3], 256, p[4], 0, p[5], need.value, NULL]

    def over(i, v, *names):
        a = list(good)
        a[i] = v
        refused(lib, lib.gc_linear_wgrad, a, names)
    over(8, p[0], "dy", "dw")
    over(8, at(p[1], 8192 * 256 - 4), "dw", "codes")
    over(10, at(p[3], 256 * 256 * 4 - 4), "dw", "db")
    over(12, at(p[0], 256), "dy", "workspace")
    over(12, p[3], "dw", "workspace")
