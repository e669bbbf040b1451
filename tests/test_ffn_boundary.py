"""The feed-forward operators' C ABI on the host: exports, refusals before anything is
enqueued, plain C use, and the binding's own checks (no GPU needed)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import perfectly_balanced_token_gb300 as mx
from perfectly_balanced_token_gb300 import _ffn, _lib

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include")
HEADER = os.path.join(INCLUDE, "moonep_ffn.h")
P = ctypes.c_void_p
OK_PTR, ODD = P(0x20000), P(0x20004)


@pytest.fixture(scope="module")
def lib():
    from perfectly_balanced_token_gb300.build import build
    build()
    return _ffn.library()


@pytest.fixture(autouse=True)
def nothing_launched(lib):
    before = mx.moonep_launch_count()
    yield
    assert mx.moonep_launch_count() == before


def test_every_declared_function_is_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(moonep_\w+)\s*\(", text)))
    assert len(names) == 10
    for n in names:
        assert hasattr(lib, n) and hasattr(mx, n), n


def linear(lib, ld, x=OK_PTR, w=OK_PTR, bias=None, residual=None, out=OK_PTR, z=None, status=OK_PTR):
    return lib.moonep_linear(ctypes.byref(ld) if ld else None, x, w, bias, residual, out, z, status, None)


def dx(lib, ld, d_z=OK_PTR, w=OK_PTR, d_x=OK_PTR, status=OK_PTR):
    return lib.moonep_linear_dx(ctypes.byref(ld) if ld else None, d_z, w, d_x, status, None)


def dw(lib, ld, x=OK_PTR, d_z=OK_PTR, d_w=OK_PTR, acc=0, status=OK_PTR):
    return lib.moonep_linear_dw(ctypes.byref(ld) if ld else None, x, d_z, d_w, acc, status, None)


def test_linear_sizes_are_checked(lib):
    big = (1 << 31) - 512
    bad = {_lib.ERR_ARG: [dict(T=-1), dict(K=0), dict(N=0), dict(K=-8)],
           _lib.ERR_SHAPE: [dict(K=12), dict(N=12), dict(N=24, act="swiglu"), dict(T=big),
                            dict(K=big + 504), dict(N=big + 504), dict(T=big - 8, N=1 << 20)]}
    for code, cases in bad.items():
        for c in cases:
            ld = mx.linear_dims(**{**dict(T=10, K=64, N=64), **c})
            for call in (linear, dx, dw):
                assert call(lib, ld) == code, (c, call)
    for field, value in (("act", -1), ("act", 5), ("out_f32", 2)):
        ld = mx.linear_dims(10, 64, 64)
        setattr(ld, field, value)
        assert linear(lib, ld) == _lib.ERR_ARG
    for call in (linear, dx, dw):
        assert call(lib, None) == _lib.ERR_ARG
    assert linear(lib, mx.linear_dims(0, 64, 64), x=None, w=None, out=None, status=None) == _lib.OK
    assert dx(lib, mx.linear_dims(0, 64, 64), d_z=None, w=None, d_x=None, status=None) == _lib.OK
    assert dw(lib, mx.linear_dims(0, 64, 64), acc=1, x=None, d_z=None, status=None) == _lib.OK
    with pytest.raises(ValueError):
        mx.linear_dims(1, 64, 64, act="tanh")
    with pytest.raises(ValueError):
        mx.linear_dims(1, 64, 64, out_dtype=torch.float16)


def test_linear_pointers_are_checked(lib):
    ld = mx.linear_dims(10, 64, 64)
    for call, names in ((linear, ("x", "w", "out")), (dx, ("d_z", "w", "d_x")), (dw, ("x", "d_z", "d_w"))):
        for name in names:
            assert call(lib, ld, **{name: None}) == _lib.ERR_ARG
            assert call(lib, ld, **{name: ODD}) == _lib.ERR_ALIGN
        assert call(lib, ld, status=None) == _lib.ERR_ARG
        assert call(lib, ld, status=P(0x20002)) == _lib.ERR_ALIGN
    for name in ("bias", "residual", "z"):
        assert linear(lib, ld, **{name: ODD}) == _lib.ERR_ALIGN
    assert dw(lib, ld, acc=2) == _lib.ERR_ARG


def act(lib, rows=4, cols=64, act=3, z=OK_PTR, d_out=OK_PTR, d_z=OK_PTR, d_bias=None, acc=0, scratch=None):
    return lib.moonep_act_backward(rows, cols, act, z, d_out, d_z, d_bias, acc, scratch, None)


def grouped_act(lib, d, ws=OK_PTR, act=3, z=OK_PTR, d_out=OK_PTR, d_z=OK_PTR, d_bias=None, acc=0,
                scratch=None):
    return lib.moonep_grouped_act_backward(ctypes.byref(d), ws, act, z, d_out, d_z, d_bias, acc, scratch,
                                           None)


def test_act_backward_is_checked(lib):
    d = mx.dims(1, 8, 0, 2, 16, 64, 64, 1)
    assert act(lib, rows=-1) == _lib.ERR_ARG
    assert act(lib, cols=0) == _lib.ERR_ARG
    assert act(lib, cols=12) == _lib.ERR_SHAPE
    assert act(lib, cols=24, act=4) == _lib.ERR_SHAPE
    assert act(lib, rows=1 << 40) == _lib.ERR_SHAPE
    assert act(lib, cols=(1 << 31) - 256) == _lib.ERR_SHAPE
    assert grouped_act(lib, mx.dims(1, 2, 0, 1, 1, 64, 1 << 26, 1)) == _lib.ERR_SHAPE
    for call in (act, lambda lib, **kw: grouped_act(lib, d, **kw)):
        for bad in (-1, 5):
            assert call(lib, act=bad) == _lib.ERR_ARG
        for name in ("z", "d_out", "d_z"):
            assert call(lib, **{name: None}) == _lib.ERR_ARG
            assert call(lib, **{name: ODD}) == _lib.ERR_ALIGN
        assert call(lib, d_bias=OK_PTR) == _lib.ERR_ARG  # no scratch
        assert call(lib, d_bias=OK_PTR, scratch=ODD) == _lib.ERR_ALIGN
        assert call(lib, d_bias=ODD, scratch=OK_PTR) == _lib.ERR_ALIGN
        assert call(lib, acc=2) == _lib.ERR_ARG
        assert call(lib, act=0, z=None, d_z=None) == _lib.ERR_ARG  # nothing to write
    assert grouped_act(lib, d, ws=None) == _lib.ERR_ARG
    assert grouped_act(lib, mx.dims(1, 8, 0, 2, 16, 64, 96, 1)) == _lib.ERR_SHAPE
    assert act(lib, rows=0, z=None, d_out=None, d_z=None) == _lib.OK
    assert act(lib, rows=0, d_bias=OK_PTR, acc=1) == _lib.OK
    assert mx.moonep_act_backward_workspace_bytes(0, 64) == 64 * 4
    assert mx.moonep_act_backward_workspace_bytes(129, 64) == 3 * 64 * 4
    assert lib.moonep_act_backward_workspace_bytes(4, 64, None) == _lib.ERR_ARG
    assert lib.moonep_grouped_act_backward_workspace_bytes(ctypes.byref(d), None) == _lib.ERR_ARG
    # a tile of the plan's list and one of a column of sums each
    assert mx.moonep_grouped_act_backward_workspace_bytes(d) == (1 + 8) * 64 * 4
    with pytest.raises(mx.MoonepError):
        mx.moonep_grouped_act_backward_workspace_bytes(mx.dims(3, 8, 0, 2, 16, 64, 64, 1))


def gemm(lib, d, ws=OK_PTR, act=0, recv=OK_PTR, home=OK_PTR, slot=None, bias=None, y=OK_PTR, z=None):
    return lib.moonep_grouped_gemm_act(ctypes.byref(d), ws, act, recv, home, slot, bias, y, z, None)


def test_grouped_gemm_act_is_checked(lib):
    d = mx.dims(1, 8, 0, 2, 16, 64, 64, 1)
    for name in ("ws", "recv", "home", "y"):
        assert gemm(lib, d, **{name: None}) == _lib.ERR_ARG
        assert gemm(lib, d, **{name: ODD}) == _lib.ERR_ALIGN
    for name in ("bias", "z"):
        assert gemm(lib, d, **{name: ODD}) == _lib.ERR_ALIGN
    for bad in (-1, 5):
        assert gemm(lib, d, act=bad) == _lib.ERR_ARG
    assert gemm(lib, mx.dims(1, 8, 8, 2, 16, 64, 64)) == _lib.ERR_ARG  # slots, but no weights for them
    assert gemm(lib, mx.dims(1, 8, 0, 2, 16, 96, 64, 1)) == _lib.ERR_SHAPE
    assert gemm(lib, mx.dims(1, 1, 0, 1, 16, (1 << 31) - 64, 64, 1)) == _lib.ERR_SHAPE  # E*H too large


def combine(lib, d, ws=OK_PTR, y=OK_PTR, gates=OK_PTR, residual=None, out=OK_PTR, p=0.5, rng=OK_PTR):
    return lib.moonep_combine_dropout(ctypes.byref(d), ws, y, gates, residual, out, p, rng, None)


def combine_back(lib, d, ws=OK_PTR, y=OK_PTR, gates=OK_PTR, d_out=OK_PTR, d_y=OK_PTR, d_gates=OK_PTR,
                 p=0.5, rng=OK_PTR):
    return lib.moonep_combine_dropout_backward(ctypes.byref(d), ws, y, gates, d_out, d_y, d_gates, p, rng,
                                               None)


def test_combine_dropout_is_checked(lib):
    d = mx.dims(1, 8, 0, 2, 16, 64, 64, 1)
    for call, names in ((combine, ("ws", "y", "gates", "out")),
                        (combine_back, ("ws", "y", "gates", "d_out", "d_y", "d_gates"))):
        for name in names + ("rng",):
            assert call(lib, d, **{name: None}) == _lib.ERR_ARG
            assert call(lib, d, **{name: ODD}) == _lib.ERR_ALIGN
        for p in (-0.1, 1.0, 1.5, float("nan"), 1 - 2.0 ** -18):
            assert call(lib, d, p=p) == _lib.ERR_ARG, p
    assert combine(lib, d, residual=ODD) == _lib.ERR_ALIGN
    assert combine_back(lib, mx.dims(1, 256, 0, 129, 16, 64, 64, 1)) == _lib.ERR_SHAPE
    assert combine_back(lib, mx.dims(1, 8, 0, 2, 16, 64, 8256, 1)) == _lib.ERR_SHAPE


def test_binding_checks_its_arguments():
    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    ld = mx.linear_dims(4, 64, 64)
    with pytest.raises(ValueError, match="CUDA"):
        mx.moonep_linear(ld, t, t, t, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="act must be"):
        mx.moonep_act_backward(t, t, t, act="tanh")
    with pytest.raises(ValueError, match="tensor of rows"):
        mx.moonep_act_backward(t, torch.zeros(()), t)
    with pytest.raises(ValueError, match="scratch has"):
        _ffn._scratch(torch.zeros(8, dtype=torch.uint8), 16)
    with pytest.raises(ValueError, match="scratch is required"):
        _ffn._scratch(None, 16)


def test_plain_c_client(tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "client.c"
    src.write_text('''
#include <stdio.h>
#include "moonep_ffn.h"
#include "moonep_ops.h"
int main(void) {
  moonep_linear_dims d = {4, 64, 64, MOONEP_ACT_SWIGLU, 0};
  size_t n = 0;
  int32_t status = 0;
  uint16_t b[8];
  if (moonep_act_backward_workspace_bytes(300, 64, &n) != MOONEP_OK || n != 5 * 64 * 4) return 1;
  if (moonep_linear(&d, NULL, b, NULL, NULL, b, NULL, &status, NULL) != MOONEP_ERR_ARG) return 2;
  d.K = 65;
  if (moonep_linear_dx(&d, b, b, b, &status, NULL) != MOONEP_ERR_SHAPE) return 3;
  printf("ok\\n");
  return 0;
}
''')
    exe = tmp_path / "client"
    r = subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", INCLUDE, "-o", str(exe), str(src),
                        _lib.LIB_PATH, f"-Wl,-rpath,{os.path.dirname(_lib.LIB_PATH)}"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == "ok\n", (r.returncode, r.stdout, r.stderr)
