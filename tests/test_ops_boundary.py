"""The operators' C ABI on the host: exports, refusals before anything is
enqueued, plain C use, and the binding's own checks (no GPU needed)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import perfectly_balanced_token_gb300 as mx
from perfectly_balanced_token_gb300 import _lib, _ops

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include")
HEADER = os.path.join(INCLUDE, "moonep_ops.h")
P = ctypes.c_void_p
OK_PTR, ODD = P(0x20000), P(0x20004)


@pytest.fixture(scope="module")
def lib():
    from perfectly_balanced_token_gb300.build import build
    build()
    return _ops.library()


@pytest.fixture(autouse=True)
def nothing_launched(lib):
    before = mx.moonep_launch_count()
    yield
    assert mx.moonep_launch_count() == before


def test_every_declared_function_is_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(moonep_\w+)\s*\(", text)))
    assert len(names) == 9
    for n in names:
        assert hasattr(lib, n) and hasattr(mx, n), n


def forward(lib, rd, logits=OK_PTR, mask=None, idx=OK_PTR, gates=OK_PTR, ws=None, counts=None,
            psum=None, tokens=None, loss=None):
    return lib.moonep_router_forward(ctypes.byref(rd) if rd else None, logits, mask, idx, gates, ws,
                                     counts, psum, tokens, loss, None)


def test_router_sizes_are_checked(lib):
    bad = {_lib.ERR_ARG: [dict(T=0), dict(E=0), dict(K=0), dict(T=-1), dict(segment=-1),
                          dict(scale=float("nan")), dict(scale=float("inf"))],
           _lib.ERR_SHAPE: [dict(K=65), dict(E=4097), dict(E=200, K=129), dict(segment=101),
                            dict(T=1 << 28, K=8)]}
    for code, cases in bad.items():
        for c in cases:
            rd = mx.router_dims(**{**dict(T=100, E=64, K=4), **c})
            assert forward(lib, rd) == code, c
            with pytest.raises(mx.MoonepError) as ei:
                mx.moonep_router_workspace_bytes(rd)
            assert ei.value.status == code
    for field in ("score", "normalise", "dtype"):
        rd = mx.router_dims(100, 64, 4)
        setattr(rd, field, 2)
        assert forward(lib, rd) == _lib.ERR_ARG
    assert forward(lib, None) == _lib.ERR_ARG
    assert lib.moonep_router_workspace_bytes(ctypes.byref(mx.router_dims(9, 8, 2)), None) == _lib.ERR_ARG
    with pytest.raises(ValueError):
        mx.router_dims(9, 8, 2, score="relu")
    with pytest.raises(ValueError):
        mx.router_dims(9, 8, 2, dtype=torch.float16)


def test_router_pointers_are_checked(lib):
    rd = mx.router_dims(100, 64, 4)
    for name in ("logits", "idx", "gates"):
        assert forward(lib, rd, **{name: None}) == _lib.ERR_ARG
        assert forward(lib, rd, **{name: ODD}) == _lib.ERR_ALIGN
    assert forward(lib, rd, mask=P(0x20001)) == _lib.ERR_ALIGN
    balance = dict(ws=OK_PTR, counts=OK_PTR, psum=OK_PTR, tokens=OK_PTR, loss=OK_PTR)
    for name in balance:  # all or none
        assert forward(lib, rd, **{**balance, name: None}) == _lib.ERR_ARG
        assert forward(lib, rd, **{name: OK_PTR}) == _lib.ERR_ARG
        if name != "loss":
            assert forward(lib, rd, **{**balance, name: ODD}) == _lib.ERR_ALIGN
    assert forward(lib, rd, **{**balance, "loss": P(0x20002)}) == _lib.ERR_ALIGN

    def backward(logits=OK_PTR, mask=None, idx=OK_PTR, dg=OK_PTR, counts=None, tokens=None,
                 dl=None, out=OK_PTR):
        return lib.moonep_router_backward(ctypes.byref(rd), logits, mask, idx, dg, counts, tokens,
                                          dl, out, None)

    for name in ("logits", "idx", "out"):
        assert backward(**{name: None}) == _lib.ERR_ARG
        assert backward(**{name: ODD}) == _lib.ERR_ALIGN
    assert backward(dg=None) == _lib.ERR_ARG  # no gradient at all
    assert backward(dg=ODD) == _lib.ERR_ALIGN
    assert backward(mask=ODD) == _lib.ERR_ALIGN
    for name in ("counts", "tokens", "dl"):
        assert backward(**{name: OK_PTR}) == _lib.ERR_ARG
    assert backward(counts=OK_PTR, tokens=OK_PTR, dl=P(0x20002)) == _lib.ERR_ALIGN


def test_mxfp4_arguments_are_checked(lib):
    for fn in (lib.moonep_mxfp4_quantize, lib.moonep_mxfp4_dequantize):
        assert fn(4, 33, OK_PTR, OK_PTR, OK_PTR, None) == _lib.ERR_SHAPE
        assert fn(1 << 40, 32, OK_PTR, OK_PTR, OK_PTR, None) == _lib.ERR_SHAPE
        assert fn(-1, 32, OK_PTR, OK_PTR, OK_PTR, None) == _lib.ERR_ARG
        assert fn(4, 0, OK_PTR, OK_PTR, OK_PTR, None) == _lib.ERR_ARG
        assert fn(0, 32, None, None, None, None) == _lib.OK  # nothing to do
        for i in range(3):
            ptrs = [OK_PTR] * 3
            ptrs[i] = None
            assert fn(4, 32, *ptrs, None) == _lib.ERR_ARG
            ptrs[i] = ODD
            assert fn(4, 32, *ptrs, None) == _lib.ERR_ALIGN
    w = lib.moonep_mxfp4_quantize_weights
    assert w(2, 96, 64, OK_PTR, OK_PTR, OK_PTR, None) == _lib.ERR_SHAPE
    assert w(2, 64, 96, OK_PTR, OK_PTR, OK_PTR, None) == _lib.ERR_SHAPE
    assert w(2, 0, 64, OK_PTR, OK_PTR, OK_PTR, None) == _lib.ERR_ARG
    assert w(-1, 64, 64, OK_PTR, OK_PTR, OK_PTR, None) == _lib.ERR_ARG
    assert w(2, 64, 64, None, OK_PTR, OK_PTR, None) == _lib.ERR_ARG
    assert w(2, 64, 64, OK_PTR, ODD, OK_PTR, None) == _lib.ERR_ALIGN


def test_mxfp4_layer_calls_are_checked(lib):
    d = mx.dims(4, 8, 2, 2, 16, 64, 128)
    D, ws = ctypes.byref(d), P(0x10000)
    o = OK_PTR
    calls = [(lib.moonep_mxfp4_prefetch_weights, 4), (lib.moonep_mxfp4_dispatch, 3),
             (lib.moonep_mxfp4_grouped_gemm, 7)]
    for fn, n in calls:
        assert fn(None, ws, *[o] * n, None) == _lib.ERR_ARG
        assert fn(D, None, *[o] * n, None) == _lib.ERR_ARG
        assert fn(D, P(0x10008), *[o] * n, None) == _lib.ERR_ALIGN
        for i in range(n):
            args = [o] * n
            args[i] = None
            assert fn(D, ws, *args, None) == _lib.ERR_ARG
            args[i] = ODD
            assert fn(D, ws, *args, None) == _lib.ERR_ALIGN
        bad = mx.dims(4, 8, 1, 2, 16, 64, 128)
        assert fn(ctypes.byref(bad), ws, *[o] * n, None) == _lib.ERR_SLOTS
    # more weight rows than a 32-bit coordinate reaches
    wide = mx.dims(1, 4096, 0, 1, 1, 64, 1 << 19, 1)
    assert lib.moonep_mxfp4_grouped_gemm(ctypes.byref(wide), ws, o, o, o, o, None, None, o,
                                         None) == _lib.ERR_SHAPE


def test_binding_checks_its_tensors(lib):
    rd = mx.router_dims(4, 8, 2)
    host = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        mx.moonep_router_forward(rd, host, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    with pytest.raises(ValueError):
        mx.moonep_mxfp4_quantize(torch.zeros(4, 64, dtype=torch.bfloat16),
                                 torch.zeros(4, 32, dtype=torch.uint8),
                                 torch.zeros(4, 16, dtype=torch.uint8))
    with pytest.raises(ValueError):
        mx.moonep_mxfp4_quantize_weights(torch.zeros(64, 64, dtype=torch.bfloat16), None, None)


def test_kept_sizes_do_not_pile_up(lib):
    # a program whose token count never repeats
    sizes = [(mx.moonep_router_workspace_bytes(mx.router_dims(64, 64, 4, n)),
              mx.moonep_plan_workspace_bytes(mx.dims(1, 8, 0, 2, 100 + n, 64, 64, 1)))
             for n in range(1, 65)]
    for n in range(3000):
        mx.moonep_router_workspace_bytes(mx.router_dims(100 + n, 64, 4))
        mx.moonep_plan_workspace_bytes(mx.dims(1, 8, 0, 2, 200 + n, 64, 64, 1))
    assert len(_ops._sizes) <= 1024 and len(_lib._workspace_bytes) <= 1024
    # and the answers stay what they were
    assert sizes == [(mx.moonep_router_workspace_bytes(mx.router_dims(64, 64, 4, n)),
                      mx.moonep_plan_workspace_bytes(mx.dims(1, 8, 0, 2, 100 + n, 64, 64, 1)))
                     for n in range(1, 65)]


C_CLIENT = r"""
#include <stdio.h>
#include <string.h>
#include "moonep_ops.h"

int main(void) {
  moonep_router_dims d;
  size_t bytes = 0;
  memset(&d, 0, sizeof d);
  d.T = 1024; d.E = 64; d.K = 4; d.scale = 1.0f;
  if (moonep_router_workspace_bytes(&d, &bytes) != MOONEP_OK || bytes == 0) return 1;
  d.K = 65;
  if (moonep_router_workspace_bytes(&d, &bytes) != MOONEP_ERR_SHAPE) return 2;
  if (MOONEP_MXFP4_SCALE_PITCH(64) != 16 || MOONEP_MXFP4_SCALE_PITCH(544) != 32) return 3;
  if (moonep_mxfp4_quantize(1, 48, 0, 0, 0, 0) != MOONEP_ERR_SHAPE) return 4;
  printf("sizeof %zu\n", sizeof(moonep_router_dims));
  return 0;
}
"""


def test_header_is_plain_c_and_links(tmp_path, lib):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    from perfectly_balanced_token_gb300.build import LIB
    src, exe = tmp_path / "client.c", tmp_path / "client"
    offsets = "".join(f'  printf("{n} %zu\\n", offsetof(moonep_router_dims, {n}));\n'
                      for n, _ in _ops.moonep_router_dims._fields_)
    src.write_text(C_CLIENT.replace("  return 0;\n}", offsets + "  return 0;\n}"))
    r = subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", INCLUDE, str(src), LIB,
                        f"-Wl,-rpath,{os.path.dirname(LIB)}", "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, (r.returncode, r.stderr)
    got = dict(ln.split() for ln in r.stdout.splitlines())
    assert int(got.pop("sizeof")) == ctypes.sizeof(_ops.moonep_router_dims)
    assert {k: int(v) for k, v in got.items()} == {
        n: getattr(_ops.moonep_router_dims, n).offset for n, _ in _ops.moonep_router_dims._fields_}
