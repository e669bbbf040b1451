"""The feed-forward operators' launchers on the host, against a CUDA runtime that launches nothing
(fake_runtime_ffn.cpp): what they keep for a device holds for that device alone."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    from perfectly_balanced_token_gb300 import build as b
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    b.build()
    headers = os.path.join(os.path.dirname(os.path.dirname(b._nvcc())), "include")
    exe = str(tmp_path_factory.mktemp("fake") / "fake")
    objects = [os.path.join(b.OUT_DIR, s.replace(".cu", ".o")) for s in b.SOURCES]
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-I", headers, "-o", exe,
                        os.path.join(HERE, "fake_runtime_ffn.cpp"), *objects, "-lpthread"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(*args):
        r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stdout + r.stderr
        return r.stdout.splitlines()
    return run


@pytest.mark.parametrize("call,kernels", [("linear", 1), ("linear_few", 1), ("linear_dx", 1), ("linear_dw", 1),
                                          ("act_backward", 2), ("grouped_gemm_act", 2)])
def test_each_device_is_set_up(fake, call, kernels):
    # the second device has half the multiprocessors and an opt-in of its own
    lines = fake(call, 0, 1, 0)
    assert [ln for ln in lines if ln.startswith("returned")] == ["returned 0"] * 3, lines
    grids = [(int(m[1]), int(m[2])) for m in (re.match(r"device (\d) \S+ grid (\d+) ok", ln)
                                              for ln in lines) if m]
    assert [g[0] for g in grids] == [0] * kernels + [1] * kernels + [0] * kernels, lines
    assert grids[:kernels] == grids[2 * kernels:], lines
    if call in ("linear", "linear_dx", "linear_dw", "grouped_gemm_act"):  # one CTA a multiprocessor
        assert all(g[1] == (152, 76)[g[0]] for g in grids), lines
