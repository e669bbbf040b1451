"""The library's launchers on the host, against a CUDA runtime that launches nothing
(fake_runtime.cpp): what they keep for a device holds for that device alone."""
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
    work = tmp_path_factory.mktemp("fake")
    exe = str(work / "fake")
    objects = [os.path.join(b.OUT_DIR, s.replace(".cu", ".o")) for s in b.SOURCES]
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-I", headers, "-o", exe,
                        os.path.join(HERE, "fake_runtime.cpp"), *objects, "-lpthread"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(*args):
        r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stdout + r.stderr
        return r.stdout.splitlines()
    return run


@pytest.mark.parametrize("call", ["mxfp4_grouped_gemm", "grouped_gemm", "grouped_gemm_dx",
                                  "grouped_gemm_dw"])
def test_each_device_is_set_up(fake, call):
    # the second device has half the multiprocessors and an opt-in of its own
    lines = fake(call, 0, 1, 0)
    assert [ln for ln in lines if ln.startswith("returned")] == ["returned 0"] * 3, lines
    grids = [(int(m[1]), int(m[2])) for m in (re.match(r"device (\d) \S+ grid (\d+) ok", ln)
                                              for ln in lines) if m]
    n = 1 if call.endswith("dw") else 2  # a kernel for each height of the plan's tiles
    assert grids == [(0, 152)] * n + [(1, 76)] * n + [(0, 152)] * n, lines


@pytest.mark.parametrize("call", ["mxfp4_grouped_gemm", "grouped_gemm", "grouped_gemm_dx",
                                  "grouped_gemm_dw"])
@pytest.mark.parametrize("offset", [0, 16, 112, 240])
def test_tensor_maps_lie_on_128_bytes(fake, call, offset):
    # the workspace may begin at any multiple of 16; the copies stay in its last bytes
    import perfectly_balanced_token_gb300 as mx
    d = mx.dims(2, 8, 4, 2, 4096, 512, 512)
    end = 0x10000000 + offset + mx.moonep_plan_workspace_bytes(d)
    lines = fake("offset", call, offset)
    maps = [(int(m[1]), int(m[2])) for m in (re.search(r"grid (\d+) ok maps (\d+)", ln)
                                             for ln in lines) if m]
    assert maps and lines[-1] == "returned 0", lines
    for ctas, at in maps:
        assert at % 128 == 0, lines
        assert end - mx.GEMM_SCRATCH_BYTES <= at and at + ctas * 8 * 2 * 128 <= end, lines
