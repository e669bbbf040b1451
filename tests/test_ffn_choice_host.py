"""What the feed-forward operators' launchers choose by size, on the host, against a CUDA runtime that
launches nothing (fake_runtime_choice.cpp)."""
import os
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
                        os.path.join(HERE, "fake_runtime_choice.cpp"), *objects, "-lpthread"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(device, *args):
        r = subprocess.run([exe, str(device), *map(str, args)], capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stdout + r.stderr
        return r.stdout.splitlines()
    return run


def test_widest_bias_sums_of_experts(fake):
    # 65535 blocks of 1024 columns are launched, more are refused before anything is
    lines = fake(0, "act_bias", 2, 65535 * 1024)
    assert len(lines) == 3 and lines[1].split()[1:3] == ["2", "65535"], lines
    assert lines[2] == "returned 0 refused 0", lines
    for Hp in (65535 * 1024 + 64, (1 << 26) - 64, 1 << 26):
        assert fake(0, "act_bias", 2, Hp) == ["returned 4 refused 0"], Hp


def first(lines):
    """Kernel, grid and tile columns of the first launch."""
    name, x, _, columns = lines[0].split()
    return name, int(x), int(columns)


@pytest.mark.parametrize("sizes,columns", [((5000, 2048, 1024), (192, 256)), ((9984, 2048, 1288), (192, 256)),
                                           ((8192, 2048, 4096), (256, 256))])
def test_tile_width_goes_by_the_devices_pairs(fake, sizes, columns):
    # 76 pairs, and 38: 80 wide tiles are 2 rounds and 3, 120 of 192 columns 2 and 4 (0.88 of the time each)
    for device in (0, 1):
        name, _, got = first(fake(device, "linear", *sizes, 0, 0))
        assert "k_product" in name and got == columns[device], (device, name, got)


def test_the_pair_kernels_tests_reach_it(fake):
    from tests import test_gpu_ffn_pair as t
    acts = ["none", "relu", "gelu", "silu", "swiglu"]
    calls = [(("linear", T, K, N, acts.index(act), f32), width)
             for f32, table in ((0, t.FORWARD), (1, t.FORWARD_F32)) for T, K, N, width, of in table for act in of]
    calls += [((what, T, K, N), width) for what, table in (("dx", t.INPUT), ("dw", t.WEIGHT))
              for T, K, N, width in table]
    calls += [(("experts", *s.values(), act), 128) for s in t.EXPERTS for act in (0, 4)]
    for call, width in calls:
        lines = fake(0, *call)
        launches = [ln.split() for ln in lines[:-1]]
        assert len(launches) == (2 if call[0] == "experts" else 1) and lines[-1].startswith("returned 0"), (call, lines)
        for name, _, _, columns in launches:
            assert "k_product_split" not in name and "k_product" in name and int(columns) == width, (call, name, columns)
