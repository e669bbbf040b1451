"""Calls of the feed-forward operators that their documentation allows and that lie at its edges."""
import numpy as np
import pytest
import torch

import perfectly_balanced_token_gb300 as mx
from oracle import ffn
from perfectly_balanced_token_gb300 import synthetic as syn
from tests.test_gpu_ffn import BF16, F32, Plan, assert_within, np64
from tests.gpu_harness import ensure_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_library()


@pytest.mark.parametrize("K,Hp", [(2, 192), (4, 512), (8, 256), (3, 1024), (2, 2048), (5, 1088), (3, 4096), (9, 7168)])
def test_dropped_values_reach_no_gradient(K, Hp):
    # infinities and NaN of y, of d_out and of a gate, where the element was dropped
    pl = Plan(R=2, E=16, B=8, K=K, S=37, H=64, Hp=Hp)
    d, T, p, seed, offset = pl.d, 74, 0.5, 31, 5
    rng = torch.tensor([seed, offset], device="cuda")
    f = ffn.dropout_factor(T * Hp, p, seed, offset).reshape(T, Hp)
    y, dout = syn.normal_bf16((d.N, Hp), 1.0, 1), syn.normal_bf16((T, Hp), 1.0, 2)
    gates = pl.gates.reshape(T, K).clone()
    bad = [float("inf"), float("-inf"), float("nan")]
    for t in range(0, T, 3):
        gone = np.nonzero(f[t] == 0)[0]
        for i, v in enumerate(bad):
            y[pl.dst[t, i % K], gone[i::7]] = v
        dout[t, gone[::5]] = bad[t % 3]
    gates[1, 0], gates[4, K - 1], gates[7, 1] = bad[0], bad[2], bad[1]
    y[pl.dst[10, 0], np.nonzero(f[10] != 0)[0][3]] = bad[2]  # and one that was kept
    d_y, d_g = torch.empty(d.N, Hp, dtype=BF16, device="cuda"), torch.empty(T, K, dtype=F32, device="cuda")
    mx.moonep_combine_dropout_backward(d, pl.ws.buf, y.cuda(), gates, dout.cuda(), d_y, d_g, p=p, rng=rng)
    y64, g64, d64 = np64(y), np64(gates), np64(dout)
    want_y, want_g = ffn.combine_dropout_backward(y64, pl.dst, g64, d64, f)
    finite = np.isfinite(want_g)
    assert (~finite).sum() == 1 and np.array_equal(np.isfinite(np64(d_g)), finite)
    # (dropped values, whatever they are, have no part in the bound either)
    size = ffn.combine_dropout_backward(np.abs(y64), pl.dst, g64, np.abs(d64), f)[1]
    assert_within(np64(d_g)[finite], want_g[finite], (Hp + 2) * 2.0 ** -24 * size[finite], "d_gates")
    got = np64(d_y)
    odd = ~np.isfinite(want_y)
    assert odd.any() and np.array_equal(np.isnan(got), np.isnan(want_y))
    assert np.array_equal(got[odd], want_y[odd], equal_nan=True)
    assert_within(got[~odd], want_y[~odd], (2.0 ** -8 + 2.0 ** -22) * np.abs(want_y[~odd]), "d_y")
