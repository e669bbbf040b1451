"""What the binding of the feed-forward operators refuses by itself (no GPU needed)."""
import pytest
import torch

import perfectly_balanced_token_gb300 as mx
from perfectly_balanced_token_gb300 import _ffn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from perfectly_balanced_token_gb300.build import build
    build()


def one_row(cols):
    """A tensor of one row of any length, with no memory behind it."""
    return torch.empty(1, cols, dtype=torch.bfloat16, device="meta")


def test_sizes_past_32_bits_are_refused(monkeypatch):
    # (an int32 argument would take their low bits: 2^32 + 64 columns would run as 64)
    for wide in ((1 << 32) + 64, 1 << 31, -(1 << 31) - 8):
        with pytest.raises(ValueError, match="past 32 bits"):
            mx.moonep_act_backward_workspace_bytes(4, wide)
        for sizes in ((wide, 64, 64), (4, wide, 64), (4, 64, wide)):
            with pytest.raises(ValueError, match="past 32 bits"):
                mx.linear_dims(*sizes)
    with pytest.raises(mx.MoonepError):  # within 32 bits, and too large for the library
        mx.moonep_act_backward_workspace_bytes(4, (1 << 31) - 8)
    monkeypatch.setattr(_ffn, "_ptr", lambda *a, **k: 0x20000)
    before = mx.moonep_launch_count()
    for act, cols in (("relu", (1 << 32) + 64), ("swiglu", (1 << 31) + 64)):
        with pytest.raises(ValueError, match="past 32 bits"):
            mx.moonep_act_backward(None, one_row(cols), None, act=act)
    assert mx.moonep_launch_count() == before
