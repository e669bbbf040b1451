"""The 64-bit definitions of the feed-forward operators, by known values and by differences."""
import numpy as np
import pytest

from oracle import ffn


def test_philox_known_answers():
    # the published known answers of philox4x32-10
    full = (1 << 64) - 1
    assert [int(v) for v in ffn.philox(0, 0, np.array([0]))[0]] == [
        0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert [int(v) for v in ffn.philox(full, full, np.array([full], np.uint64))[0]] == [
        0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    seed, offset = 0x299F31D0A4093822, 0x0370734413198A2E
    assert [int(v) for v in ffn.philox(seed, offset, np.array([0x85A308D3243F6A88], np.uint64))[0]] == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9])
def test_dropout_keeps_its_share(p):
    f = ffn.dropout_factor(1 << 20, p, 7, 3)
    kept = (f != 0).mean()
    # a binomial's standard deviation is at most 2^-11 at 2^20 draws: five of them
    assert abs(kept - (1 - p)) < 5 * 2.0 ** -11 + 2.0 ** -17
    assert abs(f.mean() - 1) < 5 * 2.0 ** -11 / max(1 - p, 1e-9) + 2.0 ** -15
    assert p == 0 or not np.array_equal(f, ffn.dropout_factor(1 << 20, p, 7, 4))


def test_activation_values():
    z = np.array([-1.0, 0.0, 2.0])
    assert np.allclose(ffn.activation(z, "relu"), [0, 0, 2])
    assert np.allclose(ffn.activation(z, "silu"), [-0.2689414213699951, 0, 1.7615941559557649])
    assert np.allclose(ffn.activation(z, "gelu"), [-0.15865525393145707, 0, 1.9544997361036416])
    assert np.allclose(ffn.activation(np.array([[2.0, -1.0, 3.0, 5.0]]), "swiglu"),
                       [[3 * 1.7615941559557649, -5 * 0.2689414213699951]])


@pytest.mark.parametrize("act", ffn.ACTIVATIONS)
def test_activation_gradient_by_differences(act):
    rng = np.random.default_rng(1)
    z = rng.standard_normal((5, 12)) * 2
    d = rng.standard_normal((5, 6 if act == "swiglu" else 12))
    got = ffn.activation_backward(z, d, act)
    h = 1e-6
    for i in range(z.shape[1]):
        up, down = z.copy(), z.copy()
        up[:, i] += h
        down[:, i] -= h
        want = ((ffn.activation(up, act) - ffn.activation(down, act)) * d).sum(-1) / (2 * h)
        assert np.allclose(got[:, i], want, rtol=1e-6, atol=1e-8), i


def test_combine_gradient_by_differences():
    rng = np.random.default_rng(2)
    T, K, H = 4, 2, 8
    y, gates = rng.standard_normal((T * K, H)), rng.random((T, K))
    dst = rng.permutation(T * K).reshape(T, K)
    f = ffn.dropout_factor(T * H, 0.4, 5, 1).reshape(T, H)
    d = rng.standard_normal((T, H))
    d_y, d_gates = ffn.combine_dropout_backward(y, dst, gates, d, f)
    total = lambda y, g: (ffn.combine_dropout(y, dst, g, None, f) * d).sum()  # noqa: E731
    h = 1e-6
    for i in np.ndindex(y.shape):
        e = np.zeros_like(y)
        e[i] = h
        assert abs((total(y + e, gates) - total(y - e, gates)) / (2 * h) - d_y[i]) < 1e-7
    for i in np.ndindex(gates.shape):
        e = np.zeros_like(gates)
        e[i] = h
        assert abs((total(y, gates + e) - total(y, gates - e)) / (2 * h) - d_gates[i]) < 1e-7
