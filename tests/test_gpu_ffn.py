"""The feed-forward operators on the GPU against their 64-bit definitions.

Bound of a product: the instruction adds 16 exact products to the fp32 accumulator and rounds or cuts
each of the 17 terms at 2^-24 of the largest magnitude, which the sum of magnitudes bounds, so K of
them are off by at most 17/16 K 2^-24 of the sum of magnitudes; K 2^-23 is used.  The bias adds one
rounding (2^-24 of the value).  An activation moves by its slope times that (oracle.ffn.sensitivity,
twice for what is not first order), and its own evaluation is off by at most 2^-20 of its result plus
2^-22 of its factors.  Rounding to bf16 is off by 2^-8 of the value, doubled nowhere.
"""
import numpy as np
import pytest
import torch

import perfectly_balanced_token_gb300 as mx
from oracle import ffn
from perfectly_balanced_token_gb300 import synthetic as syn
from tests.gpu_harness import ensure_library

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
BF16_STEP, FLOOR = 2.0 ** -8, 1e-37  # half a step of bf16; below the smallest normal numbers


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_library()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def np64(t):
    return t.detach().double().cpu().numpy()


class Guarded:
    """A buffer with canaries of 256 elements on both sides."""

    def __init__(self, shape, dtype, fill=None):
        n = int(np.prod(shape))
        self.whole = torch.empty(n + 512, dtype=dtype, device="cuda")
        self.bits = self.whole.view(torch.int16 if dtype == BF16 else torch.int32)
        self.bits.fill_(0x7F7F)
        self.t = self.whole[256:256 + n].view(*shape)
        if fill is not None:
            self.t.copy_(fill)

    def check(self):
        assert bool((self.bits[:256] == 0x7F7F).all()) and bool((self.bits[-256:] == 0x7F7F).all())


def assert_within(got, want, bound, what):
    got = np64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~(np.abs(got - want) <= bound + FLOOR)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first at {i}: got {got[i]}, "
                             f"want {want[i]} within {np.broadcast_to(bound, got.shape)[i]}")


def product_bounds(x, w, bias, K):
    """z in 64 bits and how far fp32 sums may be from it."""
    z = x @ w
    err = K * 2.0 ** -23 * (np.abs(x) @ np.abs(w))
    if bias is not None:
        z = z + bias
        err = err + 2.0 ** -24 * np.abs(z)
    return z, err


def act_error(z, act, err):
    e = 2 * ffn.sensitivity(z, act, err)
    if act == "none":
        return err
    if act == "swiglu":
        f = z.shape[-1] // 2
        second = err[..., :f] * err[..., f:]
        return e + 2.0 ** -20 * np.abs(ffn.activation(z, act)) + second
    # (second order: the activations' slopes change by at most 1.2 over a unit)
    return e + 2.0 ** -20 * np.abs(ffn.activation(z, act)) + err ** 2 * 1.2


LINEAR = [  # T, K, N
    (1, 8, 8), (1, 64, 256), (1, 7168, 512), (2, 2048, 1000), (3, 72, 24), (5, 128, 4096), (7, 200, 328),
    (16, 1032, 264), (17, 512, 1024), (31, 640, 520), (64, 4096, 384), (65, 256, 2048), (127, 96, 128),
    (128, 1024, 512), (129, 64, 136), (200, 2056, 1000), (255, 320, 256), (256, 256, 256),
    (257, 264, 272), (511, 136, 640), (777, 1032, 520), (1024, 512, 384), (2049, 72, 1032)]


@pytest.mark.parametrize("T,K,N", LINEAR)
@pytest.mark.parametrize("act,bias,residual,f32,z", [
    ("none", False, False, False, False), ("none", True, True, True, True),
    ("swiglu", True, False, False, True), ("silu", False, True, False, True),
    ("gelu", True, True, True, False), ("relu", True, False, False, False),
    ("swiglu", False, True, True, False)])
def test_linear(T, K, N, act, bias, residual, f32, z):
    if act == "swiglu":
        N *= 2  # (halves of any multiple of 8)
    cols = N // 2 if act == "swiglu" else N
    x, w = syn.normal_bf16((T, K), 1.0, 1), syn.normal_bf16((K, N), K ** -0.5, 2)
    b = torch.randn(N, generator=torch.Generator().manual_seed(3)) if bias else None
    r = syn.normal_bf16((T, cols), 1.0, 4) if residual else None
    out, zz = Guarded((T, cols), F32 if f32 else BF16), Guarded((T, N), BF16) if z else None
    st = status()
    mx.moonep_linear(mx.linear_dims(T, K, N, act=act, out_dtype=F32 if f32 else BF16), x.cuda(), w.cuda(),
                     out.t, st, bias=b.cuda() if bias else None, residual=r.cuda() if residual else None,
                     z=zz.t if z else None)
    assert int(st) == 0
    want_z, err = product_bounds(np64(x), np64(w), np64(b) if bias else None, K)
    want, e = ffn.activation(want_z, act), act_error(want_z, act, err)
    if residual:
        want = want + np64(r)
        e = e + 2.0 ** -24 * np.abs(want)
    assert_within(out.t, want, e + (0 if f32 else BF16_STEP * (np.abs(want) + e)), "out")
    out.check()
    if z:
        assert_within(zz.t, want_z, err + BF16_STEP * (np.abs(want_z) + err), "z")
        zz.check()


@pytest.mark.parametrize("T,K,N", [(1, 8, 8), (3, 72, 24), (64, 512, 1024), (65, 264, 272), (129, 1032, 520),
                                   (257, 256, 256), (777, 1000, 136), (1030, 640, 2048)])
def test_linear_gradients(T, K, N):
    x, w, d = (syn.normal_bf16(s, 1.0, i) for i, s in enumerate([(T, K), (K, N), (T, N)]))
    ld, st = mx.linear_dims(T, K, N), status()
    d_x, d_w = Guarded((T, K), BF16), Guarded((K, N), F32)
    mx.moonep_linear_dx(ld, d.cuda(), w.cuda(), d_x.t, st)
    mx.moonep_linear_dw(ld, x.cuda(), d.cuda(), d_w.t, st)
    x, w, d = np64(x), np64(w), np64(d)
    want, e = product_bounds(d, w.T, None, N)
    assert_within(d_x.t, want, e + BF16_STEP * (np.abs(want) + e), "d_x")
    want, e = product_bounds(x.T, d, None, T)
    assert_within(d_w.t, want, e, "d_w")
    start = torch.randn(K, N, generator=torch.Generator().manual_seed(9))
    acc = Guarded((K, N), F32, start.cuda())
    mx.moonep_linear_dw(ld, torch.from_numpy(x).to(BF16).cuda(), torch.from_numpy(d).to(BF16).cuda(), acc.t,
                        st, accumulate=True)
    want = want + np64(start)
    assert_within(acc.t, want, e + 2.0 ** -24 * (np.abs(want) + e), "d_w added to")
    for g in (d_x, d_w, acc):
        g.check()
    assert int(st) == 0


def test_linear_without_rows():
    ld, st = mx.linear_dims(0, 64, 64), status()
    e, w = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.ones(64, 64, dtype=BF16, device="cuda")
    d_w = torch.ones(64, 64, device="cuda")
    mx.moonep_linear(ld, e, w, e, st)
    mx.moonep_linear_dw(ld, e, e, d_w, st, accumulate=True)
    assert bool((d_w == 1).all())
    mx.moonep_linear_dw(ld, e, e, d_w, st)
    assert bool((d_w == 0).all())


def test_linear_with_a_status_writes_nothing():
    T, K, N = 300, 128, 256
    x, w = syn.normal_bf16((T, K), 1.0, 1).cuda(), syn.normal_bf16((K, N), 1.0, 2).cuda()
    for rows in (3, T):
        st = torch.full((1,), 0x400, dtype=torch.int32, device="cuda")
        out = torch.full((rows, N), 7.0, dtype=BF16, device="cuda")
        mx.moonep_linear(mx.linear_dims(rows, K, N), x[:rows], w, out, st)
        assert bool((out == 7).all()) and int(st) == 0x400


def test_linear_infinities_and_nan():
    # a NaN or an infinity of x stays in its row, one of w in its column
    for T in (4, 300):
        K, N = 128, 264
        x, w = syn.normal_bf16((T, K), 1.0, 1).cuda(), syn.normal_bf16((K, N), 1.0, 2).cuda()
        x[1, 5], x[2, 6], w[7, 11] = float("nan"), float("inf"), float("nan")
        out = torch.empty(T, N, dtype=BF16, device="cuda")
        mx.moonep_linear(mx.linear_dims(T, K, N), x, w, out, status())
        bad = torch.zeros(T, N, dtype=torch.bool, device="cuda")
        bad[1], bad[2], bad[:, 11] = True, True, True
        assert bool(((~torch.isfinite(out)) == bad).all())
        relu = torch.empty_like(out)
        mx.moonep_linear(mx.linear_dims(T, K, N, act="relu"), x, w, relu, status())
        assert bool(torch.isnan(relu[1]).all()) and bool(torch.isnan(relu[:, 11]).all())


ACT_VALUES = [0.0, -0.0, 1e-30, -1e-30, 0.5, -0.5, 5.0, -5.0, 12.0, -12.0, 40.0, -40.0, 80.0, -80.0, 100.0,
              -100.0, 3e4, -3e4]


@pytest.mark.parametrize("act", ffn.ACTIVATIONS)
@pytest.mark.parametrize("rows,N", [(1, 8), (5, 24), (128, 256), (129, 264), (1000, 136), (257, 4096),
                                    (4099, 520)])
def test_act_backward(act, rows, N):
    if act == "swiglu":
        N *= 2
    cols = N // 2 if act == "swiglu" else N
    z, d = syn.normal_bf16((rows, N), 1.5, 1), syn.normal_bf16((rows, cols), 1.0, 2)
    if rows > 4:
        z[2] = torch.tensor(ACT_VALUES).to(BF16).repeat(N // len(ACT_VALUES) + 1)[:N]
    d_z, d_b = Guarded((rows, N), BF16), Guarded((N,), F32)
    scratch = Guarded((mx.moonep_act_backward_workspace_bytes(rows, N) // 4,), F32)
    raw = scratch.t.view(torch.uint8)
    mx.moonep_act_backward(z.cuda(), d.cuda(), d_z.t, act=act, d_bias=d_b.t, scratch=raw)
    z, d = np64(z), np64(d)
    want = ffn.activation_backward(z, d, act)
    # factors: d_out, the other half (swiglu), and slopes of at most 1.2 |.| + z-dependent terms that are
    # off by 2^-20 of themselves and of the two parts they are the sum of
    up = np.concatenate([z[:, cols:], z[:, :cols]], -1) if act == "swiglu" else 1.0
    dd = np.concatenate([d, d], -1) if act == "swiglu" else d
    e = 2.0 ** -20 * (np.abs(want) + np.abs(dd * up) * (1.0 if act != "none" else 0.0))
    assert_within(d_z.t, want, e + BF16_STEP * np.abs(want), "d_z")
    sums = want.sum(0)
    slack = e.sum(0) + rows * 2.0 ** -24 * np.abs(want).sum(0)
    assert_within(d_b.t, sums, slack, "d_bias")
    again = Guarded((N,), F32, torch.ones(N, device="cuda"))
    other = torch.empty_like(d_z.t)
    mx.moonep_act_backward(torch.from_numpy(z).to(BF16).cuda(), torch.from_numpy(d).to(BF16).cuda(), other,
                           act=act, d_bias=again.t, scratch=raw, accumulate=True)
    assert torch.equal(other.view(torch.int16), d_z.t.view(torch.int16))
    assert torch.equal(again.t, d_b.t + 1)  # the same sums, in the same order
    for g in (d_z, d_b, again, scratch):
        g.check()
    mx.moonep_act_backward(torch.from_numpy(z).to(BF16).cuda(), torch.from_numpy(d).to(BF16).cuda(), other,
                           act=act)
    assert torch.equal(other.view(torch.int16), d_z.t.view(torch.int16))
    if act == "none":
        mx.moonep_act_backward(None, torch.from_numpy(d).to(BF16).cuda(), None, d_bias=again.t, scratch=raw)
        assert torch.equal(again.t, d_b.t)


def test_act_backward_without_rows():
    e, b = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.ones(64, device="cuda")
    scratch = torch.empty(64 * 4, dtype=torch.uint8, device="cuda")
    mx.moonep_act_backward(e, e, e, act="gelu", d_bias=b, scratch=scratch, accumulate=True)
    assert bool((b == 1).all())
    mx.moonep_act_backward(e, e, e, act="gelu", d_bias=b, scratch=scratch)
    assert bool((b == 0).all())


class Plan:
    """A plan with the expert of each row of the receive buffers."""

    def __init__(self, R, E, B, K, S, H, Hp, mode=0, rows=0, alpha=1.0, seed=1):
        self.d = mx.dims(R, E, B, K, S, H, Hp, mode, 0, rows)
        self.ws = mx.PlanWorkspace(self.d)
        rt = syn.gumbel_topk_routing(R, S, K, E, alpha=alpha, seed=seed)
        self.idx, self.gates = torch.from_numpy(rt.idx).cuda(), torch.from_numpy(rt.gates).cuda()
        mx.moonep_plan(self.d, self.idx, self.ws.buf)
        t = self.ws.tables()
        assert int(t["status"][0]) == 0
        self.dst = t["dst"].reshape(R * S, K)
        self.expert = np.empty(self.d.N, np.int64)
        self.expert[self.dst.reshape(-1)] = rt.idx.reshape(-1)
        self.slot_expert = t["slot_expert"]

    def weights(self, seed=2, size=None):
        d = self.d
        home = syn.normal_bf16((d.E, d.H, d.Hp), size or d.H ** -0.5, seed).cuda()
        slot = torch.full((max(d.R * d.B, 1), d.H, d.Hp), float("nan"), dtype=BF16, device="cuda")
        if d.B:
            mx.moonep_prefetch_weights(d, self.ws.buf, home, slot)
        return home, slot if d.B else None


PLANS = [dict(R=1, E=8, B=0, K=2, S=64, H=64, Hp=128, mode=1), dict(R=2, E=8, B=4, K=2, S=200, H=128, Hp=256),
         dict(R=4, E=16, B=4, K=3, S=333, H=192, Hp=640), dict(R=4, E=16, B=1, K=2, S=150, H=256, Hp=512, mode=1),
         dict(R=8, E=64, B=8, K=4, S=128, H=128, Hp=384), dict(R=1, E=3, B=0, K=1, S=1, H=64, Hp=128, mode=1),
         dict(R=2, E=4, B=2, K=4, S=700, H=64, Hp=1024)]


# few rows a rank: the depth is split over clusters where that makes few tiles
FEW = [dict(R=1, E=14, B=0, K=2, S=1, H=2432, Hp=416 * 2, mode=1), dict(R=1, E=16, B=0, K=7, S=1, H=256, Hp=384, mode=1),
       dict(R=2, E=8, B=4, K=3, S=5, H=1024, Hp=1152), dict(R=4, E=16, B=4, K=2, S=17, H=512, Hp=640),
       dict(R=1, E=5, B=0, K=3, S=16, H=1024, Hp=3200, mode=1), dict(R=1, E=4, B=0, K=1, S=128, H=192, Hp=128, mode=1),
       dict(R=2, E=4, B=2, K=4, S=32, H=4096, Hp=256), dict(R=1, E=2, B=0, K=2, S=40, H=7168, Hp=128, mode=1),
       dict(R=8, E=64, B=8, K=8, S=1, H=4096, Hp=1024)]


@pytest.mark.parametrize("sizes", PLANS + FEW, ids=lambda s: "-".join(str(v) for v in s.values()))
@pytest.mark.parametrize("rows", [128, 256, 0])
@pytest.mark.parametrize("act,bias,z", [("swiglu", True, True), ("none", False, False), ("gelu", True, True),
                                        ("silu", False, True), ("swiglu", False, False), ("relu", True, False)])
def test_grouped_gemm_act(sizes, rows, act, bias, z):
    p = Plan(**sizes, rows=rows)
    d = p.d
    cols = d.Hp // 2 if act == "swiglu" else d.Hp
    home, slot = p.weights()
    recv = syn.normal_bf16((d.N, d.H), 1.0, 3)
    b = torch.randn(d.E, d.Hp, generator=torch.Generator().manual_seed(4)) if bias else None
    y, zz = Guarded((d.N, cols), BF16), Guarded((d.N, d.Hp), BF16) if z else None
    mx.moonep_grouped_gemm_act(d, p.ws.buf, recv.cuda(), home, slot, y.t, act=act,
                               bias=b.cuda() if bias else None, z=zz.t if z else None)
    assert mx.moonep_read_status(d, p.ws.buf) == 0
    x, w = np64(recv), np64(home)
    want_z, err = np.empty((d.N, d.Hp)), np.empty((d.N, d.Hp))
    for e in range(d.E):
        at = np.nonzero(p.expert == e)[0]
        want_z[at], err[at] = product_bounds(x[at], w[e], np64(b)[e] if bias else None, d.H)
    want, e = ffn.activation(want_z, act), act_error(want_z, act, err)
    assert_within(y.t, want, e + BF16_STEP * (np.abs(want) + e), "y")
    y.check()
    if z:
        assert_within(zz.t, want_z, err + BF16_STEP * (np.abs(want_z) + err), "z")
        zz.check()
    if act == "none" and not bias and d.C > 128:
        # bit for bit the call that it stands beside (with fewer rows a rank the depth may be split, and
        # sums in another order are as good as the bound above says)
        plain = torch.empty_like(y.t)
        mx.moonep_grouped_gemm(d, p.ws.buf, recv.cuda(), home, slot, plain)
        assert torch.equal(plain, y.t)


@pytest.mark.parametrize("sizes", PLANS, ids=lambda s: "-".join(str(v) for v in s.values()))
@pytest.mark.parametrize("act", ["gelu", "swiglu", "none"])
def test_grouped_act_backward(sizes, act):
    p = Plan(**sizes)
    d = p.d
    cols = d.Hp // 2 if act == "swiglu" else d.Hp
    z, dy = syn.normal_bf16((d.N, d.Hp), 1.5, 1), syn.normal_bf16((d.N, cols), 1.0, 2)
    d_z, d_b = Guarded((d.N, d.Hp), BF16), Guarded((d.E, d.Hp), F32)
    scratch = Guarded((mx.moonep_grouped_act_backward_workspace_bytes(d) // 4,), F32)
    raw = scratch.t.view(torch.uint8)
    mx.moonep_grouped_act_backward(d, p.ws.buf, z.cuda(), dy.cuda(), d_z.t, act=act, d_bias=d_b.t, scratch=raw)
    plain = torch.empty_like(d_z.t)
    mx.moonep_act_backward(z.cuda(), dy.cuda(), plain, act=act)
    assert torch.equal(plain.view(torch.int16), d_z.t.view(torch.int16))
    other = torch.empty_like(d_z.t)
    mx.moonep_grouped_act_backward(d, p.ws.buf, z.cuda(), dy.cuda(), other, act=act)
    assert torch.equal(other.view(torch.int16), d_z.t.view(torch.int16))
    want = ffn.activation_backward(np64(z), np64(dy), act)
    sums, size = np.zeros((d.E, d.Hp)), np.zeros((d.E, d.Hp))
    np.add.at(sums, p.expert, want)
    np.add.at(size, p.expert, np.abs(want) + np.abs(np64(dy)).max() * 10 * 2.0 ** -4)
    assert_within(d_b.t, sums, (d.N * 2.0 ** -24 + 2.0 ** -20) * size, "d_bias")
    again = Guarded((d.E, d.Hp), F32, torch.ones(d.E, d.Hp, device="cuda"))
    mx.moonep_grouped_act_backward(d, p.ws.buf, z.cuda(), dy.cuda(), other, act=act, d_bias=again.t,
                                   scratch=raw, accumulate=True)
    assert_within(again.t, sums + 1, (d.N * 2.0 ** -24 + 2.0 ** -20) * size + 2.0 ** -23, "d_bias added to")
    for g in (d_z, d_b, scratch, again):
        g.check()


COMBINE = [dict(R=1, E=8, B=0, K=2, S=3, H=64, Hp=64, mode=1), dict(R=2, E=8, B=4, K=3, S=100, H=64, Hp=1088),
           dict(R=4, E=16, B=4, K=8, S=65, H=64, Hp=4096), dict(R=1, E=40, B=0, K=17, S=70, H=64, Hp=7168, mode=1),
           dict(R=1, E=200, B=0, K=128, S=9, H=64, Hp=8192, mode=1), dict(R=1, E=8, B=0, K=1, S=1, H=64, Hp=128, mode=1)]


@pytest.mark.parametrize("sizes", COMBINE, ids=lambda s: "-".join(str(v) for v in s.values()))
@pytest.mark.parametrize("p,residual", [(0.0, False), (0.1, True), (0.5, False), (0.0, True), (0.99, True)])
def test_combine_dropout(sizes, p, residual):
    pl = Plan(**sizes)
    d, T = pl.d, pl.d.R * pl.d.S
    y, dout = syn.normal_bf16((d.N, d.Hp), 1.0, 5), syn.normal_bf16((T, d.Hp), 1.0, 6)
    r = syn.normal_bf16((T, d.Hp), 1.0, 7) if residual else None
    seed, offset = 0x123456789ABCDEF, (1 << 62) + 12345
    rng = torch.tensor([seed, offset], device="cuda") if p else None
    out, d_y, d_g = Guarded((T, d.Hp), BF16), Guarded((d.N, d.Hp), BF16), Guarded((T, d.K), F32)
    g = pl.gates.reshape(T, d.K)
    mx.moonep_combine_dropout(d, pl.ws.buf, y.cuda(), g, out.t, residual=r.cuda() if residual else None, p=p,
                              rng=rng)
    mx.moonep_combine_dropout_backward(d, pl.ws.buf, y.cuda(), g, dout.cuda(), d_y.t, d_g.t, p=p, rng=rng)
    f = ffn.dropout_factor(T * d.Hp, p, seed, offset).reshape(T, d.Hp)
    y64, g64 = np64(y), np64(g)
    res = np64(r) if residual else None
    want = ffn.combine_dropout(y64, pl.dst, g64, res, f)
    size = ffn.combine_dropout(np.abs(y64), pl.dst, np.abs(g64), None, f)
    e = (d.K + 2) * 2.0 ** -24 * size + 2.0 ** -24 * np.abs(want)
    assert_within(out.t, want, e + BF16_STEP * (np.abs(want) + e), "out")
    want_y, want_g = ffn.combine_dropout_backward(y64, pl.dst, g64, np64(dout), f)
    assert_within(d_y.t, want_y, (BF16_STEP + 2.0 ** -22) * np.abs(want_y), "d_y")
    _, size = ffn.combine_dropout_backward(np.abs(y64), pl.dst, g64, np.abs(np64(dout)), f)
    assert_within(d_g.t, want_g, (d.Hp + 2) * 2.0 ** -24 * size, "d_gates")
    for b in (out, d_y, d_g):
        b.check()
    if p == 0 and not residual:  # bit for bit the calls that it stands beside
        plain = torch.empty_like(out.t)
        mx.moonep_combine(d, pl.ws.buf, y.cuda(), g, plain)
        assert torch.equal(plain, out.t)


def test_dropped_values_are_zero_whatever_they_were():
    pl = Plan(R=1, E=8, B=0, K=2, S=64, H=64, Hp=512, mode=1)
    d, T = pl.d, 64
    y = torch.full((d.N, d.Hp), float("inf"), dtype=BF16, device="cuda")
    rng = torch.tensor([3, 4], device="cuda")
    out = torch.empty(T, d.Hp, dtype=BF16, device="cuda")
    mx.moonep_combine_dropout(d, pl.ws.buf, y, pl.gates.view(T, 2), out, p=0.5, rng=rng)
    f = ffn.dropout_factor(T * d.Hp, 0.5, 3, 4).reshape(T, d.Hp)
    assert np.array_equal(np64(out), np.where(f != 0, np.inf, 0.0))


def test_failed_plan_writes_nothing():
    pl = Plan(R=2, E=8, B=4, K=2, S=32, H=64, Hp=128)
    d, T = pl.d, 64
    bad = pl.idx.clone()
    bad[0, 0, 0] = 99
    mx.moonep_plan(d, bad, pl.ws.buf)
    home, slot = torch.zeros(8, 64, 128, dtype=BF16, device="cuda"), torch.zeros(8, 64, 128, dtype=BF16, device="cuda")
    z = torch.zeros(d.N, 128, dtype=BF16, device="cuda")
    recv = torch.zeros(d.N, 64, dtype=BF16, device="cuda")
    outs = [torch.full((n, 128), 7.0, dtype=BF16, device="cuda") for n in (d.N, d.N, T, d.N)]
    b, dg = torch.full((8, 128), 7.0, device="cuda"), torch.full((T, 2), 7.0, device="cuda")
    scratch = torch.empty(mx.moonep_grouped_act_backward_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    mx.moonep_grouped_gemm_act(d, pl.ws.buf, recv, home, slot, outs[0])
    mx.moonep_grouped_act_backward(d, pl.ws.buf, z, z, outs[1], act="silu", d_bias=b, scratch=scratch)
    mx.moonep_combine_dropout(d, pl.ws.buf, z, pl.gates.view(T, 2), outs[2])
    mx.moonep_combine_dropout_backward(d, pl.ws.buf, z, pl.gates.view(T, 2), outs[2].clone(), outs[3], dg)
    assert all(bool((t == 7).all()) for t in outs + [b, dg])
    assert mx.moonep_read_status(d, pl.ws.buf) == 0x100
