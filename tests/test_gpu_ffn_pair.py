"""The dense products on tiles of CTA pairs, and the experts' product on the narrowest of them, against
64 bits.  (Small products split the depth over clusters; that these sizes do not is tested on the host,
in test_ffn_choice_host.py.)

Bounds: as in test_gpu_ffn.py, a sum of K exact products is off by at most K 2^-23 of the sum of their
magnitudes S.  Where the output is fp32 the depth is summed in parts of 768, each off by 768 2^-23 of its own
magnitudes, and one rounding of 2^-24 S at most joins each: (768 2^-23 + parts 2^-24) S.  relu, silu and gelu
move by at most 1, 1.1 and 1.13 times what z moves by, swiglu by 1.1 |up| of the gate's and |silu(gate)| of
the up half's and 1.1 of the product of both; their own evaluation is off by 2^-20 of the result.  A bf16
rounding is off by 2^-8 of the value.
"""
import math

import pytest
import torch

import perfectly_balanced_token_gb300 as mx
import tests.test_gpu_ffn as base
from perfectly_balanced_token_gb300 import synthetic as syn
from tests.gpu_harness import ensure_library
from tests.test_gpu_ffn import BF16, F32, FLOOR, Guarded, status

pytestmark = pytest.mark.gpu

# T, K, N, columns of a tile, activations; fp32 outputs have a part for each 768 of the depth
FORWARD = [(2049, 72, 2056, 192, ("none", "gelu")), (4100, 1032, 1288, 192, ("none", "relu", "gelu", "silu")),
           (4096, 2048, 1024, 256, ("none", "relu", "gelu", "silu")), (40000, 200, 120, 128, ("none", "silu", "gelu")),
           (5000, 1032, 1296, 256, ("swiglu",)), (2500, 128, 2064, 256, ("swiglu",)), (40000, 136, 112, 128, ("swiglu",))]
FORWARD_F32 = [(8200, 1032, 376, 192, ("none",)), (4100, 1608, 2056, 192, ("none", "gelu")),
               (5000, 2056, 1032, 192, ("none", "relu", "silu")), (4096, 2048, 1024, 256, ("none", "gelu", "silu")),
               (4100, 1608, 2064, 256, ("swiglu",)), (2500, 128, 2064, 256, ("swiglu",))]
INPUT = [(4096, 2048, 1024, 256), (5000, 1032, 1288, 192), (2049, 2064, 72, 192), (4100, 2056, 200, 192),
         (40000, 120, 200, 128)]
WEIGHT = [(4096, 2048, 1024, 192), (1000, 2056, 2056, 192), (72, 2056, 2056, 192), (2000, 1032, 5000, 192),
          (1800, 3080, 2312, 256)]
EXPERTS = [dict(R=2, E=4, B=2, K=4, S=700, H=64, Hp=128), dict(R=4, E=48, B=12, K=3, S=777, H=64, Hp=64),
           dict(R=2, E=8, B=4, K=2, S=900, H=1024, Hp=128)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_library()


def within(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound + FLOOR)
    if bool(bad.any()):
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {float(got[i])}, "
                             f"want {float(want[i])} within {float(bound[i])}")


def exact_sum(x, w, f32=False):
    """x w in 64 bits and how far the kernel's sums may be from it."""
    K = x.shape[1]
    part = 768 if f32 else K
    step = min(part, K) * 2.0 ** -23 + (math.ceil(K / part) * 2.0 ** -24 if f32 else 0)
    return x.double() @ w.double(), step * (x.double().abs() @ w.double().abs())


def rounded(want, e):
    return e + 2.0 ** -8 * (want.abs() + e)


def activation(z, err, act):
    if act == "swiglu":
        f = z.shape[1] // 2
        s, u = z[:, :f] * torch.sigmoid(z[:, :f]), z[:, f:]
        eg, eu = err[:, :f], err[:, f:]
        a, e = s * u, 1.1 * eg * u.abs() + s.abs() * eu + 1.1 * eg * eu
    elif act == "gelu":
        a, e = 0.5 * z * torch.erfc(-z / math.sqrt(2)), 1.13 * err
    elif act == "silu":
        a, e = z * torch.sigmoid(z), 1.1 * err
    elif act == "relu":
        a, e = z.clamp(min=0), err
    else:
        return z, err
    return a, e + 2.0 ** -20 * a.abs()


def forward(T, K, N, act, f32, bias, residual, keep):
    cols = N // 2 if act == "swiglu" else N
    dtype = F32 if f32 else BF16
    x, w = syn.normal_bf16((T, K), 1.0, 1).cuda(), syn.normal_bf16((K, N), K ** -0.5, 2).cuda()
    b = torch.randn(N, generator=torch.Generator().manual_seed(3)).cuda() if bias else None
    r = syn.normal_bf16((T, cols), 1.0, 4).cuda() if residual else None
    out, z = Guarded((T, cols), dtype), Guarded((T, N), BF16) if keep else None
    st, ld = status(), mx.linear_dims(T, K, N, act=act, out_dtype=dtype)
    mx.moonep_linear(ld, x, w, out.t, st, bias=b, residual=r, z=z.t if keep else None)
    want_z, err = exact_sum(x, w, f32)
    if bias:
        want_z = want_z + b.double()
        err = err + 2.0 ** -24 * (want_z.abs() + err)
    want, e = activation(want_z, err, act)
    if residual:
        want = want + r.double()
        e = e + 2.0 ** -24 * (want.abs() + e)
    within(out.t, want, e if f32 else rounded(want, e), "out")
    out.check()
    if keep:
        within(z.t, want_z, rounded(want_z, err), "z")
        z.check()
    again = torch.empty_like(out.t)
    mx.moonep_linear(ld, x, w, again, st, bias=b, residual=r, z=z.t if keep else None)
    assert torch.equal(again, out.t) and int(st) == 0


def cases(table):
    return [(T, K, N, act) for T, K, N, _, acts in table for act in acts]


@pytest.mark.parametrize("T,K,N,act", cases(FORWARD))
@pytest.mark.parametrize("bias,residual,keep", [(False, False, False), (True, True, True), (True, False, True),
                                                (False, True, False)])
def test_linear(T, K, N, act, bias, residual, keep):
    forward(T, K, N, act, False, bias, residual, keep)


@pytest.mark.parametrize("T,K,N,act", cases(FORWARD_F32))
@pytest.mark.parametrize("bias,residual,keep", [(False, False, False), (True, True, True), (True, False, True)])
def test_linear_in_32_bits(T, K, N, act, bias, residual, keep):
    forward(T, K, N, act, True, bias, residual, keep)


@pytest.mark.parametrize("T,K,N", [s[:3] for s in INPUT])
def test_input_gradient(T, K, N):
    w, d = syn.normal_bf16((K, N), 1.0, 1).cuda(), syn.normal_bf16((T, N), 1.0, 2).cuda()
    d_x, st, ld = Guarded((T, K), BF16), status(), mx.linear_dims(T, K, N)
    mx.moonep_linear_dx(ld, d, w, d_x.t, st)
    want, e = exact_sum(d, w.t())
    within(d_x.t, want, rounded(want, e), "d_x")
    again = torch.empty_like(d_x.t)
    mx.moonep_linear_dx(ld, d, w, again, st)
    assert torch.equal(again, d_x.t) and int(st) == 0
    d_x.check()


@pytest.mark.parametrize("T,K,N", [s[:3] for s in WEIGHT])
def test_weight_gradient(T, K, N):
    x, d = syn.normal_bf16((T, K), 1.0, 1).cuda(), syn.normal_bf16((T, N), 1.0, 2).cuda()
    d_w, st, ld = Guarded((K, N), F32), status(), mx.linear_dims(T, K, N)
    mx.moonep_linear_dw(ld, x, d, d_w.t, st)
    want, e = exact_sum(x.t(), d, True)
    within(d_w.t, want, e, "d_w")
    start = torch.randn(K, N, generator=torch.Generator().manual_seed(9)).cuda()
    acc = Guarded((K, N), F32, start)
    mx.moonep_linear_dw(ld, x, d, acc.t, st, accumulate=True)
    assert torch.equal(acc.t, start + d_w.t)  # one addition to the same sums
    again = torch.empty_like(d_w.t)
    mx.moonep_linear_dw(ld, x, d, again, st)
    assert torch.equal(again, d_w.t) and int(st) == 0
    for g in (d_w, acc):
        g.check()


def test_a_status_stops_the_stores():
    st = torch.full((1,), 0x400, dtype=torch.int32, device="cuda")
    for T, K, N, _, acts in FORWARD + FORWARD_F32:
        x, w = torch.ones(T, K, dtype=BF16, device="cuda"), torch.ones(K, N, dtype=BF16, device="cuda")
        cols = N // 2 if acts[0] == "swiglu" else N
        dtype = F32 if (T, K, N, _, acts) in FORWARD_F32 else BF16
        out, z = torch.full((T, cols), 7.0, dtype=dtype, device="cuda"), torch.full((T, N), 7.0, dtype=BF16, device="cuda")
        mx.moonep_linear(mx.linear_dims(T, K, N, act=acts[0], out_dtype=dtype), x, w, out, st, z=z)
        assert bool((out == 7).all()) and bool((z == 7).all())
    for T, K, N, _ in INPUT:
        d_x = torch.full((T, K), 7.0, dtype=BF16, device="cuda")
        mx.moonep_linear_dx(mx.linear_dims(T, K, N), torch.ones(T, N, dtype=BF16, device="cuda"),
                            torch.ones(K, N, dtype=BF16, device="cuda"), d_x, st)
        assert bool((d_x == 7).all())
    for T, K, N, _ in WEIGHT:
        d_w = torch.full((K, N), 7.0, device="cuda")
        for add in (False, True):
            mx.moonep_linear_dw(mx.linear_dims(T, K, N), torch.ones(T, K, dtype=BF16, device="cuda"),
                                torch.ones(T, N, dtype=BF16, device="cuda"), d_w, st, accumulate=add)
        assert bool((d_w == 7).all())
    assert int(st) == 0x400


@pytest.mark.parametrize("T,K,N,act", [(4100, 1032, 1288, "none"), (40000, 200, 120, "relu"), (4096, 2048, 1024, "silu"),
                                       (2500, 128, 2064, "swiglu")])
def test_infinities_and_nan_stay_in_their_row_or_column(T, K, N, act):
    x, w = syn.normal_bf16((T, K), 1.0, 1).cuda(), syn.normal_bf16((K, N), 1.0, 2).cuda()
    clean = torch.empty(T, N // 2 if act == "swiglu" else N, dtype=BF16, device="cuda")
    out, z, st, ld = torch.empty_like(clean), torch.empty(T, N, dtype=BF16, device="cuda"), status(), mx.linear_dims(T, K, N, act=act)
    mx.moonep_linear(ld, x, w, clean, st)
    x[T - 1, 5], x[300, K - 1], w[7, 11] = float("nan"), float("inf"), float("nan")
    mx.moonep_linear(ld, x, w, out, st, z=z)
    bad = torch.zeros(T, N, dtype=torch.bool, device="cuda")
    bad[T - 1], bad[300], bad[:, 11] = True, True, True
    assert torch.equal(~torch.isfinite(z), bad)
    same = ~bad[:, :clean.shape[1]]
    assert torch.equal(out[same], clean[same])
    assert bool(torch.isnan(out[T - 1]).all()) and bool(torch.isnan(out[:, 11]).all())


def test_infinities_and_nan_in_the_gradients():
    T, K, N = 5000, 1032, 1288  # the input gradient's; of the weight's x and d_z change places
    w, d = syn.normal_bf16((K, N), 1.0, 1).cuda(), syn.normal_bf16((T, N), 1.0, 2).cuda()
    d[4999, 1287], w[1031, 0] = float("nan"), float("inf")
    d_x = torch.empty(T, K, dtype=BF16, device="cuda")
    mx.moonep_linear_dx(mx.linear_dims(T, K, N), d, w, d_x, status())
    bad = torch.zeros(T, K, dtype=torch.bool, device="cuda")
    bad[4999], bad[:, 1031] = True, True
    assert torch.equal(~torch.isfinite(d_x), bad)
    T, K, N = 1000, 2056, 2056
    x, d = syn.normal_bf16((T, K), 1.0, 1).cuda(), syn.normal_bf16((T, N), 1.0, 2).cuda()
    x[999, 2055], d[0, 3] = float("nan"), float("inf")
    d_w = torch.empty(K, N, device="cuda")
    mx.moonep_linear_dw(mx.linear_dims(T, K, N), x, d, d_w, status())
    bad = torch.zeros(K, N, dtype=torch.bool, device="cuda")
    bad[2055], bad[:, 3] = True, True
    assert torch.equal(~torch.isfinite(d_w), bad)


@pytest.mark.parametrize("sizes", EXPERTS, ids=lambda s: "-".join(str(v) for v in s.values()))
@pytest.mark.parametrize("rows", [128, 256, 0])
@pytest.mark.parametrize("act,bias,z", [("swiglu", True, True), ("none", False, False), ("gelu", True, True),
                                        ("relu", True, False), ("swiglu", False, False)])
def test_experts_on_the_narrowest_tiles(sizes, rows, act, bias, z):
    base.test_grouped_gemm_act(sizes, rows, act, bias, z)
