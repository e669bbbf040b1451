"""MXFP4 on the GPU against the 64-bit definition: codes, scales and values
exactly; the grouped product within the error of its fp32 sums and bf16 result.

Bound of the product: products of codes and scales are exact; an fp32 sum over
H/64 instructions is off by at most (H/64 + 1) 2^-22 of the sum of magnitudes
(each instruction rounds or cuts once, twice the unit for the sum inside it), and
the bf16 result by 2^-9 of itself (2^-8 is used: the sum's error moves it).
"""
import numpy as np
import pytest
import torch

import perfectly_balanced_token_gb300 as mx
from oracle import ops
from perfectly_balanced_token_gb300 import synthetic as syn
from tests.gpu_harness import ensure_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_library()


def bf16(x) -> torch.Tensor:
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def rows_with_everything(rows, cols, seed):
    """Values over all bf16 exponents, ties, zeros of both signs, infinities, NaN."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-30, 30, (rows, cols // 32)).repeat(32, 1))
    grid = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7, 7.9, 0.0], (rows, cols))
    x = np.where(rng.random((rows, 1)) < 0.4, grid * rng.choice([-1.0, 1.0], (rows, cols)), x)
    t = bf16(x)
    if rows > 3:
        t[1] = 0.0
        t[2] *= 2.0 ** -120  # subnormal values and the smallest scales
        t[0, :32] = torch.tensor([3e38, -1e-38] * 16, dtype=torch.bfloat16)
        t[3, cols - 1] = float("nan")
        t[3, 5] = float("-inf")
    return t


@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 64), (3, 96), (7, 512), (5, 544), (64, 1088),
                                       (33, 7168), (3000, 480), (2, 16384)])
def test_quantize_and_back(rows, cols):
    x = rows_with_everything(rows, cols, rows + cols)
    codes = torch.full((rows, cols // 2), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, mx.mxfp4_scale_pitch(cols)), 0xEE, dtype=torch.uint8, device="cuda")
    mx.moonep_mxfp4_quantize(x.cuda(), codes, scales)
    want_c, want_s = ops.mxfp4_quantize(x.double().numpy())
    assert np.array_equal(codes.cpu().numpy(), want_c)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    back = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    mx.moonep_mxfp4_dequantize(codes, scales, back)
    assert np.array_equal(back.double().cpu().numpy(), ops.mxfp4_values(want_c, want_s),
                          equal_nan=True)


def test_every_code_and_scale_back():
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)  # 512 values a row
    s = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16)
    out = torch.empty(256, 512, dtype=torch.bfloat16, device="cuda")
    mx.moonep_mxfp4_dequantize(codes.cuda(), s.cuda(), out)
    want = ops.mxfp4_values(codes.numpy(), s.numpy())
    want = np.where(np.abs(want) > 3.3895e38, np.sign(want) * np.inf, want)
    assert np.array_equal(out.double().cpu().numpy(), want, equal_nan=True)


def test_offsets_past_32_bits():
    rows, cols = 640_000, 7168  # 4.6e9 values
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = rows_with_everything(4, cols, 1)
    x[-4:] = tail.cuda()
    codes = torch.full((rows, cols // 2), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, mx.mxfp4_scale_pitch(cols)), 0xEE, dtype=torch.uint8, device="cuda")
    mx.moonep_mxfp4_quantize(x, codes, scales)
    want_c, want_s = ops.mxfp4_quantize(tail.double().numpy())
    assert np.array_equal(codes[-4:].cpu().numpy(), want_c)
    assert np.array_equal(scales[-4:].cpu().numpy(), want_s)
    assert not codes[:-4].any() and not scales[:-4].any()
    x.fill_(7.0)
    mx.moonep_mxfp4_dequantize(codes, scales, x)
    assert np.array_equal(x[-4:].double().cpu().numpy(), ops.mxfp4_values(want_c, want_s),
                          equal_nan=True)
    assert not x[:-4].any()


def test_product_with_offsets_past_32_bits():
    # 1.3 million rows of 3584 bytes of codes; the last rows' outputs against the definition
    w = syn.Workload("long", R=1, E=2, B=0, K=1, S=1_300_000, H=7168, Hp=64, mode=1)
    d = mx.dims(w.R, w.E, w.B, w.K, w.S, w.H, w.Hp, w.mode)
    ids = torch.ones(w.N, dtype=torch.int32, device="cuda")
    ids[: w.N // 2] = 0
    ws = mx.PlanWorkspace(d)
    mx.moonep_plan(d, ids, ws.buf)
    x = torch.zeros(w.S, w.H, dtype=torch.bfloat16, device="cuda")
    tail = syn.normal_bf16((6, w.H), 1.0, 5)
    x[-6:] = tail.cuda()
    wt = syn.normal_bf16((2, w.H, w.Hp), 0.05, 6)
    u8 = dict(dtype=torch.uint8, device="cuda")
    pitch = mx.mxfp4_scale_pitch(w.H)
    hq, hs = torch.empty(2, w.Hp, w.H // 2, **u8), torch.empty(2, w.Hp, pitch, **u8)
    mx.moonep_mxfp4_quantize_weights(wt.cuda(), hq, hs)
    rq, rs = torch.full((w.N, w.H // 2), 0xEE, **u8), torch.full((w.N, pitch), 0xEE, **u8)
    y = torch.full((w.N, w.Hp), 7.0, dtype=torch.bfloat16, device="cuda")
    mx.moonep_mxfp4_dispatch(d, ws.buf, x, rq, rs)
    mx.moonep_mxfp4_grouped_gemm(d, ws.buf, rq, rs, hq, hs, None, None, y)
    torch.cuda.synchronize()
    assert mx.moonep_read_status(d, ws.buf) == 0
    xv = ops.mxfp4_values(*ops.mxfp4_quantize(tail.double().numpy()))
    wv = ops.mxfp4_values(*ops.mxfp4_quantize(wt[1].double().numpy().T.copy()))
    want, size = xv @ wv.T, np.abs(xv) @ np.abs(wv.T)
    err = np.abs(y[-6:].double().cpu().numpy() - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + (w.H / 64 + 1) * 2.0 ** -22 * size).all()
    assert not y[:-6].any()


def test_no_rows():
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    u = torch.empty(0, 32, dtype=torch.uint8, device="cuda")
    s = torch.empty(0, 16, dtype=torch.uint8, device="cuda")
    mx.moonep_mxfp4_quantize(e, u, s)
    mx.moonep_mxfp4_dequantize(u, s, e)


@pytest.mark.parametrize("n,H,Hp", [(1, 64, 64), (3, 192, 128), (2, 256, 320), (2, 1088, 64),
                                    (5, 448, 192)])
def test_quantize_weights(n, H, Hp):
    w = rows_with_everything(n * H, Hp, n + H).view(n, H, Hp)
    codes = torch.full((n, Hp, H // 2), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((n, Hp, mx.mxfp4_scale_pitch(H)), 0xEE, dtype=torch.uint8, device="cuda")
    mx.moonep_mxfp4_quantize_weights(w.cuda(), codes, scales)
    want_c, want_s = ops.mxfp4_quantize(w.double().transpose(1, 2).reshape(n * Hp, H).numpy())
    assert np.array_equal(codes.cpu().numpy().reshape(n * Hp, -1), want_c)
    assert np.array_equal(scales.cpu().numpy().reshape(n * Hp, -1), want_s)


# ------------------------------------------------------------------------- the layer's calls
def guarded(n, dtype=torch.uint8, pad=256):
    t = torch.full((n + 2 * pad,), 0x5A, dtype=torch.uint8, device="cuda") if dtype == torch.uint8 \
        else torch.full((n + 2 * pad,), -77.0, dtype=dtype, device="cuda")
    return t, t[pad:pad + n]


def untouched(t, n, pad=256):
    v = t[:pad].float()
    assert bool((v == v[0]).all()) and bool((t[pad + n:].float() == v[0]).all())


def run_layer(w, idx, gemm_rows, x=None, wt=None, seed=3):
    """plan, prefetch, dispatch and product; returns what the checks need."""
    d = mx.dims(w.R, w.E, w.B, w.K, w.S, w.H, w.Hp, w.mode, 0, gemm_rows)
    pitch = mx.mxfp4_scale_pitch(w.H)
    x = syn.normal_bf16((w.R * w.S, w.H), 1.0, seed) if x is None else x
    wt = syn.normal_bf16((w.E, w.H, w.Hp), 0.05, seed + 1) if wt is None else wt
    home_q = torch.empty(w.E, w.Hp, w.H // 2, dtype=torch.uint8, device="cuda")
    home_s = torch.empty(w.E, w.Hp, pitch, dtype=torch.uint8, device="cuda")
    mx.moonep_mxfp4_quantize_weights(wt.cuda(), home_q, home_s)
    nb = w.R * w.B * w.Hp
    slot_q = torch.full((nb * (w.H // 2),), 0xFF, dtype=torch.uint8, device="cuda") if w.B else None
    slot_s = torch.full((nb * pitch,), 0xFF, dtype=torch.uint8, device="cuda") if w.B else None
    rq_full, rq = guarded(w.N * (w.H // 2))
    rs_full, rs = guarded(w.N * pitch)
    y_full, y = guarded(w.N * w.Hp, torch.bfloat16)
    ws = mx.PlanWorkspace(d)
    mx.moonep_plan(d, torch.from_numpy(np.ascontiguousarray(idx)).cuda(), ws.buf)
    mx.moonep_mxfp4_prefetch_weights(d, ws.buf, home_q, home_s, slot_q, slot_s)
    mx.moonep_mxfp4_dispatch(d, ws.buf, x.cuda(), rq, rs)
    mx.moonep_mxfp4_grouped_gemm(d, ws.buf, rq, rs, home_q, home_s, slot_q, slot_s, y)
    torch.cuda.synchronize()
    assert mx.moonep_read_status(d, ws.buf) == 0
    untouched(rq_full, rq.numel())
    untouched(rs_full, rs.numel())
    untouched(y_full, y.numel())
    tabs = ws.tables()
    return dict(d=d, ws=ws, tabs=tabs, x=x, wt=wt, rq=rq, rs=rs, y=y, slot_q=slot_q, slot_s=slot_s,
                home_q=home_q, home_s=home_s)


def check_layer(w, idx, r):
    inv = r["tabs"]["inverse"]  # copy of each row
    token, expert = inv // w.K, idx.reshape(-1)[inv]
    xc, xs = ops.mxfp4_quantize(r["x"].double().numpy())
    assert np.array_equal(r["rq"].cpu().numpy().reshape(w.N, -1), xc[token])
    assert np.array_equal(r["rs"].cpu().numpy().reshape(w.N, -1), xs[token])
    xv = ops.mxfp4_values(xc, xs)
    if w.B:  # occupied slots hold their experts' rows, the others what they held
        slots = r["tabs"]["slot_expert"].reshape(-1)
        sq = r["slot_q"].view(w.R * w.B, -1)
        for s, e in enumerate(slots):
            if e >= 0:
                assert torch.equal(sq[s], r["home_q"][e].reshape(-1))
                assert torch.equal(r["slot_s"].view(w.R * w.B, -1)[s], r["home_s"][e].reshape(-1))
            else:
                assert bool((sq[s] == 0xFF).all())
    y = r["y"].double().cpu().numpy().reshape(w.N, w.Hp)
    for e in np.unique(expert):
        at = np.nonzero(expert == e)[0]
        wc, wsc = ops.mxfp4_quantize(r["wt"][e].double().numpy().T.copy())
        wv = ops.mxfp4_values(wc, wsc)
        want = xv[token[at]] @ wv.T
        size = np.abs(xv[token[at]]) @ np.abs(wv.T)
        tol = 2.0 ** -8 * np.abs(want) + (w.H / 64 + 1) * 2.0 ** -22 * size + 1e-30
        err = np.abs(y[at] - want)
        assert np.array_equal(np.isnan(y[at]), np.isnan(want)), f"expert {e}"
        ok = (err <= tol) | np.isnan(want)
        assert ok.all(), (f"expert {e}", int((~ok).sum()), np.nanmax(err), np.nanmax(err / tol))


def routed(w, seed, alpha=0.6):
    return syn.gumbel_topk_routing(w.R, w.S, w.K, w.E, alpha=alpha, seed=seed).idx


# one token on one rank to several tiles a group; widths inside and past one tile and
# one stage (K of 256), N of 64 to more than 256; slots used, missing and overflowing
WORKLOADS = [
    syn.Workload("one", R=1, E=4, B=0, K=1, S=1, H=64, Hp=64, mode=1),
    syn.Workload("one-all", R=1, E=4, B=0, K=4, S=1, H=256, Hp=256, mode=1),
    syn.Workload("short", R=2, E=4, B=2, K=2, S=5, H=128, Hp=128),
    syn.Workload("tail", R=2, E=6, B=3, K=3, S=67, H=192, Hp=320),
    syn.Workload("one-stage", R=1, E=3, B=0, K=1, S=300, H=256, Hp=512, mode=1),
    syn.Workload("odd", R=4, E=12, B=3, K=3, S=111, H=1088, Hp=320),
    syn.Workload("overflow", R=4, E=16, B=1, K=2, S=200, H=448, Hp=192, mode=1),
    syn.Workload("no-slots", R=4, E=16, B=0, K=2, S=200, H=576, Hp=256, mode=1),
    syn.Workload("deep", R=2, E=4, B=2, K=2, S=256, H=4160, Hp=512),
    syn.Workload("wide", R=2, E=8, B=4, K=2, S=700, H=512, Hp=1088),
    syn.Workload("many-k", R=2, E=48, B=24, K=40, S=30, H=128, Hp=64),
]


@pytest.mark.parametrize("gemm_rows", [0, 128, 256])
@pytest.mark.parametrize("w", WORKLOADS, ids=lambda w: w.name)
def test_layer_calls(w, gemm_rows):
    idx = routed(w, 5)
    check_layer(w, idx, run_layer(w, idx, gemm_rows))


@pytest.mark.parametrize("gemm_rows", [128, 256])
def test_skewed_routing_uses_the_slots(gemm_rows):
    w = syn.SMALL
    idx = syn.routing_for(w, 5.0, seed=0).idx
    r = run_layer(w, idx, gemm_rows)
    assert (r["tabs"]["slot_expert"] >= 0).any()
    check_layer(w, idx, r)


@pytest.mark.parametrize("gemm_rows", [128, 256])
def test_what_is_not_finite_stays_in_its_row_and_column(gemm_rows):
    w = syn.Workload("nan", R=2, E=4, B=2, K=2, S=90, H=320, Hp=192)
    idx = routed(w, 1)
    x = syn.normal_bf16((w.R * w.S, w.H), 1.0, 1)
    x[7, 200] = float("nan")
    x[50, 319] = float("inf")
    wt = syn.normal_bf16((w.E, w.H, w.Hp), 0.05, 2)
    wt[2, 33, 100] = float("-inf")
    r = run_layer(w, idx, gemm_rows, x, wt)
    check_layer(w, idx, r)


def test_largest_and_smallest_scales():
    w = syn.Workload("scales", R=1, E=2, B=0, K=1, S=40, H=128, Hp=64, mode=1)
    rng = np.random.default_rng(0)
    x = bf16(rng.standard_normal((40, 128)) * np.exp2(rng.integers(-100, 60, (40, 4)).repeat(32, 1)))
    wt = bf16(rng.standard_normal((2, 128, 64)) * np.exp2(rng.integers(-30, 60, (2, 4, 1)).repeat(32, 1)))
    idx = rng.integers(0, 2, (1, 40, 1)).astype(np.int32)
    check_layer(w, idx, run_layer(w, idx, 0, x, wt))


def test_same_bits_again_and_on_another_stream_and_in_a_graph():
    w = syn.Workload("again", R=2, E=8, B=4, K=2, S=500, H=704, Hp=512)
    idx = routed(w, 9)
    r = run_layer(w, idx, 0)
    d, first = r["d"], r["y"].clone()
    args = (d, r["ws"].buf, r["rq"], r["rs"], r["home_q"], r["home_s"], r["slot_q"], r["slot_s"], r["y"])
    r["y"].zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mx.moonep_mxfp4_grouped_gemm(*args, stream=side)
    side.synchronize()
    assert torch.equal(first, r["y"])
    r["y"].zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.moonep_mxfp4_grouped_gemm(*args)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, r["y"])


@pytest.mark.parametrize("S,E,K,H,Hp,launches", [(16, 96, 8, 7168, 2048, 2000),
                                                 (2400, 64, 4, 4096, 1024, 2000),
                                                 (300, 12, 3, 1088, 320, 3000)])
def test_launch_after_launch_gives_the_same_bits(S, E, K, H, Hp, launches):
    # rows and scales that differ from stage to stage: a stage that takes another's shows
    d = mx.dims(1, E, 0, K, S, H, Hp, 1)
    g = torch.Generator(device="cuda").manual_seed(S)
    ids = torch.topk(torch.randn(S, E, generator=g, device="cuda"), K).indices.int()
    ws = mx.PlanWorkspace(d)
    mx.moonep_plan(d, ids, ws.buf)
    pitch = mx.mxfp4_scale_pitch(H)

    def codes_and_scales(rows):
        q = torch.randint(0, 256, (rows, H // 2), generator=g, device="cuda", dtype=torch.uint8)
        s = torch.randint(120, 130, (rows, pitch), generator=g, device="cuda", dtype=torch.uint8)
        return q, s

    rq, rs = codes_and_scales(d.N)
    hq, hs = codes_and_scales(E * Hp)
    y = torch.empty(d.N, Hp, dtype=torch.bfloat16, device="cuda")
    run = lambda: mx.moonep_mxfp4_grouped_gemm(d, ws.buf, rq, rs, hq, hs, None, None, y)  # noqa: E731
    run()
    first = y.clone()
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(launches):
        run()
        differ += (y != first).any()
    assert int(differ) == 0 and mx.moonep_read_status(d, ws.buf) == 0


def test_a_failed_plan_writes_nothing():
    w = syn.TINY
    d = mx.dims(w.R, w.E, w.B, w.K, w.S, w.H, w.Hp)
    bad = syn.bad_routing_duplicate(w.R, w.S, w.K, w.E)
    ws = mx.PlanWorkspace(d)
    mx.moonep_plan(d, torch.from_numpy(bad).cuda(), ws.buf)
    pitch = mx.mxfp4_scale_pitch(w.H)
    u8 = dict(dtype=torch.uint8, device="cuda")
    hq, hs = torch.zeros(w.E * w.Hp * w.H // 2, **u8), torch.zeros(w.E * w.Hp * pitch, **u8)
    sq = torch.full((w.R * w.B * w.Hp * w.H // 2,), 9, **u8)
    ss = torch.full((w.R * w.B * w.Hp * pitch,), 9, **u8)
    rq, rs = torch.full((w.N * w.H // 2,), 9, **u8), torch.full((w.N * pitch,), 9, **u8)
    y = torch.full((w.N * w.Hp,), 9.0, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(w.R * w.S * w.H, dtype=torch.bfloat16, device="cuda")
    mx.moonep_mxfp4_prefetch_weights(d, ws.buf, hq, hs, sq, ss)
    mx.moonep_mxfp4_dispatch(d, ws.buf, x, rq, rs)
    mx.moonep_mxfp4_grouped_gemm(d, ws.buf, rq, rs, hq, hs, sq, ss, y)
    torch.cuda.synchronize()
    assert mx.moonep_read_status(d, ws.buf) == mx._lib.ERR_ROUTING
    for t in (sq, ss, rq, rs, y):
        assert bool((t == 9).all())


@pytest.mark.parametrize("gemm_rows", [128, 256])
def test_workspace_at_any_multiple_of_16(gemm_rows):
    # groups that end inside tiles, so tensor maps are edited in the workspace
    w = syn.Workload("offset", R=2, E=8, B=4, K=2, S=500, H=512, Hp=512)
    idx = routed(w, 9)
    r = run_layer(w, idx, gemm_rows)
    d, n = r["d"], r["ws"].buf.numel()
    x = r["x"].cuda()
    for offset in (16, 112):
        ws = torch.zeros(n + 256, dtype=torch.uint8, device="cuda")[offset:offset + n]
        mx.moonep_plan(d, torch.from_numpy(np.ascontiguousarray(idx)).cuda(), ws)
        y = torch.full_like(r["y"], 7.0)
        mx.moonep_mxfp4_grouped_gemm(d, ws, r["rq"], r["rs"], r["home_q"], r["home_s"], r["slot_q"],
                                     r["slot_s"], y)
        assert torch.equal(y, r["y"])
        # the bf16 weight gradient, on the same plan in both workspaces
        recv = torch.empty(w.N * w.H, dtype=torch.bfloat16, device="cuda")
        mx.moonep_dispatch(d, ws, x, recv)
        got = []
        for buf in (r["ws"].buf, ws):
            g_home = torch.zeros(w.E * w.H * w.Hp, device="cuda")
            g_slot = torch.zeros(w.R * w.B * w.H * w.Hp, device="cuda")
            mx.moonep_grouped_gemm_dw(d, buf, recv, y, g_home, g_slot)
            got.append((g_home, g_slot))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
        assert mx.moonep_read_status(d, ws) == 0


def test_whole_layer_repeats_itself_between_other_inputs():
    # from the router's logits to the combined output, on the same buffers with other inputs
    # between: bit for bit, and the gated sum of its own y to within the rounding of the output
    # (K + 1 fp32 roundings of the sum of magnitudes and 2^-9 of the value)
    w = syn.Workload("layer", R=4, E=16, B=4, K=3, S=300, H=512, Hp=320)
    T, pitch = w.R * w.S, mx.mxfp4_scale_pitch(w.H)
    d, rd = mx.dims(w.R, w.E, w.B, w.K, w.S, w.H, w.Hp), mx.router_dims(T, w.E, w.K, w.S)
    ws = mx.PlanWorkspace(d)
    u8 = dict(dtype=torch.uint8, device="cuda")
    home = torch.empty(w.E * w.Hp, w.H // 2, **u8), torch.empty(w.E * w.Hp, pitch, **u8)
    mx.moonep_mxfp4_quantize_weights(syn.normal_bf16((w.E, w.H, w.Hp), 0.05, 4).cuda(), *home)
    nb = w.R * w.B * w.Hp
    slot = torch.empty(nb, w.H // 2, **u8), torch.empty(nb, pitch, **u8)
    recv = torch.empty(w.N, w.H // 2, **u8), torch.empty(w.N, pitch, **u8)
    rws = torch.empty(mx.moonep_router_workspace_bytes(rd), **u8)
    idx = torch.empty(T, w.K, dtype=torch.int32, device="cuda")
    gates = torch.empty(T, w.K, device="cuda")
    balance = dict(counts=torch.empty(w.R, w.E, dtype=torch.int32, device="cuda"),
                   prob_sum=torch.empty(w.R, w.E, device="cuda"),
                   seg_tokens=torch.empty(w.R, dtype=torch.int32, device="cuda"),
                   loss=torch.empty(1, device="cuda"))
    y = torch.empty(w.N, w.Hp, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(T, w.Hp, dtype=torch.bfloat16, device="cuda")

    def layer(seed):
        g = torch.Generator().manual_seed(seed)
        skew = 0.7 * torch.log1p(torch.arange(w.E).float())
        logits = (torch.randn(T, w.E, generator=g) - skew).cuda()
        x = syn.normal_bf16((T, w.H), 1.0, seed).cuda()
        mx.moonep_router_forward(rd, logits, idx, gates, ws=rws, **balance)
        mx.moonep_plan(d, idx, ws.buf)
        mx.moonep_mxfp4_prefetch_weights(d, ws.buf, *home, *slot)
        mx.moonep_mxfp4_dispatch(d, ws.buf, x, *recv)
        mx.moonep_mxfp4_grouped_gemm(d, ws.buf, *recv, *home, *slot, y)
        mx.moonep_combine(d, ws.buf, y, gates, out)
        return [t.clone() for t in (idx, gates, *balance.values(), y, out)]

    first = layer(1)
    rows = ws.tables()["dst"].reshape(T, w.K)
    terms = y.double().cpu().numpy()[rows] * gates.double().cpu().numpy()[..., None]
    want, size = terms.sum(1), np.abs(terms).sum(1)
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + (w.K + 1) * 2.0 ** -24 * size).all()
    for other in (2, 3):
        layer(other)
        assert all(torch.equal(a, b) for a, b in zip(first, layer(1)))
    assert mx.moonep_read_status(d, ws.buf) == 0


@pytest.mark.parametrize("name,R,E,B,K,S,H,Hp", [("narrow", 2, 6, 3, 3, 67, 384, 320),
                                                 ("wide", 4, 16, 4, 2, 300, 512, 256)])
def test_gradients_of_the_quantised_product(name, R, E, B, K, S, H, Hp):
    """moonep_grouped_gemm_dx and _dw on the dequantised operands, as the header describes, against
    the chain rule in 64 bits through y = recv_q W_q^T.  fp32 sums of n terms: n 2^-24 of the sum
    of magnitudes (twice that is allowed), the bf16 input gradient 2^-8 of itself."""
    w = syn.Workload(name, R=R, E=E, B=B, K=K, S=S, H=H, Hp=Hp)
    idx = routed(w, 4)
    r = run_layer(w, idx, 0)
    d, ws, bf = r["d"], r["ws"].buf, torch.bfloat16
    recv = torch.empty(w.N, H, dtype=bf, device="cuda")
    mx.moonep_mxfp4_dequantize(r["rq"], r["rs"], recv)
    turned = torch.empty(E, Hp, H, dtype=bf, device="cuda")
    mx.moonep_mxfp4_dequantize(r["home_q"], r["home_s"], turned)
    w_home = turned.transpose(1, 2).contiguous()
    w_slot = torch.zeros(R * B * H * Hp, dtype=bf, device="cuda")
    mx.moonep_prefetch_weights(d, ws, w_home, w_slot)
    rng = np.random.default_rng(1)
    gates = torch.from_numpy(rng.random(w.N).astype(np.float32)).cuda()
    d_out = syn.normal_bf16((R * S, Hp), 1.0, 8).cuda()
    d_y, d_gates = torch.empty_like(r["y"]).contiguous(), torch.empty(w.N, device="cuda")
    mx.moonep_combine_backward(d, ws, r["y"], gates, d_out, d_y, d_gates)
    d_recv = torch.empty(w.N, H, dtype=bf, device="cuda")
    mx.moonep_grouped_gemm_dx(d, ws, d_y, w_home, w_slot, d_recv)
    g_home = torch.zeros(E, H, Hp, device="cuda")
    g_slot = torch.zeros(R * B * H * Hp, device="cuda")
    mx.moonep_grouped_gemm_dw(d, ws, recv, d_y, g_home, g_slot)
    mx.moonep_reduce_grad(d, ws, g_home, g_slot)
    assert mx.moonep_read_status(d, ws) == 0
    inv = r["tabs"]["inverse"]
    token, expert = inv // K, idx.reshape(-1)[inv]
    xv = ops.mxfp4_values(*ops.mxfp4_quantize(r["x"].double().numpy()))[token]
    dy = d_y.double().cpu().numpy().reshape(w.N, Hp)
    want_dy = gates.double().cpu().numpy()[inv, None] * d_out.double().cpu().numpy()[token]
    assert (np.abs(dy - want_dy) <= 2.0 ** -8 * np.abs(want_dy)).all()
    dx, dw = d_recv.double().cpu().numpy(), g_home.double().cpu().numpy()
    for e in range(E):
        at = np.nonzero(expert == e)[0]
        wv = ops.mxfp4_values(*ops.mxfp4_quantize(r["wt"][e].double().numpy().T.copy()))
        want, size = dy[at] @ wv, np.abs(dy[at]) @ np.abs(wv)
        assert (np.abs(dx[at] - want) <= 2.0 ** -8 * np.abs(want) + Hp * 2.0 ** -23 * size).all(), e
        want, size = xv[at].T @ dy[at], np.abs(xv[at].T) @ np.abs(dy[at])
        assert (np.abs(dw[e] - want) <= (len(at) + 8) * 2.0 ** -23 * size).all(), e
