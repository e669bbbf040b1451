"""The router on the GPU against its 64-bit definition: ids, counts and token
numbers exactly; gates, sums, loss and gradient within bounds derived below.

Rounding: an exponential of x is off by at most (3 + 1.2 |x|) 2^-23 of itself
(|x| <= 40 here where it counts: 51 ulp = 6.1e-6), a sum of n terms by n 2^-24
of the sum of magnitudes in the worst order (a lane adds at most 128 of them and
5 levels across the warp: 8e-6).  A gate takes an exponential, a sum and a
division: RTOL = 2e-5 covers 6.1e-6 twice and 8e-6.  The balance sums also
round each warp's part to 2^-shift, shift = 46 at these lengths: nothing beside
ATOL = 1e-10.  A bf16 gradient adds 2^-9 of its value.
"""
import numpy as np
import pytest
import torch

import perfectly_balanced_token_gb300 as mx
from oracle import ops
from tests.gpu_harness import ensure_library

pytestmark = pytest.mark.gpu
RTOL, ATOL = 2e-5, 1e-10


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_library()


def draw(T, E, seed, dtype=torch.float32, ties=False, off=0, spread=2.0):
    rng = np.random.default_rng(seed)
    l = rng.standard_normal((T, E)) * spread
    if ties:  # many equal logits, zeros of both signs among them
        l = np.round(l)
        l[l == 0] = np.where(rng.random((l == 0).sum()) < 0.5, -0.0, 0.0)
    if off:
        l[:, rng.permutation(E)[:off]] = -np.inf
    return torch.from_numpy(l.astype(np.float32)).to(dtype)


def forward(rd, logits, mask=None, loss=True, stream=None):
    dev = "cuda"
    out = dict(topk_idx=torch.full((rd.T, rd.K), -7, dtype=torch.int32, device=dev),
               gates=torch.full((rd.T, rd.K), 7e7, dtype=torch.float32, device=dev))
    if loss:
        out.update(counts=torch.full((rd.G, rd.E), -7, dtype=torch.int32, device=dev),
                   prob_sum=torch.full((rd.G, rd.E), 7e7, dtype=torch.float32, device=dev),
                   seg_tokens=torch.full((rd.G,), -7, dtype=torch.int32, device=dev),
                   loss=torch.full((1,), 7e7, dtype=torch.float32, device=dev))
        ws = torch.full((mx.moonep_router_workspace_bytes(rd),), 0xA5, dtype=torch.uint8, device=dev)
        mx.moonep_router_forward(rd, logits, out["topk_idx"], out["gates"], token_mask=mask, ws=ws,
                                 stream=stream, **{k: out[k] for k in ("counts", "prob_sum",
                                                                       "seg_tokens", "loss")})
    else:
        mx.moonep_router_forward(rd, logits, out["topk_idx"], out["gates"], token_mask=mask,
                                 stream=stream)
    return out


def close(got, want, what, rtol=RTOL, atol=ATOL):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), what
    err = np.abs(got - want)[~nan]
    bad = err > (atol + rtol * np.abs(want))[~nan]
    assert not bad.any(), (what, int(bad.sum()), err.max())


def check(rd, logits, mask_np=None, score="softmax", loss=True):
    x = logits.double().numpy()
    live = None if mask_np is None else mask_np != 0
    mask = None if mask_np is None else torch.from_numpy(mask_np).cuda()
    out = {k: v.cpu().numpy() for k, v in forward(rd, logits.cuda(), mask, loss).items()}
    scale = float(np.float32(rd.scale))
    ids, gates, counts, sums, tokens, value = ops.router(
        x, rd.K, rd.segment or rd.T, score, bool(rd.normalise), scale, live)
    assert np.array_equal(out["topk_idx"], ids)
    close(out["gates"], gates, "gates")
    if loss:
        assert np.array_equal(out["counts"], counts)
        assert np.array_equal(out["seg_tokens"], tokens)
        close(out["prob_sum"], sums, "prob_sum")
        close(out["loss"][0], value, "loss")
    return out


# T, E, K, segment: one token to several blocks a segment, experts from fewer than
# lanes to 4096 and off every vector width, K from 1 to E and beyond 32, ragged segments
SHAPES = [(1, 1, 1, 0), (1, 8, 8, 0), (7, 20, 3, 3), (33, 31, 31, 32), (64, 33, 2, 1),
          (130, 71, 5, 50), (257, 127, 7, 0), (64, 128, 8, 16), (300, 132, 4, 7),
          (1000, 257, 6, 999), (513, 384, 8, 128), (100, 384, 40, 0), (77, 640, 9, 20),
          (1300, 896, 16, 600), (64, 1023, 12, 0), (40, 1024, 128, 9), (19, 1500, 10, 0),
          (21, 2048, 33, 5), (23, 4096, 16, 11), (9, 4093, 100, 4), (5000, 64, 6, 5000),
          (20000, 96, 4, 9000)]


@pytest.mark.parametrize("T,E,K,segment", SHAPES)
@pytest.mark.parametrize("score,normalise,dtype", [("softmax", True, torch.float32),
                                                   ("sigmoid", False, torch.bfloat16),
                                                   ("softmax", False, torch.bfloat16),
                                                   ("sigmoid", True, torch.float32)])
def test_forward(T, E, K, segment, score, normalise, dtype):
    rd = mx.router_dims(T, E, K, segment, score, normalise, 2.5, dtype)
    logits = draw(T, E, T + E + K, dtype)
    mask = (np.random.default_rng(T).random(T) > 0.2).astype(np.uint8)
    with_loss = check(rd, logits, mask, score)
    # the form without the loss gives the same ids and gates
    bare = forward(rd, logits.cuda(), torch.from_numpy(mask).cuda(), loss=False)
    assert np.array_equal(bare["topk_idx"].cpu().numpy(), with_loss["topk_idx"])
    assert np.array_equal(bare["gates"].cpu().numpy(), with_loss["gates"])


@pytest.mark.parametrize("T,E,K", [(50, 384, 8), (50, 71, 16), (20, 1500, 8), (20, 32, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_and_experts_switched_off(T, E, K, score):
    rd = mx.router_dims(T, E, K, 0, score, True, 1.0)
    check(rd, draw(T, E, 1, ties=True), score=score)
    check(rd, torch.zeros(T, E), score=score)  # every logit equal
    check(rd, draw(T, E, 2, off=E // 2), score=score)
    check(rd, draw(T, E, 3, off=E - 3), score=score)  # fewer than K left


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [24, 384])
def test_rows_of_infinities_and_nan(score, E):
    T, K = 12, 6
    l = draw(T, E, 5)
    l[1] = -np.inf
    l[3, 4] = np.nan
    l[4] = np.nan
    l[5] = -np.inf
    l[5, 7] = np.nan
    l[6] = torch.finfo(torch.float32).min
    l[7] = torch.finfo(torch.float32).max
    l[8, 2] = torch.finfo(torch.float32).max
    if score == "sigmoid":
        l[9, 3] = np.inf
    rd = mx.router_dims(T, E, K, 4, score, True, 1.0)
    check(rd, l, score=score)
    # a masked token's NaN reaches no sum
    mask = np.ones(T, np.uint8)
    mask[[3, 4, 5]] = 0
    out = check(rd, l, mask, score)
    assert np.isfinite(out["loss"]).all()


def test_very_low_logits_keep_their_shares():
    l = draw(6, 40, 4)
    l[0] -= 100.0    # sigmoids below the smallest float
    l[1] -= 1e6
    l[2] += 100.0
    l[3] = -3e38
    for score in ("softmax", "sigmoid"):
        check(mx.router_dims(6, 40, 3, 2, score, True, 1.0), l, score=score)
        check(mx.router_dims(6, 40, 3, 2, score, False, 1.0), l, score=score)


def test_segments_without_tokens():
    rd = mx.router_dims(40, 64, 4, 8, "softmax", True, 1.0)
    mask = np.ones(40, np.uint8)
    mask[8:24] = 0
    check(rd, draw(40, 64, 0), mask)
    check(rd, draw(40, 64, 0), np.zeros(40, np.uint8))
    big = mx.router_dims(4000, 64, 4, 2000, "softmax", True, 1.0)
    mask = np.ones(4000, np.uint8)
    mask[:2000] = 0
    check(big, draw(4000, 64, 0), mask)


def test_same_bits_in_every_run_and_on_another_stream():
    rd = mx.router_dims(30000, 384, 8, 10000, "softmax", True, 1.0)
    l = draw(30000, 384, 9).cuda()
    first = forward(rd, l)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = forward(rd, l)
    third = forward(rd, l, stream=side)
    torch.cuda.synchronize()
    for k in first:
        assert torch.equal(first[k], second[k]) and torch.equal(first[k], third[k]), k


@pytest.mark.parametrize("E,K,score,dtype", [(384, 8, "softmax", torch.float32),
                                             (896, 16, "sigmoid", torch.bfloat16)])
def test_launch_after_launch_gives_the_same_bits(E, K, score, dtype):
    T = 20000
    rd = mx.router_dims(T, E, K, 3000, score, True, 1.0, dtype)
    l = draw(T, E, 12, dtype).cuda()
    want = forward(rd, l)
    got = {k: torch.zeros_like(v) for k, v in want.items()}
    ws = torch.empty(mx.moonep_router_workspace_bytes(rd), dtype=torch.uint8, device="cuda")
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(500):
        mx.moonep_router_forward(rd, l, got["topk_idx"], got["gates"], ws=ws,
                                 **{k: got[k] for k in ("counts", "prob_sum", "seg_tokens", "loss")})
        for k in want:
            differ += (got[k] != want[k]).any()
    assert int(differ) == 0


def test_in_a_graph():
    rd = mx.router_dims(5000, 384, 8, 1700, "sigmoid", True, 1.0)
    l = draw(5000, 384, 10).cuda()
    want = forward(rd, l)
    outs = {}
    ws = torch.full((mx.moonep_router_workspace_bytes(rd),), 0xA5, dtype=torch.uint8, device="cuda")
    got = {k: torch.zeros_like(v) for k, v in want.items()}
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        mx.moonep_router_forward(rd, l, got["topk_idx"], got["gates"], ws=ws,
                                 **{k: got[k] for k in ("counts", "prob_sum", "seg_tokens", "loss")})
    for _ in range(3):
        for v in got.values():
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        outs = {k: torch.equal(got[k], want[k]) for k in want}
        assert all(outs.values()), outs


def test_offsets_past_32_bits():
    T, E, K = 4_900_000, 896, 2  # 4.4e9 logits
    rd = mx.router_dims(T, E, K, 0, "softmax", True, 1.0, torch.bfloat16)
    l = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    tail = draw(5, E, 3, torch.bfloat16)
    l[-5:] = tail.cuda()
    idx = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
    gates = torch.full((T, K), 7e7, device="cuda")
    mx.moonep_router_forward(rd, l, idx, gates)
    ids, want, *_ = ops.router(tail.double().numpy(), K, 5, "softmax", True, 1.0)
    assert np.array_equal(idx[-5:].cpu().numpy(), ids)
    close(gates[-5:].cpu().numpy(), want, "gates")
    assert bool((idx[:-5] == torch.arange(K, device="cuda", dtype=torch.int32)).all())
    dg = torch.zeros(T, K, device="cuda")
    dg[-5:, 0] = 1.0
    got = torch.full_like(l, 7.0)
    mx.moonep_router_backward(rd, l, idx, got, d_gates=dg)
    grad, size = ops.router_backward(tail.double().numpy(), ids, 5, "softmax", True, 1.0, None,
                                     dg[-5:].cpu().numpy(), 0.0)
    err = np.abs(got[-5:].double().cpu().numpy() - grad)
    assert (err <= 3 * RTOL * size + 2.0 ** -8 * np.abs(grad) + 1e-12).all()
    assert not got[:-5].any()


def test_ids_feed_the_plan():
    d = mx.dims(4, 64, 16, 4, 100, 64, 64)
    rd = mx.router_dims(400, 64, 4, 100)
    out = forward(rd, draw(400, 64, 3).cuda())
    ws = mx.PlanWorkspace(d)
    mx.moonep_plan(d, out["topk_idx"], ws.buf)
    tabs = ws.tables()
    assert tabs["status"][0] == 0
    assert np.array_equal(tabs["T"], out["counts"].sum(0).cpu().numpy())


# ------------------------------------------------------------------------- gradient
# Each factor of the gradient (a score, a gate's share, the sums over the row) is
# within RTOL of its own, so the element is within 3 RTOL of the sum of magnitudes
# that make it up; bf16 results are rounded once more.
@pytest.mark.parametrize("T,E,K,segment", [(1, 1, 1, 0), (7, 20, 3, 3), (33, 31, 31, 32),
                                           (64, 33, 2, 1), (130, 71, 5, 50), (64, 128, 8, 16),
                                           (60, 384, 8, 25), (40, 384, 40, 0), (30, 896, 16, 30),
                                           (9, 1023, 12, 0), (9, 1024, 128, 4), (5, 2047, 9, 2),
                                           (3, 4096, 16, 0)])
@pytest.mark.parametrize("score,normalise,dtype", [("softmax", True, torch.float32),
                                                   ("sigmoid", False, torch.bfloat16),
                                                   ("softmax", False, torch.float32),
                                                   ("sigmoid", True, torch.bfloat16)])
@pytest.mark.parametrize("parts", ["both", "gates", "loss"])
def test_backward(T, E, K, segment, score, normalise, dtype, parts):
    rd = mx.router_dims(T, E, K, segment, score, normalise, 1.5, dtype)
    off = E // 3 if E > 3 * K else 0
    logits = draw(T, E, T + E, dtype, off=off)
    rng = np.random.default_rng(E)
    live = rng.random(T) > 0.2
    mask = torch.from_numpy(live.astype(np.uint8)).cuda()
    fwd = forward(rd, logits.cuda(), mask)
    dg = rng.standard_normal((T, K)).astype(np.float32) if parts != "loss" else None
    dl = float(np.float32(rng.random() * T + 1)) if parts != "gates" else 0.0
    got = torch.full((T, E), 7.0, dtype=dtype, device="cuda")
    extra = {}
    if dg is not None:
        extra["d_gates"] = torch.from_numpy(dg).cuda()
    if dl:
        extra.update(counts=fwd["counts"], seg_tokens=fwd["seg_tokens"],
                     d_loss=torch.tensor([dl], device="cuda"))
    mx.moonep_router_backward(rd, logits.cuda(), fwd["topk_idx"], got, token_mask=mask, **extra)
    want, size = ops.router_backward(logits.double().numpy(), fwd["topk_idx"].cpu().numpy(),
                                     segment or T, score, normalise, 1.5, live, dg, dl)
    tol = 3 * RTOL * size + 1e-12 + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), (err.max(), (err / tol).max())
    assert not got[torch.from_numpy(~live).cuda()].any()


def test_backward_of_rows_without_weight():
    T, E, K = 6, 40, 3
    for score in ("softmax", "sigmoid"):
        rd = mx.router_dims(T, E, K, 3, score, True, 1.0)
        l = draw(T, E, 8)
        l[2] = -np.inf
        fwd = forward(rd, l.cuda())
        got = torch.full((T, E), 7.0, device="cuda")
        mx.moonep_router_backward(rd, l.cuda(), fwd["topk_idx"], got,
                                  d_gates=torch.ones(T, K, device="cuda"), counts=fwd["counts"],
                                  seg_tokens=fwd["seg_tokens"], d_loss=torch.ones(1, device="cuda"))
        assert torch.isfinite(got).all() and not got[2].any()


# Rows with NaN and infinities at chosen and at unchosen experts: NaN where the formula has it
# (sigmoid gates without the loss depend on the chosen logits alone) and nowhere else.
@pytest.mark.parametrize("E,K,dtype", [(24, 6, torch.float32), (71, 5, torch.bfloat16),
                                       (384, 8, torch.float32), (896, 16, torch.bfloat16),
                                       (1500, 10, torch.float32), (64, 40, torch.float32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalise", [True, False])
@pytest.mark.parametrize("parts", ["both", "gates", "loss"])
def test_backward_of_rows_of_infinities_and_nan(E, K, dtype, score, normalise, parts):
    T = 16
    l = draw(T, E, 15, dtype)
    top = l[:, :].float().argsort(1, descending=True)
    l[1, top[1, E - 1]] = np.nan            # never chosen
    l[2, top[2, [K + 1, E - 2]]] = np.nan   # just below the chosen ones
    l[3] = np.nan
    l[4] = np.nan
    l[4, 7] = 1.0                           # NaN among the chosen
    l[5, : E - K + 1] = np.nan              # one chosen NaN
    l[6, top[6, 0]] = np.inf                # chosen
    l[7, top[7, : K + 1]] = np.inf          # one of them not chosen
    l[8, top[8, E // 2:]] = -np.inf
    l[9] = -np.inf
    l[9, 3] = 2.0                           # -inf among the chosen
    l[10] = -np.inf
    l[10, 5] = np.nan
    l[11, 0], l[11, E - 1] = np.inf, -np.inf
    rd = mx.router_dims(T, E, K, 5, score, normalise, 1.5, dtype)
    live = np.ones(T, bool)
    live[2] = parts != "both"               # a masked token's gradient is 0, whatever its row holds
    mask = torch.from_numpy(live.astype(np.uint8)).cuda()
    fwd = forward(rd, l.cuda(), mask)
    rng = np.random.default_rng(E)
    dg = rng.standard_normal((T, K)).astype(np.float32) if parts != "loss" else None
    dl = 3.0 if parts != "gates" else 0.0
    extra = {}
    if dg is not None:
        extra["d_gates"] = torch.from_numpy(dg).cuda()
    if dl:
        extra.update(counts=fwd["counts"], seg_tokens=fwd["seg_tokens"],
                     d_loss=torch.tensor([dl], device="cuda"))
    got = torch.full((T, E), 7.0, dtype=dtype, device="cuda")
    mx.moonep_router_backward(rd, l.cuda(), fwd["topk_idx"], got, token_mask=mask, **extra)
    with np.errstate(invalid="ignore"):
        want, size = ops.router_backward(l.double().numpy(), fwd["topk_idx"].cpu().numpy(), 5, score,
                                         normalise, 1.5, live, dg, dl)
    got = got.double().cpu().numpy()
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), np.nonzero((np.isnan(got) != nan).any(1))[0]
    tol = 3 * RTOL * size + 1e-12 + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0)
    err = np.abs(got - want)
    assert (err <= tol)[~nan].all(), err[~nan].max()


def test_gradient_against_differences_on_the_gpu():
    """d_logits against differences of the forward pass's own fp32 gates and loss.  Their
    rounding is RTOL of values below 3, so a difference over 2 h is off by 6 RTOL / (2 h),
    and the formula's third derivative adds at most h^2 (all terms below 10)."""
    T, E, K, h = 4, 24, 4, 0.05
    rd = mx.router_dims(T, E, K, 2, "softmax", True, 1.0)
    l = draw(T, E, 21, spread=1.0)
    dg = torch.randn(T, K, generator=torch.Generator().manual_seed(1)).cuda()
    fwd = forward(rd, l.cuda())
    got = torch.empty(T, E, device="cuda")
    mx.moonep_router_backward(rd, l.cuda(), fwd["topk_idx"], got, d_gates=dg, counts=fwd["counts"],
                              seg_tokens=fwd["seg_tokens"], d_loss=torch.ones(1, device="cuda"))

    def value(x):
        out = forward(rd, x.cuda())
        if not torch.equal(out["topk_idx"], fwd["topk_idx"]):
            return None
        return float((out["gates"] * dg).double().sum()) + float(out["loss"])

    seen = 0
    for t in range(T):
        for e in range(E):
            up, down = l.clone(), l.clone()
            up[t, e] += h
            down[t, e] -= h
            a, b = value(up), value(down)
            if a is None or b is None:
                continue  # the step changed the choice of experts
            seen += 1
            assert abs((a - b) / (2 * h) - float(got[t, e])) <= 6 * RTOL / (2 * h) + 10 * h * h
    assert seen > T * E // 2


# Several tokens a warp, blocks with whole segments and parts of others, and rows that
# lie in vectors, short and long.
@pytest.mark.parametrize("T,E,K,segment", [(2000, 896, 16, 7), (2000, 896, 16, 24),
                                           (5000, 640, 8, 37), (12000, 516, 6, 1000),
                                           (16000, 384, 8, 900)])
@pytest.mark.parametrize("score,dtype", [("sigmoid", torch.bfloat16), ("softmax", torch.float32)])
def test_many_tokens_and_segment_borders(T, E, K, segment, score, dtype):
    rd = mx.router_dims(T, E, K, segment, score, True, 1.5, dtype)
    logits = draw(T, E, T + segment, dtype)
    live = np.random.default_rng(E).random(T) > 0.2
    fwd = check(rd, logits, live.astype(np.uint8), score)
    dg = np.random.default_rng(K).standard_normal((T, K)).astype(np.float32)
    dl = float(T)
    got = torch.full((T, E), 7.0, dtype=dtype, device="cuda")
    cuda = {k: torch.from_numpy(fwd[k]).cuda() for k in ("topk_idx", "counts", "seg_tokens")}
    mx.moonep_router_backward(rd, logits.cuda(), cuda["topk_idx"], got,
                              token_mask=torch.from_numpy(live.astype(np.uint8)).cuda(),
                              d_gates=torch.from_numpy(dg).cuda(), counts=cuda["counts"],
                              seg_tokens=cuda["seg_tokens"],
                              d_loss=torch.tensor([dl], device="cuda"))
    want, size = ops.router_backward(logits.double().numpy(), fwd["topk_idx"], segment, score, True,
                                     1.5, live, dg, dl)
    tol = 3 * RTOL * size + 1e-12 + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), (err.max(), (err / tol).max())
    assert not got[torch.from_numpy(~live).cuda()].any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [24, 384, 900])
def test_bf16_rows_of_infinities_nan_and_ties(score, E):
    T, K = 14, 6
    l = draw(T, E, 6, torch.bfloat16)
    l[1] = -np.inf
    l[3, 4] = np.nan
    l[4] = np.nan
    l[5] = -np.inf
    l[5, 7] = np.nan
    l[6] = torch.finfo(torch.bfloat16).min
    l[7] = torch.finfo(torch.bfloat16).max
    l[8, 2] = torch.finfo(torch.bfloat16).max
    l[9] = torch.finfo(torch.bfloat16).tiny
    l[10, E - 3:] = 7.0
    l[11] = 2.0 ** -133
    l[11, 5] = 0.0
    l[11, 9] = 2 * 2.0 ** -133
    check(mx.router_dims(T, E, K, 4, score, True, 1.0, torch.bfloat16), l, score=score)
    rd = mx.router_dims(50, E, K, 0, score, True, 1.0, torch.bfloat16)
    check(rd, draw(50, E, 1, torch.bfloat16, ties=True), score=score)
    check(rd, torch.zeros(50, E, dtype=torch.bfloat16), score=score)
    check(rd, draw(50, E, 2, torch.bfloat16, off=E // 2), score=score)
    check(rd, draw(50, E, 3, torch.bfloat16, off=E - 3), score=score)


# Blocks that have several short segments to themselves and share their first and last one
# with a neighbour: whole segments, joins and the last block's loss in the same block.
@pytest.mark.parametrize("E,K,score,dtype", [(384, 8, "softmax", torch.float32),
                                             (896, 16, "sigmoid", torch.bfloat16),
                                             (64, 4, "softmax", torch.float32)])
@pytest.mark.parametrize("segment", [5, 37])
def test_short_segments_launch_after_launch(E, K, score, dtype, segment):
    T = 20000
    rd = mx.router_dims(T, E, K, segment, score, True, 1.0, dtype)
    l = draw(T, E, 13, dtype)
    check(rd, l, score=score)
    l = l.cuda()
    want = forward(rd, l)
    got = {k: torch.zeros_like(v) for k, v in want.items()}
    ws = torch.empty(mx.moonep_router_workspace_bytes(rd), dtype=torch.uint8, device="cuda")
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        mx.moonep_router_forward(rd, l, got["topk_idx"], got["gates"], ws=ws,
                                 **{k: got[k] for k in ("counts", "prob_sum", "seg_tokens", "loss")})
        for k in want:
            differ += (got[k] != want[k]).any()
    assert int(differ) == 0


# So many tokens that the blocks run in several rounds (a block takes 64 tokens a warp, a
# multiprocessor holds 64 warps at most): the same few rows again and again, so that all that
# repeats has to be equal and the sums are those of one turn times the turns.
# Sums: a warp's 64 tokens in fp32 add 64 2^-24 to RTOL, 24 warps half as much; a block rounds
# once to steps of 2^-41 at up to 2^21 tokens.
@pytest.mark.parametrize("E,K,turns,score,dtype", [(64, 4, 1304, "softmax", torch.float32),
                                                   (71, 5, 1304, "sigmoid", torch.bfloat16),
                                                   (384, 8, 700, "softmax", torch.float32),
                                                   (896, 16, 500, "sigmoid", torch.bfloat16)])
@pytest.mark.parametrize("segment_turns", [0, 37])
def test_blocks_in_several_rounds(E, K, turns, score, dtype, segment_turns):
    n = 997
    T = n * turns
    few = draw(n, E, 31, dtype)
    live = np.random.default_rng(3).random(n) > 0.2
    rd = mx.router_dims(T, E, K, segment_turns * n, score, True, 1.5, dtype)
    l = few.cuda().repeat(turns, 1)
    mask = torch.from_numpy(live.astype(np.uint8)).cuda().repeat(turns)
    fwd = forward(rd, l, mask)
    ids, gates, counts, sums, tokens, loss = ops.router(few.double().numpy(), K, n, score, True, 1.5,
                                                        live)
    idx, g = fwd["topk_idx"].view(turns, n, K), fwd["gates"].view(turns, n, K)
    assert np.array_equal(idx[0].cpu().numpy(), ids) and bool((idx == idx[0]).all())
    close(g[0].cpu().numpy(), gates, "gates")
    assert bool((g == g[0]).all())
    per = segment_turns or turns
    r = np.minimum(per, turns - np.arange(rd.G) * per)[:, None]  # turns of each segment
    assert np.array_equal(fwd["counts"].cpu().numpy(), r * counts)
    assert np.array_equal(fwd["seg_tokens"].cpu().numpy(), r[:, 0] * tokens)
    close(fwd["prob_sum"].cpu().numpy(), r * sums, "prob_sum", RTOL + 96 * 2.0 ** -24,
          (T / 512 + 1) * 2.0 ** -42)
    close(fwd["loss"][0].cpu().numpy(), loss, "loss", RTOL + 96 * 2.0 ** -24)
    again = forward(rd, l, mask)
    assert all(torch.equal(fwd[k], again[k]) for k in fwd)
    if segment_turns:
        return
    dg = torch.randn(n, K, generator=torch.Generator().manual_seed(2))
    got = torch.full((T, E), 7.0, dtype=dtype, device="cuda")
    mx.moonep_router_backward(rd, l, fwd["topk_idx"], got, token_mask=mask,
                              d_gates=dg.cuda().repeat(turns, 1), counts=fwd["counts"],
                              seg_tokens=fwd["seg_tokens"],
                              d_loss=torch.tensor([float(T)], device="cuda"))
    got = got.view(turns, n, E)
    assert bool((got == got[0]).all())
    # counts and tokens of all turns: the weights of one turn's over the turns
    want, size = ops.router_backward(few.double().numpy(), ids, n, score, True, 1.5, live,
                                     dg.numpy(), float(T) / turns)
    tol = 3 * RTOL * size + 1e-12 + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0)
    err = np.abs(got[0].double().cpu().numpy() - want)
    assert (err <= tol).all(), (err.max(), (err / tol).max())


# Logits within 4 of 0, so that exponents are at most 8 long: an exponential is then within
# 2 2^-23 + 8 2^-24 + 8 2^-25 (instruction, product, constant) = 9.6e-7 of itself, a sum over the
# row within 17 2^-24 (12 values a lane, 5 steps over the warp) = 1e-6 more.  Gate: two
# exponentials, the chosen scores in steps of 2^-24 (8 halves of a step over 1/2: 4.8e-7), a
# reciprocal and four products (3.6e-7): 2.8e-6.  prob_sum: the score (sigmoid: and a reciprocal,
# 1.2e-6), the row's sum of such scores (2.2e-6), a reciprocal and up to 13 additions (9e-7): 4.3e-6.
@pytest.mark.parametrize("E", [64, 384])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalise", [True, False])
def test_rounding_of_moderate_logits(E, score, normalise):
    T, K, tight = 300, 8, 5e-6
    l = torch.from_numpy(np.random.default_rng(E).uniform(-4, 4, (T, E)).astype(np.float32))
    rd = mx.router_dims(T, E, K, 100, score, normalise, 1.0)
    out = {k: v.cpu().numpy() for k, v in forward(rd, l.cuda()).items()}
    ids, gates, counts, sums, _, loss = ops.router(l.double().numpy(), K, 100, score, normalise, 1.0)
    assert np.array_equal(out["topk_idx"], ids) and np.array_equal(out["counts"], counts)
    close(out["gates"], gates, "gates", tight, 0)
    close(out["prob_sum"], sums, "prob_sum", tight)
    close(out["loss"][0], loss, "loss", tight)
