"""The feed-forward operators together, as a layer runs them, and where they run: other streams,
captured graphs, beside one another, and past 2^31 elements."""
import numpy as np
import pytest
import torch

import perfectly_balanced_token_gb300 as mx
from oracle import ffn
from perfectly_balanced_token_gb300 import synthetic as syn
from tests.gpu_harness import ensure_library

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_library()


def bf(*shape):
    return torch.empty(*shape, dtype=BF16, device="cuda")


def f32(*shape):
    return torch.zeros(*shape, device="cuda")


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


class Layer:
    """Router, routed experts of two projections, a shared expert, dropout and residual."""

    def __init__(self, R=4, E=16, B=4, K=2, S=96, H=128, F=256, Fs=192, p=0.1, seed=1):
        self.R, self.E, self.B, self.K, self.S, self.H, self.F, self.Fs, self.p = R, E, B, K, S, H, F, Fs, p
        self.T, self.N = R * S, R * S * K
        T, N = self.T, self.N
        self.d1, self.d2 = mx.dims(R, E, B, K, S, H, 2 * F), mx.dims(R, E, B, K, S, F, H)
        self.ws = mx.PlanWorkspace(self.d1)
        self.rd = mx.router_dims(T, E, K)
        w = lambda i, *s: syn.normal_bf16(s, s[-2] ** -0.5, seed + i).cuda()  # noqa: E731
        self.wr, self.w1, self.w2 = w(1, H, E), w(2, E, H, 2 * F), w(3, E, F, H)
        self.s1, self.s2 = w(4, H, 2 * Fs), w(5, Fs, H)
        g = torch.Generator().manual_seed(seed)
        self.b1 = (0.3 * torch.randn(E, 2 * F, generator=g)).cuda()
        self.bs = (0.3 * torch.randn(2 * Fs, generator=g)).cuda()
        self.slot1, self.slot2 = bf(R * B, H, 2 * F), bf(R * B, F, H)
        self.status, self.rng = word(), torch.tensor([seed, 77], device="cuda")
        self.logits, self.idx = f32(T, E), torch.empty(T, K, dtype=torch.int32, device="cuda")
        self.gates, self.out = f32(T, K), bf(T, H)
        self.recv, self.h, self.z, self.y = bf(N, H), bf(N, F), bf(N, 2 * F), bf(N, H)
        self.hs, self.zs, self.res = bf(T, Fs), bf(T, 2 * Fs), bf(T, H)
        # gradients
        self.dy, self.dgates, self.dh, self.dz, self.drecv = bf(N, H), f32(T, K), bf(N, F), bf(N, 2 * F), bf(N, H)
        self.dx_routed, self.dx_shared, self.dx_router = bf(T, H), bf(T, H), bf(T, H)
        self.dlogits, self.dhs, self.dzs = f32(T, E), bf(T, Fs), bf(T, 2 * Fs)
        self.g1, self.g2, self.g1s, self.g2s = f32(E, H, 2 * F), f32(E, F, H), f32(R * B, H, 2 * F), f32(R * B, F, H)
        self.gb1, self.gbs, self.gr = f32(E, 2 * F), f32(2 * Fs), f32(H, E)
        self.gs1, self.gs2 = f32(H, 2 * Fs), f32(Fs, H)
        self.scratch = torch.empty(mx.moonep_grouped_act_backward_workspace_bytes(self.d1), dtype=torch.uint8,
                                   device="cuda")
        self.scratch_s = torch.empty(mx.moonep_act_backward_workspace_bytes(T, 2 * Fs), dtype=torch.uint8,
                                     device="cuda")
        self.lr = mx.linear_dims(T, H, E, out_dtype=F32)
        self.l1, self.l2 = mx.linear_dims(T, H, 2 * Fs, act="swiglu"), mx.linear_dims(T, Fs, H)

    def forward(self, x):
        d1, d2, ws = self.d1, self.d2, self.ws.buf
        mx.moonep_linear(self.lr, x, self.wr, self.logits, self.status)
        mx.moonep_router_forward(self.rd, self.logits, self.idx, self.gates)
        mx.moonep_plan(d1, self.idx, ws)
        mx.moonep_prefetch_weights(d1, ws, self.w1, self.slot1)
        mx.moonep_prefetch_weights(d2, ws, self.w2, self.slot2)
        mx.moonep_linear(self.l1, x, self.s1, self.hs, self.status, bias=self.bs, z=self.zs)
        mx.moonep_linear(self.l2, self.hs, self.s2, self.res, self.status, residual=x)
        mx.moonep_dispatch(d1, ws, x, self.recv)
        mx.moonep_grouped_gemm_act(d1, ws, self.recv, self.w1, self.slot1, self.h, act="swiglu", bias=self.b1,
                                   z=self.z)
        mx.moonep_grouped_gemm(d2, ws, self.h, self.w2, self.slot2, self.y)
        mx.moonep_combine_dropout(d2, ws, self.y, self.gates, self.out, residual=self.res, p=self.p, rng=self.rng)
        return self.out

    def backward(self, x, d_out):
        d1, d2, ws = self.d1, self.d2, self.ws.buf
        mx.moonep_combine_dropout_backward(d2, ws, self.y, self.gates, d_out, self.dy, self.dgates, p=self.p,
                                           rng=self.rng)
        mx.moonep_grouped_gemm_dw(d2, ws, self.h, self.dy, self.g2, self.g2s)
        mx.moonep_grouped_gemm_dx(d2, ws, self.dy, self.w2, self.slot2, self.dh)
        mx.moonep_grouped_act_backward(d1, ws, self.z, self.dh, self.dz, act="swiglu", d_bias=self.gb1,
                                       scratch=self.scratch)
        mx.moonep_grouped_gemm_dw(d1, ws, self.recv, self.dz, self.g1, self.g1s)
        mx.moonep_grouped_gemm_dx(d1, ws, self.dz, self.w1, self.slot1, self.drecv)
        mx.moonep_dispatch_backward(d1, ws, self.drecv, self.dx_routed)
        mx.moonep_reduce_grad(d1, ws, self.g1, self.g1s)
        mx.moonep_reduce_grad(d2, ws, self.g2, self.g2s)
        mx.moonep_router_backward(self.rd, self.logits, self.idx, self.dlogits, d_gates=self.dgates)
        dl = self.dlogits.to(BF16)
        mx.moonep_linear_dw(self.lr, x, dl, self.gr, self.status)
        mx.moonep_linear_dx(self.lr, dl, self.wr, self.dx_router, self.status)
        mx.moonep_linear_dw(self.l2, self.hs, d_out, self.gs2, self.status)
        mx.moonep_linear_dx(self.l2, d_out, self.s2, self.dhs, self.status)
        mx.moonep_act_backward(self.zs, self.dhs, self.dzs, act="swiglu", d_bias=self.gbs, scratch=self.scratch_s)
        mx.moonep_linear_dw(self.l1, x, self.dzs, self.gs1, self.status)
        mx.moonep_linear_dx(self.l1, self.dzs, self.s1, self.dx_shared, self.status)

    def reference(self, x, d_out):
        """The layer in 64 bits by automatic differentiation, with the routing that was chosen."""
        F, Fs, T, K = self.F, self.Fs, self.T, self.K
        names = ("wr", "w1", "w2", "s1", "s2", "b1", "bs")
        v = {n: getattr(self, n).double().requires_grad_(True) for n in names}
        xx = x.double().requires_grad_(True)
        silu = torch.nn.functional.silu
        picked = (xx @ v["wr"]).gather(1, self.idx.long())
        gates = torch.softmax(picked, -1)
        zs = xx @ v["s1"] + v["bs"]
        res = xx + (silu(zs[:, :Fs]) * zs[:, Fs:]) @ v["s2"]
        total = torch.zeros(T, self.H, dtype=torch.float64, device="cuda")
        for e in range(self.E):
            t, k = torch.nonzero(self.idx == e, as_tuple=True)
            z = xx[t] @ v["w1"][e] + v["b1"][e]
            y = (silu(z[:, :F]) * z[:, F:]) @ v["w2"][e]
            total = total.index_add(0, t, gates[t, k, None] * y)
        seed, offset = self.rng.tolist()
        f = torch.from_numpy(ffn.dropout_factor(T * self.H, self.p, seed, offset).reshape(T, self.H)).cuda()
        out = res + total * f
        (out * d_out.double()).sum().backward()
        return out.detach(), xx.grad, {n: t.grad for n, t in v.items()}


def far(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("sizes", [dict(), dict(R=2, E=8, B=4, K=3, S=333, H=256, F=128, Fs=64, p=0.5),
                                   dict(R=1, E=8, B=8, K=2, S=5, H=128, F=128, Fs=72, p=0.0)],
                         ids=["small", "ragged", "few tokens"])
def test_layer_and_its_gradients(sizes):
    m = Layer(**sizes)
    x, d_out = syn.normal_bf16((m.T, m.H), 1.0, 11).cuda(), syn.normal_bf16((m.T, m.H), 1.0, 12).cuda()
    m.forward(x)
    m.backward(x, d_out)
    assert mx.moonep_read_status(m.d1, m.ws.buf) == 0 and int(m.status) == 0
    out, dx, g = m.reference(x, d_out)
    # Every bf16 tensor on the way from an input to an output is rounded once, by at most 2^-8 of each
    # value and so of its norm; a random linear map keeps relative errors, an activation's slope or a
    # product of two rounded factors at most doubles them.  Tensors on the longest ways: out 3 (h, y,
    # out), two of them behind or before a product: 6; a gradient of w1: dy, dh, dz and z, recv: 10.
    step = 2.0 ** -8
    assert far(m.out, out) < 6 * step
    for got, want in ((m.g2, "w2"), (m.g1, "w1"), (m.gb1, "b1"), (m.gbs, "bs"), (m.gs1, "s1"), (m.gs2, "s2"),
                      (m.gr, "wr")):
        assert far(got, g[want]) < 10 * step, want
    total = d_out.double() + m.dx_routed.double() + m.dx_shared.double() + m.dx_router.double()
    assert far(total, dx) < 10 * step


def snapshot(m):
    return [t.clone() for t in (m.out, m.y, m.z, m.dx_routed, m.dx_shared, m.dx_router, m.gb1, m.gbs, m.gr, m.gs1,
                                m.gs2, m.dgates)]


def test_layer_repeats_itself_with_other_inputs_between():
    m = Layer()
    x, d = syn.normal_bf16((m.T, m.H), 1.0, 11).cuda(), syn.normal_bf16((m.T, m.H), 1.0, 12).cuda()
    other = syn.normal_bf16((m.T, m.H), 3.0, 13).cuda()
    m.forward(x)
    m.backward(x, d)
    first = snapshot(m)
    m.forward(other)
    m.backward(other, x)
    m.forward(x)
    m.backward(x, d)
    for a, b in zip(first, snapshot(m)):
        assert torch.equal(a, b)


def test_layer_in_a_graph_on_another_stream():
    m = Layer()
    x, d = syn.normal_bf16((m.T, m.H), 1.0, 11).cuda(), syn.normal_bf16((m.T, m.H), 1.0, 12).cuda()
    m.forward(x)
    m.backward(x, d)
    first = snapshot(m)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        m.forward(x)
        m.backward(x, d)
    for t in (m.out, m.y, m.z, m.gb1):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, snapshot(m)):
        assert torch.equal(a, b)
    # other tokens and other random numbers through the same graph
    x.copy_(syn.normal_bf16((m.T, m.H), 1.0, 21).cuda())
    m.rng.copy_(torch.tensor([5, 1 << 40], device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    got = snapshot(m)
    m.forward(x)
    m.backward(x, d)
    for a, b in zip(got, snapshot(m)):
        assert torch.equal(a, b)
    assert not torch.equal(got[0], first[0])


def test_two_layers_beside_one_another():
    layers = [Layer(seed=1), Layer(seed=2, p=0.5)]
    xs = [syn.normal_bf16((m.T, m.H), 1.0, 30 + i).cuda() for i, m in enumerate(layers)]
    for m, x in zip(layers, xs):
        m.forward(x)
        m.backward(x, x)
    alone = [snapshot(m) for m in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(5):
        for m, x, s in zip(layers, xs, streams):
            with torch.cuda.stream(s):
                m.forward(x)
                m.backward(x, x)
    torch.cuda.synchronize()
    for m, want in zip(layers, alone):
        for a, b in zip(want, snapshot(m)):
            assert torch.equal(a, b)


def test_stream_argument():
    T, K, N = 70, 256, 512
    x, w, out = syn.normal_bf16((T, K), 1.0, 1).cuda(), syn.normal_bf16((K, N), 0.1, 2).cuda(), bf(T, N)
    want = bf(T, N)
    mx.moonep_linear(mx.linear_dims(T, K, N), x, w, want, word())
    s = torch.cuda.Stream()
    st = word()
    torch.cuda.synchronize()
    mx.moonep_linear(mx.linear_dims(T, K, N), x, w, out, st, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


def test_tensors_of_another_device_are_refused(monkeypatch):
    from perfectly_balanced_token_gb300 import _ffn
    x, w, out, st = bf(4, 64), bf(64, 64), bf(4, 64), word()
    monkeypatch.setattr(_ffn, "_device", lambda: 1)  # as if another device were the current one
    before = mx.moonep_launch_count()
    with pytest.raises(ValueError, match="x is on device 0, the current one is 1"):
        mx.moonep_linear(mx.linear_dims(4, 64, 64), x, w, out, st)
    assert mx.moonep_launch_count() == before


@pytest.mark.parametrize("T,K,N", [(1, 2048, 2048), (40, 7168, 384), (1000, 1032, 520), (6000, 512, 1032)])
def test_products_repeat_launch_after_launch(T, K, N):
    # launches overlap the end of the one before: each writes what one alone does
    ld, st = mx.linear_dims(T, K, N), word()
    xs = [syn.normal_bf16((T, K), 1.0, i).cuda() for i in range(3)]
    w, d = syn.normal_bf16((K, N), 0.05, 9).cuda(), syn.normal_bf16((T, N), 1.0, 10).cuda()
    alone = []
    for x in xs:
        o, g, dx = bf(T, N), f32(K, N), bf(T, K)
        mx.moonep_linear(ld, x, w, o, st)
        torch.cuda.synchronize()
        mx.moonep_linear_dw(ld, x, d, g, st)
        torch.cuda.synchronize()
        mx.moonep_linear_dx(ld, o, w, dx, st)
        torch.cuda.synchronize()
        alone.append((o, g, dx))
    outs = [[(bf(T, N), f32(K, N), bf(T, K)) for _ in xs] for _ in range(40)]
    for row in outs:
        for x, (o, g, dx) in zip(xs, row):
            mx.moonep_linear(ld, x, w, o, st)
            mx.moonep_linear_dx(ld, o, w, dx, st)  # reads what the launch before it writes
            mx.moonep_linear_dw(ld, x, d, g, st)
    for row in outs:
        for got, want in zip(row, alone):
            for a, b in zip(got, want):
                assert torch.equal(a, b)
    assert int(st) == 0


def test_product_past_32_bit_offsets():
    T, K, N = 70000, 64, 32768  # 2.3e9 elements of out and z
    x, w = syn.normal_bf16((T, K), 1.0, 1).cuda(), syn.normal_bf16((K, N), 0.125, 2).cuda()
    out, z, st = bf(T, N // 2), bf(T, N), word()
    mx.moonep_linear(mx.linear_dims(T, K, N, act="swiglu"), x, w, out, st, z=z)
    rows = torch.tensor([0, 1, 255, 256, 32767, 32768, 65535, 65536, 69999], device="cuda")
    want = x[rows].double() @ w.double()
    err = K * 2.0 ** -23 * (x[rows].double().abs() @ w.double().abs())
    assert bool(((z[rows].double() - want).abs() <= err + 2.0 ** -8 * (want.abs() + err)).all())
    g, u = want[:, :N // 2], want[:, N // 2:]
    act = torch.nn.functional.silu(g) * u
    e = 4 * err[:, :N // 2] * (1 + u.abs() + g.abs()) + 2.0 ** -20 * act.abs()
    assert bool(((out[rows].double() - act).abs() <= e + 2.0 ** -8 * (act.abs() + e)).all())
    assert int(st) == 0
    # its activation's gradient and the product's, where d_z has as many elements
    d_z, d_b = bf(T, N), f32(N)
    scratch = torch.empty(mx.moonep_act_backward_workspace_bytes(T, N), dtype=torch.uint8, device="cuda")
    mx.moonep_act_backward(z, out, d_z, act="swiglu", d_bias=d_b, scratch=scratch)
    zz, dd = z[rows].double().cpu().numpy(), out[rows].double().cpu().numpy()
    want = ffn.activation_backward(zz, dd, "swiglu")
    size = np.abs(np.concatenate([dd, dd], -1) * np.concatenate([zz[:, N // 2:], zz[:, :N // 2]], -1))
    got = d_z[rows].double().cpu().numpy()
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * (np.abs(want) + size) + 1e-37)
    d_x = bf(T, K)
    mx.moonep_linear_dx(mx.linear_dims(T, K, N), d_z, w, d_x, st)
    want = d_z[rows].double() @ w.double().T
    err = N * 2.0 ** -23 * (d_z[rows].double().abs() @ w.double().abs().T)
    assert bool(((d_x[rows].double() - want).abs() <= err + 2.0 ** -8 * (want.abs() + err)).all())


def test_combine_past_32_bit_offsets():
    T, K, Hp = 150000, 2, 7168  # 2.15e9 elements of y and d_y, counters past 2^27
    d = mx.dims(1, 8, 0, K, T, 64, Hp, 1)
    ws = mx.PlanWorkspace(d)
    rt = syn.gumbel_topk_routing(1, T, K, 8, alpha=0.5, seed=3)
    idx, gates = torch.from_numpy(rt.idx).cuda(), torch.from_numpy(rt.gates).cuda().view(T, K)
    mx.moonep_plan(d, idx, ws.buf)
    y = bf(T * K, Hp)
    y.view(torch.int16).random_(0x3F00, 0x4000)  # 0.5 .. 2
    out, rng = bf(T, Hp), torch.tensor([9, 8], device="cuda")
    mx.moonep_combine_dropout(d, ws.buf, y, gates, out, p=0.25, rng=rng)
    d_y, d_g = bf(T * K, Hp), f32(T, K)
    mx.moonep_combine_dropout_backward(d, ws.buf, y, gates, out, d_y, d_g, p=0.25, rng=rng)
    dst = ws.tables()["dst"].reshape(T, K)
    for t in (0, 1, 74999, 149999):
        n = t * Hp // 8
        w = ffn.philox(9, 8, np.arange(n, n + Hp // 8))
        numbers = np.stack([w & np.uint32(0xFFFF), w >> np.uint32(16)], -1).reshape(-1)
        f = np.where(numbers >= 16384, 4.0 / 3.0, 0.0)
        rows = y[torch.from_numpy(dst[t]).long().cuda()].double().cpu().numpy()
        g = gates[t].double().cpu().numpy()
        want = (rows * g[:, None]).sum(0) * f
        assert np.all(np.abs(out[t].double().cpu().numpy() - want) <= (2.0 ** -8 + 2.0 ** -20) * want)
        dd = out[t].double().cpu().numpy() * f
        got = d_y[torch.from_numpy(dst[t]).long().cuda()].double().cpu().numpy()
        assert np.all(np.abs(got - g[:, None] * dd) <= (2.0 ** -8 + 2.0 ** -20) * g[:, None] * dd)
        want = (rows * dd).sum(-1)
        assert np.all(np.abs(d_g[t].double().cpu().numpy() - want) <= Hp * 2.0 ** -23 * want)


def test_grouped_product_at_the_width_of_the_pages():
    # wide products on pair tiles: a sample of rows of every expert
    R, E, B, K, S, H, Hp = 2, 8, 4, 2, 2000, 7168, 4096
    d = mx.dims(R, E, B, K, S, H, Hp)
    ws = mx.PlanWorkspace(d)
    rt = syn.gumbel_topk_routing(R, S, K, E, alpha=1.0, seed=4)
    mx.moonep_plan(d, torch.from_numpy(rt.idx).cuda(), ws.buf)
    home = syn.normal_bf16((E, H, Hp), H ** -0.5, 2, "cuda")
    slot = bf(R * B, H, Hp)
    mx.moonep_prefetch_weights(d, ws.buf, home, slot)
    recv, bias = syn.normal_bf16((d.N, H), 1.0, 3, "cuda"), torch.randn(E, Hp, device="cuda")
    y, z = bf(d.N, Hp // 2), bf(d.N, Hp)
    mx.moonep_grouped_gemm_act(d, ws.buf, recv, home, slot, y, act="swiglu", bias=bias, z=z)
    expert = np.empty(d.N, np.int64)
    expert[ws.tables()["dst"].reshape(-1)] = rt.idx.reshape(-1)
    for e in range(E):
        at = np.nonzero(expert == e)[0]
        at = torch.from_numpy(at[np.linspace(0, len(at) - 1, 40).astype(int)]).cuda()
        x, w = recv[at].double(), home[e].double()
        want = x @ w + bias[e].double()
        err = H * 2.0 ** -23 * (x.abs() @ w.abs()) + 2.0 ** -24 * want.abs()
        assert bool(((z[at].double() - want).abs() <= err + 2.0 ** -8 * (want.abs() + err)).all()), e
        g, u = want[:, :Hp // 2], want[:, Hp // 2:]
        act = torch.nn.functional.silu(g) * u
        eg, eu = err[:, :Hp // 2], err[:, Hp // 2:]
        b = 2 * (1.2 * u.abs() * eg + g.abs() * eu) + eg * eu + 2.0 ** -20 * act.abs()
        assert bool(((y[at].double() - act).abs() <= b + 2.0 ** -8 * (act.abs() + b)).all()), e
    assert mx.moonep_read_status(d, ws.buf) == 0
