"""The operators around the expert product, as cases to measure: the router with its balance loss,
its gradient, MXFP4 quantisation, the grouped product on MXFP4 operands, and the layer they form.

``own = False`` computes each operator in a plain form (elementary torch operations in 32 bits,
rounded once at the end); ``own = True`` makes the calls a user of the framework makes.

MXFP4: blocks of 32 values along the contraction share a scale 2^(b - 127), b one byte (255: a block
that holds a value that is not finite); a value is a 4-bit code, sign and the magnitudes
0, 0.5, 1, 1.5, 2, 3, 4, 6, two to a byte with the even column in the low half.  A row of `cols`
values takes cols/2 bytes of codes and cols/32 scale bytes, padded to a multiple of 16.
"""
import math

import torch

own = False

BF16 = torch.bfloat16
F32 = torch.float32


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one decoding step's tokens through the router: latency alone
        dict(name="router 8 tokens", op="router", T=8, E=384, K=8, segment=0, score="softmax",
             normalise=True, bf16=False, masked=0.0, off=0),
        # a training micro-batch of 8 ranks x 8192 tokens, loss per rank
        dict(name="router 65536x384", op="router", T=65536, E=384, K=8, segment=8192,
             score="softmax", normalise=True, bf16=False, masked=0.0, off=0),
        # 64 ranks x 1024 tokens, many experts, padding tokens and switched-off experts
        dict(name="router 65536x896 bf16 masked", op="router", T=65536, E=896, K=16, segment=1024,
             score="sigmoid", normalise=True, bf16=True, masked=0.1, off=32),
        # the gradient of that micro-batch
        dict(name="router backward 65536x384", op="router_backward", T=65536, E=384, K=8,
             segment=8192, score="softmax", normalise=True, bf16=False, masked=0.0, off=0),
        # sequences of 1000 tokens with a ragged last one, an expert count no vector width divides
        dict(name="router backward 4099x71 odd", op="router_backward", T=4099, E=71, K=5,
             segment=1000, score="sigmoid", normalise=False, bf16=True, masked=0.2, off=0),
        # activations of one micro-batch rounded to MXFP4 and back (quantisation-aware training)
        dict(name="quantize 32768x7168", op="quantize", rows=32768, cols=7168),
        # expert weights laid out for serving: quantised along H, so transposed
        dict(name="quantize weights 16x4096x1024", op="quantize_weights", E=16, H=4096, Hp=1024),
        # a decoding step: a few copies an expert, the weights are what is read
        dict(name="product decode 16 tokens", op="product", T=16, E=384, K=8, H=7168, Hp=2048,
             skew=0.3),
        # odd sizes: groups and both widths end inside the tiles
        dict(name="product odd 777", op="product", T=777, E=12, K=3, H=1088, Hp=320, skew=0.5),
        # prefill: about 2000 rows an expert
        dict(name="product 262144 rows", op="product", T=32768, E=128, K=8, H=7168, Hp=2048,
             skew=0.3),
        # the whole forward layer from the router's logits, small
        dict(name="layer r8-e64", op="layer", R=8, E=64, K=4, S=1024, H=1024, Hp=512, skew=0.5),
        # and at the width of the pages' benchmark
        dict(name="layer r8-e128 wide", op="layer", R=8, E=128, K=8, S=2048, H=7168, Hp=2048,
             skew=0.3),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, most):
    """A multiple of 64 up to 64 * most."""
    n = _log_int(rng, 1, most)
    return 64 * (n if n != 48 else 47)


def draw(rng):
    op = rng.choice(["router", "router", "router_backward", "quantize", "quantize_weights",
                     "product", "product", "layer"])
    if op in ("router", "router_backward"):
        E = _log_int(rng, 16, 896)
        T = _log_int(rng, 1 if op == "router" else 16, 65536)
        K = rng.randint(1, min(16, E // 2))
        segment = rng.choice([0, T, max(1, T // 8), max(1, T // 3)])
        if op == "router_backward" and segment == 0:
            segment = T
        return dict(op=op, T=T, E=E, K=K, segment=segment, score=rng.choice(["softmax", "sigmoid"]),
                    normalise=rng.random() < 0.7, bf16=rng.random() < 0.5,
                    masked=rng.choice([0.0, 0.1, 0.3]), off=rng.choice([0, 0, E // 8]))
    if op == "quantize":
        return dict(op=op, rows=_log_int(rng, 1, 32768), cols=_width(rng, 112))
    if op == "quantize_weights":
        return dict(op=op, E=_log_int(rng, 1, 16), H=_width(rng, 64),
                    Hp=_width(rng, 16))
    if op == "product":
        E = _log_int(rng, 4, 128)
        return dict(op=op, T=_log_int(rng, 1, 16384), E=E, K=rng.randint(1, min(8, E)),
                    H=_width(rng, 112), Hp=_width(rng, 32),
                    skew=rng.choice([0.0, 0.3, 0.6]))
    R = rng.choice([1, 2, 4, 8])
    E = R * _log_int(rng, 2, 16)
    return dict(op=op, R=R, E=E, K=rng.randint(1, min(8, E)), S=_log_int(rng, 1, 2048),
                H=_width(rng, 64), Hp=_width(rng, 32),
                skew=rng.choice([0.0, 0.5]))


# ------------------------------------------------------------------------------ MXFP4, plain
def _pitch(cols):
    return (cols // 32 + 15) // 16 * 16


def _plain_blocks(v):
    """fp32 [..., cols] -> scale bytes int32 [..., cols/32] and the scaled values [..., cols/32, 32]."""
    v = v.unflatten(-1, (-1, 32))
    amax = v.abs().amax(-1)
    biased = amax.view(torch.int32) >> 23
    b = torch.where(biased == 255, 255, (biased - 2).clamp(min=0))
    inv = ((254 - b.clamp(max=253)) << 23).view(F32)
    return b, v * inv.unsqueeze(-1)


def _plain_power(b):
    """2^(b - 127) of scale bytes b (int32), not a number for 255."""
    s = torch.where(b == 0, 1 << 22, b << 23).view(F32)
    return torch.where(b == 255, float("nan"), s)


def _plain_round(a):
    """Nearest E2M1 magnitude of a >= 0, ties to the even code, at most 6."""
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(a / step) * step).clamp(max=6.0)


def _plain_fake(x):
    """x rounded to MXFP4 along its last axis, as fp32 values."""
    b, v = _plain_blocks(x.float())
    q = torch.copysign(_plain_round(v.abs()), v)
    return (q * _plain_power(b).unsqueeze(-1)).flatten(-2)


def _plain_codes(x):
    """x along its last axis -> (codes uint8 [..., cols/2], scales uint8 [..., pitch])."""
    b, v = _plain_blocks(x.float())
    r = _plain_round(v.abs())
    mag = torch.where(r < 2, 2 * r, torch.where(r < 4, r + 2, r / 2 + 4)).to(torch.uint8)
    c = (mag | (torch.signbit(v).to(torch.uint8) << 3)).flatten(-2)
    codes = c[..., 0::2] | (c[..., 1::2] << 4)
    cols = x.shape[-1]
    scales = torch.zeros(*x.shape[:-1], _pitch(cols), dtype=torch.uint8, device=x.device)
    scales[..., :cols // 32] = b.to(torch.uint8)
    return codes, scales


def _table(dtype):
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=dtype, device="cuda")
    val = torch.cat([mag, -mag])
    byte = torch.arange(256, device="cuda")
    return torch.stack([val[byte & 15], val[byte >> 4]], -1)


def _plain_values(table, codes, scales, cols):
    """Codes and scales -> the fp32 values they stand for."""
    v = table[codes.int()].flatten(-2)
    f = _plain_power(scales[..., :cols // 32].int())
    return (v.unflatten(-1, (-1, 32)) * f.unsqueeze(-1)).flatten(-2)


# ------------------------------------------------------------------------------ the router, plain
def _plain_router(st):
    c, l = st["case"], st["logits"].float()
    T, E, K = c["T"], c["E"], c["K"]
    idx = torch.sort(l, dim=-1, descending=True, stable=True).indices[:, :K]
    if c["score"] == "softmax":
        e = torch.exp(l - l.amax(-1, keepdim=True))
        s = e / e.sum(-1, keepdim=True)
        q = s
    else:
        s = 1 / (1 + torch.exp(-l))
        q = s / s.sum(-1, keepdim=True)
    g = s.gather(1, idx)
    if c["normalise"]:
        g = g / g.sum(-1, keepdim=True)
    g = g * c.get("scale", 2.5)
    live = st["mask"] if st["mask"] is not None else torch.ones(T, dtype=torch.uint8, device="cuda")
    g = torch.where(live.unsqueeze(-1) != 0, g, 0.0)
    out = {"topk_idx": idx.int(), "gates": g}
    if c["segment"]:
        n = c["segment"]
        G = (T + n - 1) // n
        seg = torch.arange(T, device="cuda") // n
        tokens = torch.zeros(G, dtype=torch.int32, device="cuda").index_add_(0, seg, live.int())
        flat = (seg.unsqueeze(-1) * E + idx).flatten()
        counts = torch.zeros(G * E, dtype=torch.int32, device="cuda").index_add_(
            0, flat, live.int().repeat_interleave(K)).view(G, E)
        full = torch.zeros(G * n, E, dtype=F32, device="cuda")
        full[:T] = torch.where(live.unsqueeze(-1) != 0, q, 0.0)
        psum = full.view(G, n, E).sum(1)
        nt = tokens.clamp(min=1).float()
        per = E / (K * nt * nt) * (counts.float() * psum).sum(-1)
        out.update(counts=counts, prob_sum=psum, seg_tokens=tokens, loss=(per.sum() / G).view(1))
    return out


def _plain_router_backward(st):
    c, l = st["case"], st["logits"].float()
    T, E, K, n = c["T"], c["E"], c["K"], c["segment"]
    G = (T + n - 1) // n
    seg = torch.arange(T, device="cuda") // n
    idx, dg = st["topk_idx"].long(), st["d_gates"]
    nt = st["seg_tokens"].clamp(min=1).float()
    w = (st["d_loss"] * E / (G * K * nt * nt)).unsqueeze(-1) * st["counts"].float()
    w = w[seg]
    if c["score"] == "softmax":
        e = torch.exp(l - l.amax(-1, keepdim=True))
        s = e / e.sum(-1, keepdim=True)
    else:
        s = 1 / (1 + torch.exp(-l))
    sk = s.gather(1, idx)
    dk = c.get("scale", 2.5) * dg
    if c["normalise"]:
        total = sk.sum(-1, keepdim=True)
        dk = (dk - (dk * sk).sum(-1, keepdim=True) / total) / total
    ds = torch.zeros_like(s).scatter_(1, idx, dk)
    if c["score"] == "softmax":
        ds = ds + w
        dl = s * (ds - (s * ds).sum(-1, keepdim=True))
    else:
        total = s.sum(-1, keepdim=True)
        ds = ds + (w - (s * w).sum(-1, keepdim=True) / total) / total
        dl = ds * s * (1 - s)
    if st["mask"] is not None:
        dl = torch.where(st["mask"].unsqueeze(-1) != 0, dl, 0.0)
    return {"d_logits": dl.to(st["logits"].dtype)}


# ------------------------------------------------------------------------------ the product, plain
def _plain_grouped(values, weights, expert, place, most):
    """values [N, H] fp32, row i in slot place[i] of expert[i] (of the weights [n, Hp, H])."""
    a = torch.zeros(weights.shape[0], most, values.shape[1], dtype=F32, device="cuda")
    a[expert, place] = values
    return torch.bmm(a, weights.transpose(1, 2))[expert, place]


def _plain_product(st):
    c, H = st["case"], st["case"]["H"]
    a = _plain_values(st["table"], st["recv_q"], st["recv_s"], H)
    w = _plain_values(st["table"], st["w_q"][st["active"]], st["w_s"][st["active"]], H)
    y = _plain_grouped(a, w, st["expert"], st["place"], st["most"])
    return {"y": y.to(BF16)}


def _plain_layer(st):
    c = st["case"]
    K, H = c["K"], c["H"]
    out = _plain_router(st)
    w = _plain_values(st["table"], st["w_q"][st["active"]], st["w_s"][st["active"]], H)
    x = _plain_fake(st["x"])
    y = _plain_grouped(x[st["token"]], w, st["expert"], st["place"], st["most"])
    back = torch.empty_like(y)
    back[st["order"]] = y
    y = back.view(-1, K, c["Hp"])
    out["out"] = (y * out["gates"].unsqueeze(-1)).sum(1).to(BF16)
    return out


# ------------------------------------------------------------------------------ prepare
def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed((seed * 1000003 + salt) & 0x7FFFFFFF)


def _logits(case, T, seed, skew):
    """Router logits: normal noise on a popularity that falls off as a power of the rank."""
    E = case["E"]
    rank = torch.randperm(E, generator=_gen(seed, 1), device="cuda").float()
    l = torch.randn(T, E, generator=_gen(seed, 2), device="cuda") - skew * torch.log1p(rank)
    if case.get("off"):
        l[:, rank >= E - case["off"]] = -math.inf
    return l.to(BF16) if case.get("bf16") else l


def _router_state(case, seed):
    T = case["T"]
    st = {"case": case, "logits": _logits(case, T, seed, 0.5), "mask": None}
    if case["masked"]:
        st["mask"] = (torch.rand(T, generator=_gen(seed, 3), device="cuda")
                      >= case["masked"]).to(torch.uint8)
    return st


def _router_buffers(st):
    c = st["case"]
    T, E, K = c["T"], c["E"], c["K"]
    i32 = dict(dtype=torch.int32, device="cuda")
    st["out"] = {"topk_idx": torch.empty(T, K, **i32),
                 "gates": torch.empty(T, K, dtype=F32, device="cuda")}
    if c["segment"]:
        G = (T + c["segment"] - 1) // c["segment"]
        st["out"].update(counts=torch.empty(G, E, **i32),
                         prob_sum=torch.empty(G, E, dtype=F32, device="cuda"),
                         seg_tokens=torch.empty(G, **i32),
                         loss=torch.empty(1, dtype=F32, device="cuda"))


def _activations(rows, cols, seed):
    """Normal values with a size of each row's own and a few large columns."""
    x = torch.randn(rows, cols, generator=_gen(seed, 4), device="cuda")
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=_gen(seed, 5), device="cuda"))
    big = torch.rand(cols, generator=_gen(seed, 6), device="cuda") < 0.01
    return torch.where(big, x * 20, x).to(BF16)


def _weights(case, seed):
    """Quantised expert weights: codes [E, Hp, H/2] and scales [E, Hp, pitch]."""
    E, H, Hp = case["E"], case["H"], case["Hp"]
    q = torch.empty(E, Hp, H // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, Hp, _pitch(H), dtype=torch.uint8, device="cuda")
    g = _gen(seed, 7)
    step = max(1, (1 << 27) // (H * Hp))
    for e in range(0, E, step):
        n = min(step, E - e)
        w = torch.randn(n, Hp, H, generator=g, device="cuda") * 0.02
        q[e:e + n], s[e:e + n] = _plain_codes(w.to(BF16))
    return q, s


def _groups(st, ids, E, K):
    """Copies sorted by expert (ascending copy inside one): where the plain form puts each row."""
    flat = ids.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    count = torch.bincount(flat, minlength=E)
    start = torch.cumsum(count, 0) - count
    expert = flat[order]
    active = torch.nonzero(count).flatten()
    rename = torch.zeros(E, dtype=torch.long, device="cuda")
    rename[active] = torch.arange(active.numel(), device="cuda")
    st.update(order=order, token=order // K, active=active, expert=rename[expert],
              place=torch.arange(flat.numel(), device="cuda") - start[expert],
              most=int(count.max()), table=_table(F32))


def prepare(case, seed):
    op = case["op"]
    if op == "router":
        st = _router_state(case, seed)
        _router_buffers(st)
        if own:
            _own_router_handle(st)
        return st
    if op == "router_backward":
        st = _router_state(case, seed)
        fwd = _plain_router(st)
        st.update({k: fwd[k] for k in ("topk_idx", "counts", "seg_tokens")})
        st["d_gates"] = torch.randn(case["T"], case["K"], generator=_gen(seed, 8), device="cuda")
        # the loss coefficient a training program multiplies in, large enough to show
        st["d_loss"] = torch.rand(1, generator=_gen(seed, 9), device="cuda") * case["T"]
        st["d_logits"] = torch.empty_like(st["logits"])
        if own:
            _own_router_handle(st)
        return st
    if op == "quantize":
        st = {"case": case, "x": _activations(case["rows"], case["cols"], seed)}
        st["values"] = torch.empty_like(st["x"])
        st["q"] = torch.empty(case["rows"], case["cols"] // 2, dtype=torch.uint8, device="cuda")
        st["s"] = torch.empty(case["rows"], _pitch(case["cols"]), dtype=torch.uint8, device="cuda")
        return st
    if op == "quantize_weights":
        E, H, Hp = case["E"], case["H"], case["Hp"]
        w = (torch.randn(E, H, Hp, generator=_gen(seed, 7), device="cuda") * 0.02).to(BF16)
        return {"case": case, "w": w, "values": torch.empty(E, Hp, H, dtype=BF16, device="cuda"),
                "q": torch.empty(E, Hp, H // 2, dtype=torch.uint8, device="cuda"),
                "s": torch.empty(E, Hp, _pitch(H), dtype=torch.uint8, device="cuda")}
    if op == "product":
        T, E, K, H, Hp = (case[k] for k in ("T", "E", "K", "H", "Hp"))
        ids = torch.topk(_logits(case, T, seed, case["skew"]), K).indices.int()
        st = {"case": case, "ids": ids}
        _groups(st, ids, E, K)
        x_q, x_s = _plain_codes(_activations(T, H, seed))
        st["recv_q"], st["recv_s"] = x_q[st["token"]], x_s[st["token"]]
        st["w_q"], st["w_s"] = _weights(case, seed)
        st["y"] = torch.empty(T * K, Hp, dtype=BF16, device="cuda")
        if own:
            _own_plan_handle(st, dict(R=1, E=E, B=0, K=K, S=T, H=H, Hp=Hp, mode=1))
            _own().moonep_plan(st["d"], ids, st["ws"])
        return st
    R, E, K, S, H, Hp = (case[k] for k in ("R", "E", "K", "S", "H", "Hp"))
    T = R * S
    router = dict(case, T=T, segment=S, score="softmax", normalise=True, scale=1.0, masked=0.0)
    st = {"case": router, "logits": _logits(case, T, seed, case["skew"]), "mask": None,
          "x": _activations(T, H, seed)}
    _router_buffers(st)
    ids = torch.sort(st["logits"], dim=-1, descending=True, stable=True).indices[:, :K]
    _groups(st, ids, E, K)
    st["w_q"], st["w_s"] = _weights(case, seed)
    st["layer_out"] = torch.empty(T, Hp, dtype=BF16, device="cuda")
    if own:
        B = E // R
        _own_router_handle(st)
        _own_plan_handle(st, dict(R=R, E=E, B=B, K=K, S=S, H=H, Hp=Hp, mode=0))
        u8 = dict(dtype=torch.uint8, device="cuda")
        st["slot_q"] = torch.empty(R * B, Hp, H // 2, **u8)
        st["slot_s"] = torch.empty(R * B, Hp, _pitch(H), **u8)
        st["recv_q"] = torch.empty(T * K, H // 2, **u8)
        st["recv_s"] = torch.empty(T * K, _pitch(H), **u8)
        st["y"] = torch.empty(T * K, Hp, dtype=BF16, device="cuda")
    return st


# ------------------------------------------------------------------------------ the framework's calls
def _own():
    import perfectly_balanced_token_gb300 as mx
    return mx


def _own_router_handle(st):
    mx, c = _own(), st["case"]
    st["rd"] = mx.router_dims(c["T"], c["E"], c["K"], segment=c["segment"], score=c["score"],
                              normalise=c["normalise"], scale=c.get("scale", 2.5),
                              dtype=st["logits"].dtype)
    st["router_ws"] = torch.empty(mx.moonep_router_workspace_bytes(st["rd"]), dtype=torch.uint8,
                                  device="cuda")


def _own_plan_handle(st, sizes):
    mx = _own()
    st["d"] = mx.dims(**sizes)
    st["ws"] = torch.empty(mx.moonep_plan_workspace_bytes(st["d"]), dtype=torch.uint8, device="cuda")


def _own_router(st):
    o = st["out"]
    if "loss" in o:
        _own().moonep_router_forward(st["rd"], st["logits"], o["topk_idx"], o["gates"],
                                     token_mask=st["mask"], ws=st["router_ws"], counts=o["counts"],
                                     prob_sum=o["prob_sum"], seg_tokens=o["seg_tokens"],
                                     loss=o["loss"])
    else:
        _own().moonep_router_forward(st["rd"], st["logits"], o["topk_idx"], o["gates"],
                                     token_mask=st["mask"])
    return dict(o)


def _own_run(st):
    mx, op = _own(), st["case"]["op"]
    if op == "router":
        return _own_router(st)
    if op == "router_backward":
        mx.moonep_router_backward(st["rd"], st["logits"], st["topk_idx"], st["d_logits"],
                                  d_gates=st["d_gates"], token_mask=st["mask"],
                                  counts=st["counts"], seg_tokens=st["seg_tokens"],
                                  d_loss=st["d_loss"])
        return {"d_logits": st["d_logits"]}
    if op == "quantize":
        mx.moonep_mxfp4_quantize(st["x"], st["q"], st["s"])
        mx.moonep_mxfp4_dequantize(st["q"], st["s"], st["values"])
        return {"values": st["values"]}
    if op == "quantize_weights":
        mx.moonep_mxfp4_quantize_weights(st["w"], st["q"], st["s"])
        mx.moonep_mxfp4_dequantize(st["q"], st["s"], st["values"])
        return {"values": st["values"]}
    d, ws = st["d"], st["ws"]
    if op == "product":
        mx.moonep_mxfp4_grouped_gemm(d, ws, st["recv_q"], st["recv_s"], st["w_q"], st["w_s"],
                                     None, None, st["y"])
        return {"y": st["y"]}
    out = _own_router(st)
    mx.moonep_plan(d, out["topk_idx"], ws)
    mx.moonep_mxfp4_prefetch_weights(d, ws, st["w_q"], st["w_s"], st["slot_q"], st["slot_s"])
    mx.moonep_mxfp4_dispatch(d, ws, st["x"], st["recv_q"], st["recv_s"])
    mx.moonep_mxfp4_grouped_gemm(d, ws, st["recv_q"], st["recv_s"], st["w_q"], st["w_s"],
                                 st["slot_q"], st["slot_s"], st["y"])
    mx.moonep_combine(d, ws, st["y"], out["gates"], st["layer_out"])
    out["out"] = st["layer_out"]
    return out


def run(st):
    if own:
        return _own_run(st)
    op = st["case"]["op"]
    if op == "router":
        return _plain_router(st)
    if op == "router_backward":
        return _plain_router_backward(st)
    if op == "quantize":
        return {"values": _plain_fake(st["x"]).to(BF16)}
    if op == "quantize_weights":
        return {"values": _plain_fake(st["w"].transpose(1, 2)).to(BF16)}
    if op == "product":
        return _plain_product(st)
    return _plain_layer(st)


# ------------------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op in ("router", "router_backward", "layer"):
        T = case["T"] if op != "layer" else case["R"] * case["S"]
        E, K = case["E"], case["K"]
        n = case["segment"] if op != "layer" else case["S"]
        G = (T + n - 1) // n if n else 0
        lb = 2 if case.get("bf16") else 4
        router = T * E * lb + T * K * 8 + G * E * 8 + (T if case.get("masked") else 0)
    if op == "router":  # per value a compare, a subtraction, an exponential, two sums
        return {"bytes": router, "flops": 5 * T * E}
    if op == "router_backward":
        return {"bytes": router + T * E * lb - G * E * 4, "flops": 8 * T * E}
    if op == "quantize":  # bf16 in, the codes and scales out and in again, bf16 out
        n = case["rows"] * case["cols"]
        return {"bytes": 4 * n + 2 * n * (1 / 2 + 1 / 32), "flops": 4 * n}
    if op == "quantize_weights":
        n = case["E"] * case["H"] * case["Hp"]
        return {"bytes": 4 * n + 2 * n * (1 / 2 + 1 / 32), "flops": 4 * n}
    E, K, H, Hp = case["E"], case["K"], case["H"], case["Hp"]
    T = case["T"] if op == "product" else case["R"] * case["S"]
    N = T * K
    active = E * (1 - (1 - K / E) ** T)  # experts that some token picks, were they alike
    weights = active * Hp * H * (1 / 2 + 1 / 32)
    flops = 2 * N * H * Hp
    if op == "product":
        return {"bytes": N * H * (1 / 2 + 1 / 32) + weights + N * Hp * 2, "flops": flops}
    return {"bytes": router + T * H * 2 + weights + T * Hp * 2, "flops": flops}


# ------------------------------------------------------------------------------ 64 bits
def _exact_router(st):
    c = st["case"]
    l = st["logits"].double()
    T, E, K = c["T"], c["E"], c["K"]
    rank = torch.argsort(-l, dim=-1, stable=True)[:, :K]
    chosen = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_(1, rank, 1.0)
    if c["score"] == "softmax":
        s = torch.softmax(l, -1)
        q = s
    else:
        s = torch.sigmoid(l)
        q = s / s.sum(-1, keepdim=True)
    live = torch.ones(T, 1, dtype=torch.float64, device="cuda")
    if st["mask"] is not None:
        live = st["mask"].double().view(T, 1)
    weight = s / (s * chosen).sum(-1, keepdim=True) if c["normalise"] else s
    gates = (weight * live).gather(1, rank) * c.get("scale", 2.5)
    return chosen, s, q, live, rank, gates


def _exact_loss(st, chosen, q, live):
    c = st["case"]
    n = c["segment"]
    G = (c["T"] + n - 1) // n
    counts, sums, losses = [], [], []
    for g in range(G):
        part = slice(g * n, min(c["T"], (g + 1) * n))
        tokens = live[part].sum()
        f = (chosen[part] * live[part]).sum(0)
        p = (q[part] * live[part]).sum(0)
        counts.append(f)
        sums.append(p)
        losses.append(torch.where(tokens > 0, c["E"] * (f * p).sum()
                                  / (c["K"] * tokens.clamp(min=1) ** 2), 0.0))
    return torch.stack(counts), torch.stack(sums), torch.stack(losses).mean().view(1)


def _exact_router_outputs(st):
    chosen, s, q, live, rank, gates = _exact_router(st)
    out = {"topk_idx": None, "gates": gates}
    if st["case"]["segment"]:
        _, sums, loss = _exact_loss(st, chosen, q, live)
        out.update(counts=None, prob_sum=sums, seg_tokens=None, loss=loss)
    return out


def _exact_router_backward(st):
    """The gradient of <d_gates, gates> + d_loss * loss by automatic differentiation, with the
    choice of experts and their counts held fixed."""
    c = st["case"]
    l = st["logits"].double().requires_grad_(True)
    idx = st["topk_idx"].long()
    s = torch.softmax(l, -1) if c["score"] == "softmax" else torch.sigmoid(l)
    q = s / s.sum(-1, keepdim=True)
    live = torch.ones(c["T"], 1, dtype=torch.float64, device="cuda")
    if st["mask"] is not None:
        live = st["mask"].double().view(-1, 1)
    g = s.gather(1, idx)
    if c["normalise"]:
        g = g / g.sum(-1, keepdim=True)
    n = c["segment"]
    G = (c["T"] + n - 1) // n
    total = (g * c.get("scale", 2.5) * live * st["d_gates"].double()).sum()
    for k in range(G):
        part = slice(k * n, min(c["T"], (k + 1) * n))
        tokens = st["seg_tokens"][k].double().clamp(min=1)
        p = (q[part] * live[part]).sum(0)
        total = total + st["d_loss"].double()[0] * c["E"] / (G * c["K"] * tokens ** 2) * (
            st["counts"][k].double() * p).sum()
    return {"d_logits": torch.autograd.grad(total, l)[0]}


def _two_to(n):
    """2^n in 64 bits, exactly, for whole n."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _exact_fake(x):
    """Nearest MXFP4 values along the last axis, by comparison with the midpoints."""
    v = x.double().unflatten(-1, (-1, 32))
    top = v.abs().amax(-1, keepdim=True)
    _, e = torch.frexp(top)  # top = m 2^e, 1/2 <= m < 1
    power = torch.where(top > 0, (e - 3).clamp(min=-127), -127)
    a = v.abs() * _two_to(-power)
    code = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    return (grid[code] * torch.sign(v) * _two_to(power)).flatten(-2)


def _exact_codes(codes, scales, cols):
    lo, hi = (codes & 15).long(), (codes >> 4).long()
    c = torch.stack([lo, hi], -1).flatten(-2)
    m = (c & 7).double()
    big = _two_to((c & 7) // 2 - 1) * (1 + 0.5 * (c & 1))
    v = torch.where(m < 2, m / 2, big) * (1 - 2 * (c >> 3)).double()
    s = _two_to(scales[..., :cols // 32].long() - 127)
    return v * s.repeat_interleave(32, -1)


def _exact_product(st, rows_of):
    c = st["case"]
    y = torch.empty(st["expert"].numel(), c["Hp"], dtype=torch.float64, device="cuda")
    for i, e in enumerate(st["active"].tolist()):
        at = torch.nonzero(st["expert"] == i).flatten()
        w = _exact_codes(st["w_q"][e], st["w_s"][e], c["H"])
        y[at] = rows_of(at) @ w.T
    return y


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "router":
        return _exact_router_outputs(st)
    if op == "router_backward":
        return _exact_router_backward(st)
    if op == "quantize":
        return {"values": torch.cat([_exact_fake(p) for p in st["x"].split(4096)])}
    if op == "quantize_weights":
        return {"values": torch.stack([_exact_fake(w.T.contiguous()) for w in st["w"]])}
    if op == "product":
        return {"y": _exact_product(st, lambda at: _exact_codes(st["recv_q"][at], st["recv_s"][at],
                                                                case["H"]))}
    out = _exact_router_outputs(st)
    y = _exact_product(st, lambda at: _exact_fake(st["x"][st["token"][at]]))
    back = torch.empty_like(y)
    back[st["order"]] = y
    out["out"] = (back.view(-1, case["K"], case["Hp"]) * out["gates"].unsqueeze(-1)).sum(1)
    return out
