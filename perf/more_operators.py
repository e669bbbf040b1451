"""The feed-forward network of the experts and the end of the layer, as cases to measure: a product
with bias, activation and residual (a shared expert, the router's logits), its gradient, the
activation's gradient with that of the bias, the experts' product with bias and activation, and the
combine with dropout and residual, forward and backward.

``own = False`` computes each operator in a plain form (elementary torch operations in 32 bits,
rounded once at the end); ``own = True`` makes the calls a user of the framework makes.

Activations of z = x w + bias: none, relu, gelu (by the error function), silu, and swiglu, where the
first half of z's columns are gates and a = silu(gate) * second half.

Dropout of the element i of an output counted row by row: Philox4x32 of ten rounds (Salmon, Moraes,
Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) with the seed as its key and
(i / 8 in 64 bits, offset in 64 bits) as its counter gives four words, so eight 16-bit numbers, low
halves first; the i % 8-th of them is below round(65536 p) for an element that is dropped.  What stays
is multiplied by 65536 / (65536 - round(65536 p)).
"""
import math

import torch

own = False

BF16 = torch.bfloat16
F32 = torch.float32
F64 = torch.float64


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # a shared expert's gate and up projections for one decoded token: the weights are what is read
        dict(name="linear 1 token swiglu", op="linear", T=1, K=7168, N=4096, act="swiglu", bias=False,
             residual=False, f32=False, z=False),
        # the router's logits of a rank's micro-batch, in 32 bits
        dict(name="linear router logits 8192x384", op="linear", T=8192, K=7168, N=384, act="none",
             bias=True, residual=False, f32=True, z=False),
        # a down projection added to the layer's input, sizes that end inside every tile
        dict(name="linear odd 777 residual", op="linear", T=777, K=2056, N=1000, act="none", bias=True,
             residual=True, f32=False, z=False),
        # the gate and up projections of eight ranks x 8192 tokens in training (z kept for the gradient)
        dict(name="linear 65536 swiglu", op="linear", T=65536, K=7168, N=4096, act="swiglu", bias=True,
             residual=False, f32=False, z=True),
        # gradients of a small projection
        dict(name="linear backward 1000 odd", op="linear_backward", T=1000, K=1032, N=520),
        # gradients of the shared expert's up projection
        dict(name="linear backward 32768", op="linear_backward", T=32768, K=7168, N=4096),
        # through the shared expert's activation, with the bias's gradient
        dict(name="activation backward 32768x4096 swiglu", op="act_backward", T=32768, E=0, K=1,
             N=4096, act="swiglu", skew=0.0),
        # through the routed experts' activation: a bias and so a sum for each expert
        dict(name="activation backward 64 experts gelu", op="act_backward", T=8192, E=64, K=4, N=2048,
             act="gelu", skew=0.5),
        # a decoding step of the experts' gate and up projections: a few copies an expert
        dict(name="experts decode 16 tokens", op="experts", T=16, E=128, K=8, H=7168, Hp=4096,
             act="swiglu", bias=False, z=False, skew=0.3),
        # the width of a small configuration, few rows an expert, z kept
        dict(name="experts 3000 x 60 experts gelu", op="experts", T=3000, E=60, K=4, H=1024, Hp=576,
             act="gelu", bias=True, z=True, skew=0.5),
        # a training micro-batch: about 2000 rows an expert
        dict(name="experts 131072 rows swiglu", op="experts", T=16384, E=64, K=8, H=7168, Hp=4096,
             act="swiglu", bias=True, z=True, skew=0.3),
        # the end of the layer and its gradient, four ranks x 8192 tokens of the widest configuration
        dict(name="combine dropout 32768x7168", op="combine_dropout", T=32768, E=64, K=8, Hp=7168,
             p=0.1, residual=True, skew=0.3),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _log_step(rng, lo, hi, step):
    return step * _log_int(rng, lo // step, hi // step)


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "act_backward", "experts", "experts",
                     "combine_dropout"])
    act = rng.choice(["none", "relu", "gelu", "silu", "swiglu", "swiglu"])
    half = rng.random() < 0.5
    if op in ("linear", "linear_backward"):
        K, N = _log_step(rng, 64, 7168, 8), _log_step(rng, 64, 4096, 16)
        T = _log_int(rng, 1, 65536 if op == "linear" else 32768)
        if op == "linear_backward":
            return dict(op=op, T=T, K=K, N=N)
        return dict(op=op, T=T, K=K, N=N, act=act, bias=rng.random() < 0.5,
                    residual=rng.random() < 0.5, f32=rng.random() < 0.3, z=half)
    if op == "act_backward":
        E = rng.choice([0, _log_int(rng, 2, 128)])
        K = rng.randint(1, min(8, E)) if E else 1
        return dict(op=op, T=_log_int(rng, 1, 32768 // K), E=E, K=K,
                    N=_log_step(rng, 128, 4096, 128), act=act if act != "none" else "silu",
                    skew=rng.choice([0.0, 0.5]))
    E = _log_int(rng, 4, 64)
    K = rng.randint(1, min(8, E))
    if op == "experts":
        return dict(op=op, T=_log_int(rng, 1, 16384), E=E, K=K, H=_log_step(rng, 64, 7168, 64),
                    Hp=_log_step(rng, 128, 4096, 128), act=act, bias=rng.random() < 0.5, z=half,
                    skew=rng.choice([0.0, 0.3, 0.6]))
    return dict(op=op, T=_log_int(rng, 1, 32768), E=E, K=K, Hp=_log_step(rng, 64, 7168, 64),
                p=rng.choice([0.0, 0.1, 0.25, 0.5]), residual=half, skew=rng.choice([0.0, 0.5]))


# ------------------------------------------------------------------------------ plain forms
def _plain_act(z, act):
    """The activation of z in 32 bits."""
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "swiglu":
        g, u = z.chunk(2, -1)
        return g / (1 + torch.exp(-g)) * u
    return z


def _plain_slope(z, act):
    """d act / d z of the activations that take one value."""
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi)))
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def _plain_act_grad(z, d_out, act):
    if act != "swiglu":
        return d_out * _plain_slope(z, act)
    g, u = z.chunk(2, -1)
    s = 1 / (1 + torch.exp(-g))
    return torch.cat([d_out * u * _plain_slope(g, "silu"), d_out * g * s], -1)


def _plain_linear(st):
    c = st["case"]
    z = st["x"].float() @ st["w"].float()
    if c["bias"]:
        z = z + st["bias"]
    y = _plain_act(z, c["act"])
    if c["residual"]:
        y = y + st["residual"].float()
    out = {"out": y.to(F32 if c["f32"] else BF16)}
    if c["z"]:
        out["z"] = z.to(BF16)
    return out


def _plain_linear_backward(st):
    d_z = st["d_z"].float()
    return {"d_x": (d_z @ st["w"].float().t()).to(BF16), "d_w": st["x"].float().t() @ d_z}


def _plain_act_backward(st):
    c = st["case"]
    d_z = _plain_act_grad(st["z"].float(), st["d_out"].float(), c["act"])
    if not c["E"]:
        return {"d_z": d_z.to(BF16), "d_bias": d_z.sum(0)}
    sums = torch.zeros(c["E"], c["N"], dtype=F32, device="cuda")
    for e, a, b in st["groups"]:
        sums[e] = d_z[a:b].sum(0)
    return {"d_z": d_z.to(BF16), "d_bias": sums}


def _plain_experts(st):
    c = st["case"]
    cols = c["Hp"] // 2 if c["act"] == "swiglu" else c["Hp"]
    rows = c["T"] * c["K"]
    y = torch.empty(rows, cols, dtype=BF16, device="cuda")
    z = torch.empty(rows, c["Hp"], dtype=BF16, device="cuda") if c["z"] else None
    for e, a, b in st["groups"]:
        v = st["recv"][a:b].float() @ st["w"][e].float()
        if c["bias"]:
            v = v + st["bias"][e]
        y[a:b] = _plain_act(v, c["act"]).to(BF16)
        if c["z"]:
            z[a:b] = v.to(BF16)
    return {"y": y, "z": z} if c["z"] else {"y": y}


_M32 = 0xFFFFFFFF


def _plain_numbers(rng, start, n):
    """n 16-bit random numbers (a multiple of 8) from element `start` (another) on, int64."""
    g = torch.arange(start // 8, (start + n) // 8, device="cuda")
    offset = rng[1] & 0x7FFFFFFFFFFFFFFF
    c = [g & _M32, g >> 32, (offset & _M32).expand_as(g), (offset >> 32).expand_as(g)]
    k0, k1 = rng[0] & _M32, (rng[0] >> 32) & _M32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((b >> 32) & _M32) ^ c[1] ^ k0, b & _M32, ((a >> 32) & _M32) ^ c[3] ^ k1, a & _M32]
        k0, k1 = (k0 + 0x9E3779B9) & _M32, (k1 + 0xBB67AE85) & _M32
    w = torch.stack(c, -1)
    return torch.stack([w & 0xFFFF, w >> 16], -1).view(-1)


def _plain_combine_dropout(st):
    c = st["case"]
    T, K, Hp = c["T"], c["K"], c["Hp"]
    cut = int(math.floor(c["p"] * 65536 + 0.5))
    scale = 65536.0 / (65536 - cut)
    out = torch.empty(T, Hp, dtype=BF16, device="cuda")
    d_y = torch.empty(T * K, Hp, dtype=BF16, device="cuda")
    d_gates = torch.empty(T, K, dtype=F32, device="cuda")
    step = 2048
    for t in range(0, T, step):
        n = min(step, T - t)
        rows = st["dst"][t:t + n].view(-1)
        y = st["y"][rows].float().view(n, K, Hp)
        gates = st["gates"][t:t + n].unsqueeze(-1)
        o = (y * gates).sum(1)
        d = st["d_out"][t:t + n].float()
        if cut:
            keep = _plain_numbers(st["rng"], t * Hp, n * Hp).view(n, Hp) >= cut
            o = torch.where(keep, o * scale, 0.0)
            d = torch.where(keep, d * scale, 0.0)
        if c["residual"]:
            o = o + st["residual"][t:t + n].float()
        out[t:t + n] = o.to(BF16)
        d_gates[t:t + n] = (y * d.unsqueeze(1)).sum(-1)
        d_y[rows] = (d.unsqueeze(1) * gates).to(BF16).view(-1, Hp)
    return {"out": out, "d_y": d_y, "d_gates": d_gates}


# ------------------------------------------------------------------------------ prepare
def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed((seed * 1000003 + salt) & 0x7FFFFFFF)


def _normal(seed, salt, *shape, size=1.0, dtype=BF16):
    """Normal values, drawn in pieces of 2^27."""
    n = math.prod(shape)
    out, g = torch.empty(n, dtype=dtype, device="cuda"), _gen(seed, salt)
    for a in range(0, n, 1 << 27):
        b = min(n, a + (1 << 27))
        out[a:b] = torch.randn(b - a, generator=g, device="cuda") * size
    return out.view(*shape)


def _activations(seed, rows, cols):
    """Normal values with a size of each row's own and a few large columns."""
    out = torch.empty(rows, cols, dtype=BF16, device="cuda")
    g = _gen(seed, 1)
    size = torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 8.0, 1.0)
    for a in range(0, rows, 16384):
        b = min(rows, a + 16384)
        row = torch.exp(0.3 * torch.randn(b - a, 1, generator=g, device="cuda"))
        out[a:b] = torch.randn(b - a, cols, generator=g, device="cuda") * row * size
    return out


def _routing(st, seed):
    """K experts of every token, by a popularity that falls off as a power of the rank; the copies
    sorted by expert, ascending inside one, are the rows of the experts' buffers."""
    c = st["case"]
    T, E, K = c["T"], c["E"], c["K"]
    rank = torch.randperm(E, generator=_gen(seed, 2), device="cuda").float()
    like = torch.randn(T, E, generator=_gen(seed, 3), device="cuda") - c["skew"] * torch.log1p(rank)
    st["ids"] = torch.topk(like, K).indices.int()
    flat = st["ids"].reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    ends = torch.cumsum(torch.bincount(flat, minlength=E), 0).tolist()
    st["groups"] = [(e, a, b) for e, (a, b) in enumerate(zip([0] + ends[:-1], ends)) if b > a]
    st["order"] = order
    dst = torch.empty_like(order)
    dst[order] = torch.arange(order.numel(), device="cuda")
    st["dst"] = dst.view(T, K)


def prepare(case, seed):
    op, st = case["op"], {"case": case}
    if op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        cols = N // 2 if case["act"] == "swiglu" else N
        st.update(x=_activations(seed, T, K), w=_normal(seed, 4, K, N, size=1 / math.sqrt(K)),
                  bias=_normal(seed, 5, N, size=0.5, dtype=F32) if case["bias"] else None,
                  residual=_normal(seed, 6, T, cols) if case["residual"] else None)
        if own:
            st.update(out=torch.empty(T, cols, dtype=F32 if case["f32"] else BF16, device="cuda"),
                      z=torch.empty(T, N, dtype=BF16, device="cuda") if case["z"] else None,
                      d=_own().linear_dims(T, K, N, act=case["act"],
                                           out_dtype=F32 if case["f32"] else BF16),
                      status=torch.zeros(1, dtype=torch.int32, device="cuda"))
        return st
    if op == "linear_backward":
        T, K, N = case["T"], case["K"], case["N"]
        st.update(x=_activations(seed, T, K), w=_normal(seed, 4, K, N, size=1 / math.sqrt(K)),
                  d_z=_normal(seed, 7, T, N))
        if own:
            st.update(d_x=torch.empty(T, K, dtype=BF16, device="cuda"),
                      d_w=torch.empty(K, N, dtype=F32, device="cuda"),
                      d=_own().linear_dims(T, K, N),
                      status=torch.zeros(1, dtype=torch.int32, device="cuda"))
        return st
    if op == "act_backward":
        T, E, K, N = case["T"], case["E"], case["K"], case["N"]
        rows = T * K
        st.update(z=_normal(seed, 8, rows, N, size=1.5),
                  d_out=_normal(seed, 9, rows, N // 2 if case["act"] == "swiglu" else N))
        if E:
            _routing(st, seed)
        if own:
            st.update(d_z=torch.empty(rows, N, dtype=BF16, device="cuda"),
                      d_bias=torch.empty(max(E, 1) * N, dtype=F32, device="cuda").view(
                          (E, N) if E else (N,)))
            if E:
                # (the experts' products' depth, which a plan needs and this operator does not)
                _own_plan(st, dict(R=1, E=E, B=0, K=K, S=T, H=64, Hp=N, mode=1))
                size = _own().moonep_grouped_act_backward_workspace_bytes(st["d"])
            else:
                size = _own().moonep_act_backward_workspace_bytes(rows, N)
            st["scratch"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        return st
    if op == "experts":
        T, E, K, H, Hp = (case[k] for k in ("T", "E", "K", "H", "Hp"))
        _routing(st, seed)
        st["recv"] = _activations(seed, T, H)[st["order"] // K]
        st["w"] = _normal(seed, 4, E, H, Hp, size=1 / math.sqrt(H))
        st["bias"] = _normal(seed, 5, E, Hp, size=0.5, dtype=F32) if case["bias"] else None
        if own:
            cols = Hp // 2 if case["act"] == "swiglu" else Hp
            st["y"] = torch.empty(T * K, cols, dtype=BF16, device="cuda")
            st["z"] = torch.empty(T * K, Hp, dtype=BF16, device="cuda") if case["z"] else None
            _own_plan(st, dict(R=1, E=E, B=0, K=K, S=T, H=H, Hp=Hp, mode=1))
        return st
    T, E, K, Hp = (case[k] for k in ("T", "E", "K", "Hp"))
    _routing(st, seed)
    gates = torch.rand(T, K, generator=_gen(seed, 10), device="cuda") + 0.05
    st.update(y=_normal(seed, 11, T * K, Hp), gates=gates / gates.sum(-1, keepdim=True),
              d_out=_normal(seed, 12, T, Hp),
              residual=_normal(seed, 6, T, Hp) if case["residual"] else None,
              rng=torch.randint(0, 1 << 62, (2,), generator=_gen(seed, 13), device="cuda"))
    if own:
        st.update(out=torch.empty(T, Hp, dtype=BF16, device="cuda"),
                  d_y=torch.empty(T * K, Hp, dtype=BF16, device="cuda"),
                  d_gates=torch.empty(T, K, dtype=F32, device="cuda"))
        _own_plan(st, dict(R=1, E=E, B=0, K=K, S=T, H=64, Hp=Hp, mode=1))
    return st


# ------------------------------------------------------------------------------ the framework's calls
def _own():
    import perfectly_balanced_token_gb300 as mx
    return mx


def _own_plan(st, sizes):
    mx = _own()
    st["d"] = mx.dims(**sizes)
    st["ws"] = torch.empty(mx.moonep_plan_workspace_bytes(st["d"]), dtype=torch.uint8, device="cuda")
    mx.moonep_plan(st["d"], st["ids"], st["ws"])


def _own_run(st):
    mx, c = _own(), st["case"]
    if c["op"] == "linear":
        mx.moonep_linear(st["d"], st["x"], st["w"], st["out"], st["status"], bias=st["bias"],
                         residual=st["residual"], z=st["z"])
        return {"out": st["out"], "z": st["z"]} if c["z"] else {"out": st["out"]}
    if c["op"] == "linear_backward":
        mx.moonep_linear_dx(st["d"], st["d_z"], st["w"], st["d_x"], st["status"])
        mx.moonep_linear_dw(st["d"], st["x"], st["d_z"], st["d_w"], st["status"])
        return {"d_x": st["d_x"], "d_w": st["d_w"]}
    if c["op"] == "act_backward":
        if c["E"]:
            mx.moonep_grouped_act_backward(st["d"], st["ws"], st["z"], st["d_out"], st["d_z"],
                                           act=c["act"], d_bias=st["d_bias"], scratch=st["scratch"])
        else:
            mx.moonep_act_backward(st["z"], st["d_out"], st["d_z"], act=c["act"],
                                   d_bias=st["d_bias"], scratch=st["scratch"])
        return {"d_z": st["d_z"], "d_bias": st["d_bias"]}
    if c["op"] == "experts":
        mx.moonep_grouped_gemm_act(st["d"], st["ws"], st["recv"], st["w"], None, st["y"],
                                   act=c["act"], bias=st["bias"], z=st["z"])
        return {"y": st["y"], "z": st["z"]} if c["z"] else {"y": st["y"]}
    mx.moonep_combine_dropout(st["d"], st["ws"], st["y"], st["gates"], st["out"],
                              residual=st["residual"], p=c["p"], rng=st["rng"])
    mx.moonep_combine_dropout_backward(st["d"], st["ws"], st["y"], st["gates"], st["d_out"],
                                       st["d_y"], st["d_gates"], p=c["p"], rng=st["rng"])
    return {"out": st["out"], "d_y": st["d_y"], "d_gates": st["d_gates"]}


def run(st):
    if own:
        return _own_run(st)
    return {"linear": _plain_linear, "linear_backward": _plain_linear_backward,
            "act_backward": _plain_act_backward, "experts": _plain_experts,
            "combine_dropout": _plain_combine_dropout}[st["case"]["op"]](st)


# ------------------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    cols = case.get("N", case.get("Hp"))
    outs = cols // 2 if case.get("act") == "swiglu" else cols
    if op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        b = 2 * T * K + 2 * K * N + T * outs * (4 if case["f32"] else 2)
        b += 4 * N * case["bias"] + 2 * T * outs * case["residual"] + 2 * T * N * case["z"]
        return {"bytes": b, "flops": 2 * T * K * N}
    if op == "linear_backward":  # x, w and d_z in, d_x and d_w out
        T, K, N = case["T"], case["K"], case["N"]
        return {"bytes": 4 * T * K + 2 * T * N + 6 * K * N, "flops": 4 * T * K * N}
    rows = case["T"] * case["K"]
    if op == "act_backward":  # about ten operations a value
        return {"bytes": rows * (4 * cols + 2 * outs) + 4 * max(case["E"], 1) * cols,
                "flops": 10 * rows * cols}
    if op == "experts":
        E, K, T = case["E"], case["K"], case["T"]
        active = E * (1 - (1 - K / E) ** T)  # experts that some token picks, were they alike
        b = rows * (2 * case["H"] + 2 * outs + 2 * cols * case["z"])
        b += active * cols * (2 * case["H"] + 4 * case["bias"])
        return {"bytes": b, "flops": 2 * rows * case["H"] * cols}
    T = case["T"]  # y read by either pass, d_y written; out, d_out and the residual; gates, d_gates
    b = 6 * rows * cols + T * cols * (4 + 2 * case["residual"]) + 12 * rows + 8 * rows
    return {"bytes": b, "flops": 5 * rows * cols}


# ------------------------------------------------------------------------------ 64 bits
def _exact_sigmoid(z):
    return 0.5 * (1 + torch.tanh(0.5 * z))


def _exact_act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if act == "silu":
        return z * _exact_sigmoid(z)
    if act == "swiglu":
        f = z.shape[-1] // 2
        return z[..., :f] * _exact_sigmoid(z[..., :f]) * z[..., f:]
    return z


def _exact_numbers(rng, start, n):
    """The same 16-bit numbers, by products of 16-bit halves."""
    def wide(a, m):  # a < 2^32 times the constant m: (high word, low word)
        lo, hi = a * (m & 0xFFFF), a * (m >> 16)
        s = (lo >> 16) + hi
        return s >> 16, ((s & 0xFFFF) << 16) | (lo & 0xFFFF)

    seed, offset = (int(v) for v in rng.tolist())
    g = torch.arange(start // 8, (start + n) // 8, device="cuda")
    x = [g % (1 << 32), g // (1 << 32), torch.full_like(g, offset % (1 << 32)),
         torch.full_like(g, offset >> 32)]
    for r in range(10):
        k0 = (seed + r * 0x9E3779B9) % (1 << 32)
        k1 = ((seed >> 32) + r * 0xBB67AE85) % (1 << 32)
        h0, l0 = wide(x[0], 0xD2511F53)
        h1, l1 = wide(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ k0, l1, h0 ^ x[3] ^ k1, l0]
    parts = []
    for w in x:
        parts += [w % 65536, w // 65536]
    return torch.stack(parts, 1).reshape(-1)


def _exact_combine_dropout(st):
    c = st["case"]
    T, K, Hp = c["T"], c["K"], c["Hp"]
    cut = round(c["p"] * 65536)
    out = torch.empty(T, Hp, dtype=F64, device="cuda")
    d_y = torch.empty(T * K, Hp, dtype=F64, device="cuda")
    d_gates = torch.empty(T, K, dtype=F64, device="cuda")
    step = 1024
    for t in range(0, T, step):
        n = min(step, T - t)
        factor = torch.ones(n, Hp, dtype=F64, device="cuda")
        if cut:
            r = _exact_numbers(st["rng"], t * Hp, n * Hp).view(n, Hp)
            factor = (r >= cut).double() * (65536 / (65536 - cut))
        o = torch.zeros(n, Hp, dtype=F64, device="cuda")
        d = st["d_out"][t:t + n].double() * factor
        for k in range(K):
            at = st["dst"][t:t + n, k]
            y, g = st["y"][at].double(), st["gates"][t:t + n, k].double().unsqueeze(-1)
            o += g * y
            d_y[at] = g * d
            d_gates[t:t + n, k] = (y * d).sum(-1)
        o *= factor
        if c["residual"]:
            o += st["residual"][t:t + n].double()
        out[t:t + n] = o
    return {"out": out, "d_y": d_y, "d_gates": d_gates}


def _exact_act_backward(st):
    """By automatic differentiation, in pieces of rows."""
    c = st["case"]
    d_z = torch.empty(st["z"].shape, dtype=F64, device="cuda")
    for a in range(0, d_z.shape[0], 8192):
        z = st["z"][a:a + 8192].double().requires_grad_(True)
        total = (_exact_act(z, c["act"]) * st["d_out"][a:a + 8192].double()).sum()
        d_z[a:a + 8192] = torch.autograd.grad(total, z)[0]
    if not c["E"]:
        return {"d_z": d_z, "d_bias": d_z.sum(0)}
    sums = [d_z[0:0].sum(0)] * c["E"]
    for e, a, b in st["groups"]:
        sums[e] = d_z[a:b].sum(0)
    return {"d_z": d_z, "d_bias": torch.stack(sums)}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        w = st["w"].double()
        outs, zs = [], []
        for a in range(0, case["T"], 16384):
            z = st["x"][a:a + 16384].double() @ w
            if case["bias"]:
                z += st["bias"].double()
            y = _exact_act(z, case["act"])
            if case["residual"]:
                y = y + st["residual"][a:a + 16384].double()
            outs.append(y)
            zs.append(z if case["z"] else None)
        out = {"out": torch.cat(outs)}
        if case["z"]:
            out["z"] = torch.cat(zs)
        return out
    if op == "linear_backward":
        d_z = st["d_z"].double()
        return {"d_x": torch.mm(d_z, st["w"].double().T),
                "d_w": torch.mm(st["x"].double().T, d_z)}
    if op == "act_backward":
        return _exact_act_backward(st)
    if op == "experts":
        ys, zs = [], []
        for e, a, b in st["groups"]:
            z = st["recv"][a:b].double() @ st["w"][e].double()
            if case["bias"]:
                z += st["bias"][e].double()
            ys.append(_exact_act(z, case["act"]))
            if case["z"]:
                zs.append(z)
        return {"y": torch.cat(ys), "z": torch.cat(zs)} if case["z"] else {"y": torch.cat(ys)}
    return _exact_combine_dropout(st)
