"""One MoE layer with its router: top-K and balance loss, the balanced plan, the expert
product in MXFP4, and the gradient back to the router's weights.

    python examples/mxfp4_layer.py [--steps N]

The router starts out skewed towards a few experts.  Each step runs

    router_forward -> plan -> mxfp4_prefetch_weights -> mxfp4_dispatch
      -> mxfp4_grouped_gemm -> combine
    combine_backward -> router_backward

and lets the router's weights follow the gradient of <out, out>/2 - <out, target>
plus the balance loss.  Prints, per step, the balance loss, the load of the busiest
expert over the mean one, and how far the output is from the one of the bf16 calls.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import perfectly_balanced_token_gb300 as mx  # noqa: E402
from perfectly_balanced_token_gb300 import synthetic as syn  # noqa: E402


class Layer:
    """Buffers of one layer, kept from step to step as a training program keeps them."""

    def __init__(self, w: syn.Workload, seed=0):
        self.w, dev, bf = w, "cuda", torch.bfloat16
        T, pitch = w.R * w.S, mx.mxfp4_scale_pitch(w.H)
        self.d = mx.dims(w.R, w.E, w.B, w.K, w.S, w.H, w.Hp)
        self.ws = mx.PlanWorkspace(self.d)
        self.rd = mx.router_dims(T, w.E, w.K, segment=w.S, score="softmax")
        u8 = dict(dtype=torch.uint8, device=dev)
        self.router_ws = torch.empty(mx.moonep_router_workspace_bytes(self.rd), **u8)
        # tokens have a mean of 0.5 (see main), so the second term adds -0.7 log(rank) to an
        # expert's logits
        rank = torch.randperm(w.E, device=dev).float()
        self.w_router = (torch.randn(w.H, w.E, device=dev) / w.H ** 0.5
                         - 0.7 / (0.5 * w.H) * torch.log1p(rank))
        self.w_home = syn.normal_bf16((w.E, w.H, w.Hp), w.H ** -0.5, seed + 2, dev)
        self.w_slot = torch.zeros(w.R * w.B * w.H * w.Hp, dtype=bf, device=dev)
        # the experts' weights are quantised once
        self.home = (torch.empty(w.E, w.Hp, w.H // 2, **u8), torch.empty(w.E, w.Hp, pitch, **u8))
        mx.moonep_mxfp4_quantize_weights(self.w_home, *self.home)
        nb = w.R * w.B * w.Hp
        self.slot = (torch.empty(nb, w.H // 2, **u8), torch.empty(nb, pitch, **u8))
        self.recv = (torch.empty(w.N, w.H // 2, **u8), torch.empty(w.N, pitch, **u8))
        self.idx = torch.empty(T, w.K, dtype=torch.int32, device=dev)
        self.gates = torch.empty(T, w.K, device=dev)
        self.balance = dict(counts=torch.empty(w.R, w.E, dtype=torch.int32, device=dev),
                            prob_sum=torch.empty(w.R, w.E, device=dev),
                            seg_tokens=torch.empty(w.R, dtype=torch.int32, device=dev),
                            loss=torch.empty(1, device=dev))
        self.y, self.d_y = (torch.empty(w.N, w.Hp, dtype=bf, device=dev) for _ in range(2))
        self.out = torch.empty(T, w.Hp, dtype=bf, device=dev)
        self.d_gates = torch.empty(T, w.K, device=dev)
        self.d_logits = torch.empty(T, w.E, device=dev)

    def forward(self, x):
        d, ws = self.d, self.ws.buf
        self.logits = x.float() @ self.w_router
        mx.moonep_router_forward(self.rd, self.logits, self.idx, self.gates, ws=self.router_ws,
                                 **self.balance)
        mx.moonep_plan(d, self.idx, ws)
        mx.moonep_mxfp4_prefetch_weights(d, ws, *self.home, *self.slot)
        mx.moonep_mxfp4_dispatch(d, ws, x, *self.recv)
        mx.moonep_mxfp4_grouped_gemm(d, ws, *self.recv, *self.home, *self.slot, self.y)
        mx.moonep_combine(d, ws, self.y, self.gates, self.out)
        return self.out

    def forward_bf16(self, x):
        """The same routing through the bf16 calls."""
        w, d, ws = self.w, self.d, self.ws.buf
        recv = torch.empty(w.N, w.H, dtype=torch.bfloat16, device="cuda")
        y, out = torch.empty_like(self.y), torch.empty_like(self.out)
        mx.moonep_prefetch_weights(d, ws, self.w_home, self.w_slot)
        mx.moonep_dispatch(d, ws, x, recv)
        mx.moonep_grouped_gemm(d, ws, recv, self.w_home, self.w_slot, y)
        mx.moonep_combine(d, ws, y, self.gates, out)
        return out

    def router_gradient(self, x, d_out, balance_weight):
        """Gradient of the output's loss and of the balance loss at the router's weights."""
        mx.moonep_combine_backward(self.d, self.ws.buf, self.y, self.gates, d_out, self.d_y,
                                   self.d_gates)
        d_loss = torch.full((1,), balance_weight, device="cuda")
        mx.moonep_router_backward(self.rd, self.logits, self.idx, self.d_logits,
                                  d_gates=self.d_gates, counts=self.balance["counts"],
                                  seg_tokens=self.balance["seg_tokens"], d_loss=d_loss)
        return x.float().T @ self.d_logits


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rate", type=float, default=0.003, help="step size of the router's weights")
    args = ap.parse_args(argv)
    torch.manual_seed(0)
    layer = Layer(syn.SMALL)
    w = layer.w
    T = w.R * w.S
    x = syn.normal_bf16((T, w.H), 1.0, 1, "cuda")
    x += 0.5
    target = syn.normal_bf16((T, w.Hp), 1.0, 3, "cuda")
    history = []
    for step in range(args.steps):
        out = layer.forward(x)
        far = (out.float() - layer.forward_bf16(x).float()).norm() / out.float().norm()
        d_out = ((out - target).float() / T).to(torch.bfloat16)
        grad = layer.router_gradient(x, d_out, balance_weight=0.05)
        layer.w_router -= args.rate * grad
        counts = layer.balance["counts"].sum(0).float()
        status = mx.moonep_read_status(layer.d, layer.ws.buf)
        if status:
            raise mx.MoonepError(status, "layer")
        history.append((float(layer.balance["loss"]), float(counts.max() / counts.mean()), float(far)))
        print("step %2d  balance loss %.4f  busiest expert %.2f x mean  MXFP4 from bf16 %.3f"
              % (step, *history[-1]))
    return history


if __name__ == "__main__":
    main()
