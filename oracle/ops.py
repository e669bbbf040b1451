"""Plain 64-bit definitions of the operators around the layer path: the router
with its balance loss and gradient, and MXFP4 quantisation.

Test infrastructure, written from the formulas; nothing is shared with the
CUDA path.
"""
from __future__ import annotations

import numpy as np


def top_k(logits: np.ndarray, K: int) -> np.ndarray:
    """Ids of the K largest logits of every row, largest first, equal ones by
    ascending id; NaN after everything else."""
    key = np.where(np.isnan(logits), np.inf, -logits)
    nan = np.isnan(logits)
    ids = np.broadcast_to(np.arange(logits.shape[1]), logits.shape)
    return np.lexsort((ids, key, nan), axis=-1)[:, :K].astype(np.int32)


def scores(logits: np.ndarray, kind: str):
    """(s, q): the gates' scores and the balance loss's probabilities."""
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if kind == "softmax":
            m = np.fmax.reduce(logits, axis=-1, keepdims=True)
            m = np.where(np.isneginf(m), 0.0, m)
            s = np.exp(logits - m)
            total = s.sum(-1, keepdims=True)
            s = np.where(total == 0, 0.0, s / total)
            return s, s
        s = 1.0 / (1.0 + np.exp(-logits))
        return s, _share(_log_sigmoid(logits))


def _log_sigmoid(x):
    return -np.logaddexp(0.0, -x)


def _share(logs: np.ndarray) -> np.ndarray:
    """e^logs over its sum along the row, whatever the size of logs; 0 for a row of -inf."""
    m = np.fmax.reduce(logs, axis=-1, keepdims=True)
    e = np.exp(logs - np.where(np.isneginf(m), 0.0, m))
    total = e.sum(-1, keepdims=True)
    return np.where(total == 0, 0.0, e / total)


def gates_of(logits, kind: str, ids: np.ndarray, normalise: bool, scale: float, live: np.ndarray):
    at = ids.astype(np.int64)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if not normalise:
            g = np.take_along_axis(scores(logits, kind)[0], at, 1)
        else:
            chosen = np.take_along_axis(logits, at, 1)
            g = _share(chosen if kind == "softmax" else _log_sigmoid(chosen))
            if kind == "softmax":  # a NaN or an infinity in the row is in every score
                bad = np.isnan(scores(logits, kind)[0]).any(-1, keepdims=True)
                g = np.where(bad, np.nan, g)
    return np.where(live[:, None], scale * g, 0.0)


def balance(q: np.ndarray, ids: np.ndarray, live: np.ndarray, segment: int):
    """counts, prob_sum, seg_tokens and the loss."""
    T, E = q.shape
    K = ids.shape[1]
    G = -(-T // segment)
    counts = np.zeros((G, E), np.int64)
    sums = np.zeros((G, E))
    tokens = np.zeros(G, np.int64)
    parts = np.zeros(G)
    for g in range(G):
        rows = np.arange(g * segment, min(T, (g + 1) * segment))
        rows = rows[live[rows]]
        tokens[g] = len(rows)
        counts[g] = np.bincount(ids[rows].reshape(-1), minlength=E)
        sums[g] = q[rows].sum(0)
        if len(rows):
            parts[g] = E * np.sum(counts[g] * sums[g]) / (K * float(len(rows)) ** 2)
    return counts, sums, tokens, parts.mean()


def router(logits, K, segment, kind, normalise, scale, live=None):
    T = logits.shape[0]
    live = np.ones(T, bool) if live is None else live
    ids = top_k(logits, K)
    s, q = scores(logits, kind)
    gates = gates_of(logits, kind, ids, normalise, scale, live)
    return ids, gates, *balance(q, ids, live, segment)


def router_backward(logits, ids, segment, kind, normalise, scale, live, d_gates, d_loss):
    """Gradient of sum(d_gates * gates) + d_loss * loss for fixed ids, by the chain
    rule through the matrices ds/dl and dq/dl; and a bound on the size of what is
    summed for each element (what rounding errors are relative to)."""
    T, E = logits.shape
    K = ids.shape[1]
    live = np.ones(T, bool) if live is None else live
    s, q = scores(logits, kind)
    counts, _, tokens, _ = balance(np.nan_to_num(q), ids, live, segment)
    G = len(tokens)
    grad, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        if not live[t]:
            continue
        g = t // segment
        ds = np.zeros(E)
        if d_gates is not None:
            sk = s[t, ids[t]]
            dg = scale * d_gates[t]
            if normalise:
                total = sk.sum()
                dg = (dg - (dg * sk).sum() / total) / total if total else 0 * dg
            ds[ids[t]] = dg
        w = d_loss * E / (G * K * float(tokens[g]) ** 2) * counts[g] if d_loss else np.zeros(E)
        if kind == "softmax":
            jac = np.diag(s[t]) - np.outer(s[t], s[t])  # ds/dl, and dq/dl
            grad[t] = jac @ (ds + w)
            size[t] = s[t] * (np.abs(ds) + np.abs(w) + (s[t] * (np.abs(ds) + np.abs(w))).sum())
        else:
            total = s[t].sum()
            inner = np.zeros(E)
            if total:
                inner = (w - (q[t] * w).sum()) / total
            grad[t] = s[t] * (1 - s[t]) * (ds + inner)
            size[t] = s[t] * (1 - s[t]) * (np.abs(ds) + np.abs(w) / max(total, 1e-300)
                                           + (q[t] * np.abs(w)).sum() / max(total, 1e-300))
            if not d_loss:  # the gates are functions of the chosen logits alone
                chosen = np.isin(np.arange(E), ids[t])
                grad[t] = np.where(chosen, s[t] * (1 - s[t]) * ds, 0.0)
                size[t] = np.where(chosen, s[t] * (1 - s[t]) * np.abs(ds), 0.0)
        if d_gates is not None and normalise:  # what cancels inside a normalised gate's gradient
            sk = s[t, ids[t]]
            n = sk / sk.sum() if sk.sum() else sk
            size[t, ids[t]] += scale * n * (np.abs(d_gates[t]) + (n * np.abs(d_gates[t])).sum())
    return grad, size


# ---------------------------------------------------------------------------- MXFP4
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def mxfp4_pitch(cols: int) -> int:
    return -(-(cols // 32) // 16) * 16


def mxfp4_quantize(x: np.ndarray):
    """x [rows][cols] -> (codes [rows][cols/2], scales [rows][pitch]), uint8."""
    rows, cols = x.shape
    b = x.reshape(rows, cols // 32, 32)
    finite = np.isfinite(b).all(-1)
    safe = np.where(finite[..., None], b, 0.0)
    top = np.abs(safe).max(-1)
    exp = np.where(top > 0, np.frexp(top)[1] - 1, -127)  # top = f 2^exp, 1 <= f < 2
    shared = np.maximum(exp - 2, -127)
    v = np.abs(np.ldexp(safe, -shared[..., None]))
    d = np.abs(v[..., None] - GRID)  # nearest magnitude, ties to the even code
    best = d.min(-1, keepdims=True)
    tied = d == best
    first = tied.argmax(-1)
    last = 7 - tied[..., ::-1].argmax(-1)
    code = np.where(first % 2 == 0, first, last) | (np.signbit(safe).astype(np.int64) << 3)
    code = np.where(finite[..., None], code, 0).reshape(rows, cols).astype(np.uint8)
    scales = np.zeros((rows, mxfp4_pitch(cols)), np.uint8)
    scales[:, :cols // 32] = np.where(finite, shared + 127, 255)
    return code[:, 0::2] | (code[:, 1::2] << 4), scales


def mxfp4_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    rows, half = codes.shape
    c = np.stack([codes & 15, codes >> 4], -1).reshape(rows, half * 2)
    v = np.where(c & 8, -1.0, 1.0) * GRID[c & 7]
    s = scales[:, :half * 2 // 32].astype(np.int64)
    f = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return v * np.repeat(f, 32, 1)
