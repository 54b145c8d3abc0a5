"""Plain CPU oracle, in float64, of the operators around the expert block: the
balanced gate and its gradient, the norms before and after the block with
their gate and residual and their gradients, and the clip of many gradients
by one norm. Test infrastructure only, like the rest of this package; written
from the definitions, one token or one tensor at a time.
"""
from __future__ import annotations

import math

import numpy as np

F32_MAX = float(np.finfo(np.float32).max)


def _logit(v: float) -> float:
    """NaN counts as -inf, +inf as the largest float."""
    return -math.inf if math.isnan(v) else min(v, F32_MAX)


def _sigmoid(v: float) -> float:
    if v == -math.inf:
        return 0.0
    return 1.0 / (1.0 + math.exp(-v)) if v > -700.0 else math.exp(v)


def _scores(row, score):
    if score == "sigmoid":
        return [_sigmoid(v) for v in row]
    top = max(row)
    if top == -math.inf:
        return [0.0] * len(row)
    ex = [math.exp(v - top) for v in row]
    total = math.fsum(ex)
    return [v / total for v in ex]


def _best(values, among, count):
    """The count indices of `among` with the largest values, ties to the lower index."""
    return sorted(among, key=lambda i: (-values[i], i))[:count]


def _weights(row, scores, live, ids, score, renormalise):
    """(scores of the chosen, weights before the scale)."""
    s = [scores[e] if live[e] else 0.0 for e in ids]
    if not renormalise:
        return s, list(s)
    if score == "softmax":
        chosen = [row[e] if live[e] else -math.inf for e in ids]
        top = max(chosen)
        u = [0.0 if v == -math.inf else math.exp(v - top) for v in chosen]
    else:
        u = s
    total = math.fsum(u)
    return s, [v / total if total > 0.0 else 0.0 for v in u]


def route_gate(logits, k, bias=None, score="softmax", n_group=1, topk_group=1, group_topk=1,
               renormalise=True, scale=1.0):
    """(ids int32 [T, k], weights float64 [T, k], counts int32 [E], offsets int32 [E+1])."""
    lg = np.asarray(logits, dtype=np.float64)
    T, E = lg.shape
    ids = np.zeros((T, k), dtype=np.int32)
    w = np.zeros((T, k))
    b = [0.0] * E if bias is None else [_logit(float(v)) for v in np.asarray(bias, np.float64)]
    size = E // n_group
    for t in range(T):
        row = [_logit(v) for v in lg[t].tolist()]
        s = _scores(row, score)
        live = [l != -math.inf and c != -math.inf for l, c in zip(row, b)]
        v = [a + c if ok else -math.inf for a, c, ok in zip(s, b, live)]
        among = range(E)
        if n_group > 1:
            group = []
            for g in range(n_group):
                top = [v[e] for e in _best(v, range(g * size, (g + 1) * size), group_topk)
                       if live[e]]
                group.append(math.fsum(top) if top else -math.inf)
            kept = set(_best(group, range(n_group), topk_group))
            among = [e for e in range(E) if e // size in kept]
        rank = v if bias is not None else row
        chosen = _best(rank, among, k)
        ids[t] = chosen
        w[t] = [scale * u for u in _weights(row, s, live, chosen, score, renormalise)[1]]
    counts = np.bincount(ids.reshape(-1), minlength=E).astype(np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return ids, w, counts, offsets


def route_gate_backward(dprobs, logits, ids, bias=None, score="softmax", renormalise=True,
                        scale=1.0):
    """dlogits float64 [T, E]."""
    lg, dp = np.asarray(logits, np.float64), np.asarray(dprobs, np.float64)
    T, E = lg.shape
    b = [0.0] * E if bias is None else [_logit(float(v)) for v in np.asarray(bias, np.float64)]
    out = np.zeros((T, E))
    for t in range(T):
        row = [_logit(v) for v in lg[t].tolist()]
        s = _scores(row, score)
        live = [l != -math.inf and c != -math.inf for l, c in zip(row, b)]
        chosen = [int(e) for e in ids[t]]
        sj, u = _weights(row, s, live, chosen, score, renormalise)
        d = math.fsum(g * x for g, x in zip(dp[t], u))
        if score == "softmax" and not renormalise:
            out[t] = [-p * d for p in s]
        for j, e in enumerate(chosen):
            if not live[e]:
                continue
            g = dp[t, j]
            far = _sigmoid(-row[e])                       # 1 - sigmoid, without cancellation
            if score == "softmax":
                out[t, e] += u[j] * (g - d) if renormalise else sj[j] * g
            else:
                out[t, e] += u[j] * far * (g - d) if renormalise else sj[j] * far * g
    return scale * out


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def gate_rows(gate, T):
    """The gate row of every token."""
    if gate is None:
        return np.ones((T, 1))
    gate = np.atleast_2d(gate)
    return np.repeat(gate, T // gate.shape[0], axis=0)


def norm_residual(x, y=None, w_post=None, gate=None, w_next=None, eps=1e-6, residual_scale=1.0,
                  branch_scale=1.0):
    """dict(out, n, rstd_y, rstd_out) in float64, None where not computed."""
    x, y, w_post, gate, w_next = (_f64(a) for a in (x, y, w_post, gate, w_next))
    got = dict(out=None, n=None, rstd_y=None, rstd_out=None)
    out = x
    if y is not None:
        z = y
        if w_post is not None:
            got["rstd_y"] = 1.0 / np.sqrt(np.mean(y * y, axis=1) + eps)
            z = y * got["rstd_y"][:, None] * w_post
        out = residual_scale * x + branch_scale * gate_rows(gate, x.shape[0]) * z
        got["out"] = out
    if w_next is not None:
        got["rstd_out"] = 1.0 / np.sqrt(np.mean(out * out, axis=1) + eps)
        got["n"] = out * got["rstd_out"][:, None] * w_next
    return got


def norm_residual_backward(d_out, d_n, out, y=None, w_post=None, gate=None, w_next=None,
                           rstd_y=None, rstd_out=None, residual_scale=1.0, branch_scale=1.0):
    """dict(dx, dy, dw_post, dgate, dw_next) in float64, None where there is no such input."""
    d_out, d_n, out, y, w_post, gate, w_next, rstd_y, rstd_out = (
        _f64(a) for a in (d_out, d_n, out, y, w_post, gate, w_next, rstd_y, rstd_out))
    got = dict(dx=None, dy=None, dw_post=None, dgate=None, dw_next=None)
    D = np.zeros_like(out) if d_out is None else d_out
    T = D.shape[0]
    if d_n is not None:
        o = out * rstd_out[:, None]
        q = d_n * w_next
        D = D + rstd_out[:, None] * (q - o * np.mean(q * o, axis=1, keepdims=True))
        got["dw_next"] = np.sum(d_n * o, axis=0)
    if y is None:
        got["dx"] = D
        return got
    got["dx"] = residual_scale * D
    g = gate_rows(gate, T)
    yh = y if w_post is None else y * rstd_y[:, None]
    w = 1.0 if w_post is None else w_post
    if gate is not None:
        rows = np.atleast_2d(gate).shape[0]
        terms = branch_scale * w * D * yh
        got["dgate"] = terms.reshape(rows, T // rows, -1).sum(axis=1).reshape(gate.shape)
    p = branch_scale * g * w * D
    if w_post is not None:
        got["dw_post"] = np.sum(branch_scale * g * D * yh, axis=0)
        p = rstd_y[:, None] * (p - yh * np.mean(p * yh, axis=1, keepdims=True))
    got["dy"] = p
    return got


def clip_grad_norm(grads, max_norm, norm_type=2.0, eps=1e-6):
    """(norm, coef, the scaled gradients in float64)."""
    grads = [_f64(g) for g in grads]
    with np.errstate(invalid="ignore", over="ignore"):
        if norm_type == math.inf:
            norm = max([0.0] + [float(np.max(np.abs(g))) for g in grads if g.size],
                       key=lambda v: math.inf if math.isnan(v) else v)
            if any(np.isnan(g).any() for g in grads):
                norm = math.nan
        else:
            norm = math.sqrt(sum(float(np.sum(g * g)) for g in grads))
        coef = 1.0
        if max_norm is not None:
            c = max_norm / (norm + eps) if norm + eps != 0.0 else \
                (math.inf if max_norm > 0 else math.nan)
            coef = 1.0 if c >= 1.0 else c
        return norm, coef, [g * coef for g in grads]
