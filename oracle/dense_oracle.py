"""Plain CPU oracle, in float64, of the dense half of a layer: the gated
feed-forward block and its gradients, low-rank adapters beside a projection
and theirs, and dropout with a mask made from a counter. Test infrastructure
only, like the rest of this package; written from the definitions.
"""
from __future__ import annotations

import math

import numpy as np

from .moe_oracle import bf16

_erf = np.vectorize(math.erf, otypes=[np.float64])
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _tanh_share(z, sign=1.0):
    """(1 + sign tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 as a logistic function, which
    keeps its tail where 1 + tanh would cancel."""
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-sign * math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3)))


def act(z, kind):
    """act(z) in float64."""
    z = np.asarray(z, dtype=np.float64)
    if kind == "silu":
        with np.errstate(over="ignore"):
            return z / (1.0 + np.exp(-z))
    if kind == "gelu":
        return z * 0.5 * _erfc(-z / math.sqrt(2.0))
    if kind == "gelu_tanh":
        return z * _tanh_share(z)
    return np.maximum(z, 0.0)


def act_grad(z, kind):
    """act'(z) in float64; relu has 0 at 0."""
    z = np.asarray(z, dtype=np.float64)
    if kind == "silu":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if kind == "gelu":
        return 0.5 * _erfc(-z / math.sqrt(2.0)) + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        s, inner = _tanh_share(z), math.sqrt(8.0 / math.pi) * (1.0 + 3 * 0.044715 * z * z)
        return s + z * s * _tanh_share(z, -1.0) * inner
    return (z > 0.0).astype(np.float64)


def gated_ffn(x, w_gate, w_up, w_down, kind="silu", add=None, rounded=True):
    """dict(y, a_gate, a_up, h); h is rounded to bf16 as the block rounds it unless
    rounded is false. y, a_gate and a_up are not rounded."""
    a_gate, a_up = x @ w_gate, x @ w_up
    h = act(a_gate, kind) * a_up
    if rounded:
        h = bf16(h)
    y = h @ w_down
    return dict(y=y if add is None else add + y, a_gate=a_gate, a_up=a_up, h=h)


def gated_ffn_backward(dy, x, w_gate, w_up, w_down, a_gate, a_up, kind="silu", add=None,
                       rounded=True):
    """dict(dx, dw_gate, dw_up, dw_down, h, da_gate, da_up), the last three rounded to
    bf16 as the block rounds them unless rounded is false."""
    f, d = act(a_gate, kind), act_grad(a_gate, kind)
    dh = dy @ w_down.T
    h, dg, du = f * a_up, dh * a_up * d, dh * f
    if rounded:
        h, dg, du = bf16(h), bf16(dg), bf16(du)
    dx = dg @ w_gate.T + du @ w_up.T
    return dict(dx=dx if add is None else add + dx, dw_gate=x.T @ dg, dw_up=x.T @ du,
                dw_down=h.T @ dy, h=h, da_gate=dg, da_up=du)


def lora_plan(ids, n):
    """(order, offsets): the rows of each adapter in turn, those without one last."""
    rows = [[t for t, i in enumerate(ids) if i == a] for a in range(n)]
    rest = [t for t, i in enumerate(ids) if not 0 <= i < n]
    offsets = np.concatenate([[0], np.cumsum([len(r) for r in rows])])
    return (np.array([t for r in rows for t in r] + rest, dtype=np.int32),
            offsets.astype(np.int32))


def lora(x, a, b, ids, scales=None, base=None):
    """(out, v), one row at a time."""
    T, (n, r, _) = x.shape[0], a.shape
    out = np.zeros((T, b.shape[2])) if base is None else np.array(base, dtype=np.float64)
    v = np.zeros((T, r))
    for t, i in enumerate(ids):
        if 0 <= i < n:
            v[t] = a[i] @ x[t]
            out[t] += (1.0 if scales is None else scales[i]) * (v[t] @ b[i])
    return out, v


def lora_backward(dy, x, v, a, b, ids, scales=None, base=None):
    """dict(dx, da, db, dv), one row at a time."""
    n, r, _ = a.shape
    dx = np.zeros(x.shape) if base is None else np.array(base, dtype=np.float64)
    da, db, dv = np.zeros(a.shape), np.zeros(b.shape), np.zeros((x.shape[0], r))
    for t, i in enumerate(ids):
        if 0 <= i < n:
            s = 1.0 if scales is None else scales[i]
            dv[t] = s * (b[i] @ dy[t])
            dx[t] += dv[t] @ a[i]
            da[i] += np.outer(dv[t], x[t])
            db[i] += s * np.outer(v[t], dy[t])
    return dict(dx=dx, da=da, db=db, dv=dv)


def philox4x32(counter, key):
    """Ten rounds of Philox 4x32 on plain integers: four words of a counter of four
    and a key of two."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(q >> 32) ^ c[1] ^ k[0], q & 0xFFFFFFFF, (p >> 32) ^ c[3] ^ k[1], p & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def dropout_threshold(p):
    """The least of the 65536 numbers that is kept."""
    return min(65535, int(np.rint(float(np.float32(p)) * 65536.0)))


def dropout_kept(numel, seed, draw, p):
    """bool [numel]: which elements are kept."""
    words = []
    lo = 0xFFFFFFFF
    for block in range((numel + 7) // 8):
        for w in philox4x32([block & lo, block >> 32, draw & lo, (draw >> 32) & lo],
                            [seed & lo, (seed >> 32) & lo]):
            words += [w & 0xFFFF, w >> 16]
    return np.array(words[:numel], dtype=np.int64) >= dropout_threshold(p)


def dropout_residual(y, kept, p, x=None, a=1.0, b=1.0):
    """a x + f kept y of flat arrays."""
    f = b / (1.0 - dropout_threshold(p) / 65536.0)
    out = np.where(kept, f * np.asarray(y, dtype=np.float64), 0.0)
    return out if x is None else out + a * np.asarray(x, dtype=np.float64)
