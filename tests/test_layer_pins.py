"""CPU pins of the operators around the expert block: the oracle's formulas
against hand-worked values and finite differences, and the host-side checks
of the entry points, which answer before any launch."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle as orc


# ------------------------------------------------------------------ the oracle's formulas

def test_gate_defaults_are_the_plain_top_k_gate():
    rng = np.random.default_rng(1)
    logits = rng.standard_normal((50, 12)).astype(np.float32)
    ids, w, counts, offsets = orc.route_gate(logits, 3)
    rid, rw, rc, ro = orc.route_topk(logits, 3)
    assert np.array_equal(ids, rid) and np.array_equal(counts, rc) and np.array_equal(offsets, ro)
    np.testing.assert_allclose(w, rw, rtol=1e-14)


def test_gate_by_hand():
    # scores 0.5, 0.75, 0.25, 0.9 in two groups of two
    logits = np.log(np.array([[1.0, 3.0, 1.0 / 3.0, 9.0]]))
    ids, w, _, _ = orc.route_gate(logits, 2, score="sigmoid", scale=2.0)
    assert ids.tolist() == [[3, 1]]
    np.testing.assert_allclose(w, [[2 * 0.9 / 1.65, 2 * 0.75 / 1.65]])
    # the best two of each group sum to 1.25 and 1.15: only the first group is kept
    ids, w, _, _ = orc.route_gate(logits, 2, score="sigmoid", n_group=2, topk_group=1,
                                  group_topk=2, renormalise=False)
    assert ids.tolist() == [[1, 0]]
    np.testing.assert_allclose(w, [[0.75, 0.5]])
    # by their best one the second is
    ids, _, _, _ = orc.route_gate(logits, 2, score="sigmoid", n_group=2, topk_group=1)
    assert ids.tolist() == [[3, 2]]
    # a bias moves the choice and not the weight
    ids, w, _, _ = orc.route_gate(logits, 1, bias=[0.0, 0.0, 1.0, 0.0], score="sigmoid",
                                  renormalise=False)
    assert ids.tolist() == [[2]] and abs(w[0, 0] - 0.25) < 1e-15


def test_gate_masks_by_hand():
    inf = math.inf
    logits = np.array([[-inf, -inf, -inf, -inf], [2.0, -inf, math.nan, 1.0], [inf, 0.0, 0.0, 0.0]])
    ids, w, counts, _ = orc.route_gate(logits, 3)
    assert ids.tolist() == [[0, 1, 2], [0, 3, 1], [0, 1, 2]]
    assert w[0].tolist() == [0.0, 0.0, 0.0] and w[1, 2] == 0.0 and w[2, 0] == 1.0
    assert counts.sum() == 9
    ids, w, _, _ = orc.route_gate(np.zeros((1, 4)), 2, bias=[-inf, -inf, math.nan, 0.0],
                                  score="sigmoid")
    assert ids.tolist() == [[3, 0]] and w.tolist() == [[1.0, 0.0]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_gate_gradient_against_differences(score, renormalise):
    rng = np.random.default_rng(3)
    T, E, k, scale = 4, 7, 3, 1.5
    logits, dp = rng.standard_normal((T, E)) * 2.0, rng.standard_normal((T, k))
    bias = rng.standard_normal(E) * 0.1
    kw = dict(bias=bias, score=score, renormalise=renormalise, scale=scale)
    ids, _, _, _ = orc.route_gate(logits, k, **kw)
    got = orc.route_gate_backward(dp, logits, ids, **kw)

    def loss(lg):
        i2, w, _, _ = orc.route_gate(lg, k, **kw)
        assert np.array_equal(i2, ids)
        return float((w * dp).sum())

    h = 1e-6
    for t in range(T):
        for e in range(E):
            up, dn = logits.copy(), logits.copy()
            up[t, e] += h
            dn[t, e] -= h
            assert abs((loss(up) - loss(dn)) / (2 * h) - got[t, e]) < 1e-8


NORM_FORMS = [
    dict(y=True, post=True, rows=1, nxt=True), dict(y=True, post=True, rows=3, nxt=True),
    dict(y=True, post=True, rows=0, nxt=False), dict(y=True, post=False, rows=6, nxt=True),
    dict(y=True, post=False, rows=0, nxt=True), dict(y=False, post=False, rows=0, nxt=True),
]


@pytest.mark.parametrize("form", NORM_FORMS)
def test_norm_gradient_against_differences(form):
    rng = np.random.default_rng(5)
    T, H, a, b = 6, 5, 0.7, 1.3
    v = dict(x=rng.standard_normal((T, H)))
    if form["y"]:
        v["y"] = rng.standard_normal((T, H))
    if form["post"]:
        v["w_post"] = rng.standard_normal(H)
    if form["rows"]:
        v["gate"] = rng.standard_normal((form["rows"], H))
    if form["nxt"]:
        v["w_next"] = rng.standard_normal(H)
    d_out = rng.standard_normal((T, H))
    d_n = rng.standard_normal((T, H)) if form["nxt"] else None
    sc = dict(residual_scale=a, branch_scale=b)

    def loss(values):
        f = orc.norm_residual(**values, **sc)
        out = values["x"] if f["out"] is None else f["out"]
        return float((out * d_out).sum() + (0.0 if d_n is None else (f["n"] * d_n).sum()))

    f = orc.norm_residual(**v, **sc)
    rest = {key: v.get(key) for key in ("y", "w_post", "gate", "w_next")}
    got = orc.norm_residual_backward(d_out, d_n, v["x"] if f["out"] is None else f["out"], **rest,
                                     rstd_y=f["rstd_y"], rstd_out=f["rstd_out"], **sc)
    h = 1e-6
    for key, name in (("x", "dx"), ("y", "dy"), ("w_post", "dw_post"), ("gate", "dgate"),
                      ("w_next", "dw_next")):
        if key not in v:
            assert got[name] is None
            continue
        for i in np.ndindex(v[key].shape):
            up, dn = v[key].copy(), v[key].copy()
            up[i] += h
            dn[i] -= h
            diff = (loss({**v, key: up}) - loss({**v, key: dn})) / (2 * h)
            assert abs(diff - got[name][i]) < 1e-7, (name, i)


def test_clip_by_hand():
    norm, coef, out = orc.clip_grad_norm([[3.0], [4.0]], 1.0, eps=0.0)
    assert norm == 5.0 and coef == 0.2 and np.allclose(out, [[0.6], [0.8]])
    norm, coef, out = orc.clip_grad_norm([[3.0, -4.0]], 8.0, norm_type=math.inf, eps=0.0)
    assert norm == 4.0 and coef == 1.0 and out[0].tolist() == [3.0, -4.0]
    norm, coef, _ = orc.clip_grad_norm([[math.inf, 1.0]], 1.0)
    assert norm == math.inf and coef == 0.0
    for kind in (2.0, math.inf):
        norm, coef, _ = orc.clip_grad_norm([[1.0], [math.nan]], 1.0, norm_type=kind)
        assert math.isnan(norm) and math.isnan(coef)
    assert orc.clip_grad_norm([], 1.0)[:2] == (0.0, 1.0)


# ------------------------------------------------------------------ host-side checks

@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    import moe_expert_dispatch_gb300
    return moe_expert_dispatch_gb300


def test_config_defaults(m):
    g = m.moe_gate_config(9, 9, 9, 9, 9, 9.0)
    m._lib.moe_gate_config_init(ctypes.byref(g))
    assert (g.score, g.n_group, g.topk_group, g.group_topk, g.renormalise, g.scale) == \
        (0, 1, 1, 1, 1, 1.0)
    n = m.moe_norm_config(9.0, 9.0, 9.0, 9, 9)
    m._lib.moe_norm_config_init(ctypes.byref(n))
    assert (n.residual_scale, n.branch_scale, n.stream_type, n.weight_type) == (1.0, 1.0, 1, 1)
    m._lib.moe_gate_config_init(None)
    m._lib.moe_norm_config_init(None)


def test_workspace_sizes(m):
    L = m._lib
    assert L.moe_route_gate_workspace_size(4096, 8, 256) > 0
    assert L.moe_route_gate_workspace_size(4, 8, 256) == 0        # one cluster needs none
    assert L.moe_route_gate_workspace_size(1 << 62, 32, 64) == 0
    assert L.moe_route_gate_workspace_size(-1, 2, 8) == 0
    assert L.moe_norm_residual_backward_workspace_size(4096, 4096, 1) > 0
    assert L.moe_norm_residual_backward_workspace_size(1 << 62, 4096, 1) == 0
    assert L.moe_norm_residual_backward_workspace_size(16, 0, 0) == 0
    assert L.moe_norm_residual_backward_workspace_size(16, 65537, 0) == 0
    assert L.moe_clip_grad_norm_workspace_size() > 0


def test_entry_points_refuse_before_any_launch(m):
    # each call is wrong in one way the host can see. P is a fake, aligned
    # device address that no check dereferences; with a GPU present the test
    # does not run, so a missing check could never hand it to a kernel.
    if torch.cuda.is_available():
        pytest.skip("host-only: the cases carry fake device addresses")
    L = m._lib
    P = ctypes.c_void_p(1 << 20)
    U = ctypes.c_void_p((1 << 20) + 8)          # not 16-byte aligned
    O = ctypes.c_void_p((1 << 20) + 1)          # not aligned to any element  # noqa: E741
    INV, UNS, WS = 1, 2, 4
    F, B = 0, 1
    WSB = 1 << 30

    def gate(logits=P, lt=F, bias=None, T=4, E=8, k=2, cfg=None, ids=P, probs=P, counts=P,
             offsets=P, ws=P, wsb=WSB):
        return L.moe_route_gate(logits, lt, bias, T, E, k, cfg, ids, probs, counts, offsets, ws,
                                wsb, None)

    def gcfg(score=0, n_group=1, topk_group=1, group_topk=1, renorm=1, scale=1.0):
        return m.moe_gate_config(score, n_group, topk_group, group_topk, renorm, scale)

    def gate_b(dp=P, logits=P, lt=F, ids=P, T=4, E=8, k=2, cfg=None, dl=P):
        return L.moe_route_gate_backward(dp, logits, lt, None, ids, T, E, k, cfg, dl, None)

    def ncfg(eps=1e-6, a=1.0, b=1.0, st=B, wt=B):
        return m.moe_norm_config(eps, a, b, st, wt)

    def norm(x=P, y=P, wp=P, gate=None, rows=0, wn=P, T=4, H=64, cfg=None, out=P, n=P):
        return L.moe_norm_residual(x, y, wp, gate, rows, wn, T, H, cfg, out, n, P, P, None)

    def norm_b(d_out=P, d_n=P, out=P, y=P, wp=P, gate=None, rows=0, wn=P, ry=P, ro=P, T=4, H=64,
               cfg=None, dx=P, dy=P, dwp=P, dg=None, dwn=P, ws=P, wsb=WSB):
        return L.moe_norm_residual_backward(d_out, d_n, out, y, wp, gate, rows, wn, ry, ro, T, H,
                                            cfg, dx, dy, dwp, dg, dwn, 0, ws, wsb, None)

    def clip(grads=((1 << 20),), outs=None, numels=(4,), types=(F,), n=None, max_norm=1.0, kind=0,
             eps=1e-6, nc=P, ws=P, wsb=WSB):
        k = len(grads)
        return L.moe_clip_grad_norm(
            (ctypes.c_void_p * k)(*grads),
            None if outs is None else (ctypes.c_void_p * k)(*outs),
            (ctypes.c_int64 * k)(*numels), (ctypes.c_int * k)(*types), k if n is None else n,
            max_norm, kind, eps, nc, ws, wsb, None)

    nan, inf = math.nan, math.inf
    cases = [
        ("gate: no logits", INV, lambda: gate(logits=None)),
        ("gate: logits' type", INV, lambda: gate(lt=2)),
        ("gate: unaligned logits", INV, lambda: gate(logits=O)),
        ("gate: T < 0", INV, lambda: gate(T=-1)),
        ("gate: E = 0", INV, lambda: gate(E=0)),
        ("gate: E > 1024", INV, lambda: gate(E=1025)),
        ("gate: k = 0", INV, lambda: gate(k=0)),
        ("gate: k > E", INV, lambda: gate(k=9)),
        ("gate: k > 32", INV, lambda: gate(E=64, k=33)),
        ("gate: T k past int32", INV, lambda: gate(T=1 << 31)),
        ("gate: score", INV, lambda: gate(cfg=gcfg(score=2))),
        ("gate: n_group = 0", INV, lambda: gate(cfg=gcfg(n_group=0))),
        ("gate: n_group does not divide E", INV, lambda: gate(cfg=gcfg(n_group=3, topk_group=3))),
        ("gate: n_group > 32", INV, lambda: gate(E=64, cfg=gcfg(n_group=64, topk_group=64))),
        ("gate: topk_group > n_group", INV, lambda: gate(cfg=gcfg(n_group=2, topk_group=3))),
        ("gate: too few experts kept", INV,
         lambda: gate(k=3, cfg=gcfg(n_group=4, topk_group=1))),
        ("gate: group_topk = 3", INV, lambda: gate(cfg=gcfg(group_topk=3))),
        ("gate: scale", INV, lambda: gate(cfg=gcfg(scale=inf))),
        ("gate: no counts", INV, lambda: gate(counts=None)),
        ("gate: no workspace", WS, lambda: gate(T=9999, ws=None)),
        ("gate: small workspace", WS, lambda: gate(T=9999, wsb=8)),
        ("gate: unaligned workspace", WS, lambda: gate(T=9999, ws=U)),
        ("gate backward: no ids", INV, lambda: gate_b(ids=None)),
        ("gate backward: no dlogits", INV, lambda: gate_b(dl=None)),
        ("gate backward: unaligned dlogits", INV, lambda: gate_b(dl=O)),
        ("gate backward: k > E", INV, lambda: gate_b(k=9)),
        ("gate backward: T = 0 does nothing", 0, lambda: gate_b(T=0, dp=None)),
        ("norm: no x", INV, lambda: norm(x=None)),
        ("norm: nothing to compute", INV, lambda: norm(y=None, wp=None, wn=None, out=None)),
        ("norm: w_post without y", INV, lambda: norm(y=None, out=None)),
        ("norm: out without y", INV, lambda: norm(y=None, wp=None)),
        ("norm: no out", INV, lambda: norm(out=None)),
        ("norm: no n", INV, lambda: norm(n=None)),
        ("norm: gate rows do not divide T", INV, lambda: norm(gate=P, rows=3)),
        ("norm: gate without rows", INV, lambda: norm(gate=P, rows=0)),
        ("norm: rows without a gate", INV, lambda: norm(rows=1)),
        ("norm: unaligned x", INV, lambda: norm(x=U)),
        ("norm: H = 0", INV, lambda: norm(H=0)),
        ("norm: H > 65536", UNS, lambda: norm(H=65537)),
        ("norm: T < 0", INV, lambda: norm(T=-1)),
        ("norm: T past 2^32", INV, lambda: norm(T=1 << 32)),
        ("norm: eps", INV, lambda: norm(cfg=ncfg(eps=nan))),
        ("norm: negative eps", INV, lambda: norm(cfg=ncfg(eps=-1.0))),
        ("norm: residual scale", INV, lambda: norm(cfg=ncfg(a=inf))),
        ("norm: stream type", INV, lambda: norm(cfg=ncfg(st=2))),
        ("norm: weight type", INV, lambda: norm(cfg=ncfg(wt=-1))),
        ("norm: T = 0 does nothing", 0, lambda: norm(T=0, x=None, out=None)),
        ("norm backward: no gradient", INV, lambda: norm_b(d_out=None, d_n=None, dwn=None)),
        ("norm backward: d_n without w_next", INV, lambda: norm_b(wn=None)),
        ("norm backward: no dx", INV, lambda: norm_b(dx=None)),
        ("norm backward: no dy", INV, lambda: norm_b(dy=None)),
        ("norm backward: no dw_post", INV, lambda: norm_b(dwp=None)),
        ("norm backward: dw_post without w_post", INV, lambda: norm_b(wp=None)),
        ("norm backward: no dgate", INV, lambda: norm_b(gate=P, rows=1)),
        ("norm backward: dgate without a gate", INV, lambda: norm_b(dg=P)),
        ("norm backward: no dw_next", INV, lambda: norm_b(dwn=None)),
        ("norm backward: no rstd_out", INV, lambda: norm_b(ro=None)),
        ("norm backward: no rstd_y", INV, lambda: norm_b(ry=None)),
        ("norm backward: no out", INV, lambda: norm_b(out=None)),
        ("norm backward: no workspace", WS, lambda: norm_b(ws=None)),
        ("norm backward: small workspace", WS, lambda: norm_b(wsb=64)),
        ("clip: no tensors' list", INV,
         lambda: L.moe_clip_grad_norm(None, None, None, None, 2, 1.0, 0, 1e-6, P, P, WSB, None)),
        ("clip: n < 0", INV, lambda: clip(n=-1)),
        ("clip: null gradient", INV, lambda: clip(grads=(None,))),
        ("clip: unaligned gradient", INV, lambda: clip(grads=((1 << 20) + 2,))),
        ("clip: null output", INV, lambda: clip(outs=(None,))),
        ("clip: negative size", INV, lambda: clip(numels=(-1,))),
        ("clip: type", INV, lambda: clip(types=(2,))),
        ("clip: kind", INV, lambda: clip(kind=2)),
        ("clip: eps", INV, lambda: clip(eps=-1.0)),
        ("clip: NaN max_norm", INV, lambda: clip(max_norm=nan)),
        ("clip: no result", INV, lambda: clip(nc=None)),
        ("clip: no workspace", WS, lambda: clip(ws=None)),
        ("clip: small workspace", WS, lambda: clip(wsb=8)),
    ]
    for name, want, call in cases:
        assert call() == want, name


def test_binding_refuses_before_the_library(m):
    f32, bf = torch.float32, torch.bfloat16
    logits, x = torch.zeros((4, 8)), torch.zeros((4, 64), dtype=bf)
    for call in (lambda: m.moe_route_gate(logits, 2),
                 lambda: m.moe_route_gate_backward(torch.zeros((4, 2)), logits,
                                                   torch.zeros((4, 2), dtype=torch.int32)),
                 lambda: m.moe_norm_residual(x, x),
                 lambda: m.moe_norm_residual_backward(x, None, x),
                 lambda: m.moe_clip_grad_norm([logits], 1.0)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="norm_type"):
        m.moe_clip_grad_norm([logits], 1.0, norm_type=1.0)
    with pytest.raises(ValueError, match="max_norm"):
        m.moe_clip_grad_norm([logits], -1.0)
    with pytest.raises(ValueError, match="no gradients"):
        m.moe_clip_grad_norm([], 1.0)
    with pytest.raises(ValueError, match="contiguous"):
        m.moe_clip_grad_norm([torch.zeros((4, 8)).t()], 1.0)
    with pytest.raises(ValueError, match=r"grads\[1\]"):
        m.moe_clip_grad_norm([logits, logits.double()], 1.0)
    with pytest.raises(ValueError, match="max_norm is None"):
        m.moe_clip_grad_norm([logits], None, out=[logits])
    with pytest.raises(ValueError, match="score"):
        m._gate_config("tanh", 1, 1, 1, True, 1.0)
    with pytest.raises(ValueError, match="bfloat16"):
        m._typed(logits.double(), "logits")
    with pytest.raises(ValueError, match="shape"):
        m._shaped(torch.zeros(3, dtype=f32), "bias", 8)
