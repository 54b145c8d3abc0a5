"""CPU pins of the dense half of a layer: the oracle's formulas against
hand-worked values, torch and finite differences, and the host-side checks of
the entry points, which answer before any launch."""
import ctypes
import functools
import math

import numpy as np
import pytest
import torch

import oracle as orc

ACTS = ["silu", "gelu", "gelu_tanh", "relu"]


def _torch_act(z, kind):
    F = torch.nn.functional
    return {"silu": F.silu, "gelu": F.gelu, "relu": F.relu,
            "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}[kind](z)


# ------------------------------------------------------------------ the oracle's formulas

@pytest.mark.parametrize("kind", ACTS)
def test_activations_are_torchs(kind):
    z = torch.linspace(-9, 9, 361, dtype=torch.float64, requires_grad=True)
    f = _torch_act(z, kind)
    f.sum().backward()
    np.testing.assert_allclose(orc.act(z.detach().numpy(), kind), f.detach().numpy(), rtol=1e-12,
                               atol=1e-15)
    np.testing.assert_allclose(orc.act_grad(z.detach().numpy(), kind), z.grad.numpy(), rtol=1e-10,
                               atol=1e-14)


def test_gelu_tanh_far_out():
    # (1 + tanh u) / 2 in 180 digits, where doubles would cancel: -9.5 gives 7.4e-34 of it
    from decimal import Decimal, localcontext

    with localcontext() as c:
        c.prec = 180
        k = (Decimal(2) / Decimal("3.14159265358979323846264338327950288419716939937510582097494459")).sqrt()

        def f(z):
            e = (2 * k * (z + Decimal("0.044715") * z ** 3)).exp()
            return z * (1 + (e - 1) / (e + 1)) / 2

        for v in (-12.0, -9.5, -6.0, -1.0, 0.5, 3.0, 9.0):
            z, d = Decimal(v), Decimal("1e-30")
            got = orc.act(np.array([v]), "gelu_tanh")[0], orc.act_grad(np.array([v]), "gelu_tanh")[0]
            for have, want in zip(got, (f(z), (f(z + d) - f(z - d)) / (2 * d))):
                assert abs(have - float(want)) <= 1e-11 * abs(float(want)), (v, have, float(want))
    far = np.array([-3e4, -1e3, 1e3, 3e4])
    assert orc.act(far, "gelu_tanh").tolist() == [0.0, 0.0, 1e3, 3e4]
    assert orc.act_grad(far, "gelu_tanh").tolist() == [0.0, 0.0, 1.0, 1.0]


def test_ffn_by_hand():
    # one token, two hidden units: A_g = (1, -2), A_u = (3, 5); relu keeps the first
    x, wg, wu = np.array([[1.0, 2.0]]), np.array([[1.0, 0.0], [0.0, -1.0]]), np.array([[1.0, 1.0],
                                                                                     [1.0, 2.0]])
    wd = np.array([[2.0, -1.0], [7.0, 7.0]])
    f = orc.gated_ffn(x, wg, wu, wd, "relu", add=np.array([[10.0, 10.0]]))
    assert f["h"].tolist() == [[3.0, 0.0]] and f["y"].tolist() == [[16.0, 7.0]]
    b = orc.gated_ffn_backward(np.array([[1.0, 1.0]]), x, wg, wu, wd, f["a_gate"], f["a_up"],
                               "relu")
    # dh = (1, 14): dA_g = (3, 0), dA_u = (1, 0)
    assert b["da_gate"].tolist() == [[3.0, 0.0]] and b["da_up"].tolist() == [[1.0, 0.0]]
    assert b["dx"].tolist() == [[4.0, 1.0]]
    assert b["dw_down"].tolist() == [[3.0, 3.0], [0.0, 0.0]]
    assert b["dw_gate"].tolist() == [[3.0, 0.0], [6.0, 0.0]]
    assert b["dw_up"].tolist() == [[1.0, 0.0], [2.0, 0.0]]


@pytest.mark.parametrize("kind", ACTS)
def test_ffn_gradient_against_differences(kind):
    rng = np.random.default_rng(4)
    T, H, F = 3, 4, 5
    v = dict(x=rng.standard_normal((T, H)), w_gate=rng.standard_normal((H, F)),
             w_up=rng.standard_normal((H, F)), w_down=rng.standard_normal((F, H)))
    dy = rng.standard_normal((T, H))

    def loss(p):
        return float((orc.gated_ffn(**p, kind=kind, rounded=False)["y"] * dy).sum())

    f = orc.gated_ffn(**v, kind=kind, rounded=False)
    got = orc.gated_ffn_backward(dy, **v, a_gate=f["a_gate"], a_up=f["a_up"], kind=kind,
                                 rounded=False)
    e = 1e-6
    for key, name in (("x", "dx"), ("w_gate", "dw_gate"), ("w_up", "dw_up"),
                      ("w_down", "dw_down")):
        for at in np.ndindex(v[key].shape):
            hi, lo = {k: a.copy() for k, a in v.items()}, {k: a.copy() for k, a in v.items()}
            hi[key][at] += e
            lo[key][at] -= e
            assert abs((loss(hi) - loss(lo)) / (2 * e) - got[name][at]) < 1e-6, (name, at)


def test_lora_by_hand():
    a = np.array([[[1.0, 1.0]], [[1.0, -1.0]]])             # n 2, r 1, H 2
    b = np.array([[[1.0, 2.0, 3.0]], [[10.0, 0.0, 0.0]]])
    x = np.array([[2.0, 1.0], [5.0, 1.0], [1.0, 1.0]])
    out, v = orc.lora(x, a, b, [1, -1, 0], scales=[2.0, 0.5], base=np.ones((3, 3)))
    assert v.tolist() == [[1.0], [0.0], [2.0]]
    assert out.tolist() == [[6.0, 1.0, 1.0], [1.0, 1.0, 1.0], [5.0, 9.0, 13.0]]
    order, offsets = orc.lora_plan([1, -1, 0, 1, -1], 3)
    assert order.tolist() == [2, 0, 3, 1, 4] and offsets.tolist() == [0, 1, 3, 3]


def test_lora_gradient_against_differences():
    rng = np.random.default_rng(5)
    T, H, N, n, r = 6, 4, 5, 3, 2
    ids = [2, -1, 0, 2, 2, 0]
    v = dict(x=rng.standard_normal((T, H)), a=rng.standard_normal((n, r, H)),
             b=rng.standard_normal((n, r, N)))
    scales, dy = [0.5, 3.0, 2.0], rng.standard_normal((T, N))

    def loss(p):
        return float((orc.lora(p["x"], p["a"], p["b"], ids, scales)[0] * dy).sum())

    kept = orc.lora(v["x"], v["a"], v["b"], ids, scales)[1]
    got = orc.lora_backward(dy, v["x"], kept, v["a"], v["b"], ids, scales)
    e = 1e-6
    for key, name in (("x", "dx"), ("a", "da"), ("b", "db")):
        for at in np.ndindex(v[key].shape):
            hi, lo = {k: t.copy() for k, t in v.items()}, {k: t.copy() for k, t in v.items()}
            hi[key][at] += e
            lo[key][at] -= e
            assert abs((loss(hi) - loss(lo)) / (2 * e) - got[name][at]) < 1e-7, (name, at)
    assert not got["da"][1].any() and not got["db"][1].any()      # no row has that adapter


def test_philox_known_answers():
    # the generator's published test vectors (Random123: kat_vectors, philox4x32 10)
    assert orc.philox4x32([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert orc.philox4x32([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2) == [
        0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert orc.philox4x32([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344],
                          [0xA4093822, 0x299F31D0]) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_dropout_share_and_streams():
    kept = orc.dropout_kept(40000, 11, 3, 0.25)
    # a binomial of 40000 tries: six standard deviations
    assert abs(kept.mean() - 0.75) < 6 * math.sqrt(0.75 * 0.25 / 40000)
    assert np.array_equal(kept, orc.dropout_kept(40000, 11, 3, 0.25))
    for other in (orc.dropout_kept(40000, 12, 3, 0.25), orc.dropout_kept(40000, 11, 4, 0.25)):
        # two independent masks agree in 0.75^2 + 0.25^2 of the places
        assert abs((kept == other).mean() - 0.625) < 6 * math.sqrt(0.625 * 0.375 / 40000)
    assert orc.dropout_kept(100, 1, 1, 0.0).all()
    assert orc.dropout_threshold(0.1) == 6554 and orc.dropout_threshold(0.9999999) == 65535
    # the mean of what is kept is that of the input
    out = orc.dropout_residual(np.ones(40000), kept, 0.25)
    assert abs(out.mean() - 1.0) < 0.02


# ------------------------------------------------------------------ host-side checks

@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    import moe_expert_dispatch_gb300
    return moe_expert_dispatch_gb300


P = ctypes.c_void_p(1 << 20)             # fake, aligned addresses that no check reads
U = ctypes.c_void_p((1 << 20) + 2)
Q, R = ctypes.c_void_p(1 << 21), ctypes.c_void_p(1 << 22)
INV, UNS, WS = 1, 2, 4
BIG = 1 << 40


def test_lora_takes_rows_one_by_one_as_measured(m):
    # no workspace: a cluster a row. With every slot in use the first of each pair is faster
    # so; the second is faster by units when one or 16 of the slots are in use
    size = m._lib.moe_lora_workspace_size
    for T, n, r in ((128, 32, 16), (256, 32, 16), (512, 512, 16), (1000, 512, 16), (64, 1024, 64),
                    (1800, 1024, 16)):
        assert size(T, n, r) == 0, (T, n, r)
    for T, n, r in ((512, 16, 16), (512, 32, 16), (1000, 256, 16), (1800, 512, 16), (4096, 1024, 16),
                    (1000, 512, 64), (600, 256, 64)):
        assert size(T, n, r) > 0, (T, n, r)


def test_dense_workspace_sizes(m):
    L = m._lib
    assert L.moe_gated_ffn_workspace_size(3, 64, 40) == 256
    assert L.moe_gated_ffn_workspace_size(1000, 64, 4096) == 1000 * 4096 * 2
    assert L.moe_gated_ffn_backward_workspace_size(1000, 64, 4096) == 3 * 1000 * 4096 * 2
    assert L.moe_gated_ffn_workspace_size(0, 64, 40) == 0
    for bad in ((-1, 64, 64), (4, 60, 64), (4, 64, 60), (4, 0, 64), (4, 64, -8)):
        assert L.moe_gated_ffn_workspace_size(*bad) == 0, bad
        assert L.moe_gated_ffn_backward_workspace_size(*bad) == 0, bad
    # images of units of 128 rows, 16 KB to 64 columns of two parts; none for few rows
    assert L.moe_lora_workspace_size(1000, 4, 16) == (8 + 4) * 16384
    assert L.moe_lora_workspace_size(1000, 4, 128) == (8 + 4) * 4 * 16384
    assert L.moe_lora_workspace_size(64, 4, 16) == 0
    assert L.moe_lora_backward_workspace_size(1000, 4, 16) > 2 * (8 + 4) * 16384
    for bad in ((100, 4, 129), (-1, 4, 16), (100, 0, 16), (100, 1025, 16), (100, 4, 0)):
        assert L.moe_lora_workspace_size(*bad) == 0
        assert L.moe_lora_backward_workspace_size(*bad) == 0
    c = m.moe_dropout_config()
    L.moe_dropout_config_init(c)
    assert abs(c.p - 0.1) < 1e-7 and c.residual_scale == 1.0 and c.branch_scale == 1.0
    assert c.stream_type == 1 and c.branch_type == 1


def test_dense_entry_points_refuse_before_any_launch(m):
    if torch.cuda.is_available():
        pytest.skip("host-only: the cases carry fake device addresses")
    L = m._lib

    def ffn(x=P, wg=P, wu=P, wd=P, add=None, T=4, H=64, F=64, act=0, y=P, ag=None, au=None, ws=P,
            n=BIG):
        return L.moe_gated_ffn(x, wg, wu, wd, add, T, H, F, act, y, ag, au, ws, n, None)

    def ffn_b(dy=P, x=P, wg=P, wu=P, wd=P, ag=P, au=P, add=None, T=4, H=64, F=64, act=0, dx=P,
              dg=P, du=P, dd=P, dt=1, acc=0, ws=P, n=BIG):
        return L.moe_gated_ffn_backward(dy, x, wg, wu, wd, ag, au, add, T, H, F, act, dx, dg, du,
                                        dd, dt, acc, ws, n, None)

    assert ffn(T=0, x=None) == 0
    for kw in (dict(x=None), dict(wg=None), dict(wu=None), dict(wd=None), dict(y=None),
               dict(ag=P), dict(au=P), dict(act=4), dict(act=-1), dict(T=-1), dict(T=1 << 31),
               dict(H=0), dict(F=-8), dict(x=U), dict(wg=U), dict(wu=U), dict(wd=U), dict(add=U),
               dict(y=U), dict(ag=U, au=P), dict(ag=P, au=U)):
        assert ffn(**kw) == INV, kw
    for kw in (dict(H=60), dict(F=4), dict(H=100, F=100)):
        assert ffn(**kw) == UNS, kw
    for kw in (dict(ws=None), dict(n=255), dict(ws=U)):
        assert ffn(**kw) == WS, kw
    for kw in (dict(dy=None), dict(x=None), dict(wg=None), dict(wu=None), dict(wd=None),
               dict(ag=None), dict(au=None), dict(dx=None), dict(dg=None), dict(du=None),
               dict(dd=None), dict(dt=2), dict(act=9), dict(T=-2), dict(dy=U), dict(dx=U),
               dict(add=U), dict(dg=U), dict(dd=U), dict(ag=U), dict(dx=Q, dy=Q),
               dict(dx=Q, x=Q)):
        assert ffn_b(**dict(dict(dx=R), **kw)) == INV, kw
    assert ffn_b(H=60) == UNS and ffn_b(acc=1) == UNS
    ffn_b = functools.partial(ffn_b, dx=R)
    assert ffn_b(T=0, acc=1, dt=0) == 0 and ffn_b(T=0, dg=None, du=None, dd=None) == 0
    for kw in (dict(ws=None), dict(n=3 * 512 - 1), dict(ws=U)):
        assert ffn_b(**kw) == WS, kw

    def plan(ids=P, T=4, n=2, order=P, off=P):
        return L.moe_lora_plan(ids, T, n, order, off, None)

    for kw in (dict(ids=None), dict(order=None), dict(off=None), dict(n=0), dict(n=1025),
               dict(T=-1), dict(T=1 << 31)):
        assert plan(**kw) == INV, kw

    def lora(x=P, a=P, b=P, ids=P, order=P, off=P, s=None, base=None, T=4, H=64, N=64, n=2, r=8,
             out=P, v=P, ws=P, nb=BIG):
        return L.moe_lora(x, a, b, ids, order, off, s, base, T, H, N, n, r, out, v, ws, nb, None)

    assert lora(T=0, x=None) == 0
    for kw in (dict(x=None), dict(a=None), dict(b=None), dict(ids=None), dict(order=None),
               dict(off=None), dict(out=None), dict(v=None), dict(n=0), dict(n=1025), dict(r=0),
               dict(T=-1), dict(H=0), dict(N=-8), dict(x=U), dict(a=U), dict(b=U), dict(base=U),
               dict(out=U)):
        assert lora(**kw) == INV, kw
    for kw in (dict(H=60), dict(N=12), dict(r=129)):
        assert lora(**kw) == UNS, kw

    for kw in (dict(ws=None), dict(nb=255), dict(ws=U)):
        assert lora(T=500, **kw) == WS, kw

    def lora_b(dy=P, x=P, v=P, a=P, b=P, order=P, off=P, s=None, base=None, T=4, H=64, N=64, n=2,
               r=8, dx=P, da=P, db=P, acc=0, ws=P, nb=BIG):
        return L.moe_lora_backward(dy, x, v, a, b, order, off, s, base, T, H, N, n, r, dx, da, db,
                                   acc, ws, nb, None)

    assert lora_b(T=0, acc=1) == 0
    for kw in (dict(dy=None), dict(x=None), dict(v=None), dict(a=None), dict(b=None),
               dict(order=None), dict(off=None), dict(dx=None), dict(da=None), dict(db=None),
               dict(dy=U), dict(base=U), dict(da=U), dict(db=U), dict(n=0), dict(r=0),
               dict(dx=Q, dy=Q), dict(dx=Q, x=Q)):
        assert lora_b(**dict(dict(dx=R), **kw)) == INV, kw
    assert lora_b(r=129) == UNS and lora_b(H=4) == UNS
    for kw in (dict(ws=None), dict(nb=255), dict(ws=U)):
        assert lora_b(dx=R, **kw) == WS, kw

    def drop(y=P, x=None, k=10, rng=P, p=0.1, a=1.0, b=1.0, st=1, bt=1, out=P):
        return L.moe_dropout_residual(y, x, k, rng, m.moe_dropout_config(p, a, b, st, bt), out,
                                      None)

    def drop_b(d=P, k=10, rng=P, p=0.1, a=1.0, b=1.0, st=1, bt=1, dx=None, dy=P):
        return L.moe_dropout_residual_backward(d, k, rng, m.moe_dropout_config(p, a, b, st, bt),
                                               dx, dy, None)

    odd = ctypes.c_void_p((1 << 20) + 1)
    assert drop(k=0, y=None, rng=None) == 0 and drop_b(k=0, d=None, rng=None) == 0
    for kw in (dict(y=None), dict(out=None), dict(rng=None), dict(p=1.0), dict(p=-0.1),
               dict(p=math.nan), dict(a=math.inf), dict(b=math.nan), dict(st=2), dict(bt=-1),
               dict(k=-1), dict(k=1 << 40), dict(y=odd), dict(x=odd), dict(out=odd),
               dict(y=U, bt=0), dict(x=U, st=0), dict(rng=U)):
        assert drop(**kw) == INV, kw
    for kw in (dict(d=None), dict(dy=None), dict(rng=None), dict(p=1.0), dict(st=3), dict(k=-1),
               dict(d=odd), dict(dx=odd), dict(dy=odd), dict(dx=U, st=0)):
        assert drop_b(**kw) == INV, kw


def test_dense_entry_points_refuse_what_would_overlap_or_overflow(m):
    if torch.cuda.is_available():
        pytest.skip("host-only: the cases carry fake device addresses")
    L = m._lib

    def drop(y=P, x=None, numel=64, out=Q, p=0.5, b=1.0, st=0, bt=1):
        return L.moe_dropout_residual(y, x, numel, R, m.moe_dropout_config(p, 1.0, b, st, bt), out,
                                      None)

    def drop_b(d_out=P, numel=64, dx=None, dy=Q, st=0, bt=1):
        return L.moe_dropout_residual_backward(d_out, numel, R,
                                               m.moe_dropout_config(0.5, 1.0, 1.0, st, bt), dx, dy,
                                               None)

    assert drop(out=P) == INV and drop_b(dy=P) == INV
    assert drop_b(dy=P, dx=Q, bt=0) == INV and drop_b(dx=Q, dy=Q, bt=0) == INV
    # the factor is rounded to float: 3e38 / (1 - 1/2) is past its range
    assert drop(b=3e38) == INV and drop(b=-3e38) == INV and drop(b=3e38, numel=0) == INV

    T = 2 ** 27
    assert m._lib.moe_lora_workspace_size(T, 3, 4) > 0
    assert m._lib.moe_lora_workspace_size(T + 1, 3, 4) == 0
    assert m._lib.moe_lora_backward_workspace_size(T + 1, 3, 4) == 0
    assert L.moe_lora(P, P, P, P, P, P, None, None, T + 1, 8, 8, 3, 4, P, P, P, BIG, None) == UNS
    assert L.moe_lora_backward(P, P, P, P, P, P, P, None, None, T + 1, 8, 8, 3, 4, R, P, P, 0, P,
                               BIG, None) == UNS


def test_dense_binding_refuses_before_the_library(m):
    bf = torch.bfloat16
    x, w, wd = torch.zeros(4, 16, dtype=bf), torch.zeros(16, 8, dtype=bf), torch.zeros(8, 16, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_gated_ffn(x, w, w, wd)
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_gated_ffn_backward(x, x, w, w, wd, torch.zeros(4, 8, dtype=bf),
                                 torch.zeros(4, 8, dtype=bf))
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_lora_plan(torch.zeros(4, dtype=torch.int32), 2)
    with pytest.raises(ValueError, match="shape"):
        m.moe_lora_plan(torch.zeros(4, 1, dtype=torch.int32), 2)
    a, b = torch.zeros(2, 4, 16, dtype=bf), torch.zeros(2, 4, 8, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_lora(x, a, b, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="shapes"):
        m.moe_lora(x, a, b[0], torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="shapes"):
        m.moe_lora(x, a, b[:1], torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_dropout_residual(x, torch.zeros(2, dtype=torch.int64), 0.1)
    with pytest.raises(ValueError, match="float32 or torch.bfloat16"):
        m.moe_dropout_residual(x.half(), torch.zeros(2, dtype=torch.int64), 0.1)
    with pytest.raises(ValueError, match="act must"):
        m._act("swish")
