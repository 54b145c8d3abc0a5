"""The gated feed-forward block on the GPU against the float64 oracle.

Two kinds of input. Small integers through relu: every product and partial sum
is an integer below 2^24, exact in the float accumulators, and h and dA are
rounded from equal numbers, so every output has to be bit-equal to the oracle's
rounding. Gaussian values through every activation: a bf16 rounding is off by
at most 2^-8 of the value; h and dA may besides land one step (2^-7) away where
the float value before the rounding (2^-14 of it off at most: the sums' 2^-24 a
term, __expf and the reciprocal) crosses a boundary. So each output lies within
2^-8 of itself plus (2^-7 + 2^-14) of the sum of its terms' magnitudes."""
import numpy as np
import pytest
import torch

import oracle as orc
from gpu_util import dev

pytestmark = pytest.mark.gpu
m = pytest.importorskip("moe_expert_dispatch_gb300")

BF = torch.bfloat16
ACTS = ["silu", "gelu", "gelu_tanh", "relu"]
# one tile, tails of every tile dimension, a K shorter than a block and not a multiple of it
SHAPES = [(1, 8, 8), (1, 64, 64), (2, 2048, 768), (3, 72, 136), (16, 512, 1024), (17, 128, 64),
          (33, 1000, 328), (64, 264, 2056), (65, 64, 520), (127, 256, 384), (129, 136, 72),
          (256, 128, 640), (257, 200, 1000), (300, 1000, 328), (513, 512, 1032),
          # few tiles of a long K: its parts in several clusters
          (130, 4096, 136), (200, 1104, 2056), (513, 1032, 1544), (140, 72, 4104)]


def _np(t):
    return t.detach().double().cpu().numpy()


def _bf(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(BF)


def _ints(T, H, F, seed, add=True):
    """Values in {-1, 0, 1}, sparse enough that |A| stays small."""
    rng = np.random.default_rng(seed)

    def tri(shape, share):
        return rng.choice([-1.0, 0.0, 1.0], shape, p=[share / 2, 1 - share, share / 2])

    share = min(1.0, 24.0 / H)
    v = dict(x=tri((T, H), 0.7), w_gate=tri((H, F), share), w_up=tri((H, F), share),
             w_down=tri((F, H), min(1.0, 24.0 / F)))
    return v, (tri((T, H), 0.9) * 5 if add else None), tri((T, H), 0.6)


def _forward(v, add, act, **kw):
    d = {k: dev(_bf(t)) for k, t in v.items()}
    a = None if add is None else dev(_bf(add))
    return d, a, m.moe_gated_ffn(**d, act=act, add=a, **kw)


def _equal(got, ref, what):
    want = _bf(ref).double().numpy() if got.dtype == BF else ref
    assert np.array_equal(_np(got), want), (what, np.argwhere(_np(got) != want)[:3])


@pytest.mark.parametrize("T,H,F", SHAPES)
@pytest.mark.parametrize("add", [False, True])
def test_ffn_forward_integers(T, H, F, add):
    v, a, _ = _ints(T, H, F, T + H + F, add)
    ref = orc.gated_ffn(**v, kind="relu", add=a)
    for save in (False, True):
        _, _, got = _forward(v, a, "relu", save_for_backward=save)
        assert m.moe_get_error() == 0
        _equal(got["y"], ref["y"], "y")
        if save:
            _equal(got["a_gate"], ref["a_gate"], "a_gate")
            _equal(got["a_up"], ref["a_up"], "a_up")
        else:
            assert got["a_gate"] is None and got["a_up"] is None


@pytest.mark.parametrize("T,H,F", SHAPES)
@pytest.mark.parametrize("add", [False, True])
def test_ffn_backward_integers(T, H, F, add):
    v, a, dy = _ints(T, H, F, 2 * T + H + F, add)
    fwd = orc.gated_ffn(**v, kind="relu")
    ref = orc.gated_ffn_backward(dy, **v, a_gate=fwd["a_gate"], a_up=fwd["a_up"], kind="relu",
                                 add=a)
    d = {k: dev(_bf(t)) for k, t in v.items()}
    rest = dict(a_gate=dev(_bf(fwd["a_gate"])), a_up=dev(_bf(fwd["a_up"])), act="relu",
                add=None if a is None else dev(_bf(a)))
    for dt in (BF, torch.float32):
        got = m.moe_gated_ffn_backward(dev(_bf(dy)), **d, **rest, dw_dtype=dt)
        assert m.moe_get_error() == 0
        for key in ("dx", "dw_gate", "dw_up", "dw_down"):
            assert got[key].dtype == (BF if key == "dx" else dt)
            _equal(got[key], ref[key], key)
    # added to what is there, in float
    more = {k: torch.full_like(got[k], 3.0) for k in ("dw_gate", "dw_up", "dw_down")}
    got = m.moe_gated_ffn_backward(dev(_bf(dy)), **d, **rest, **more, accumulate_dw=True)
    for key in more:
        assert got[key] is more[key]
        _equal(got[key], ref[key] + 3.0, key)
    # frozen weights
    got = m.moe_gated_ffn_backward(dev(_bf(dy)), **d, **rest, weight_grads=False)
    _equal(got["dx"], ref["dx"], "dx")
    assert got["dw_gate"] is None and got["dw_up"] is None and got["dw_down"] is None


def _within(got, ref, terms, what, step=2.0 ** -7 + 2.0 ** -14, own=2.0 ** -8):
    err = np.abs(_np(got) - ref)
    bound = own * np.abs(ref) + step * terms + 1e-30
    assert (err <= bound).all(), (what, float((err / bound).max()))


def _gauss(T, H, F, seed):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, sd=1.0):
        return (torch.randn(shape, generator=g) * sd).to(BF)

    return (dict(x=normal(T, H), w_gate=normal(H, F, sd=H ** -0.5), w_up=normal(H, F, sd=H ** -0.5),
                 w_down=normal(F, H, sd=F ** -0.5)), normal(T, H), normal(T, H, sd=0.1))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,H,F", [(1, 128, 256), (5, 72, 200), (40, 520, 392), (150, 256, 328),
                                   (300, 200, 264), (180, 1096, 1544)])
def test_ffn_gaussian(T, H, F, act):
    v, add, dy = _gauss(T, H, F, T + H)
    n = {k: _np(t) for k, t in v.items()}
    d = {k: dev(t) for k, t in v.items()}
    ref = orc.gated_ffn(**n, kind=act, add=_np(add))
    got = m.moe_gated_ffn(**d, act=act, add=dev(add), save_for_backward=True)
    size = np.abs(ref["h"]) @ np.abs(n["w_down"]) + 2.0 ** -10 * np.abs(_np(add))
    _within(got["y"], ref["y"], size, "y")
    for key, w in (("a_gate", "w_gate"), ("a_up", "w_up")):
        _within(got[key], ref[key], np.abs(n["x"]) @ np.abs(n[w]), key, step=2.0 ** -20)
    kept = {k: _np(got[k]) for k in ("a_gate", "a_up")}
    ref = orc.gated_ffn_backward(_np(dy), **n, **kept, kind=act, add=_np(add))
    back = m.moe_gated_ffn_backward(dev(dy), **d, a_gate=got["a_gate"], a_up=got["a_up"], act=act,
                                    add=dev(add))
    assert m.moe_get_error() == 0
    # dh may cancel: its own rounding goes by its terms
    dh = np.abs(_np(dy)) @ np.abs(n["w_down"]).T * 2.0 ** -10
    dg = np.abs(ref["da_gate"]) + dh * np.abs(kept["a_up"]) * 1.2
    du = np.abs(ref["da_up"]) + dh * np.abs(orc.act(kept["a_gate"], act))
    _within(back["dx"], ref["dx"], dg @ np.abs(n["w_gate"]).T + du @ np.abs(n["w_up"]).T
            + 2.0 ** -10 * np.abs(_np(add)), "dx")
    _within(back["dw_gate"], ref["dw_gate"], np.abs(n["x"]).T @ dg, "dw_gate")
    _within(back["dw_up"], ref["dw_up"], np.abs(n["x"]).T @ du, "dw_up")
    _within(back["dw_down"], ref["dw_down"], np.abs(ref["h"]).T @ np.abs(_np(dy)), "dw_down")


@pytest.mark.parametrize("T,H,F", [(20, 128, 256), (300, 136, 200)])
def test_ffn_gradient_against_differences(T, H, F):
    """The slope of a float64 forward along a random direction of each input, against
    the kernels' gradients: bf16 roundings of h, dA and the result are 2^-8 each, and
    the products of 300 x 136 random terms average them."""
    v, _, dy = _gauss(T, H, F, 3)
    n = {k: _np(t) for k, t in v.items()}
    f = m.moe_gated_ffn(**{k: dev(t) for k, t in v.items()}, act="gelu", save_for_backward=True)
    got = m.moe_gated_ffn_backward(dev(dy), **{k: dev(t) for k, t in v.items()},
                                   a_gate=f["a_gate"], a_up=f["a_up"], act="gelu",
                                   dw_dtype=torch.float32)
    rng = np.random.default_rng(9)
    e = 1e-5
    for key, name in (("x", "dx"), ("w_gate", "dw_gate"), ("w_up", "dw_up"),
                      ("w_down", "dw_down")):
        u = rng.standard_normal(n[key].shape)

        def loss(s):
            p = dict(n, **{key: n[key] + s * u})
            return float((orc.gated_ffn(**p, kind="gelu", rounded=False)["y"] * _np(dy)).sum())

        slope = (loss(e) - loss(-e)) / (2 * e)
        size = np.linalg.norm(_np(got[name]))      # a random direction's slope is about that
        assert abs(slope - float((_np(got[name]) * u).sum())) < 2.0 ** -5 * size, name


def test_ffn_rows_keep_to_themselves():
    # a NaN or an infinity in one row reaches that row alone, in every direction but
    # the weight gradients; rows of a tile past T hold nothing
    T, H, F = 70, 128, 192
    v, _, dy = _gauss(T, H, F, 1)
    clean = m.moe_gated_ffn(**{k: dev(t) for k, t in v.items()}, save_for_backward=True)
    bad = dict(v, x=v["x"].clone())
    bad["x"][13, 5] = float("nan")
    bad["x"][44, 7] = float("inf")
    got = m.moe_gated_ffn(**{k: dev(t) for k, t in bad.items()}, save_for_backward=True)
    rest = [t for t in range(T) if t not in (13, 44)]
    for key in ("y", "a_gate", "a_up"):
        assert torch.equal(got[key][rest], clean[key][rest]), key
        assert got[key][13].isnan().all()
    dyb = dy.clone()
    dyb[13] = float("nan")
    w = {k: dev(t) for k, t in v.items()}
    kept = dict(a_gate=clean["a_gate"], a_up=clean["a_up"], weight_grads=False)
    a = m.moe_gated_ffn_backward(dev(dy), **w, **kept)["dx"]
    b = m.moe_gated_ffn_backward(dev(dyb), **w, **kept)["dx"]
    assert torch.equal(a[[t for t in range(T) if t != 13]], b[[t for t in range(T) if t != 13]])
    assert b[13].isnan().all()


@pytest.mark.parametrize("act", ACTS)
def test_ffn_far_activations(act):
    # gates from -3e4 to 3e4: one input, w_gate holding them, w_up 1, w_down the unit
    # matrix, so that y is h itself; and the gradient of that
    z = torch.cat([torch.linspace(-40, 40, 161), torch.tensor([-3e4, 3e4, 1e-30, 0.0, -0.0])])
    F = 176
    z = torch.cat([z, torch.zeros(F - z.numel())]).to(BF)
    x = torch.zeros(1, 8, dtype=BF)
    x[0, 0] = 1.0
    wg, wu = torch.zeros(8, F, dtype=BF), torch.zeros(8, F, dtype=BF)
    wg[0], wu[0] = z, 1.0
    wd = torch.zeros(F, F, dtype=BF)[:, :8]
    got = m.moe_gated_ffn(dev(x), dev(wg), dev(wu), dev(wd.contiguous()), act=act,
                          save_for_backward=True)
    assert torch.equal(got["a_gate"][0].cpu(), z) and (got["y"] == 0).all()
    # dW_down = h^T dy reads h out, dA through dW_gate and dW_up (x = 1 in column 0)
    dy = torch.zeros(1, 8, dtype=BF)
    dy[0, 0] = 1.0
    one = torch.zeros(F, 8, dtype=BF)
    one[:, 0] = 1.0
    back = m.moe_gated_ffn_backward(dev(dy), dev(x), dev(wg), dev(wu), dev(one), got["a_gate"],
                                    got["a_up"], act=act, dw_dtype=torch.float32)
    z64 = z.double().numpy()
    h, dg, du = (_np(back["dw_down"])[:, 0], _np(back["dw_gate"])[0], _np(back["dw_up"])[0])
    # bf16's 2^-8 beside the float formula's own error: a few 2^-24 of |z| + 1
    small = (np.abs(z64) + 1) * 2.0 ** -20
    assert (np.abs(h - orc.act(z64, act)) <= 2.0 ** -7.9 * np.abs(orc.act(z64, act)) + small).all()
    assert (np.abs(du - orc.act(z64, act)) <= 2.0 ** -7.9 * np.abs(orc.act(z64, act)) + small).all()
    want = orc.act_grad(z64, act)
    assert (np.abs(dg - want) <= 2.0 ** -7.9 * np.abs(want) + small).all()


def test_ffn_in_place_and_empty():
    v, a, dy = _ints(90, 136, 72, 5)
    ref = orc.gated_ffn(**v, kind="relu", add=a)
    d = {k: dev(_bf(t)) for k, t in v.items()}
    y = dev(_bf(a))
    got = m.moe_gated_ffn(**d, act="relu", add=y, y=y)
    assert got["y"] is y
    _equal(y, ref["y"], "y in place")
    kept = dict(a_gate=dev(_bf(ref["a_gate"])), a_up=dev(_bf(ref["a_up"])), act="relu")
    want = orc.gated_ffn_backward(dy, **v, a_gate=ref["a_gate"], a_up=ref["a_up"], kind="relu",
                                  add=a)
    dx = dev(_bf(a))
    m.moe_gated_ffn_backward(dev(_bf(dy)), **d, **kept, add=dx, dx=dx)
    _equal(dx, want["dx"], "dx in place")
    # no tokens
    e = torch.empty(0, 136, dtype=BF, device="cuda")
    ef = torch.empty(0, 72, dtype=BF, device="cuda")
    w = dict(w_gate=d["w_gate"], w_up=d["w_up"], w_down=d["w_down"])
    assert m.moe_gated_ffn(e, **w)["y"].shape == (0, 136)
    for dt in (BF, torch.float32):
        got = m.moe_gated_ffn_backward(e, e, **w, a_gate=ef, a_up=ef, dw_dtype=dt)
        assert all((got[k] == 0).all() for k in ("dw_gate", "dw_up", "dw_down"))
    one = {k: torch.ones(got[k].shape, device="cuda") for k in ("dw_gate", "dw_up", "dw_down")}
    m.moe_gated_ffn_backward(e, e, **w, a_gate=ef, a_up=ef, accumulate_dw=True, **one)
    assert all((t == 1).all() for t in one.values())
    assert m.moe_get_error() == 0


@pytest.mark.parametrize("T", [1, 40, 300])
def test_ffn_writes_its_outputs_only(T):
    # every output in the middle of a buffer of sevens: what lies around stays
    H, F = 136, 200
    v, a, dy = _ints(T, H, F, 6)
    d = {k: dev(_bf(t)) for k, t in v.items()}

    def middle(rows, cols, dtype=BF):
        buf = torch.full((rows * cols + 4096,), 7.0, dtype=dtype, device="cuda")
        return buf, buf[2048:2048 + rows * cols].view(rows, cols)

    bufs = [middle(T, H), middle(T, F), middle(T, F)]
    m.moe_gated_ffn(**d, act="relu", save_for_backward=True, y=bufs[0][1], a_gate=bufs[1][1],
                    a_up=bufs[2][1])
    ref = orc.gated_ffn(**v, kind="relu")
    _equal(bufs[0][1], ref["y"], "y")
    back = [middle(T, H), middle(H, F), middle(H, F), middle(F, H)]
    m.moe_gated_ffn_backward(dev(_bf(dy)), **d, a_gate=bufs[1][1], a_up=bufs[2][1], act="relu",
                             dx=back[0][1], dw_gate=back[1][1], dw_up=back[2][1],
                             dw_down=back[3][1])
    assert m.moe_get_error() == 0
    for buf, mid in bufs + back:
        assert (buf[:2048] == 7).all() and (buf[2048 + mid.numel():] == 7).all()


@pytest.mark.parametrize("T", [4, 300])
def test_ffn_on_another_stream_and_in_a_graph(T):
    H, F = 256, 512
    v, add, dy = _gauss(T, H, F, 8)
    d = {k: dev(t) for k, t in v.items()}
    add, dy = dev(add), dev(dy)
    want = m.moe_gated_ffn(**d, add=add, save_for_backward=True)
    back = m.moe_gated_ffn_backward(dy, **d, a_gate=want["a_gate"], a_up=want["a_up"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = m.moe_gated_ffn(**d, add=add, save_for_backward=True, stream=s)
    s.synchronize()
    for key in want:
        assert torch.equal(got[key], want[key])
    x = d["x"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f = m.moe_gated_ffn(x, d["w_gate"], d["w_up"], d["w_down"], add=add, save_for_backward=True)
        b = m.moe_gated_ffn_backward(dy, x, d["w_gate"], d["w_up"], d["w_down"], f["a_gate"],
                                     f["a_up"])
    for _ in range(3):
        for t in list(f.values()) + list(b.values()):
            t.fill_(9.0)
        x.copy_(d["x"])
        g.replay()
    torch.cuda.synchronize()
    for key in want:
        assert torch.equal(f[key], want[key]), key
    for key in back:
        assert torch.equal(b[key], back[key]), key
    x.copy_(d["x"].flip(0))
    g.replay()
    again = m.moe_gated_ffn(x, d["w_gate"], d["w_up"], d["w_down"], add=add)
    assert torch.equal(f["y"], again["y"])
    assert m.moe_get_error() == 0


@pytest.mark.parametrize("T,H,F", [(300000, 8, 8192), (90, 2048, 264)])
def test_ffn_far_rows_and_repeats(T, H, F):
    # h and the gradients of 2.4e9 elements, rows by their own formula; the same bits again
    x = torch.zeros(T, H, dtype=BF, device="cuda")
    x[:, 3] = (torch.arange(T, device="cuda") % 5 - 2).to(BF)
    wg, wu = (torch.zeros(H, F, dtype=BF, device="cuda") for _ in range(2))
    wd = torch.zeros(F, H, dtype=BF, device="cuda")
    wg[3], wu[3] = 1.0, 2.0
    wd[F - 1, 1] = 1.0
    got = m.moe_gated_ffn(x, wg, wu, wd, act="relu", save_for_backward=True)
    xs = x[:, 3].float()
    h = xs.clamp(min=0) * 2 * xs
    assert torch.equal(got["y"][:, 1].float(), h) and torch.equal(got["a_up"][:, F - 1].float(), 2 * xs)
    assert torch.equal(m.moe_gated_ffn(x, wg, wu, wd, act="relu")["y"], got["y"])
    dy = torch.zeros(T, H, dtype=BF, device="cuda")
    dy[:, 1] = 1.0
    back = [m.moe_gated_ffn_backward(dy, x, wg, wu, wd, got["a_gate"], got["a_up"], act="relu",
                                     dw_dtype=torch.float32) for _ in range(2)]
    on = (xs > 0).float()
    # dA_g = 2 x [x > 0], dA_u = x [x > 0], in the last column alone
    assert torch.equal(back[0]["dx"][:, 3].float(), 4 * xs * on)
    assert back[0]["dw_down"][F - 1, 1] == h.double().sum()
    assert back[0]["dw_up"][3, F - 1] == (xs * xs * on).double().sum()
    for key in back[0]:
        assert torch.equal(back[0][key], back[1][key]), key
    assert m.moe_get_error() == 0


def test_ffn_two_streams_at_once():
    H, F = 512, 1024
    runs = []
    for T, seed in ((64, 1), (400, 2)):
        v, add, _ = _gauss(T, H, F, seed)
        runs.append((dict({k: dev(t) for k, t in v.items()}, add=dev(add)), torch.cuda.Stream()))
    want = [m.moe_gated_ffn(**d)["y"] for d, _ in runs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (d, s) in enumerate(runs):
            got[i].append(m.moe_gated_ffn(**d, stream=s)["y"])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])
    assert m.moe_get_error() == 0


# by few rows, by tiles, and by tiles whose K is split
@pytest.mark.parametrize("T,H", [(1, 176), (300, 176), (140, 1096)])
@pytest.mark.parametrize("act", ACTS)
def test_ffn_far_activations_in_each_form(act, T, H):
    """Gates from -3e4 to 3e4 with unit matrices around them, so that y is h, dx is dA_g or
    dA_u, and dW_down against rows of the unit matrix is h again; A_u = 1. Each is off by a
    bf16 rounding (2^-8) beside the float formula's own error, 2^-14 of each of its terms: the
    exponential's argument (up to 88, by four roundings of 2^-24) and its 2 + 1.2 * 88 ulps;
    erfc's argument (by two, which erfc multiplies by up to 13^2) and a few ulps; a quotient of
    two ulps. What is below 2^-118 may be cut to zero (a quotient by more than 2^126 is)."""
    z = torch.cat([torch.linspace(-40, 40, 161), torch.tensor([-3e4, 3e4, 1e-30, 0.0, -0.0, -88.0,
                                                               88.0, -1e3, 1e3])])
    z = torch.cat([z, torch.zeros(H - z.numel())]).to(BF)
    z64 = z.double().numpy()
    eye, zero = torch.eye(H).to(BF), torch.zeros(H, H, dtype=BF)
    x = torch.zeros(T, H, dtype=BF)
    x[:, 0] = 1.0
    wg, wu = zero.clone(), zero.clone()
    wg[0], wu[0] = z, 1.0
    got = m.moe_gated_ffn(dev(x), dev(wg), dev(wu), dev(eye), act=act, save_for_backward=True)
    assert torch.equal(got["a_gate"].cpu(), z.expand(T, H)) and (got["a_up"] == 1).all()
    f, d = orc.act(z64, act), orc.act_grad(z64, act)
    slack = 2.0 ** -8 * np.abs(f) + 2.0 ** -14 * np.abs(f) + 2.0 ** -118

    def holds(t, want, bound, what):
        err = np.abs(_np(t) - want)
        assert (err <= bound).all(), (what, z64[np.argwhere(err > bound)[0][-1]])

    holds(got["y"], f, slack, "y")
    one = torch.ones(T, H, dtype=BF)
    kept = dict(a_gate=got["a_gate"], a_up=got["a_up"], act=act, weight_grads=False)
    du = m.moe_gated_ffn_backward(dev(one), dev(x), dev(zero), dev(eye), dev(eye), **kept)["dx"]
    holds(du, f, slack, "dA_u")
    dg = m.moe_gated_ffn_backward(dev(one), dev(x), dev(eye), dev(zero), dev(eye), **kept)["dx"]
    # act' is f / z and a second term that may cancel it
    first = np.where(z64 == 0, 0.5, f / np.where(z64 == 0, 1.0, z64))
    terms = np.abs(first) + np.abs(d - first)
    holds(dg, d, 2.0 ** -8 * np.abs(d) + 2.0 ** -14 * terms + 2.0 ** -118, "dA_g")
    rows = torch.zeros(T, H, dtype=BF)
    rows[torch.arange(min(T, H)), torch.arange(min(T, H))] = 1.0
    kept.update(weight_grads=True, dw_dtype=torch.float32)
    back = m.moe_gated_ffn_backward(dev(rows), dev(x), dev(zero), dev(zero), dev(eye), **kept)
    holds(back["dw_down"].t()[:min(T, H)], f, slack, "h")
    assert m.moe_get_error() == 0


# shapes whose lists of tiles end in a way that SHAPES do not: units of dx on some of the
# clusters and gradient tiles past the rounds that those stay out of (the first three),
# several units a cluster with several column tiles (the last)
@pytest.mark.parametrize("T,H,F", [(140, 1032, 2056), (300, 1000, 2728), (1500, 520, 1544),
                                   (4700, 1096, 648)])
def test_ffn_walks_over_tiles(T, H, F):
    v, a, dy = _ints(T, H, F, T + F)
    ref = orc.gated_ffn(**v, kind="relu", add=a)
    d, add, got = _forward(v, a, "relu", save_for_backward=True)
    for key in ("y", "a_gate", "a_up"):
        _equal(got[key], ref[key], key)
    want = orc.gated_ffn_backward(dy, **v, a_gate=ref["a_gate"], a_up=ref["a_up"], kind="relu",
                                  add=a)
    for dt in (BF, torch.float32):
        back = m.moe_gated_ffn_backward(dev(_bf(dy)), **d, a_gate=got["a_gate"], a_up=got["a_up"],
                                        act="relu", add=add, dw_dtype=dt)
        for key in back:
            assert np.abs(want[key]).max() < 2 ** 24
            _equal(back[key], want[key], key)
    assert m.moe_get_error() == 0


# past the few rows: tiles of one part of K, and of several; columns that end inside a piece
TILED = [(300, 136, 72), (200, 136, 4104), (140, 1096, 1096), (513, 1032, 1544)]


@pytest.mark.parametrize("T,H,F", TILED)
def test_ffn_in_place_by_tiles(T, H, F):
    v, a, dy = _ints(T, H, F, T + 5)
    ref = orc.gated_ffn(**v, kind="relu", add=a)
    d = {k: dev(_bf(t)) for k, t in v.items()}
    y = dev(_bf(a))
    assert m.moe_gated_ffn(**d, act="relu", add=y, y=y)["y"] is y
    _equal(y, ref["y"], "y in place")
    kept = dict(a_gate=dev(_bf(ref["a_gate"])), a_up=dev(_bf(ref["a_up"])), act="relu")
    want = orc.gated_ffn_backward(dy, **v, a_gate=ref["a_gate"], a_up=ref["a_up"], kind="relu",
                                  add=a)
    for weights in (True, False):
        dx = dev(_bf(a))
        got = m.moe_gated_ffn_backward(dev(_bf(dy)), **d, **kept, add=dx, dx=dx,
                                       weight_grads=weights)
        assert got["dx"] is dx
        _equal(dx, want["dx"], "dx in place")
        if weights:
            for key in ("dw_gate", "dw_up", "dw_down"):
                _equal(got[key], want[key], key)
    assert m.moe_get_error() == 0


@pytest.mark.parametrize("T,H,F", TILED)
def test_ffn_rows_keep_to_themselves_by_tiles(T, H, F):
    v, add, dy = _gauss(T, H, F, 1)
    w = {k: dev(t) for k, t in v.items()}
    add = dev(add)
    clean = m.moe_gated_ffn(**w, add=add, save_for_backward=True)
    bad = v["x"].clone()
    bad[13, 5], bad[44, 7], bad[T - 1] = float("nan"), float("inf"), float("nan")
    got = m.moe_gated_ffn(**dict(w, x=dev(bad)), add=add, save_for_backward=True)
    rest = [t for t in range(T) if t not in (13, 44, T - 1)]
    for key in ("y", "a_gate", "a_up"):
        assert torch.equal(got[key][rest], clean[key][rest]), key
        assert got[key][13].isnan().all() and got[key][T - 1].isnan().all()
        assert not got[key][44].isfinite().all()
    bad = dy.clone()
    bad[13], bad[T - 1] = float("nan"), float("inf")
    for weights in (True, False):
        a, b = (m.moe_gated_ffn_backward(dev(t), **w, a_gate=clean["a_gate"], a_up=clean["a_up"],
                                         add=add, weight_grads=weights)["dx"] for t in (dy, bad))
        rest = [t for t in range(T) if t not in (13, T - 1)]
        assert torch.equal(a[rest], b[rest])
        assert b[13].isnan().all() and not b[T - 1].isfinite().all()
    assert m.moe_get_error() == 0


# runs of rows that end with a single block of 64, or one row, in either type
@pytest.mark.parametrize("T,H,F", [(8193, 72, 136), (16448, 8, 296), (577, 264, 72)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_ffn_gradients_of_runs_and_a_rest(T, H, F, dtype):
    v, _, dy = _ints(T, H, F, T, False)
    fwd = orc.gated_ffn(**v, kind="relu")
    want = orc.gated_ffn_backward(dy, **v, a_gate=fwd["a_gate"], a_up=fwd["a_up"], kind="relu")
    d = {k: dev(_bf(t)) for k, t in v.items()}
    args = dict(a_gate=dev(_bf(fwd["a_gate"])), a_up=dev(_bf(fwd["a_up"])), act="relu")
    got = m.moe_gated_ffn_backward(dev(_bf(dy)), **d, **args, dw_dtype=dtype)
    for key in got:
        assert np.abs(want[key]).max() < 2 ** 24
        _equal(got[key], want[key], key)
    # the same in a graph, beside a call on another stream
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    dyb = dev(_bf(dy))
    with torch.cuda.graph(g):
        again = m.moe_gated_ffn_backward(dyb, **d, **args, dw_dtype=dtype)
    for t in again.values():
        t.zero_()
    torch.cuda.synchronize()
    g.replay()
    beside = m.moe_gated_ffn_backward(dyb, **d, **args, dw_dtype=dtype, stream=s)
    torch.cuda.synchronize()
    for key in got:
        assert torch.equal(again[key], got[key]) and torch.equal(beside[key], got[key]), key
    assert m.moe_get_error() == 0


def _known_grads(T, H, F, positive, dtype, seed=0):
    """The weight gradients beside their float64 values and the sums of their terms'
    magnitudes, on inputs that leave no rounding before the sums: A_g = 1 through relu, so
    that h = A_u; a selection as W_down, so that dh is columns of dy and dA_u = dh; dA_g =
    bf16(dh A_u), of an exact product."""
    g = torch.Generator(device="cuda").manual_seed(T + seed)

    def rnd(*s):
        v = torch.randn(s, generator=g, device="cuda")
        return (v.abs() if positive else v).to(BF)

    x, dy, up = rnd(T, H), rnd(T, H), rnd(T, F)
    col = torch.arange(F, device="cuda") % H
    wd = torch.zeros(F, H, dtype=BF, device="cuda")
    wd[torch.arange(F), col] = 1.0
    w = torch.zeros(H, F, dtype=BF, device="cuda")
    args = (dy, x, w, w, wd, torch.ones_like(up), up)
    got = m.moe_gated_ffn_backward(*args, act="relu", dw_dtype=dtype)
    dh = dy[:, col]
    pairs = dict(dw_down=(up, dy), dw_gate=(x, (dh.float() * up.float()).to(BF)), dw_up=(x, dh))
    for key, (p, q) in pairs.items():
        ref = p.double().t() @ q.double()
        yield key, got[key], ref, p.double().abs().t() @ q.double().abs(), args


@pytest.mark.parametrize("T,H,F", [(8192, 256, 392), (12001, 72, 264), (16384, 264, 128)])
@pytest.mark.parametrize("positive", [True, False])
def test_ffn_float_gradients_of_many_rows(T, H, F, positive):
    """A run of 512 rows is 32 sums of 16 products and what is there; each may cut off 17
    numbers below 2^-23 of the partial sum, on the average half of the last one: 32 * 17 / 2 *
    2^-23 < 2^-14.9 of the terms. The additions of at most 32 runs round by 2^-24 each, 2^-19.
    What is cut off is half of the most that it can be in the mean: 2^-15.9 of the sums. (One
    accumulator over 8192 rows of positive numbers is off by 2^-14.7, over 16384 by 2^-13.5,
    all of it in the mean.)"""
    for key, got, ref, terms, args in _known_grads(T, H, F, positive, torch.float32):
        err = got.double() - ref
        assert (err.abs() <= (2.0 ** -14.9 + 2.0 ** -19) * terms).all(), key
        mean = (err * ref.sign()).sum().abs()
        assert mean <= (2.0 ** -15.9 + 2.0 ** -19) * (ref.abs() if positive else terms).sum(), key
    # a second pass adds the same again: x + x is exact
    one = m.moe_gated_ffn_backward(*args, act="relu", dw_dtype=torch.float32)
    more = {k: one[k].clone() for k in ("dw_gate", "dw_up", "dw_down")}
    m.moe_gated_ffn_backward(*args, act="relu", **more, accumulate_dw=True)
    for key in more:
        assert torch.equal(more[key], 2 * one[key]), key
    assert m.moe_get_error() == 0


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_ffn_gradients_of_a_million_rows(dtype):
    """By runs of 512 rows as above (2^-14.9 of the terms), with 2^11 roundings of sums that
    grow to the last one (2^-24 / 2 each on the average: 2^-14); in bf16 by runs of 8192 rows,
    512 such sums (2^-10.9), 2^7 roundings, and half a step of bf16 (2^-8 of the result). One
    accumulator over a million rows loses more than 2^-8."""
    T = 1000003
    for key, got, ref, terms, _ in _known_grads(T, 64, 40, True, dtype):
        own = 2.0 ** -10.9 + 2.0 ** -18 if dtype == BF else 2.0 ** -14.9 + 2.0 ** -14
        half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
        assert ((got.double() - ref).abs() <= half * ref.abs() + (1 + half) * own * terms).all(), key
    assert m.moe_get_error() == 0


def test_ffn_refusals():
    x, w, wd = (torch.zeros(s, dtype=BF, device="cuda") for s in ((4, 64), (64, 32), (32, 64)))
    with pytest.raises(m.MoeError, match="unsupported"):
        m.moe_gated_ffn(*(torch.zeros(s, dtype=BF, device="cuda") for s in ((4, 60), (60, 32),
                                                                          (60, 32), (32, 60))))
    with pytest.raises(ValueError, match="w_down"):
        m.moe_gated_ffn(x, w, w, wd.t())
    with pytest.raises(ValueError, match="w_up"):
        m.moe_gated_ffn(x, w, w[:, :16].contiguous(), wd)
    with pytest.raises(ValueError, match="contiguous"):
        m.moe_gated_ffn(torch.zeros(64, 4, dtype=BF, device="cuda").t(), w, w, wd)
    with pytest.raises(ValueError, match="x must be"):
        m.moe_gated_ffn(x.float(), w, w, wd)
    with pytest.raises(ValueError, match="add"):
        m.moe_gated_ffn(x, w, w, wd, add=x[:2])
    with pytest.raises(m.MoeError, match="workspace"):
        m.moe_gated_ffn(x, w, w, wd, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    a = torch.zeros(4, 32, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="accumulate_dw"):
        m.moe_gated_ffn_backward(x, x, w, w, wd, a, a, accumulate_dw=True)
    with pytest.raises(m.MoeError, match="unsupported"):
        m.moe_gated_ffn_backward(x, x, w, w, wd, a, a, accumulate_dw=True, dw_gate=w.clone(),
                                 dw_up=w.clone(), dw_down=wd.clone())
    with pytest.raises(ValueError, match="dw_up"):
        m.moe_gated_ffn_backward(x, x, w, w, wd, a, a, dw_gate=w.float(), dw_up=w.clone())
