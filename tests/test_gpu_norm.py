"""GPU parity of the norms around the block and their gradients against the
float64 oracle.

Tolerances, in half steps of float32 (H = 2^-24 relative): a row's mean of
non-negative terms is off by at most the length of its longest chain of
additions, here at most width / 256 + 16 terms a thread and lane (64 lanes at
least share a row), and its root by half of that; what a result multiplies
and adds up takes some 8 roundings more. C = 24 + width / 64 half steps
bound all of that, of the sum of the terms' magnitudes (up to 1024 elements
32 lanes may share a row: width / 32 + 5 terms, fewer than C). A column sum over T
tokens adds at most T half steps. bfloat16 results add half a step, 2^-8;
bfloat16 reads are exact."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle as orc
from gpu_util import dev

pytestmark = pytest.mark.gpu
m = pytest.importorskip("moe_expert_dispatch_gb300")

H32, BF = 2.0 ** -24, 2.0 ** -8
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _inputs(T, W, stream, weights, post, rows, nxt, y=True, seed=0):
    g = torch.Generator().manual_seed(seed * 7919 + T * 31 + W)
    rn = lambda *s, sd=1.0, mean=0.0: torch.randn(s, generator=g) * sd + mean  # noqa: E731
    st, wt = TYPES[stream], TYPES[weights]
    v = dict(x=rn(T, W).to(st), y=rn(T, W, sd=0.5).to(torch.bfloat16) if y else None,
             w_post=rn(W, sd=0.2, mean=1.0).to(wt) if post else None,
             gate=rn(rows, W, sd=0.5).to(wt) if rows else None,
             w_next=rn(W, sd=0.2, mean=1.0).to(wt) if nxt else None)
    d_out = rn(T, W, sd=0.1).to(st)
    d_n = rn(T, W, sd=0.1).to(torch.bfloat16) if nxt else None
    return v, d_out, d_n


def _near(got, ref, terms, units, what):
    """|got - ref| within units half steps of the terms' size, and half a step of its type."""
    g, ref = _np(got), np.asarray(ref)
    bound = units * H32 * terms + 1e-37
    if got.dtype == torch.bfloat16:
        bound = bound + BF * np.abs(ref)
    else:
        bound = bound + H32 * np.abs(ref)
    err = np.abs(g - ref)
    assert np.all(err <= bound), (what, float((err - bound).max()))


def _check(v, d_out, d_n, a=1.0, b=1.0, eps=1e-6):
    T, W = v["x"].shape
    c = 24 + W / 64
    sc = dict(residual_scale=a, branch_scale=b)
    n64 = {key: _np(t) for key, t in v.items()}
    ref = orc.norm_residual(**n64, eps=eps, **sc)
    d = {key: dev(t) for key, t in v.items()}
    got = m.moe_norm_residual(**d, eps=eps, **sc)
    # sizes of the terms of out, and of n
    g = orc.gate_rows(n64["gate"], T)
    res = np.abs(n64["x"])
    if v["y"] is not None:
        z = np.abs(n64["y"])
        if v["w_post"] is not None:
            _near(got["rstd_y"], ref["rstd_y"], ref["rstd_y"], c, "rstd_y")
            z = z * ref["rstd_y"][:, None] * np.abs(n64["w_post"])
        res = abs(a) * res + abs(b) * np.abs(g) * z
        _near(got["out"], ref["out"], res, c, "out")
    if v["w_next"] is not None:
        # the mean square of out is off by twice out's own error at most
        _near(got["rstd_out"], ref["rstd_out"],
              ref["rstd_out"] ** 3 * np.mean(res * res, axis=1) + ref["rstd_out"], 2 * c,
              "rstd_out")
        ro = ref["rstd_out"][:, None]
        rel = ro * ro * np.mean(res * res, axis=1, keepdims=True)
        o = np.abs(n64["x"] if ref["out"] is None else ref["out"])
        _near(got["n"], ref["n"], np.abs(n64["w_next"]) * ro * (res + o * (1 + 2 * rel)), 2 * c,
              "n")
    for key in ("out", "n", "rstd_y", "rstd_out"):
        assert (got[key] is None) == (ref[key] is None), key

    # backward, on what the forward kept
    saved = d["x"] if v["y"] is None else got["out"]
    rest = {key: d[key] for key in ("y", "w_post", "gate", "w_next")}
    stats = dict(rstd_y=got["rstd_y"], rstd_out=got["rstd_out"])
    r64 = dict(**{key: n64[key] for key in rest}, rstd_y=_np(stats["rstd_y"]),
               rstd_out=_np(stats["rstd_out"]), **sc)
    for do, dn in ((d_out, d_n), (None, d_n), (d_out, None)):
        if do is None and dn is None:
            continue
        want = orc.norm_residual_backward(_np(do), _np(dn), _np(saved), **r64)
        back = m.moe_norm_residual_backward(dev(do), dev(dn), saved, **rest, **stats, eps=eps, **sc)
        _check_grads(back, want, do, dn, saved, n64, r64, a, b, c)


def _check_grads(back, want, do, dn, saved, n64, r64, a, b, c):
    T, W = saved.shape
    D = np.zeros((T, W)) if do is None else np.abs(_np(do))
    if dn is not None:
        ro = r64["rstd_out"][:, None]
        o, q = np.abs(_np(saved)) * ro, np.abs(_np(dn) * n64["w_next"])
        D = D + ro * (q + o * np.mean(q * o, axis=1, keepdims=True))
        _near(back["dw_next"], want["dw_next"], np.sum(np.abs(_np(dn)) * o, axis=0), c + T,
              "dw_next")
    else:
        assert back["dw_next"] is None
    if n64["y"] is None:
        _near(back["dx"], want["dx"], D, c, "dx")
        assert back["dy"] is None
        return
    _near(back["dx"], want["dx"], abs(a) * D, c, "dx")
    yh = np.abs(n64["y"]) * (1.0 if n64["w_post"] is None else r64["rstd_y"][:, None])
    w = 1.0 if n64["w_post"] is None else np.abs(n64["w_post"])
    g = np.abs(orc.gate_rows(n64["gate"], T))
    if n64["gate"] is not None:
        rows = n64["gate"].shape[0]
        terms = (abs(b) * w * D * yh).reshape(rows, T // rows, W).sum(axis=1)
        _near(back["dgate"], want["dgate"], terms, 2 * c + T, "dgate")
    p = abs(b) * g * w * D
    if n64["w_post"] is not None:
        _near(back["dw_post"], want["dw_post"], np.sum(abs(b) * g * D * yh, axis=0), 2 * c + T,
              "dw_post")
        p = r64["rstd_y"][:, None] * (p + yh * np.mean(p * yh, axis=1, keepdims=True))
    _near(back["dy"], want["dy"], p, 2 * c, "dy")


FORMS = [  # post, gate rows (of T), next, with y
    (True, 1, True, True), (True, 0, True, True), (True, 3, True, True), (False, 0, True, True),
    (False, 1, False, True), (True, 0, False, True), (True, "T", True, True),
    (False, 0, True, False),
]


@pytest.mark.parametrize("T,W", [(1, 1), (3, 7), (6, 333), (9, 512), (3, 1000), (12, 2048),
                                 (3, 4096), (6, 7168), (3, 8192), (3, 10248), (3, 16384),
                                 (3, 20000), (300, 264), (1200, 128)])
@pytest.mark.parametrize("post,rows,nxt,y", FORMS)
def test_norm_against_the_definition(T, W, post, rows, nxt, y):
    rows = T if rows == "T" else rows
    if rows and T % rows:
        rows = T
    for i, (stream, weights) in enumerate((("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"),
                                           ("f32", "bf16"))):
        v, d_out, d_n = _inputs(T, W, stream, weights, post, rows, nxt, y, seed=i)
        _check(v, d_out, d_n, a=(1.0, 0.5)[i % 2], b=(1.0, 1.0, -0.75, 2.0)[i])


def test_norm_gate_rows_across_strips():
    # gate rows whose tokens begin and end inside, at and across the strips of rows
    for T, rows in ((1000, 4), (1216, 304), (912, 456), (2000, 1000), (700, 7), (305, 305)):
        v, d_out, d_n = _inputs(T, 136, "bf16", "f32", True, rows, True, seed=T)
        _check(v, d_out, d_n, a=1.0, b=0.5)


@pytest.mark.parametrize("T,W", [(1, 512), (151, 512), (2500, 512), (700, 1024), (333, 264),
                                 (170, 2304), (160, 1364), (90, 8192), (40, 10240), (500, 45)])
@pytest.mark.parametrize("stream,weights", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_norm_gate_row_for_each_token(T, W, stream, weights):
    v, d_out, d_n = _inputs(T, W, stream, weights, True, T, True, seed=3)
    _check(v, d_out, d_n, a=0.5, b=2.0)
    v, d_out, d_n = _inputs(T, W, stream, weights, False, T, False, seed=4)
    d = {key: dev(t) for key, t in v.items()}
    got = m.moe_norm_residual(**d)
    back = dict(y=d["y"], gate=d["gate"])
    one = m.moe_norm_residual_backward(dev(d_out), None, got["out"], **back)
    two = m.moe_norm_residual_backward(dev(d_out), None, got["out"], **back,
                                       dgate=torch.ones((T, W), device="cuda"),
                                       accumulate_dw=True)
    assert torch.equal(two["dgate"], one["dgate"] + 1.0)
    want = orc.norm_residual_backward(_np(d_out), None, _np(got["out"]), y=_np(v["y"]),
                                      gate=_np(v["gate"]))
    _near(one["dgate"], want["dgate"], np.abs(want["dgate"]), 24, "dgate")
    _near(one["dy"], want["dy"], np.abs(want["dy"]), 24, "dy")


@pytest.mark.parametrize("T,W,rows", [(2000, 136, 1000), (2001, 512, 667), (5000, 512, 2500),
                                      (1212, 333, 404), (999, 2048, 27)])
def test_norm_gate_rows_accumulate_and_repeat(T, W, rows):
    # rows inside strips and across them are each added to once, in the same order every time
    v, d_out, d_n = _inputs(T, W, "bf16", "bf16", True, rows, True, seed=6)
    d = {key: dev(t) for key, t in v.items()}
    f = m.moe_norm_residual(**d)
    rest = dict(y=d["y"], w_post=d["w_post"], gate=d["gate"], w_next=d["w_next"],
                rstd_y=f["rstd_y"], rstd_out=f["rstd_out"])
    one = m.moe_norm_residual_backward(dev(d_out), dev(d_n), f["out"], **rest)
    sums = {key: torch.full_like(one[key], 2.0) for key in ("dw_post", "dgate", "dw_next")}
    two = m.moe_norm_residual_backward(dev(d_out), dev(d_n), f["out"], **rest,
                                       accumulate_dw=True, **sums)
    for key in ("dx", "dy"):
        assert torch.equal(two[key], one[key]), key
    for key in sums:
        assert torch.equal(two[key], one[key] + 2.0), key


@pytest.mark.parametrize("W", [36, 1020, 1021, 1028, 8200, 16388, 20001])
@pytest.mark.parametrize("rows", [0, 1, 6, 30])
def test_norm_lengths_that_the_ring_does_not_take(W, rows):
    for stream, weights in (("bf16", "f32"), ("f32", "bf16")):
        v, d_out, d_n = _inputs(30, W, stream, weights, True, rows, True, seed=5)
        _check(v, d_out, d_n, a=1.5, b=0.5)


def test_norm_zero_rows_and_large_values():
    v, d_out, d_n = _inputs(4, 512, "f32", "f32", True, 1, True)
    v["x"][0] = 0.0
    v["y"][0] = 0.0                                # an empty row: the norm of zeros is zero
    v["x"][1] *= 1e15
    v["y"][2] *= 1e-20
    _check(v, d_out, d_n)
    got = m.moe_norm_residual(**{key: dev(t) for key, t in v.items()})
    assert torch.all(got["out"][0] == 0) and torch.all(got["n"][0] == 0)


def test_norm_infinities_and_nan_stay_in_their_row():
    v, d_out, d_n = _inputs(5, 256, "bf16", "bf16", True, 0, True)
    clean = m.moe_norm_residual(**{key: dev(t) for key, t in v.items()})
    v["x"][1, 3] = float("inf")
    v["y"][3, 5] = float("nan")
    got = m.moe_norm_residual(**{key: dev(t) for key, t in v.items()})
    for key in ("out", "n"):
        for t in (0, 2, 4):
            assert torch.equal(got[key][t], clean[key][t])
    assert torch.isnan(got["out"][3]).all() and torch.isnan(got["n"][3]).all()
    assert torch.isinf(got["out"][1, 3]) and torch.isnan(got["n"][1, 3])


def test_norm_in_place_and_accumulated():
    for W in (1024, 333):
        v, d_out, d_n = _inputs(40, W, "f32", "f32", True, 4, True)
        d = {key: dev(t) for key, t in v.items()}
        f = m.moe_norm_residual(**d)
        x = d["x"].clone()
        g = m.moe_norm_residual(**{**d, "x": x}, out=x)
        assert g["out"].data_ptr() == x.data_ptr()
        assert torch.equal(x, f["out"]) and torch.equal(g["n"], f["n"])
        rest = dict(y=d["y"], w_post=d["w_post"], gate=d["gate"], w_next=d["w_next"],
                    rstd_y=f["rstd_y"], rstd_out=f["rstd_out"])
        one = m.moe_norm_residual_backward(dev(d_out), dev(d_n), f["out"], **rest)
        dx = dev(d_out)
        sums = {key: torch.ones_like(one[key]) for key in ("dw_post", "dgate", "dw_next")}
        two = m.moe_norm_residual_backward(dx, dev(d_n), f["out"], **rest, dx=dx,
                                           accumulate_dw=True, **sums)
        assert torch.equal(dx, one["dx"]) and torch.equal(two["dy"], one["dy"])
        for key, t in sums.items():
            assert torch.equal(t, one[key] + 1.0), key
        with pytest.raises(ValueError, match="accumulate_dw"):
            m.moe_norm_residual_backward(dx, dev(d_n), f["out"], **rest, accumulate_dw=True)


def test_norm_zero_tokens():
    v, d_out, d_n = _inputs(0, 256, "bf16", "bf16", True, 1, True)
    d = {key: dev(t) for key, t in v.items()}
    f = m.moe_norm_residual(**d)
    assert f["out"].shape == (0, 256)
    rest = dict(y=d["y"], w_post=d["w_post"], gate=d["gate"], w_next=d["w_next"],
                rstd_y=f["rstd_y"], rstd_out=f["rstd_out"])
    g = m.moe_norm_residual_backward(dev(d_out), dev(d_n), f["out"], **rest)
    for key in ("dw_post", "dgate", "dw_next"):
        assert torch.all(g[key] == 0), key
        g[key].fill_(3.0)
    m.moe_norm_residual_backward(dev(d_out), dev(d_n), f["out"], **rest, dw_post=g["dw_post"],
                                 dgate=g["dgate"], dw_next=g["dw_next"], accumulate_dw=True)
    for key in ("dw_post", "dgate", "dw_next"):
        assert torch.all(g[key] == 3.0), key


def test_norm_past_two_to_the_31_elements():
    T, W = (1 << 31) // 4096 + 77, 4096
    x = torch.zeros((T, W), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros((T, W), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(W, dtype=torch.bfloat16, device="cuda")
    x[-1], y[-1], x[0], y[0] = 1.0, 2.0, 3.0, 1.0
    got = m.moe_norm_residual(x, y, w_post=w, w_next=w, eps=0.0)
    assert torch.all(got["out"][-1] == 2.0) and torch.all(got["n"][-1] == 1.0)
    assert torch.all(got["out"][0] == 4.0) and torch.all(got["n"][0] == 1.0)
    f = dict(y=y, w_post=w, w_next=w, rstd_y=torch.ones(T, device="cuda"),
             rstd_out=torch.ones(T, device="cuda"))
    out = got["out"]
    del got
    g = m.moe_norm_residual_backward(x, y, out, **f)
    ref = orc.norm_residual_backward(_np(x[-1:]), _np(y[-1:]), _np(out[-1:]), y=_np(y[-1:]),
                                     w_post=_np(w), w_next=_np(w), rstd_y=np.ones(1),
                                     rstd_out=np.ones(1))
    assert np.allclose(_np(g["dx"][-1:]), ref["dx"], rtol=2 * BF, atol=1e-4)
    # with eps = 0 the norm of a row of zeros is 0 / 0, and so is what follows from it
    assert torch.isnan(out[1:-1]).all() and torch.isnan(g["dx"][1:-1]).all()


def test_norm_on_another_stream_and_in_a_graph():
    v, d_out, d_n = _inputs(130, 2048, "bf16", "f32", True, 2, True)
    d = {key: dev(t) for key, t in v.items()}
    do, dn = dev(d_out), dev(d_n)
    f = m.moe_norm_residual(**d)
    rest = dict(y=d["y"], w_post=d["w_post"], gate=d["gate"], w_next=d["w_next"])
    g = m.moe_norm_residual_backward(do, dn, f["out"], **rest, rstd_y=f["rstd_y"],
                                     rstd_out=f["rstd_out"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    f2 = m.moe_norm_residual(**d, stream=side)
    side.synchronize()
    for key in f:
        assert torch.equal(f[key], f2[key]), key
    buf = {key: torch.empty_like(t) for key, t in f.items()}
    grads = {key: torch.empty_like(t) for key, t in g.items()}
    ws = torch.empty(m._lib.moe_norm_residual_backward_workspace_size(130, 2048, 2),
                     dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_norm_residual(**d, **buf)
        m.moe_norm_residual_backward(do, dn, buf["out"], **rest, rstd_y=buf["rstd_y"],
                                     rstd_out=buf["rstd_out"], workspace=ws, **grads)
    for _ in range(2):
        for t in (*buf.values(), *grads.values()):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for key in f:
            assert torch.equal(f[key], buf[key]), key
        for key in g:
            assert torch.equal(g[key], grads[key]), key


def test_norm_refusals():
    x = dev(torch.zeros((4, 64), dtype=torch.bfloat16))
    w = dev(torch.ones(64))
    with pytest.raises(ValueError, match="share one type"):
        m.moe_norm_residual(x, x, w_post=w, w_next=w.bfloat16())
    with pytest.raises(ValueError, match="shape"):
        m.moe_norm_residual(x, x, w_post=w[:32].clone())
    with pytest.raises(ValueError, match="gate"):
        m.moe_norm_residual(x, x, gate=dev(torch.ones((2, 32))))
    with pytest.raises(ValueError, match="bfloat16"):
        m.moe_norm_residual(x, x.float())
    for call in (lambda: m.moe_norm_residual(x),
                 lambda: m.moe_norm_residual(x, x, gate=dev(torch.ones((3, 64)))),
                 lambda: m.moe_norm_residual(x.reshape(-1)[1:129].view(2, 64), None, w_next=w),
                 lambda: m.moe_norm_residual_backward(None, None, x),
                 lambda: m.moe_norm_residual_backward(x, x, x),
                 lambda: m.moe_norm_residual_backward(x, None, x, y=x, w_post=w)):
        with pytest.raises(m.MoeError) as e:
            call()
        assert e.value.status == 1


def test_norm_of_two_lengths_from_two_threads():
    # rows of 512 and of 7168 share their kernels and differ in the shared memory that these
    # launch with; the library's own calls, back to back, so that the threads' launches mix
    import threading
    cases, wrong = [], []
    for W in (512, 7168):
        v, d_out, d_n = _inputs(160, W, "bf16", "bf16", True, 1, True)
        d = {key: dev(t) for key, t in v.items()}
        do, dn = dev(d_out), dev(d_n)
        f = m.moe_norm_residual(**d)
        rest = {key: d[key] for key in ("y", "w_post", "gate", "w_next")}
        g = m.moe_norm_residual_backward(do, dn, f["out"], **rest, rstd_y=f["rstd_y"],
                                         rstd_out=f["rstd_out"])
        got_f = {key: torch.zeros_like(t) for key, t in f.items()}
        got_g = {key: torch.zeros_like(t) for key, t in g.items()}
        need = m._lib.moe_norm_residual_backward_workspace_size(160, W, 1)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        stream = torch.cuda.Stream()
        at = lambda t: t.data_ptr()                # noqa: E731
        w = (at(d["w_post"]), at(d["gate"]), 1, at(d["w_next"]))
        there = (at(d["x"]), at(d["y"]), *w, 160, W, None, *map(at, got_f.values()),
                 stream.cuda_stream)
        back = (at(do), at(dn), at(f["out"]), at(d["y"]), *w, at(f["rstd_y"]), at(f["rstd_out"]),
                160, W, None, *map(at, got_g.values()), 0, at(ws), need, stream.cuda_stream)
        cases.append((there, back, stream, (f, got_f), (g, got_g), (d, do, dn, ws)))
    torch.cuda.synchronize()
    start = threading.Barrier(2)

    def work(there, back):
        torch.cuda.current_stream()                # the thread's device
        start.wait()
        for i in range(20000):
            status = (m._lib.moe_norm_residual(*there), m._lib.moe_norm_residual_backward(*back))
            if status != (0, 0):
                wrong.append((i, status))
                return

    threads = [threading.Thread(target=work, args=c[:2]) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong, wrong
    for case in cases:
        for want, got in case[3:5]:
            for key in want:
                assert torch.equal(want[key], got[key]), key


# groups of one warp and of several, one group a CTA and many, every form of the gate, rows
# whose last threads have no columns, forms without the first reduction
LATE = [(5000, 512, True, 0), (2000, 1024, True, 20), (700, 4096, True, 700), (160, 2048, True, 1),
        (3000, 1096, False, 0), (1500, 7168, True, 1), (1500, 2048, False, 1500)]


def _late(T, W, post, rows):
    """Calls that give their waits up, each followed by one that is right."""
    for stream in ("f32", "bf16"):
        v, d_out, d_n = _inputs(T, W, stream, "bf16", post, rows, True)
        d, do, dn = {key: dev(t) for key, t in v.items()}, dev(d_out), dev(d_n)
        f = m.moe_norm_residual(**d)
        rest = dict(**{key: d[key] for key in ("y", "w_post", "gate", "w_next")},
                    rstd_y=f["rstd_y"], rstd_out=f["rstd_out"])
        g = m.moe_norm_residual_backward(do, dn, f["out"], **rest)
        assert m.moe_get_error() == 0
        for _ in range(3):
            os.environ["MOE_GB300_GIVE_UP_WAITS"] = "1"
            m.moe_norm_residual(**d)
            assert m.moe_get_error() == 5
            m.moe_norm_residual_backward(do, dn, f["out"], **rest)
            assert m.moe_get_error() == 5
            del os.environ["MOE_GB300_GIVE_UP_WAITS"]
            f2 = m.moe_norm_residual(**d)
            g2 = m.moe_norm_residual_backward(do, dn, f["out"], **rest)
            assert m.moe_get_error() == 0
            for a, b in ((f, f2), (g, g2)):
                for key in a:
                    assert a[key] is None or torch.equal(a[key], b[key]), key


def test_norm_wait_timeout_reports_and_recovers():
    # the library's waits last microseconds of their two seconds: the debug build gives them up
    # where the environment says so
    if not m.DEBUG:
        code = "import test_gpu_norm as t; [t._late(*c) for c in t.LATE]; print('late ok')"
        here = os.path.dirname(os.path.abspath(__file__))
        path = os.pathsep.join([os.path.dirname(here), here])
        r = subprocess.run([sys.executable, "-c", code], cwd=here, capture_output=True, text=True,
                           timeout=300, env=dict(os.environ, MOE_GB300_DEBUG="1", PYTHONPATH=path))
        assert r.returncode == 0 and "late ok" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
        return
    for case in LATE:
        _late(*case)
