"""Low-rank adapters on the GPU against the float64 oracle.

Small integers: every sum is an integer below 2^24 (and v one that two bf16
numbers hold), so v, da, db and the roundings of out and dx have to be equal.
Gaussian values: v is a float sum (chains of 128 terms, float additions
beyond); out and dx lie within 2^-8 of themselves and 2^-15 of the sum
of their terms (v to 16 bits, the sums' own roundings); da and db within 2^-15
of theirs."""
import numpy as np
import pytest
import torch

import oracle as orc

pytestmark = pytest.mark.gpu
m = pytest.importorskip("moe_expert_dispatch_gb300")

BF = torch.bfloat16


def _np(t):
    return t.detach().double().cpu().numpy()


def _ids(T, n, kind, rng):
    if kind == "mixed":
        return rng.integers(-1, n, T)
    if kind == "none":
        return np.full(T, -1)
    if kind == "one":
        return np.full(T, n - 1)
    ids = np.sort(rng.integers(0, n, T))           # runs, some adapters without a row
    return rng.permutation(n)[ids]


def _draw(T, H, N, n, r, kind, seed, integers):
    rng = np.random.default_rng(seed)

    def make(*shape, sd=1.0, low=-2, high=3):
        v = rng.integers(low, high, shape).astype(np.float64) if integers \
            else rng.standard_normal(shape) * sd
        return torch.from_numpy(v.astype(np.float32)).to(BF).cuda()

    # integers: A sparse enough that v stays below 2^16
    v = dict(x=make(T, H), a=make(n, r, H, sd=H ** -0.5), b=make(n, r, N, sd=r ** -0.5))
    scales = rng.choice([0.5, 1.0, 2.0, -4.0], n) if integers else rng.uniform(0.5, 2.0, n)
    return (v, torch.from_numpy(_ids(T, n, kind, rng).astype(np.int32)).cuda(),
            torch.from_numpy(scales.astype(np.float32)).cuda(), make(T, N), make(T, H), make(T, N))


CASES = [(1, 64, 64, 1, 1, "one"), (1, 4096, 4096, 8, 16, "mixed"), (2, 8, 8, 3, 4, "mixed"),
         (5, 200, 72, 4, 13, "mixed"), (33, 512, 1000, 7, 16, "mixed"),
         (64, 264, 520, 70, 64, "mixed"), (128, 64, 136, 5, 32, "runs"),
         (129, 72, 328, 3, 16, "runs"), (200, 136, 264, 2, 17, "mixed"),
         (300, 520, 128, 9, 33, "runs"), (257, 128, 512, 4, 100, "mixed"),
         (400, 256, 200, 40, 128, "runs"), (500, 64, 64, 3, 8, "none"),
         (700, 328, 392, 1, 48, "one"), (1500, 200, 136, 6, 16, "mixed"),
         # whole units of rows that follow one another, and few rows up to their bound
         (900, 264, 392, 2, 64, "runs"), (600, 136, 200, 1, 128, "one"), (700, 72, 64, 1, 32, "one"),
         (256, 72, 2056, 9, 32, "mixed"), (129, 1000, 72, 300, 2, "mixed"),
         # many adapters of a few rows each, and as few as units still take
         (500, 72, 136, 200, 8, "mixed"), (900, 64, 72, 500, 5, "runs"),
         (700, 136, 64, 60, 64, "mixed"), (150, 64, 328, 1, 128, "one"),
         # few rows of long and short widths, of one adapter, of many and of none
         (64, 264, 520, 2, 13, "runs"), (65, 264, 520, 2, 13, "runs"), (66, 72, 64, 1, 1, "one"),
         (67, 4096, 8, 3, 16, "mixed"), (100, 136, 72, 3, 128, "mixed"), (90, 8, 4104, 80, 5, "mixed"),
         (99, 64, 2056, 4, 33, "none")]


@pytest.mark.parametrize("T,n,kind", [(0, 3, "mixed"), (1, 1, "one"), (31, 5, "mixed"),
                                      (33, 5, "runs"), (1000, 1, "none"), (1024, 1024, "mixed"),
                                      (1025, 7, "mixed"), (20000, 33, "mixed")])
def test_lora_plan(T, n, kind):
    _check_plan(T, n, kind)


# on both sides of where a cluster takes the rows, runs that end inside a CTA's share, one
# key alone and every key
@pytest.mark.parametrize("T,n,kind", [(4096, 1024, "mixed"), (4097, 1024, "mixed"),
                                      (4097, 1, "none"), (8191, 3, "runs"), (70001, 1, "one"),
                                      (65600, 1000, "mixed"), (100003, 64, "runs")])
def test_lora_plan_of_many_rows(T, n, kind):
    _check_plan(T, n, kind)


def _check_plan(T, n, kind):
    ids = _ids(T, n, kind, np.random.default_rng(T))
    order, offsets = m.moe_lora_plan(torch.from_numpy(ids.astype(np.int32)).cuda(), n)
    want = orc.lora_plan(ids.tolist(), n)
    assert np.array_equal(order.cpu().numpy(), want[0])
    assert np.array_equal(offsets.cpu().numpy(), want[1])
    assert m.moe_get_error() == 0


@pytest.mark.parametrize("T,H,N,n,r,kind", CASES)
def test_lora_integers(T, H, N, n, r, kind):
    v, ids, scales, base, dbase, dy = _draw(T, H, N, n, r, kind, T + r, True)
    n64 = {k: _np(t) for k, t in v.items()}
    rows = ids.cpu().numpy()
    plan = m.moe_lora_plan(ids, n)
    for s, bs, db_ in ((None, None, None), (scales, base, dbase)):
        s64 = None if s is None else _np(s)
        ref, rv = orc.lora(**n64, ids=rows, scales=s64, base=None if bs is None else _np(bs))
        got = m.moe_lora(**v, adapter_ids=ids, plan=plan, scales=s, base=bs)
        assert np.array_equal(_np(got["v"]), rv)
        assert torch.equal(got["out"].cpu(), torch.from_numpy(ref).float().to(BF))
        want = orc.lora_backward(_np(dy), n64["x"], rv, n64["a"], n64["b"], rows, s64,
                                 None if db_ is None else _np(db_))
        back = m.moe_lora_backward(dy, v["x"], got["v"], v["a"], v["b"], ids, plan=plan, scales=s,
                                   base=db_)
        assert m.moe_get_error() == 0
        assert np.abs(want["dv"]).max(initial=0) < 2 ** 16       # two bf16 numbers hold it
        assert torch.equal(back["dx"].cpu(), torch.from_numpy(want["dx"]).float().to(BF))
        for key in ("da", "db"):
            assert np.abs(want[key]).max() < 2 ** 24
            assert np.array_equal(_np(back[key]), want[key]), key
        more = {k: torch.full_like(back[k], 2.0) for k in ("da", "db")}
        m.moe_lora_backward(dy, v["x"], got["v"], v["a"], v["b"], ids, scales=s, base=db_, **more,
                            accumulate=True)
        for key in more:
            assert np.array_equal(_np(more[key]), want[key] + 2.0), key


# more units of rows than CTAs, and few enough that a CTA's run goes over two of them: by
# adapters, at their ends and where the rows without one begin
@pytest.mark.parametrize("T,H,N,n,r,kind", [(40000, 16, 136, 3, 4, "mixed"),
                                            (22000, 32, 2056, 20, 8, "mixed"),
                                            (20000, 64, 1032, 5, 100, "mixed"),
                                            (21000, 8, 1544, 300, 5, "runs"),
                                            (30000, 16, 520, 2, 16, "none")])
def test_lora_many_units(T, H, N, n, r, kind):
    v, ids, scales, base, _, _ = _draw(T, H, N, n, r, kind, T + r, True)
    rows = ids.cpu().numpy()
    plan = m.moe_lora_plan(ids, n)
    n64 = {k: _np(t) for k, t in v.items()}
    for bs in (base, None):
        ref, rv = orc.lora(**n64, ids=rows, scales=_np(scales), base=None if bs is None else _np(bs))
        want = torch.from_numpy(ref).float().to(BF)
        out = torch.full((T, N), float("nan"), dtype=BF, device="cuda")
        got = m.moe_lora(**v, adapter_ids=ids, plan=plan, scales=scales, base=bs, out=out)
        assert np.array_equal(_np(got["v"]), rv) and torch.equal(out.cpu(), want)
    held = base.clone()
    m.moe_lora(**v, adapter_ids=ids, plan=plan, scales=scales, base=held, out=held)
    want = orc.lora(**n64, ids=rows, scales=_np(scales), base=_np(base))[0]
    assert torch.equal(held.cpu(), torch.from_numpy(want).float().to(BF))
    assert m.moe_get_error() == 0


# slots of which one or a few are in use, on both sides of where units take the rows
@pytest.mark.parametrize("T,H,N,n,r,used", [(40, 72, 64, 1024, 16, 1), (300, 200, 136, 512, 8, 3),
                                            (1000, 136, 72, 256, 16, 1), (1900, 64, 200, 512, 16, 16),
                                            (900, 264, 72, 1024, 64, 2), (1, 64, 64, 1000, 128, 1)])
def test_lora_slots_that_are_not_in_use(T, H, N, n, r, used):
    v, _, scales, base, _, dy = _draw(T, H, N, n, r, "mixed", T + r, True)
    rng = np.random.default_rng(n)
    rows = rng.choice(rng.choice(n, used, replace=False), T)
    ids = torch.from_numpy(rows.astype(np.int32)).cuda()
    n64, s64 = {k: _np(t) for k, t in v.items()}, _np(scales)
    got = m.moe_lora(**v, adapter_ids=ids, scales=scales, base=base)
    ref, rv = orc.lora(**n64, ids=rows, scales=s64, base=_np(base))
    assert np.array_equal(_np(got["v"]), rv)
    assert torch.equal(got["out"].cpu(), torch.from_numpy(ref).float().to(BF))
    back = m.moe_lora_backward(dy, v["x"], got["v"], v["a"], v["b"], ids, scales=scales)
    want = orc.lora_backward(_np(dy), n64["x"], rv, n64["a"], n64["b"], rows, s64)
    assert torch.equal(back["dx"].cpu(), torch.from_numpy(want["dx"]).float().to(BF))
    for key in ("da", "db"):
        assert np.abs(want[key]).max() < 2 ** 24 and np.array_equal(_np(back[key]), want[key]), key
    assert m.moe_get_error() == 0


@pytest.mark.parametrize("T,H,N,n,r,kind", [(3, 1000, 264, 4, 16, "mixed"),
                                            (100, 512, 328, 6, 24, "mixed"),
                                            (400, 1032, 200, 3, 64, "runs"),
                                            (900, 136, 520, 5, 128, "mixed")])
def test_lora_gaussian(T, H, N, n, r, kind):
    v, ids, scales, base, dbase, dy = _draw(T, H, N, n, r, kind, T, False)
    n64, rows, s64 = {k: _np(t) for k, t in v.items()}, ids.cpu().numpy(), _np(scales)
    size = {k: np.abs(t) for k, t in n64.items()}
    got = m.moe_lora(**v, adapter_ids=ids, scales=scales, base=base)
    ref, rv = orc.lora(**n64, ids=rows, scales=s64, base=_np(base))
    terms, vt = orc.lora(**size, ids=rows, scales=np.abs(s64), base=np.abs(_np(base)))
    assert (np.abs(_np(got["v"]) - rv) <= 2.0 ** -17 * vt).all()
    err = np.abs(_np(got["out"]) - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -15 * terms).all()
    kept = _np(got["v"])
    back = m.moe_lora_backward(dy, v["x"], got["v"], v["a"], v["b"], ids, scales=scales,
                               base=dbase)
    want = orc.lora_backward(_np(dy), n64["x"], kept, n64["a"], n64["b"], rows, s64, _np(dbase))
    t = orc.lora_backward(np.abs(_np(dy)), size["x"], np.abs(kept), size["a"], size["b"], rows,
                          s64, np.abs(_np(dbase)))
    assert (np.abs(_np(back["dx"]) - want["dx"])
            <= 2.0 ** -8 * np.abs(want["dx"]) + 2.0 ** -15 * t["dx"]).all()
    for key in ("da", "db"):
        assert (np.abs(_np(back[key]) - want[key]) <= 2.0 ** -15 * t[key]).all(), key
    assert m.moe_get_error() == 0


def test_lora_scales_that_are_not_finite():
    # an infinite scale makes its own adapter's rows infinite or NaN, and nothing else
    for T, r in ((20, 5), (400, 20)):
        v, ids, scales, base, _, dy = _draw(T, 64, 72, 4, r, "mixed", 3, True)
        want = m.moe_lora(**v, adapter_ids=ids, scales=scales, base=base)
        bad = scales.clone()
        bad[2] = float("inf")
        got = m.moe_lora(**v, adapter_ids=ids, scales=bad, base=base)
        rest = ids != 2
        assert torch.equal(got["out"][rest], want["out"][rest])
        live = (want["out"] != base) & (ids == 2)[:, None]
        assert not torch.isfinite(got["out"][live]).any()
        a = m.moe_lora_backward(dy, v["x"], want["v"], v["a"], v["b"], ids, scales=scales)
        b = m.moe_lora_backward(dy, v["x"], want["v"], v["a"], v["b"], ids, scales=bad)
        keep = [0, 1, 3]
        assert torch.equal(a["dx"][rest], b["dx"][rest])
        assert torch.equal(a["da"][keep], b["da"][keep]) and torch.equal(a["db"][keep], b["db"][keep])


def test_lora_two_streams_at_once():
    runs = []
    for T, r in ((200, 16), (1000, 64)):
        v, ids, scales, base, dbase, dy = _draw(T, 264, 328, 5, r, "mixed", T, False)
        runs.append((v, dict(adapter_ids=ids, scales=scales), base, dy, torch.cuda.Stream()))

    def both(v, how, base, dy, stream):
        f = m.moe_lora(**v, **how, base=base, stream=stream)
        b = m.moe_lora_backward(dy, v["x"], f["v"], v["a"], v["b"], **how, stream=stream)
        return [f["out"], f["v"], b["dx"], b["da"], b["db"]]

    want = [both(*r[:4], None) for r in runs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, r in enumerate(runs):
            got[i].append(both(*r))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(p, q) for p, q in zip(g, want[i]))
    assert m.moe_get_error() == 0


def test_lora_past_two_to_the_31_elements():
    # x of 2.2e9 elements: rows far out, in runs and one by one
    T, H, N, n, r = 270000, 8192, 64, 3, 4
    x = torch.zeros(T, H, dtype=BF, device="cuda")
    x[:, 5] = (torch.arange(T, device="cuda") % 7 - 3).to(BF)
    a = torch.zeros(n, r, H, dtype=BF, device="cuda")
    a[:, 1, 5] = torch.tensor([1.0, 2.0, 3.0], device="cuda").to(BF)
    b = torch.zeros(n, r, N, dtype=BF, device="cuda")
    b[:, 1] = 1.0
    for ids in (torch.arange(T, device="cuda") * n // T, torch.arange(T, device="cuda") % n):
        got = m.moe_lora(x, a, b, ids.to(torch.int32))
        want = x[:, 5].float() * (ids + 1)
        assert torch.equal(got["v"][:, 1], want) and torch.equal(got["out"][:, 63].float(), want)
        dy = torch.zeros(T, N, dtype=BF, device="cuda")
        dy[:, 0] = 1.0
        back = m.moe_lora_backward(dy, x, got["v"], a, b, ids.to(torch.int32))
        assert torch.equal(back["dx"][:, 5].float(), (ids + 1).float())
        sums = torch.zeros(n, device="cuda").index_add_(0, ids, x[:, 5].float())
        assert torch.equal(back["da"][:, 1, 5], sums)
        assert torch.equal(back["db"][:, 1, 0], sums * torch.tensor([1.0, 2.0, 3.0], device="cuda"))
    assert m.moe_get_error() == 0


def test_lora_gradient_against_differences():
    """The slope of the float64 forward along a random direction of each input: exact
    but for the roundings of v (2^-16) and of dx (2^-8, averaged over its elements)."""
    T, H, N, n, r = 150, 64, 72, 3, 8
    v, ids, scales, _, _, dy = _draw(T, H, N, n, r, "mixed", 2, False)
    n64, rows, s64 = {k: _np(t) for k, t in v.items()}, ids.cpu().numpy(), _np(scales)
    f = m.moe_lora(**v, adapter_ids=ids, scales=scales)
    got = m.moe_lora_backward(dy, v["x"], f["v"], v["a"], v["b"], ids, scales=scales)
    rng = np.random.default_rng(1)
    for key, name in (("x", "dx"), ("a", "da"), ("b", "db")):
        u = rng.standard_normal(n64[key].shape)

        def loss(e):
            p = dict(n64, **{key: n64[key] + e * u})
            return float((orc.lora(**p, ids=rows, scales=s64)[0] * _np(dy)).sum())

        slope, size = (loss(1e-5) - loss(-1e-5)) / 2e-5, np.linalg.norm(_np(got[name]))
        assert abs(slope - float((_np(got[name]) * u).sum())) < 2.0 ** -6 * size, name


@pytest.mark.parametrize("T", [20, 300])
def test_lora_bad_ids_and_plans(T):
    v, ids, scales, base, _, dy = _draw(T, 64, 72, 4, 8, "mixed", 3, True)
    want = m.moe_lora(**v, adapter_ids=ids, base=base)["out"]
    bad = ids.clone()
    bad[3], bad[7] = 4, -2
    order, offsets = m.moe_lora_plan(bad, 4)
    assert m.moe_get_error() == 3
    got = m.moe_lora(**v, adapter_ids=bad, plan=(order, offsets), base=base)["out"]
    # those rows have no adapter, the others keep theirs
    assert torch.equal(got[[3, 7]], base[[3, 7]])
    rest = [t for t in range(T) if t not in (3, 7)]
    assert torch.equal(got[rest], want[rest])
    m.moe_get_error()
    if T <= 128:
        return
    # rows and offsets outside the batch are reported and not followed
    order, offsets = m.moe_lora_plan(ids, 4)
    for where, value in ((0, T), (5, -1), (T - 1, 2 ** 31 - 1)):
        o = order.clone()
        o[where] = value
        m.moe_lora(**v, adapter_ids=ids, plan=(o, offsets), base=base)
        assert m.moe_get_error() == 3, (where, value)
    for where, value in ((0, 1), (0, -5), (1, T + 9), (2, -1), (4, T + 1), (3, 2 ** 31 - 1),
                         (1, T), (2, 0)):
        o = offsets.clone()
        o[where] = value
        f = m.moe_lora(**v, adapter_ids=ids, plan=(order, o), base=base)
        assert m.moe_get_error() == 3, (where, value)
        m.moe_lora_backward(dy, v["x"], f["v"], v["a"], v["b"], ids, plan=(order, o))
        assert m.moe_get_error() == 3, (where, value)


def test_lora_few_rows_go_by_their_ids():
    T = 100                                        # the plan is not read: nothing of it counts
    v, ids, scales, base, _, _ = _draw(T, 64, 72, 4, 8, "mixed", 3, True)
    order, offsets = m.moe_lora_plan(ids, 4)
    want = m.moe_lora(**v, adapter_ids=ids, plan=(order, offsets), base=base)
    for where, value in ((0, T), (5, -1), (T - 1, 2 ** 31 - 1)):
        o = order.clone()
        o[where] = value
        f = offsets.clone()
        f[where % 5] = value
        got = m.moe_lora(**v, adapter_ids=ids, plan=(o, f), base=base)
        assert m.moe_get_error() == 0, (where, value)
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["v"], want["v"])


@pytest.mark.parametrize("T", [30, 400])
def test_lora_in_place_apart_and_empty(T):
    v, ids, scales, base, dbase, dy = _draw(T, 136, 200, 5, 16, "mixed", 4, True)
    want = m.moe_lora(**v, adapter_ids=ids, scales=scales, base=base)
    b2 = base.clone()
    assert m.moe_lora(**v, adapter_ids=ids, scales=scales, base=b2, out=b2)["out"] is b2
    assert torch.equal(b2, want["out"])
    back = m.moe_lora_backward(dy, v["x"], want["v"], v["a"], v["b"], ids, base=dbase)
    d2 = dbase.clone()
    m.moe_lora_backward(dy, v["x"], want["v"], v["a"], v["b"], ids, base=d2, dx=d2)
    assert torch.equal(d2, back["dx"])
    # a row's NaN stays in its row, and with its adapter
    x = v["x"].clone()
    x[2] = float("nan")
    got = m.moe_lora(x, v["a"], v["b"], ids, scales=scales, base=base)["out"]
    rest = [t for t in range(T) if t != 2]
    assert torch.equal(got[rest], want["out"][rest])
    ids2 = ids.clone()
    ids2[0], ids2[1] = -1, 3
    a = v["a"].clone()
    a[3] = float("inf")
    got = m.moe_lora(v["x"], a, v["b"], ids2, base=base)["out"]
    assert torch.equal(got[ids2 == -1], base[ids2 == -1])
    assert torch.isfinite(got[ids2 != 3]).all() and not torch.isfinite(got[1]).all()
    # around the outputs nothing is written
    buf = torch.full((T * 200 + 4096,), 7.0, dtype=BF, device="cuda")
    vb = torch.full((T * 16 + 4096,), 7.0, device="cuda")
    m.moe_lora(**v, adapter_ids=ids, scales=scales, base=base,
               out=buf[2048:2048 + T * 200].view(T, 200), v=vb[2048:2048 + T * 16].view(T, 16))
    assert torch.equal(buf[2048:2048 + T * 200].view(T, 200), want["out"])
    for t, k in ((buf, T * 200), (vb, T * 16)):
        assert (t[:2048] == 7).all() and (t[2048 + k:] == 7).all()
    # no rows
    e, i0 = torch.empty(0, 136, dtype=BF, device="cuda"), ids[:0]
    assert m.moe_lora(e, v["a"], v["b"], i0)["out"].shape == (0, 200)
    z = m.moe_lora_backward(torch.empty(0, 200, dtype=BF, device="cuda"), e,
                            torch.empty(0, 16, device="cuda"), v["a"], v["b"], i0)
    assert (z["da"] == 0).all() and (z["db"] == 0).all()
    assert m.moe_get_error() == 0


@pytest.mark.parametrize("T", [30, 400])
def test_lora_on_another_stream_and_in_a_graph(T):
    v, ids, scales, base, dbase, dy = _draw(T, 256, 328, 5, 16, "mixed", 4, False)
    want = m.moe_lora(**v, adapter_ids=ids, scales=scales, base=base)
    back = m.moe_lora_backward(dy, v["x"], want["v"], v["a"], v["b"], ids, scales=scales,
                               base=dbase)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = m.moe_lora(**v, adapter_ids=ids, scales=scales, base=base, stream=s)
    s.synchronize()
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["v"], want["v"])
    live = ids.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan = m.moe_lora_plan(live, 5)
        f = m.moe_lora(**v, adapter_ids=live, plan=plan, scales=scales, base=base)
        b = m.moe_lora_backward(dy, v["x"], f["v"], v["a"], v["b"], live, plan=plan,
                                scales=scales, base=dbase)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for key in want:
        assert torch.equal(f[key], want[key]), key
    for key in back:
        assert torch.equal(b[key], back[key]), key
    live.copy_(ids.flip(0))                        # other adapters at the replay
    g.replay()
    again = m.moe_lora(**v, adapter_ids=live, scales=scales, base=base)
    assert torch.equal(f["out"], again["out"])
    assert m.moe_get_error() == 0


@pytest.mark.parametrize("T,H,N,n,r", [(20, 64, 72, 3, 16), (200, 264, 280, 3, 32),
                                       (150, 200, 192, 70, 13), (300, 328, 392, 2, 64),
                                       (300, 328, 392, 2, 128)])
def test_lora_gradients_hold_24_bits(T, H, N, n, r):
    """v and dv of 24 bits, each alone in its sum, come through as they are; two bf16 numbers
    would hold less than 18 of them. dv = B dy has three terms, digits below 2^7 times 2^16,
    2^8 and 1; further columns of dy, and those of x, are one a row, so that da[:, t] = dv_t
    and db[:, 8 + t] = v_t for adapter ids[t]."""
    rng = np.random.default_rng(T + r)
    ids, t = rng.integers(0, n, T), np.arange(T)
    x, dy = np.zeros((T, H)), np.zeros((T, N))
    x[t, t], dy[t, 8 + t] = 1.0, 1.0
    dy[:, :3] = rng.integers(-127, 128, (T, 3)) * 2.0 ** np.array([16, 8, 0])
    a, b = np.zeros((n, r, H)), np.zeros((n, r, N))
    b[:, :, :3] = rng.choice([-1.0, 1.0], (n, r, 3))
    dv = np.einsum("tc,tjc->tj", dy[:, :3], b[ids][:, :, :3])
    assert np.abs(dv).max() < 2 ** 23 and (np.abs(dv) % 2 == 1).any()
    v = torch.from_numpy(rng.standard_normal((T, r)).astype(np.float32)).cuda()
    scales = torch.tensor(rng.choice([0.5, 1.0, -2.0], n).astype(np.float32)).cuda()

    def put(q):
        p = torch.from_numpy(q.astype(np.float32)).to(BF).cuda()
        assert np.array_equal(_np(p), q)
        return p

    got = m.moe_lora_backward(put(dy), put(x), v, put(a), put(b),
                              torch.from_numpy(ids.astype(np.int32)).cuda(), scales=scales)
    assert m.moe_get_error() == 0
    s = _np(scales)[ids][:, None]
    da, db = np.zeros((n, r, H)), np.zeros((n, r, N))
    da[ids[t], :, t] = (s * dv)[t]
    db[ids[t], :, 8 + t] = (s * _np(v))[t]
    assert np.array_equal(_np(got["da"]), da)
    assert np.array_equal(_np(got["db"])[:, :, 8:], db[:, :, 8:])


# One accumulator over the whole of these sums, 1024 additions of positive numbers, ends
# 2^-13.5 too small, all of it in the mean. A run of 128 terms is 8 additions of 16 products
# to what is there, each of which may cut off 17 numbers below 2^-23 of the partial sum, on
# the average half of the last one: 8 * 17 / 2 * 2^-23 < 2^-16.9. The 160 runs at most are
# added up in float, 2^-24 of sums that are half of the last one on the average: 2^-17.6.
# What is cut off is half of that in the mean. Together 2^-16.2, in the mean 2^-16.8.
SUM, MEAN = 2.0 ** -16.2, 2.0 ** -16.8


def _holds(got, ref, limit, mean, what):
    err = got.double() - ref
    assert (err.abs() <= limit * ref).all(), (what, float((err.abs() / ref).max()))
    assert err.sum().abs() <= mean * ref.sum(), (what, float(err.sum() / ref.sum()))


def _positive(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(sum(shape) + seed)
    return torch.randn(shape, generator=g, device="cuda").abs().to(BF)


@pytest.mark.parametrize("T,H,r", [(300, 16384, 16), (300, 16392, 30), (200, 16384, 64),
                                   (400, 16384, 128)])
def test_lora_long_sums_of_v(T, H, r):
    x, a, b = _positive(T, H), _positive(2, r, H), _positive(2, r, 64)
    ids = (torch.arange(T, device="cuda") % 2).to(torch.int32)
    got = m.moe_lora(x, a, b, ids)
    assert m.moe_get_error() == 0
    for i in range(2):
        _holds(got["v"][ids == i], x[ids == i].double() @ a[i].double().t(), SUM, MEAN, "v")


@pytest.mark.parametrize("T,H,N,r", [(16384, 64, 72, 16), (20000, 72, 264, 32),
                                     (16400, 136, 64, 50), (16384, 64, 64, 128)])
def test_lora_long_sums_of_gradients(T, H, N, r):
    # runs of rows and single rows; dv = B dy is itself such a sum, of at most 264 terms
    x, a, dy, b = _positive(T, H), _positive(1, r, H), _positive(T, N), _positive(1, r, N)
    v = torch.rand(T, r, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda")
    some = torch.zeros(T, dtype=torch.int32, device="cuda")
    some[::9] = -1
    for ids in (torch.zeros_like(some), some):
        got = m.moe_lora_backward(dy, x, v, a, b, ids)
        assert m.moe_get_error() == 0
        on = ids == 0
        X, D, V = x[on].double(), dy[on].double(), v[on].double()
        _holds(got["db"][0], V.t() @ D, SUM, MEAN, "db")
        _holds(got["da"][0], (D @ b[0].double().t()).t() @ X, 2 * SUM, 2 * MEAN, "da")


def test_lora_refusals():
    v, ids, scales, base, _, dy = _draw(10, 64, 72, 4, 8, "mixed", 3, True)
    with pytest.raises(ValueError, match="adapter_ids"):
        m.moe_lora(**v, adapter_ids=ids[:5])
    with pytest.raises(ValueError, match="adapter_ids"):
        m.moe_lora(**v, adapter_ids=ids.long())
    with pytest.raises(ValueError, match="offsets"):
        m.moe_lora(**v, adapter_ids=ids, plan=(ids, ids))
    with pytest.raises(ValueError, match="a and b must"):
        m.moe_lora(v["x"][:, :56].contiguous(), v["a"], v["b"], ids)
    with pytest.raises(ValueError, match="scales"):
        m.moe_lora(**v, adapter_ids=ids, scales=scales[:2])
    with pytest.raises(ValueError, match="base"):
        m.moe_lora(**v, adapter_ids=ids, base=base[:, :64].contiguous())
    with pytest.raises(m.MoeError, match="unsupported"):
        m.moe_lora(v["x"], torch.zeros(1, 200, 64, dtype=BF, device="cuda"),
                   torch.zeros(1, 200, 72, dtype=BF, device="cuda"), torch.zeros_like(ids))
    with pytest.raises(m.MoeError, match="unsupported"):
        m.moe_lora(v["x"], v["a"], v["b"][:, :, :70].contiguous(), ids)
    f = m.moe_lora(**v, adapter_ids=ids)
    with pytest.raises(ValueError, match="accumulate"):
        m.moe_lora_backward(dy, v["x"], f["v"], v["a"], v["b"], ids, accumulate=True)
    with pytest.raises(ValueError, match="v must"):
        m.moe_lora_backward(dy, v["x"], f["v"][:, :4].contiguous(), v["a"], v["b"], ids)
    assert m.moe_get_error() == 0
