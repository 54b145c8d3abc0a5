"""GPU parity of the clip of many gradients by one norm against float64.

Tolerances, in half steps of float32 (H = 2^-24 relative): squares are summed
in float over runs of at most 128 terms (128 H of the sum, half of that in its
root) and as pairs of floats, which lose next to nothing, beyond; norm and coef are rounded once (H each), a scaled
gradient once more, and bfloat16 results by half a step, 2^-8."""
import math

import numpy as np
import pytest
import torch

import oracle as orc

pytestmark = pytest.mark.gpu
m = pytest.importorskip("moe_expert_dispatch_gb300")

H32, BF = 2.0 ** -24, 2.0 ** -8
NORM = 65 * H32


def _grads(sizes, dtype=torch.float32, seed=0, sd=0.1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * sd).to(dtype) for n in sizes]


def _close(grads, norm, coef, outs, max_norm, kind=2.0, eps=1e-6):
    rn, rc, ro = orc.clip_grad_norm([g.double().cpu().numpy() for g in grads], max_norm,
                                    norm_type=kind, eps=eps)
    tol = H32 if kind == math.inf else NORM
    assert norm.shape == (1,) and norm.dtype == torch.float32
    assert abs(norm.item() - rn) <= tol * rn + 1e-37
    assert abs(coef.item() - rc) <= (tol + 3 * H32) * rc
    for g, o, r in zip(grads, outs, ro):
        err = np.abs(o.double().cpu().numpy() - r)
        b = (tol + 5 * H32 + (BF if o.dtype == torch.bfloat16 else 0.0)) * np.abs(r)
        assert np.all(err <= b + 1e-37)


SIZES = [[1], [7], [5, 0, 3], [1000], [16384, 16385, 1], [100000, 33, 4096], [1 << 20, 12345],
         [17] * 300]


@pytest.mark.parametrize("sizes", SIZES, ids=[str(i) for i in range(len(SIZES))])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", [2.0, math.inf])
def test_clip_against_the_definition(sizes, dtype, kind):
    for max_norm in (0.01, 1e9, 0.0):
        grads = _grads(sizes, dtype)
        keep = [g.clone() for g in grads]
        outs = [torch.full_like(g, 7.0) for g in grads]
        norm, coef = m.moe_clip_grad_norm(grads, max_norm, out=outs, norm_type=kind)
        assert all(torch.equal(a, b) for a, b in zip(grads, keep))
        _close(keep, norm, coef, outs, max_norm, kind)
        n2, c2 = m.moe_clip_grad_norm(grads, max_norm, norm_type=kind)
        assert torch.equal(norm, n2) and torch.equal(coef, c2)
        assert all(torch.equal(a, b) for a, b in zip(grads, outs))
        if max_norm == 1e9:
            assert coef.item() == 1.0 and all(torch.equal(a, b) for a, b in zip(grads, keep))


def test_clip_mixed_types_and_many_tensors():
    rng = np.random.default_rng(3)
    sizes = np.exp(rng.uniform(0, 9, 2500)).astype(int).tolist()
    f, b = _grads(sizes[::2]), _grads(sizes[1::2], torch.bfloat16, seed=1)
    grads = [t for pair in zip(f, b) for t in pair]
    outs = [torch.empty_like(g) for g in grads]
    norm, coef = m.moe_clip_grad_norm(grads, 1.0, out=outs)
    _close(grads, norm, coef, outs, 1.0)
    again = m.moe_clip_grad_norm(grads, 1.0, out=[torch.empty_like(g) for g in grads])
    assert torch.equal(norm, again[0]) and torch.equal(m.moe_grad_norm(grads), norm)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_clip_views_at_any_element(dtype):
    # parameters packed into one bucket start at any element, alike or not on the two sides
    flat = _grads([200007], dtype)[0]
    out = torch.full((200020,), 7.0, dtype=dtype, device="cuda")
    at, grads, outs, shift = 0, [], [], 0
    for i, n in enumerate((1, 2, 5, 129, 4097, 16384, 33333, 77, 100000)):
        shift += i % 3 == 2
        grads.append(flat[at:at + n])
        outs.append(out[at + shift:at + shift + n])
        at += n
    norm, coef = m.moe_clip_grad_norm(grads, 0.5, out=outs)
    _close(grads, norm, coef, outs, 0.5)
    covered = torch.zeros_like(out, dtype=torch.bool)
    for o in outs:
        covered[o.storage_offset():o.storage_offset() + o.numel()] = True
    assert torch.all(out[~covered] == 7.0)
    keep = flat.clone()
    m.moe_clip_grad_norm(grads, 0.5)
    assert all(torch.equal(g, o) for g, o in zip(grads, outs))
    assert torch.equal(flat[at:], keep[at:])


@pytest.mark.parametrize("kind", [2.0, math.inf])
def test_clip_infinities_and_nan(kind):
    for bad in (math.inf, -math.inf, math.nan):
        grads = _grads([3000, 77])
        grads[1][5] = bad
        outs = [torch.empty_like(g) for g in grads]
        norm, coef = m.moe_clip_grad_norm(grads, 1.0, out=outs, norm_type=kind)
        if math.isnan(bad):
            assert math.isnan(norm.item()) and math.isnan(coef.item())
            assert all(torch.isnan(o).all() for o in outs)
        else:
            assert norm.item() == math.inf and coef.item() == 0.0
            assert torch.all(outs[0] == 0) and torch.isnan(outs[1][5])


def test_clip_zero_and_nothing():
    grads = [torch.zeros(100, device="cuda"), torch.zeros(0, device="cuda")]
    norm, coef = m.moe_clip_grad_norm(grads, 1.0)
    assert norm.item() == 0.0 and coef.item() == 1.0
    nc = torch.full((2,), 5.0, device="cuda")
    norm, coef = m.moe_clip_grad_norm([], 1e-9, norm_coef=nc)
    assert norm.item() == 0.0 and abs(coef.item() - 1e-3) < 1e-9
    assert m.moe_grad_norm(grads[1:]).item() == 0.0


def test_clip_long_sums_keep_their_digits():
    # 50 million equal squares: a float sum would stop growing
    n = 50_000_011
    g = torch.full((n,), 0.5, device="cuda")
    norm, coef = m.moe_clip_grad_norm([g], 1.0)
    assert abs(norm.item() - 0.5 * math.sqrt(n)) <= NORM * 0.5 * math.sqrt(n)
    assert torch.all(g == g[0])
    big = torch.full((1000,), 1e17, device="cuda")
    assert abs(m.moe_grad_norm([big]).item() / (1e17 * math.sqrt(1000)) - 1) <= NORM
    small = torch.full((1000,), 1e-17, device="cuda")
    assert abs(m.moe_grad_norm([small]).item() / (1e-17 * math.sqrt(1000)) - 1) <= NORM


def test_clip_past_two_to_the_31_elements():
    n = (1 << 31) + 1027
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[0], g[-1], g[1 << 31] = 3.0, 4.0, 12.0
    norm, coef = m.moe_clip_grad_norm([g], 6.5, eps=0.0)
    assert norm.item() == 13.0 and coef.item() == 0.5
    assert g[0].item() == 1.5 and g[-1].item() == 2.0 and g[1 << 31].item() == 6.0


def test_clip_on_another_stream_and_in_a_graph():
    grads = _grads([5000, 300000, 3])
    outs = [torch.empty_like(g) for g in grads]
    want = [torch.empty_like(g) for g in grads]
    norm, coef = m.moe_clip_grad_norm(grads, 1.0, out=want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n2, c2 = m.moe_clip_grad_norm(grads, 1.0, out=outs, stream=side)
    side.synchronize()
    assert torch.equal(norm, n2) and all(torch.equal(a, b) for a, b in zip(outs, want))
    nc = torch.empty(2, device="cuda")
    ws = torch.empty(m._lib.moe_clip_grad_norm_workspace_size(), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_clip_grad_norm(grads, 1.0, out=outs, norm_coef=nc, workspace=ws)
    for scale in (1.0, 0.001, 3.0):
        src = [g.clone() for g in grads]
        for g in grads:
            g.mul_(scale)
        graph.replay()
        torch.cuda.synchronize()
        _close(grads, nc[0:1], nc[1:2], outs, 1.0)
        for g, s in zip(grads, src):
            g.copy_(s)


def test_clip_refusals():
    g = torch.zeros(8, device="cuda")
    with pytest.raises(ValueError, match=r"grads\[1\]"):
        m.moe_clip_grad_norm([g, g.half()], 1.0)
    with pytest.raises(ValueError, match=r"out\[0\]"):
        m.moe_clip_grad_norm([g], 1.0, out=[g[:4]])
    with pytest.raises(ValueError, match="holds 0"):
        m.moe_clip_grad_norm([g], 1.0, out=[])
    with pytest.raises(m.MoeError) as e:
        m.moe_clip_grad_norm([g], 1.0, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4
    with pytest.raises(m.MoeError) as e:
        m.moe_clip_grad_norm([g], 1.0, eps=-1.0)
    assert e.value.status == 1


# A thread's share of an item: four chains of nine squares at most, added up by two more
# additions, and to twice float's precision from there: 11 half steps of the sum and one to
# round it, half of that in the root, and the root's own.
ROOT = 7 * H32


@pytest.mark.parametrize("sizes", [[1000], [65536], [1 << 20, 12345], [50_000_011]])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_clip_norm_within_the_roundings_of_a_share(sizes, dtype):
    grads = _grads(sizes, dtype)
    want = math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))
    assert abs(m.moe_grad_norm(grads).item() - want) <= ROOT * want


@pytest.mark.parametrize("n", [4096, 8192, 65536, 131072, 60_000_011])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_clip_counts_the_ends_of_its_range_in_full(n, dtype):
    # one item, one cluster's items, two launches; every element as large or as small as stated
    for size in (1e18, 1e-18):
        g = torch.full((n,), size, dtype=dtype, device="cuda")
        value = g[0].double().item()
        out = torch.empty_like(g)
        norm, coef = m.moe_clip_grad_norm([g], value, out=[out], eps=0.0)
        assert abs(norm.item() / (value * math.sqrt(n)) - 1) <= ROOT
        assert abs(coef.item() * math.sqrt(n) - 1) <= ROOT + H32
        half = BF if dtype == torch.bfloat16 else 0.0
        ends = out[[0, n // 2, n - 1]].double() * (math.sqrt(n) / value)
        assert torch.all((ends - 1).abs() <= ROOT + 2 * H32 + half)
        assert torch.all(out == out[0])


def test_clip_mixes_small_gradients_with_the_largest():
    # the sum leaves float's range and comes back to what is small beside it
    n = 40_000_000
    large = torch.full((n,), 1e18, device="cuda")
    usual = _grads([100_000], seed=5)[0] * 1e15
    want = math.sqrt(n * large[0].double().item() ** 2 + float(usual.double().square().sum()))
    for grads in ([large, usual], [usual, large], [usual[:1000], large, usual[1000:]]):
        assert abs(m.moe_grad_norm(grads).item() - want) <= ROOT * want


@pytest.mark.parametrize("n", [8192, 60_000_011])
def test_clip_infinities_and_nan_among_the_largest(n):
    for at in (0, n // 2, n - 1):
        g = torch.full((n,), 1e18, device="cuda")
        g[at] = math.inf
        norm, coef = m.moe_clip_grad_norm([g], 1.0, out=[torch.empty_like(g)])
        assert norm.item() == math.inf and coef.item() == 0.0
        g[n // 3] = math.nan
        norm, coef = m.moe_clip_grad_norm([g], 1.0, out=[torch.empty_like(g)])
        assert math.isnan(norm.item()) and math.isnan(coef.item())
