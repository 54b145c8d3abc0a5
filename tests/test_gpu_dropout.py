"""Dropout of the branch on the GPU: the mask bit for bit against the oracle's
generator on plain integers, and the values within their rounding: out is one
fused multiply-add of float beside the product a x, 2 * 2^-24 of the terms, and
then half a step of its type."""
import numpy as np
import pytest
import torch

import oracle as orc

pytestmark = pytest.mark.gpu
m = pytest.importorskip("moe_expert_dispatch_gb300")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _np(t):
    return t.detach().double().cpu().numpy()


def _rng(seed, draw):
    return torch.tensor([seed, draw], dtype=torch.int64, device="cuda")


def _close(got, ref, terms, what):
    half = torch.finfo(got.dtype).eps / 2
    assert (np.abs(_np(got) - ref) <= half * np.abs(ref) + 2.0 ** -22 * terms).all(), what


@pytest.mark.parametrize("numel", [1, 7, 8, 9, 1000, 4099, 70001])
@pytest.mark.parametrize("stream,branch", [("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32"),
                                           ("bf16", "f32")])
@pytest.mark.parametrize("residual", [True, False])
def test_dropout_against_the_definition(numel, stream, branch, residual):
    p, a, b, seed, draw = 0.3, 0.5, 1.25, 0x1234567_89ABCDEF, (5 << 32) + numel
    g = torch.Generator().manual_seed(numel)
    y = torch.randn(numel, generator=g).to(DT[branch]).cuda()
    x = torch.randn(numel, generator=g).to(DT[stream]).cuda() if residual else None
    kept = orc.dropout_kept(numel, seed, draw, p)
    out = torch.empty(numel, dtype=DT[stream], device="cuda")
    got = m.moe_dropout_residual(y, _rng(seed, draw), p, x=x, residual_scale=a, branch_scale=b,
                                 out=out)
    assert got is out
    ref = orc.dropout_residual(_np(y), kept, p, None if x is None else _np(x), a, b)
    _close(out, ref, 2 * np.abs(_np(y)) + (0 if x is None else np.abs(_np(x))), "out")
    if not residual:
        assert np.array_equal(_np(out) != 0, kept & (_np(y) != 0))
    back = m.moe_dropout_residual_backward(out, _rng(seed, draw), p, residual=residual,
                                           residual_scale=a, branch_scale=b,
                                           branch_dtype=DT[branch])
    d = _np(out)
    _close(back["dy"], orc.dropout_residual(d, kept, p, b=b), 2 * np.abs(d), "dy")
    assert back["dy"].dtype == DT[branch]
    if residual:
        _close(back["dx"], a * d, np.abs(d), "dx")
    else:
        assert back["dx"] is None


@pytest.mark.parametrize("numel", [1, 8, 30, 5000])
@pytest.mark.parametrize("first", [1, 3, 8])
def test_dropout_views_at_any_element(numel, first):
    # the same elements are dropped wherever the tensors start, and nothing beside them
    # is written
    y = torch.randn(numel + 16, device="cuda").bfloat16()
    x = torch.randn(numel + 16, device="cuda")
    rng = _rng(3, 4)
    want = m.moe_dropout_residual(y[first:first + numel].clone(), rng, 0.5,
                                  x=x[first:first + numel].clone())
    out = torch.full((numel + 16,), 7.0, device="cuda")
    m.moe_dropout_residual(y[first:first + numel], rng, 0.5, x=x[first:first + numel],
                           out=out[first:first + numel])
    assert torch.equal(out[first:first + numel], want)
    assert (out[:first] == 7).all() and (out[first + numel:] == 7).all()


def test_dropout_ends_of_p():
    y = torch.randn(4096, device="cuda")
    assert torch.equal(m.moe_dropout_residual(y, _rng(1, 1), 0.0), y)
    # 0.99999 is taken to 65535 / 65536: hardly one of them stays, 65536 times as large
    out = m.moe_dropout_residual(y, _rng(1, 1), 0.99999)
    kept = torch.from_numpy(orc.dropout_kept(4096, 1, 1, 0.99999)).cuda()
    assert torch.equal(out, torch.where(kept, y * 65536.0, torch.zeros_like(y)))


def test_dropout_drops_what_is_not_finite():
    y = torch.full((800,), float("nan"), device="cuda")
    y[1::2] = float("inf")
    x = torch.ones(800, device="cuda")
    kept = torch.from_numpy(orc.dropout_kept(800, 9, 9, 0.5)).cuda()
    out = m.moe_dropout_residual(y, _rng(9, 9), 0.5, x=x)
    assert (out[~kept] == 1).all() and not out[kept].isfinite().any()
    d = m.moe_dropout_residual_backward(y, _rng(9, 9), 0.5, residual=False,
                                        branch_dtype=torch.float32)
    assert (d["dy"][~kept] == 0).all()


def test_dropout_in_place_shapes_and_nothing():
    y = torch.randn(3, 5, 7, device="cuda").bfloat16()
    x = torch.randn(3, 5, 7, device="cuda").bfloat16()
    rng = _rng(2, 2)
    want = m.moe_dropout_residual(y, rng, 0.2, x=x)
    assert want.shape == x.shape
    assert m.moe_dropout_residual(y, rng, 0.2, x=x, out=x) is x and torch.equal(x, want)
    alone = m.moe_dropout_residual(y, rng, 0.2)
    assert alone.dtype == torch.bfloat16
    m.moe_dropout_residual(y, rng, 0.2, out=y)
    assert torch.equal(y, alone)
    d = torch.randn(105, device="cuda")
    back = m.moe_dropout_residual_backward(d, rng, 0.2, residual_scale=0.5)
    d2 = d.clone()
    again = m.moe_dropout_residual_backward(d2, rng, 0.2, residual_scale=0.5, dx=d2)
    assert torch.equal(again["dy"], back["dy"]) and torch.equal(d2, back["dx"])
    e = torch.empty(0, 8, device="cuda")
    assert m.moe_dropout_residual(e, rng, 0.2).shape == (0, 8)


def test_dropout_far_elements():
    # elements past 2^32: the counter's second word, and 64-bit offsets
    n = (1 << 32) + 4096 + 3
    rng = _rng(77, 5)
    y = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    out = m.moe_dropout_residual(y, rng, 0.5, out=y)
    tail = out[n - 1003:].float().cpu().numpy()
    first = n - 1003
    lo = 0xFFFFFFFF
    kept = []
    for block in range(first // 8, (n + 7) // 8):
        for w in orc.philox4x32([block & lo, block >> 32, 5, 0], [77, 0]):
            kept += [(w & 0xFFFF) >= 32768, (w >> 16) >= 32768]
    kept = np.array(kept)[first - first // 8 * 8:][:1003]
    assert np.array_equal(tail, np.where(kept, 2.0, 0.0))


def test_dropout_replays_take_the_draw_of_their_time():
    y = torch.randn(6000, device="cuda").bfloat16()
    rng = _rng(123, 0)
    m.moe_dropout_residual(y, rng, 0.5)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = m.moe_dropout_residual(y, rng, 0.5)
        back = m.moe_dropout_residual_backward(y, rng, 0.5, residual=False)["dy"]
        rng[1] += 1
    seen = []
    for draw in range(3):
        g.replay()
        torch.cuda.synchronize()
        want = m.moe_dropout_residual(y, _rng(123, draw), 0.5)
        assert torch.equal(out, want) and torch.equal(back, want), draw
        seen.append(out.clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = m.moe_dropout_residual(y, _rng(123, 2), 0.5, stream=s)
    s.synchronize()
    assert torch.equal(other, seen[2])


def test_dropout_refusals():
    y, rng = torch.zeros(16, device="cuda"), _rng(1, 1)
    for p in (-0.1, 1.0, float("nan")):
        with pytest.raises(m.MoeError, match="invalid"):
            m.moe_dropout_residual(y, rng, p)
    with pytest.raises(ValueError, match="rng"):
        m.moe_dropout_residual(y, rng.int(), 0.1)
    with pytest.raises(ValueError, match="rng"):
        m.moe_dropout_residual(y, rng[:1], 0.1)
    with pytest.raises(ValueError, match="x must"):
        m.moe_dropout_residual(y, rng, 0.1, x=y.bfloat16(), out=y)
    with pytest.raises(ValueError, match="x must"):
        m.moe_dropout_residual(y, rng, 0.1, x=y[:8])
    with pytest.raises(ValueError, match="contiguous"):
        m.moe_dropout_residual(torch.zeros(4, 4, device="cuda").t(), rng, 0.1)
    with pytest.raises(ValueError, match="float32 or torch.bfloat16"):
        m.moe_dropout_residual(y.half(), rng, 0.1)
