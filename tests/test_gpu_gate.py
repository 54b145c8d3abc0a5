"""GPU parity of the balanced gate and its gradient against the float64
oracle. Expert ids, counts and offsets are exact.

Tolerances, in half steps of float32 (H = 2^-24 relative). A score takes an
exp (2 ulp = 4 H), the rounding of its argument (H times the argument's size,
at most the row's spread R), an addition and a division (3 H); a sum of n
non-negative terms adds at most n H; renormalising divides once more and the
scale multiplies (3 H). Together at most (20 + 2 R + k + E / 32 + 8) H, with
the sum over E taken by 32 lanes. The gradient multiplies such factors; its
difference dprobs - d is off by that share of |dprobs_j| + sum |dprobs u|.
bfloat16 results add half a step, 2^-8."""
import math

import numpy as np
import pytest
import torch

import oracle as orc
from gpu_util import dev

pytestmark = pytest.mark.gpu
m = pytest.importorskip("moe_expert_dispatch_gb300")

H32, TINY = 2.0 ** -24, 1e-36


def _units(logits, k):
    lg = logits.double().numpy()
    fin = np.where(np.isfinite(lg), lg, 0.0)
    spread = np.abs(fin).max(initial=0.0) * 2
    return (20 + 2 * spread + k + lg.shape[1] / 32 + 8) * H32


def _check(logits, k, bias=None, backward=True, **how):
    """Forward and backward of one gate on CPU logits [T, E]."""
    T, E = logits.shape
    lg = logits.float().numpy()
    b = None if bias is None else bias.numpy()
    rid, rw, rc, ro = orc.route_gate(lg, k, bias=b, **how)
    ids, w, counts, offsets = m.moe_route_gate(dev(logits), k, bias=dev(bias), **how)
    assert m.moe_get_error() == 0
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert np.array_equal(counts.cpu().numpy(), rc)
    assert np.array_equal(offsets.cpu().numpy(), ro)
    tol = _units(logits, k)
    err = np.abs(w.cpu().numpy().astype(np.float64) - rw)
    assert np.all(err <= tol * np.abs(rw) + TINY), float((err - tol * np.abs(rw)).max())
    if not backward:
        return
    kw = {key: how[key] for key in ("score", "renormalise", "scale") if key in how}
    dp = torch.randn((T, k), generator=torch.Generator().manual_seed(T + E))
    ref = orc.route_gate_backward(dp.numpy(), lg, rid, bias=b, **kw)
    got = m.moe_route_gate_backward(dev(dp), dev(logits), ids, bias=dev(bias), **kw)
    assert m.moe_get_error() == 0 and got.dtype == logits.dtype
    # |gradient| before its cancellation: the same sums with every sign positive
    a = np.abs(dp.numpy().astype(np.float64)).sum(axis=1, keepdims=True)
    size = np.zeros((T, E))
    s = abs(kw.get("scale", 1.0)) * np.abs(rw / (kw.get("scale", 1.0) or 1.0))
    np.put_along_axis(size, rid.astype(np.int64), s * 2 * a, 1)
    if kw.get("score", "softmax") == "softmax" and not kw.get("renormalise", True):
        clean = np.where(np.isnan(lg), -np.inf, np.minimum(lg, orc.F32_MAX)).astype(np.float64)
        top = np.max(clean, axis=1, keepdims=True)
        ex = np.exp(clean - np.where(np.isinf(top), 0.0, top))
        size += abs(kw.get("scale", 1.0)) * ex / np.maximum(ex.sum(axis=1, keepdims=True), TINY) * a
    bound = 2 * tol * size + TINY
    if logits.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * np.abs(ref)
    err = np.abs(got.float().cpu().numpy() - ref)
    assert np.all(err <= bound), float((err - bound).max())


def _logits(T, E, dtype=torch.float32, sd=1.5, seed=0):
    g = torch.Generator().manual_seed(seed * 7919 + T * 131 + E)
    return (torch.randn((T, E), generator=g) * sd).to(dtype)


def _bias(E, sd=0.1):
    return torch.randn(E, generator=torch.Generator().manual_seed(E)) * sd


SHAPES = [
    (1, 1, 1, 1, 1, 1), (5, 8, 2, 1, 1, 1), (67, 8, 8, 4, 4, 2), (33, 24, 3, 8, 2, 1),
    (129, 60, 4, 12, 5, 2), (64, 64, 6, 8, 3, 2), (31, 72, 8, 1, 1, 1), (200, 128, 8, 8, 4, 2),
    (77, 256, 8, 8, 4, 2), (9, 160, 6, 32, 8, 1), (3, 384, 32, 3, 2, 2), (17, 1024, 32, 32, 9, 2),
    (41, 33, 5, 11, 4, 2), (300, 7, 3, 1, 1, 1),
]


@pytest.mark.parametrize("T,E,k,n_group,topk_group,group_topk", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_gate_against_the_definition(T, E, k, n_group, topk_group, group_topk, score, biased):
    for renormalise, dtype, scale in ((True, torch.float32, 1.0), (False, torch.bfloat16, 2.5)):
        _check(_logits(T, E, dtype), k, bias=_bias(E) if biased else None, score=score,
               n_group=n_group, topk_group=topk_group, group_topk=group_topk,
               renormalise=renormalise, scale=scale)


@pytest.mark.parametrize("E,k,n_group,topk_group", [(7, 3, 1, 1), (40, 8, 4, 2), (128, 16, 8, 4),
                                                    (256, 5, 1, 1), (64, 6, 32, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_ties_masks_infinities_and_nan(E, k, n_group, topk_group, score):
    rng = np.random.default_rng(E)
    pool = np.array([-0.0, 0.0, 1.0, -1.0, 2.5, -np.inf, np.nan, np.inf, 0.5, -60.0], np.float32)
    some = torch.from_numpy(pool[rng.integers(0, pool.size, (200, E))])
    few = torch.full((40, E), -math.inf)                      # fewer open experts than k
    few[torch.arange(40), torch.from_numpy(rng.integers(0, E, 40))] = 0.25
    none = torch.full((8, E), -math.inf)
    same = torch.full((30, E), 0.75)
    logits = torch.cat([some, few, none, same])
    bias = torch.from_numpy(np.array([0.0, 0.25, -np.inf, np.nan, -0.5, np.inf],
                                     np.float32)[rng.integers(0, 6, E)])
    for b in (None, bias, torch.full((E,), -math.inf)):
        for renormalise in (True, False):
            _check(logits, k, bias=b, score=score, n_group=n_group, topk_group=topk_group,
                   group_topk=2 if E // n_group > 1 else 1, renormalise=renormalise)


def test_gate_values_that_float_cannot_tell_apart():
    # choice values s + b one part in 1e10 apart: the order is the double one
    E, k = 48, 8
    rng = np.random.default_rng(11)
    logits = torch.from_numpy(rng.standard_normal((400, E)).astype(np.float32))
    s = 1.0 / (1.0 + np.exp(-logits[:1].double().numpy()))
    level = torch.from_numpy((0.9 - s[0]).astype(np.float32))  # makes row 0's values nearly equal
    logits[1:200] = logits[0] + torch.from_numpy(
        (rng.integers(-1, 2, (199, E)) * 2.0 ** -22).astype(np.float32))
    for score in ("sigmoid", "softmax"):
        _check(logits, k, bias=level, score=score)
        _check(logits, k, bias=level, score=score, n_group=8, topk_group=3, group_topk=2)


def test_gate_extreme_scores_renormalise():
    # chosen scores far below float's range still have weights that sum to one
    logits = torch.full((6, 16), -20.0)
    logits[0, :] = torch.arange(16) * 0.25 - 120.0
    logits[1, :] = torch.arange(16) * 4.0 - 300.0
    logits[2, :] = 90.0
    logits[3, :8] = 500.0
    bias = torch.zeros(16)
    bias[:3] = 5.0                                            # forces poor experts in
    for score in ("sigmoid", "softmax"):
        for b in (None, bias):
            _check(logits, 3, bias=b, score=score, scale=1.0, backward=False)


def test_gate_defaults_equal_the_plain_gate():
    logits = dev(_logits(1000, 64))
    a, b = m.moe_route_gate(logits, 6), m.moe_route_topk(logits, 6)
    for i in (0, 2, 3):
        assert torch.equal(a[i], b[i])
    torch.testing.assert_close(a[1], b[1], rtol=40 * H32, atol=0)


def test_gate_many_tokens_and_repeats():
    logits, bias = dev(_logits(70001, 64, sd=1.0)), dev(_bias(64))
    how = dict(bias=bias, score="sigmoid", n_group=8, topk_group=4, group_topk=2, scale=2.5)
    a = m.moe_route_gate(logits, 6, **how)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda").random_()
    b = m.moe_route_gate(logits, 6, workspace=ws, **how)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    ids = a[0].cpu().numpy()
    assert np.array_equal(a[2].cpu().numpy(), np.bincount(ids.reshape(-1), minlength=64))
    assert np.array_equal(a[3].cpu().numpy()[1:], a[2].cpu().numpy().cumsum())
    s = torch.sigmoid(logits.double())
    v = (s + bias.double()).view(-1, 8, 8)
    keep = v.topk(2, dim=2).values.sum(2).topk(4, dim=1).indices
    mask = torch.zeros(v.shape[:2], dtype=torch.bool, device="cuda").scatter_(1, keep, True)
    want = v.masked_fill(~mask[:, :, None], -math.inf).view(-1, 64).topk(6, dim=1).indices
    assert torch.equal(a[0].long(), want)
    w = s.gather(1, want)
    torch.testing.assert_close(a[1].double(), 2.5 * w / w.sum(1, keepdim=True), rtol=60 * H32,
                               atol=0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gate_masks_of_the_types_lowest_value(dtype):
    # masked with finfo.min instead of -inf: real numbers, that are chosen where the
    # others run out, and with a weight of zero unless all of a row's are such
    E, k, low = 48, 8, torch.finfo(dtype).min
    logits = _logits(120, E, dtype)
    logits[40:80, 5:] = low                        # fewer open experts than k
    logits[80:, :] = low
    logits[100:, 7] = -math.inf
    for score in ("softmax", "sigmoid"):
        for b in (None, _bias(E)):
            for groups in ({}, dict(n_group=6, topk_group=2, group_topk=2)):
                how = dict(score=score, **groups)
                rid, rw, rc, _ = orc.route_gate(logits.float().numpy(), k,
                                                bias=None if b is None else b.numpy(), **how)
                ids, w, counts, _ = m.moe_route_gate(dev(logits), k, bias=dev(b), **how)
                assert np.array_equal(ids.cpu().numpy(), rid)
                assert np.array_equal(counts.cpu().numpy(), rc)
                # among themselves the masked are equal: the others' spread counts
                tol = _units(torch.where(logits == low, torch.zeros_like(logits), logits), k)
                assert np.all(np.abs(w.cpu().numpy() - rw) <= tol * np.abs(rw) + TINY)


def test_gate_past_two_to_the_31_elements():
    T, E, k, last = (1 << 21) + 77, 1024, 4, 100
    logits = torch.empty((T, E), dtype=torch.bfloat16, device="cuda").normal_()
    ids, w, counts, offsets = m.moe_route_gate(logits, k)
    assert m.moe_get_error() == 0 and int(counts.sum()) == int(offsets[-1]) == T * k
    tail = logits[-last:].clone()
    tid, tw, _, _ = m.moe_route_gate(tail, k)
    assert torch.equal(ids[-last:], tid) and torch.equal(w[-last:], tw)
    assert torch.equal(counts, torch.bincount(ids.reshape(-1), minlength=E).to(torch.int32))
    dp = torch.empty((T, k), device="cuda").normal_()
    got = m.moe_route_gate_backward(dp, logits, ids)
    assert torch.equal(got[-last:], m.moe_route_gate_backward(dp[-last:].clone(), tail, tid))


def test_gate_allocates_on_the_stream_that_it_runs_on():
    logits = dev(_logits(70001, 64))
    want = m.moe_route_gate(logits, 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(8):                             # workspaces and results of the side stream
        got.append(m.moe_route_gate(logits, 6, stream=side))
        torch.full((1 << 20,), -1, dtype=torch.int32, device="cuda")
    side.synchronize()
    for g in got:
        for x, y in zip(g, want):
            assert torch.equal(x, y)


def test_gate_zero_tokens():
    ids, w, counts, offsets = m.moe_route_gate(dev(torch.zeros((0, 12))), 3)
    assert ids.shape == (0, 3) and w.shape == (0, 3)
    assert counts.cpu().tolist() == [0] * 12 and offsets.cpu().tolist() == [0] * 13
    got = m.moe_route_gate_backward(w, dev(torch.zeros((0, 12))), ids)
    assert got.shape == (0, 12)


def test_gate_unaligned_rows():
    # rows that start at any element: odd E, and a view one element into its buffer
    for dtype in (torch.float32, torch.bfloat16):
        buf = dev(_logits(1, 40 * 64 + 1, dtype).reshape(-1))
        logits = buf[1:].view(40, 64)
        ids, w, counts, _ = m.moe_route_gate(logits, 4, score="sigmoid")
        rid, rw, rc, _ = orc.route_gate(logits.float().cpu().numpy(), 4, score="sigmoid")
        assert np.array_equal(ids.cpu().numpy(), rid) and np.array_equal(counts.cpu().numpy(), rc)
        out = torch.empty(40 * 64 + 1, dtype=dtype, device="cuda")[1:].view(40, 64)
        dp = torch.ones((40, 4), device="cuda")
        m.moe_route_gate_backward(dp, logits, ids, score="sigmoid", dlogits=out)
        assert torch.equal(out, m.moe_route_gate_backward(dp, logits.clone(), ids,
                                                          score="sigmoid"))


def test_gate_on_another_stream_and_in_a_graph():
    logits, bias = dev(_logits(500, 128)), dev(_bias(128))
    dp = dev(torch.randn((500, 8), generator=torch.Generator().manual_seed(2)))
    how = dict(bias=bias, score="sigmoid")
    want = m.moe_route_gate(logits, 8, **how)
    wgrad = m.moe_route_gate_backward(dp, logits, want[0], **how)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = m.moe_route_gate(logits, 8, stream=side, **how)
    side.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    outs = [torch.empty_like(t) for t in want]
    grad = torch.empty_like(logits)
    ws = torch.empty(m._lib.moe_route_gate_workspace_size(500, 8, 128), dtype=torch.uint8,
                     device="cuda")
    live = logits.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_route_gate(live, 8, expert_ids=outs[0], probs=outs[1], counts=outs[2],
                         offsets=outs[3], workspace=ws, **how)
        m.moe_route_gate_backward(dp, live, outs[0], dlogits=grad, **how)
    for scale in (1.0, -1.0, 1.0):
        live.copy_(logits * scale)
        graph.replay()
        torch.cuda.synchronize()
        now = m.moe_route_gate(live, 8, **how)
        for x, y in zip(outs, now):
            assert torch.equal(x, y)
    assert torch.equal(grad, wgrad)


def test_gate_backward_reports_a_bad_id():
    logits, dp = dev(_logits(3, 8)), dev(torch.ones((3, 2)))
    ids = dev(torch.tensor([[0, 1], [2, 8], [-1, 3]], dtype=torch.int32))
    got = m.moe_route_gate_backward(dp, logits, ids, score="sigmoid", renormalise=False)
    assert m.moe_get_error() == 3
    ref = orc.route_gate_backward(np.ones((3, 2)), logits.cpu().numpy(),
                                  np.array([[0, 1], [2, 0], [0, 3]]), score="sigmoid",
                                  renormalise=False)
    ref[1, 0] = ref[2, 0] = 0.0
    np.testing.assert_allclose(got.cpu().numpy(), ref, rtol=40 * H32, atol=TINY)


def test_gate_refusals():
    logits = dev(torch.zeros((4, 8)))
    for call in (lambda: m.moe_route_gate(logits, 9), lambda: m.moe_route_gate(logits, 0),
                 lambda: m.moe_route_gate(logits, 2, n_group=3, topk_group=3),
                 lambda: m.moe_route_gate(logits, 3, n_group=4, topk_group=1)):
        with pytest.raises(m.MoeError) as e:
            call()
        assert e.value.status == 1
    with pytest.raises(m.MoeError) as e:
        m.moe_route_gate(dev(torch.zeros((9999, 8))), 2, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4
    with pytest.raises(ValueError, match="contiguous"):
        m.moe_route_gate(dev(torch.zeros((8, 4))).t(), 2)
    with pytest.raises(ValueError, match="bfloat16"):
        m.moe_route_gate(logits.double(), 2)
    with pytest.raises(ValueError, match="shape"):
        m.moe_route_gate(logits, 2, bias=dev(torch.zeros(7)))


def _opposite_biases(E, n_group, B):
    """In every group +B, -B and, below these, -2 B: the two best sum to their scores alone."""
    size = E // n_group
    rng = np.random.default_rng(E + n_group)
    rows = np.full((n_group, size), -2.0 * B, np.float32)
    for row in rows:
        first, second = rng.choice(size, 2, replace=False)
        row[first], row[second] = B, -B
    return torch.from_numpy(rows.reshape(-1))


# groups that whole lanes hold, groups that lie across them, both with one and many tokens a warp
@pytest.mark.parametrize("E,k,n_group,topk_group", [(64, 6, 4, 2), (256, 8, 8, 4), (256, 8, 16, 3),
                                                    (512, 8, 32, 9), (8, 2, 4, 2), (48, 6, 8, 3),
                                                    (64, 6, 32, 9), (72, 5, 12, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_groups_whose_two_best_cancel(E, k, n_group, topk_group, score):
    for i, B in enumerate((100.0, 1000.0, 10000.0)):
        bias = _opposite_biases(E, n_group, B)
        for sd in (1e-4, 1e-2):
            logits = 0.3 + _logits(300, E, sd=sd, seed=i)
            _check(logits, k, bias=bias, score=score, n_group=n_group, topk_group=topk_group,
                   group_topk=2, backward=False)


@pytest.mark.parametrize("E", [8, 64, 256])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_groups_whose_sum_leaves_the_range_of_float(E, score):
    # a sum of two beyond float's range is not a masked group's, nor all such sums alike
    size = E // 4
    for pairs in (((-math.inf, -math.inf), (-3e38, -3e38), (-2e38, -2e38), (-2.5e38, -2.5e38)),
                  ((-math.inf, -math.inf), (-3e38, -3e38), (-math.inf, -math.inf), (-2e38, -3e38)),
                  ((3e38, 3e38), (3.2e38, 2.9e38), (3.3e38, 2e38), (2e38, 1e38)),
                  ((3e38, -3e38), (2e38, -2e38), (0.1, 0.1), (-3e38, -1e38))):
        bias = torch.full((4, size), -math.inf)
        bias[:, :2] = torch.tensor(pairs)
        for topk_group in (1, 2, 3):
            _check(_logits(70, E), 2, bias=bias.reshape(-1), score=score, n_group=4,
                   topk_group=topk_group, group_topk=2, backward=False)


@pytest.mark.parametrize("E,k", [(8, 4), (24, 6), (64, 6), (100, 8), (256, 8)])
@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_token_alone_and_among_others(E, k, renormalise, score):
    # rows masked with the type's lowest value, and rows of scores below float's range, beside
    # rows of any other kind: the others' bits do not depend on their neighbours
    logits = _logits(67, E)
    logits[5::7] = torch.finfo(torch.float32).min
    logits[9::11] -= 120.0
    logits, dp = dev(logits), dev(_logits(67, k, seed=1))
    how = dict(score=score, renormalise=renormalise, scale=2.5)
    ids, w, _, _ = m.moe_route_gate(logits, k, **how)
    grad = m.moe_route_gate_backward(dp, logits, ids, **how)
    for t in range(67):
        alone = m.moe_route_gate(logits[t:t + 1].clone(), k, **how)
        assert torch.equal(alone[0][0], ids[t]) and torch.equal(alone[1][0], w[t]), t
        one = m.moe_route_gate_backward(dp[t:t + 1].clone(), logits[t:t + 1].clone(), alone[0],
                                        **how)
        assert torch.equal(one[0], grad[t]), t
