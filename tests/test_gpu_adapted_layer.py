"""The operators of a layer's dense half together, as fine-tuning and serving use them
(examples/finetune_adapters.py): the layer's output and every gradient against the
float64 oracles chained in the same order, and a training step captured into a graph.

Tolerance: relative to the largest value, 3e-2, as the other layer's test holds: what
goes between the operators is bfloat16 (2^-8 each at most, random)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle as orc
from gpu_util import assert_rel_to_max

pytestmark = pytest.mark.gpu
m = pytest.importorskip("moe_expert_dispatch_gb300")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location(
        "finetune_adapters", os.path.join(ROOT, "examples", "finetune_adapters.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _np(t):
    return t.detach().double().cpu().numpy()


def _inputs(T, H, n, kind):
    g = torch.Generator().manual_seed(T)
    x, routed, d_out = ((torch.randn((T, H), generator=g) * sd).bfloat16().cuda()
                        for sd in (1.0, 0.5, 0.1))
    if kind == "runs":
        ids = torch.arange(T) * n // T
    else:
        ids = torch.randint(-1, n, (T,), generator=g)
    return x, routed, d_out, ids.to(torch.int32).cuda()


def _kept(rng, p, shape):
    seed, draw = (int(v) for v in rng.tolist())
    return orc.dropout_kept(int(np.prod(shape)), seed, draw, p).reshape(shape)


@pytest.mark.parametrize("T,n,r,kind", [(70, 5, 8, "mixed"), (520, 2, 16, "runs"),
                                        (300, 3, 24, "mixed")])
def test_adapted_layer_against_the_oracle(T, n, r, kind):
    H, F, p = 128, 256, 0.25
    layer = _example().AdaptedLayer(H, F, n, r, p=p, seed=T)
    x, routed, d_out, ids = _inputs(T, H, n, kind)
    out, s = layer.forward(x, ids, routed=routed)
    dx, d_routed, grads = layer.backward(d_out, s)
    assert m.moe_get_error() == 0

    x64, rows, s64 = _np(x), ids.cpu().numpy(), _np(layer.scales)
    w = [_np(t) for t in (layer.w_gate, layer.w_up, layer.w_down)]
    a, b = _np(layer.a), _np(layer.b)
    k_in, k_out = _kept(layer.rng, p, (T, H)), _kept(layer.rng_out, p, (T, H))
    pre = orc.norm_residual(x64, w_next=_np(layer.w_pre))
    f = orc.gated_ffn(pre["n"], *w, kind="silu", add=_np(routed), rounded=False)
    nd = orc.dropout_residual(pre["n"], k_in, p)
    y, v = orc.lora(nd, a, b, rows, s64, f["y"])
    want = orc.dropout_residual(y, k_out, p, x64)
    assert_rel_to_max(_np(out), want, 3e-2, "out")

    dy = orc.dropout_residual(_np(d_out), k_out, p)
    lo = orc.lora_backward(dy, nd, v, a, b, rows, s64)
    dn = orc.dropout_residual(lo["dx"], k_in, p)
    fb = orc.gated_ffn_backward(dy, pre["n"], *w, f["a_gate"], f["a_up"], kind="silu", add=dn,
                                rounded=False)
    back = orc.norm_residual_backward(_np(d_out), fb["dx"], x64, w_next=_np(layer.w_pre),
                                      rstd_out=pre["rstd_out"])
    assert_rel_to_max(_np(d_routed), dy, 3e-2, "d_routed")
    assert_rel_to_max(_np(dx), back["dx"], 3e-2, "dx")
    assert_rel_to_max(_np(grads["a"]), lo["da"], 3e-2, "a")
    assert_rel_to_max(_np(grads["b"]), lo["db"], 3e-2, "b")

    # served: no mask, the same adapters
    got, _ = layer.forward(x, ids, routed=routed, train=False)
    y, _ = orc.lora(pre["n"], a, b, rows, s64, f["y"])
    assert_rel_to_max(_np(got), x64 + y, 3e-2, "served")
    # a token by itself is what it is in the batch
    for t in (0, T - 1):
        one, _ = layer.forward(x[t:t + 1].contiguous(), ids[t:t + 1].contiguous(),
                               routed=routed[t:t + 1].contiguous(), train=False)
        assert_rel_to_max(_np(one), (x64 + y)[t:t + 1], 3e-2, "one token")


def test_adapted_layer_training_step_in_a_graph():
    H, F, n, r, T = 128, 256, 3, 8, 300
    ex = _example()
    x, _, d_out, ids = _inputs(T, H, n, "mixed")

    def step(layer):
        out, s = layer.forward(x, ids)
        dx, _, grads = layer.backward(d_out, s)
        layer.step(grads, lr=0.01)
        return out, dx

    eager, graphed = (ex.AdaptedLayer(H, F, n, r, seed=4) for _ in range(2))
    step(ex.AdaptedLayer(H, F, n, r, seed=4))          # first calls, before any capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(graphed)
    for i in range(4):
        want = step(eager)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i
    for key in eager.masters:
        assert torch.equal(eager.masters[key], graphed.masters[key]), key
    assert int(graphed.rng[1]) == 4
    assert m.moe_get_error() == 0


def test_example_runs(capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["finetune_adapters.py", "--steps", "3", "--tokens", "600"])
    _example().main()
    assert "served (5, 1024)" in capsys.readouterr().out
