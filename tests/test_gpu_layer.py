"""The operators around the block, together with it, as a training step uses
them (examples/train_moe_layer.py): the layer's output and every gradient
against the float64 oracles chained in the same order, and a clipped step.

Tolerance: relative to the largest value, 3e-2, as the MXFP8 paths are held to
and the smoke check uses: n, y and the gradients between the operators are
bfloat16 (2^-9 each, random), and a weight gradient sums them over tokens."""
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
        "train_moe_layer", os.path.join(ROOT, "examples", "train_moe_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _np(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("T,E,k,n_group", [(200, 8, 2, 4), (333, 16, 4, 4)])
def test_layer_gradients_against_the_oracle(T, E, k, n_group):
    H, F = 256, 128
    layer = _example().MoeLayer(H, F, E, k, n_group=n_group, seed=T)
    layer.bias.copy_(torch.linspace(-0.05, 0.05, E))
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, H), generator=g).bfloat16().cuda()
    d_out = (torch.randn((T, H), generator=g) * 0.1).bfloat16().cuda()
    out, s = layer.forward(x)
    dx, grads = layer.backward(d_out, s)
    assert m.moe_get_error() == 0

    p = {key: _np(t) for key, t in layer.params.items()}
    x64 = _np(x)
    pre = orc.norm_residual(x64, w_next=p["w_pre"])
    n = orc.bf16(pre["n"])
    logits = n @ p["w_router"]
    # the choice itself on the logits that the gate saw: a tie may fall either way
    ids, _, counts, _ = orc.route_gate(_np(s["logits"]), k, bias=_np(layer.bias), **layer.groups,
                                       **layer.how)
    assert np.array_equal(ids, s["ids"].cpu().numpy())
    assert np.array_equal(counts, s["counts"].cpu().numpy())
    sj = np.take_along_axis(1.0 / (1.0 + np.exp(-logits)), ids.astype(np.int64), 1)
    w = layer.how["scale"] * sj / sj.sum(axis=1, keepdims=True)
    post_in = orc.expert_forward(n, p["w_gate"], p["w_up"], p["w_down"], ids, w)
    post = orc.norm_residual(x64, post_in, w_post=p["w_post"], gate=p["gate"])
    assert_rel_to_max(_np(out), post["out"], 3e-2, "out")

    b1 = orc.norm_residual_backward(_np(d_out), None, post["out"], y=post_in, w_post=p["w_post"],
                                    gate=p["gate"], rstd_y=post["rstd_y"])
    b2 = orc.expert_backward(b1["dy"], n, p["w_gate"], p["w_up"], p["w_down"], ids, w)
    dl = orc.route_gate_backward(b2["dprobs"], logits, ids, bias=_np(layer.bias), **layer.how)
    b3 = orc.norm_residual_backward(b1["dx"], b2["dx"] + dl @ p["w_router"].T, x64,
                                    w_next=p["w_pre"], rstd_out=pre["rstd_out"])
    want = dict(w_pre=b3["dw_next"], w_post=b1["dw_post"], gate=b1["dgate"], w_router=n.T @ dl,
                w_gate=b2["dw_gate"], w_up=b2["dw_up"], w_down=b2["dw_down"])
    assert_rel_to_max(_np(dx), b3["dx"], 3e-2, "dx")
    for key, ref in want.items():
        assert_rel_to_max(_np(grads[key]), ref, 3e-2, key)

    # the clipped step
    total = float(np.sqrt(sum(float((_np(t) ** 2).sum()) for t in grads.values())))
    before = {key: t.clone() for key, t in grads.items()}
    norm = layer.step(grads, s["counts"], max_norm=0.5 * total)
    assert abs(norm.item() / total - 1) < 1e-5
    for key in grads:
        assert torch.allclose(grads[key], before[key] * 0.5, rtol=1e-4, atol=0), key


def test_layer_learns():
    layer = _example().MoeLayer(256, 256, 16, 4, seed=3)
    x = torch.randn((2048, 256), generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    target = (x.float() + 0.3 * torch.roll(x.float(), 1, dims=1)).bfloat16()
    losses = []
    for _ in range(12):
        out, s = layer.forward(x)
        diff = out.float() - target.float()
        losses.append(diff.square().mean().item())
        _, grads = layer.backward((2.0 / 256 * diff).bfloat16(), s)
        layer.step(grads, s["counts"])
    assert m.moe_get_error() == 0
    assert losses[-1] < losses[0]
