"""A transformer layer's MoE half, trained for a few steps on one GPU:

    n      = w_pre * rmsnorm(x)                       moe_norm_residual
    logits = n W_r                                    a library product
    route  = grouped sigmoid gate with a balance bias moe_route_gate
    y      = the expert block                         moe_expert_forward
    out    = x + g * (w_post * rmsnorm(y))            moe_norm_residual

then its backward in the opposite order, the gradients of all its parameters
clipped by one norm (moe_clip_grad_norm) and a plain gradient step. The bias is
not trained by gradient: it moves against the load of each expert.

    python examples/train_moe_layer.py [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_dispatch_gb300 as m  # noqa: E402


class MoeLayer:
    """Parameters, and one forward and backward over them. The expert weights
    are bfloat16, as the block takes them; the router, the norms and the gate
    are float32."""

    def __init__(self, H, F, E, k, n_group=4, topk_group=2, scale=2.5, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, sd, dtype=torch.float32):
            return (torch.randn(shape, generator=g, device=device) * sd).to(dtype)

        bf16 = torch.bfloat16
        self.k = k
        self.how = dict(score="sigmoid", scale=scale)
        self.groups = dict(n_group=n_group, topk_group=topk_group, group_topk=2)
        self.bias = torch.zeros(E, device=device)
        self.params = dict(
            w_pre=torch.ones(H, device=device), w_post=torch.ones(H, device=device),
            gate=torch.full((H,), 0.5, device=device), w_router=normal(H, E, sd=H ** -0.5),
            w_gate=normal(E, H, F, sd=H ** -0.5, dtype=bf16),
            w_up=normal(E, H, F, sd=H ** -0.5, dtype=bf16),
            w_down=normal(E, F, H, sd=F ** -0.5, dtype=bf16))

    def forward(self, x):
        """(out, what the backward needs) of x, bfloat16 [T, H]."""
        p = self.params
        pre = m.moe_norm_residual(x, w_next=p["w_pre"])
        n = pre["n"]
        logits = n.float() @ p["w_router"]
        ids, probs, counts, _ = m.moe_route_gate(logits, self.k, bias=self.bias, **self.groups,
                                                 **self.how)
        y, ws = m.moe_expert_forward(n, p["w_gate"], p["w_up"], p["w_down"], ids, probs,
                                     cfg=m.config(save_for_backward=True))
        post = m.moe_norm_residual(x, y, w_post=p["w_post"], gate=p["gate"])
        return post["out"], dict(x=x, n=n, rstd=pre["rstd_out"], logits=logits, ids=ids,
                                 probs=probs, counts=counts, y=y, ws=ws, rstd_y=post["rstd_y"],
                                 out=post["out"])

    def backward(self, d_out, s):
        """(dx, the gradients by the parameters' names) from d_out, bfloat16 [T, H]."""
        p = self.params
        post = m.moe_norm_residual_backward(d_out, None, s["out"], s["y"], w_post=p["w_post"],
                                            gate=p["gate"], rstd_y=s["rstd_y"])
        block = m.moe_expert_backward(post["dy"], s["n"], p["w_gate"], p["w_up"], p["w_down"],
                                      s["ids"], s["probs"], s["ws"])
        dlogits = m.moe_route_gate_backward(block["dprobs"], s["logits"], s["ids"],
                                            bias=self.bias, **self.how)
        dn = (block["dx"].float() + dlogits @ p["w_router"].t()).bfloat16()
        pre = m.moe_norm_residual_backward(post["dx"], dn, s["x"], w_next=p["w_pre"],
                                           rstd_out=s["rstd"])
        grads = dict(w_pre=pre["dw_next"], w_post=post["dw_post"], gate=post["dgate"],
                     w_router=s["n"].float().t() @ dlogits, w_gate=block["dw_gate"],
                     w_up=block["dw_up"], w_down=block["dw_down"])
        return pre["dx"], grads

    def step(self, grads, counts, max_norm=1.0, rate=0.05, bias_rate=1e-3):
        """Clips the gradients by one norm, steps, and moves the bias towards balance;
        returns the norm (a device tensor)."""
        names = list(self.params)
        norm, _ = m.moe_clip_grad_norm([grads[name] for name in names], max_norm)
        for name in names:
            self.params[name].sub_((rate * grads[name]).to(self.params[name].dtype))
        load = counts.float()
        self.bias.add_(bias_rate * torch.sign(load.mean() - load))
        return norm


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--ffn", type=int, default=1024)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--k", type=int, default=4)
    a = ap.parse_args()
    layer = MoeLayer(a.hidden, a.ffn, a.experts, a.k)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((a.tokens, a.hidden), generator=g, device="cuda").bfloat16()
    target = (x.float() + 0.3 * torch.roll(x.float(), 1, dims=1)).bfloat16()
    for i in range(a.steps):
        out, saved = layer.forward(x)
        diff = out.float() - target.float()
        loss = diff.square().mean()
        dx, grads = layer.backward((2.0 / a.hidden * diff).bfloat16(), saved)
        norm = layer.step(grads, saved["counts"])
        if i % 5 == 0 or i + 1 == a.steps:
            print(f"step {i:3d}  loss {loss.item():.5f}  gradient norm {norm.item():.4f}  "
                  f"busiest expert {int(saved['counts'].max())} of {a.tokens * a.k} slots")
    if m.moe_get_error():
        raise SystemExit("a kernel reported an error")


if __name__ == "__main__":
    main()
