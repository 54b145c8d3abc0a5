"""Adapters of several tenants fine-tuned beside the frozen dense half of a layer,
and served, on one GPU:

    n    = w_pre * rmsnorm(x)                       moe_norm_residual
    y    = shared expert of n (+ the routed experts' result)    moe_gated_ffn
    y    = y + s_a B_a A_a drop(n)                  moe_dropout_residual, moe_lora
    out  = x + drop(y)                              moe_dropout_residual

then its backward in the opposite order, the gradients of all adapters clipped by
one norm (moe_clip_grad_norm) and a plain gradient step of their float32 masters.
The dropout masks are made from a seed and a draw in device memory, so a training
step captured into a CUDA graph drops others at every replay. Serving runs the same
layer without dropout, each token with its own tenant's adapter.

    python examples/finetune_adapters.py [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_dispatch_gb300 as m  # noqa: E402

BF16 = torch.bfloat16


class AdaptedLayer:
    """The frozen weights (bfloat16), n adapters of rank r, and one forward and
    backward over them."""

    def __init__(self, H, F, n, r, p=0.1, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, sd):
            return torch.randn(shape, generator=g, device=device) * sd

        self.p = p
        self.act = "silu"
        self.w_pre = torch.ones(H, device=device)
        self.w_gate, self.w_up = (normal(H, F, sd=H ** -0.5).to(BF16) for _ in range(2))
        self.w_down = normal(F, H, sd=F ** -0.5).to(BF16)
        self.scales = torch.full((n,), 2.0, device=device)
        # float32 masters, and what the kernels read
        self.masters = dict(a=normal(n, r, H, sd=H ** -0.5), b=normal(n, r, H, sd=0.1))
        self.a, self.b = self.masters["a"].to(BF16), self.masters["b"].to(BF16)
        # seed and draw of the two masks of a step
        self.rng = torch.tensor([seed, 0], dtype=torch.int64, device=device)
        self.rng_out = torch.tensor([seed + 1, 0], dtype=torch.int64, device=device)

    def forward(self, x, ids, routed=None, train=True):
        """(out, what the backward needs) of x bfloat16 [T, H], ids int32 [T] (-1: no
        adapter) and the routed experts' result (bfloat16 [T, H] or None)."""
        n = m.moe_norm_residual(x, w_next=self.w_pre)
        plan = m.moe_lora_plan(ids, self.a.shape[0])
        f = m.moe_gated_ffn(n["n"], self.w_gate, self.w_up, self.w_down, act=self.act, add=routed,
                            save_for_backward=train)
        nd = m.moe_dropout_residual(n["n"], self.rng, self.p) if train else n["n"]
        y = m.moe_lora(nd, self.a, self.b, ids, plan=plan, scales=self.scales, base=f["y"],
                       out=f["y"])
        if not train:
            return m.moe_norm_residual(x, y["out"])["out"], None
        out = m.moe_dropout_residual(y["out"], self.rng_out, self.p, x=x)
        return out, dict(x=x, ids=ids, plan=plan, n=n["n"], nd=nd, rstd=n["rstd_out"], v=y["v"],
                         a_gate=f["a_gate"], a_up=f["a_up"])

    def backward(self, d_out, s):
        """(dx, gradient of the routed experts' result, {a, b}) of d_out bfloat16 [T, H]."""
        d = m.moe_dropout_residual_backward(d_out, self.rng_out, self.p)
        dy = d["dy"]                                  # reaches the routed experts as it is
        lo = m.moe_lora_backward(dy, s["nd"], s["v"], self.a, self.b, s["ids"], plan=s["plan"],
                                 scales=self.scales)
        dn = m.moe_dropout_residual_backward(lo["dx"], self.rng, self.p, residual=False)["dy"]
        dn = m.moe_gated_ffn_backward(dy, s["n"], self.w_gate, self.w_up, self.w_down, s["a_gate"],
                                      s["a_up"], act=self.act, add=dn, weight_grads=False,
                                      dx=dn)["dx"]
        dx = m.moe_norm_residual_backward(d["dx"], dn, s["x"], w_next=self.w_pre,
                                          rstd_out=s["rstd"])["dx"]
        return dx, dy, dict(a=lo["da"], b=lo["db"])

    def step(self, grads, lr=0.1, max_norm=1.0):
        """Clips the gradients by their one norm and applies them; the next step draws
        other masks."""
        norm, _ = m.moe_clip_grad_norm(list(grads.values()), max_norm)
        for key, t in self.masters.items():
            t.sub_(grads[key], alpha=lr)
        self.a.copy_(self.masters["a"])
        self.b.copy_(self.masters["b"])
        self.rng[1] += 1
        self.rng_out[1] += 1
        return norm


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=4096)
    args = ap.parse_args()
    H, F, n, r = 1024, 2048, 4, 16
    layer = AdaptedLayer(H, F, n, r)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((args.tokens, H), generator=g, device="cuda").to(BF16)
    # every tenant has a run of the batch, and a direction of its own to learn
    ids = (torch.arange(args.tokens, device="cuda") * n // args.tokens).to(torch.int32)
    want = torch.randn((n, H), generator=g, device="cuda")[ids.long()] + x.float()
    for i in range(args.steps):
        out, s = layer.forward(x, ids)
        diff = out.float() - want
        _, _, grads = layer.backward((2.0 / H * diff).to(BF16), s)
        norm = layer.step(grads)
        if i % 5 == 0 or i + 1 == args.steps:
            print(f"step {i:3d}  loss {diff.square().mean().item():.4f}  "
                  f"gradient norm {norm.item():.4f}")
    # one token of each tenant, and one without an adapter
    tok = torch.tensor([0, 1, 2, 3, -1], dtype=torch.int32, device="cuda")
    out, _ = layer.forward(x[:5].contiguous(), tok, train=False)
    assert m.moe_get_error() == 0
    print("served", tuple(out.shape))


if __name__ == "__main__":
    main()
