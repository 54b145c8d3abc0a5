"""Cases of the operators of a layer's dense half: the gated feed-forward block
(a shared expert, a dense layer), low-rank adapters beside a projection, and
dropout of the branch with a mask that is never stored.

With own false, run() computes the plain forms in elementary torch
operations; with own true it calls the library."""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of one sequence through a small shared expert: latency
        dict(name="ffn_step", op="ffn", dir="fwd", T=1, H=2048, F=768, act="silu", add=True,
             save=False),
        # a decoding step of 32 sequences through a dense layer: its weights have to be read
        dict(name="ffn_decode", op="ffn", dir="fwd", T=32, H=4096, F=14336, act="silu", add=False,
             save=False),
        # the prefill of the Mixtral-shaped workload, added to what the experts gave
        dict(name="ffn_prefill", op="ffn", dir="fwd", T=4096, H=4096, F=14336, act="silu",
             add=True, save=False),
        # the gradients of a short ragged batch with sizes that no tile divides
        dict(name="ffn_ragged_grad", op="ffn", dir="bwd", T=1021, H=1000, F=2728, act="gelu_tanh",
             add=False, save=True),
        # a training step's gradients of the widest feed-forward
        dict(name="ffn_train_grad", op="ffn", dir="bwd", T=8192, H=4096, F=14336, act="silu",
             add=True, save=True),
        # one token of one sequence with its adapter: latency
        dict(name="lora_step", op="lora", dir="fwd", T=1, H=4096, N=4096, n=8, r=16,
             rows="mixed", scales=True, base=True),
        # a decoding step of 64 sequences, each with an adapter of its own or none
        dict(name="lora_decode", op="lora", dir="fwd", T=64, H=4096, N=14336, n=32, r=16,
             rows="mixed", scales=True, base=True),
        # the prefill of sixteen requests, one run of tokens each
        dict(name="lora_prefill", op="lora", dir="fwd", T=8192, H=4096, N=4096, n=16, r=16,
             rows="runs", scales=True, base=True),
        # the gradients of four wide adapters trained at once
        dict(name="lora_train_grad", op="lora", dir="bwd", T=16384, H=4096, N=4096, n=4, r=64,
             rows="runs", scales=True, base=True),
        # the branch of a short batch of odd size, backward
        dict(name="drop_ragged_grad", op="drop", dir="bwd", numel=255 * 1001, stream="f32",
             branch="bf16", x=True, p=0.1, a=1.0, b=1.0),
        # the input of an adapter in training: no residual
        dict(name="drop_input", op="drop", dir="fwd", numel=4096 * 4096, stream="bf16",
             branch="bf16", x=False, p=0.05, a=1.0, b=1.0),
        # the branch of a training step before a float residual stream
        dict(name="drop_train", op="drop", dir="fwd", numel=16384 * 7168, stream="f32",
             branch="bf16", x=True, p=0.1, a=1.0, b=1.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "lora", "lora", "drop"])
    if op == "ffn":
        H, F = rng.choice([(512, 1024), (2048, 768), (4096, 14336), (7168, 2048), (2560, 8192),
                           (1000, 2728), (1160, 4104), (2048, 5504)])
        back = rng.random() < 0.4
        most = 8192 * 4096 * 14336 // (H * F)
        return dict(op="ffn", dir="bwd" if back else "fwd", T=_log_int(rng, 1, min(most, 16384)),
                    H=H, F=F, act=rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"]),
                    add=rng.random() < 0.5, save=back or rng.random() < 0.3)
    if op == "lora":
        return dict(op="lora", dir=rng.choice(["fwd", "fwd", "bwd"]), T=_log_int(rng, 1, 16384),
                    H=rng.choice([512, 1000, 2048, 4096, 7168]),
                    N=rng.choice([512, 1000, 2048, 4096, 6144]), n=_log_int(rng, 1, 32),
                    r=rng.choice([4, 8, 13, 16, 32, 64]), rows=rng.choice(["mixed", "runs"]),
                    scales=rng.random() < 0.7, base=rng.random() < 0.7)
    return dict(op="drop", dir=rng.choice(["fwd", "bwd"]), numel=_log_int(rng, 1000, 100000000),
                stream=rng.choice(["f32", "bf16"]), branch=rng.choice(["bf16", "bf16", "f32"]),
                x=rng.random() < 0.6, p=rng.choice([0.0, 0.05, 0.1, 0.5]),
                a=rng.choice([1.0, 1.0, 0.5]), b=rng.choice([1.0, 1.0, 0.7]))


_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SZ = {"f32": 4, "bf16": 2}


def _used(case):
    """Adapters that have a row, about: every one in runs, as many as rows at most."""
    return min(case["n"], case["T"])


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, sd=1.0, mean=0.0, dt=torch.bfloat16):
        return (torch.randn(shape, generator=g, device="cuda") * sd + mean).to(dt)

    s = dict(case=case)
    if case["op"] == "ffn":
        T, H, F = case["T"], case["H"], case["F"]
        s["x"] = randn(T, H)
        s["w_gate"], s["w_up"] = randn(H, F, sd=H ** -0.5), randn(H, F, sd=H ** -0.5)
        s["w_down"] = randn(F, H, sd=F ** -0.5)
        s["add"] = randn(T, H) if case["add"] else None
        if case["dir"] == "bwd":
            # what the forward kept, and the gradient that reaches its result
            s["a_gate"] = (s["x"].float() @ s["w_gate"].float()).to(torch.bfloat16)
            s["a_up"] = (s["x"].float() @ s["w_up"].float()).to(torch.bfloat16)
            s["dy"] = randn(T, H, sd=0.02)
            s["add"] = randn(T, H, sd=0.02) if case["add"] else None
            s["outs"] = dict(dx=torch.empty_like(s["x"]), dw_gate=torch.empty_like(s["w_gate"]),
                             dw_up=torch.empty_like(s["w_up"]),
                             dw_down=torch.empty_like(s["w_down"]))
        else:
            s["outs"] = dict(y=torch.empty_like(s["x"]))
            if case["save"]:
                s["outs"]["a_gate"] = torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
                s["outs"]["a_up"] = torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
        return s
    if case["op"] == "lora":
        T, H, N, n, r = case["T"], case["H"], case["N"], case["n"], case["r"]
        if case["rows"] == "runs":
            # requests of any length one after the other, each with its adapter
            cuts = torch.sort(torch.randint(0, T + 1, (n - 1,), generator=g, device="cuda")).values
            ids = torch.bucketize(torch.arange(T, device="cuda"), cuts, right=True)
            ids = torch.randperm(n, generator=g, device="cuda")[ids]
        else:
            # a batch of single tokens: one in n + 1 has no adapter
            ids = torch.randint(-1, n, (T,), generator=g, device="cuda")
        s["ids"] = ids.to(torch.int32)
        s["x"] = randn(T, H)
        s["a"], s["b"] = randn(n, r, H, sd=H ** -0.5), randn(n, r, N, sd=r ** -0.5)
        s["scales"] = (torch.rand(n, generator=g, device="cuda") * 1.5 + 0.5) if case["scales"] else None
        s["out"] = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
        s["base"] = randn(T, N) if case["base"] else None
        if case["dir"] == "bwd":
            # what the forward kept, the gradient that reaches its result, and the projection's dx
            s["v"] = _plain_shrink(s["x"], s["a"], s["ids"])
            s["dy"] = randn(T, N, sd=0.02)
            s["base"] = randn(T, H, sd=0.02) if case["base"] else None
            s["out"] = torch.empty_like(s["x"])
            s["da"] = torch.empty(n, r, H, dtype=torch.float32, device="cuda")
            s["db"] = torch.empty(n, r, N, dtype=torch.float32, device="cuda")
        # one order of a batch's rows serves every projection and layer: by adapter, those
        # without one last, and where each adapter's rows begin
        key = torch.where(ids < 0, n, ids)
        first = torch.bincount(key, minlength=n + 1).cumsum(0)
        s["plan"] = (torch.sort(key, stable=True).indices.to(torch.int32),
                     torch.cat([first.new_zeros(1), first[:n]]).to(torch.int32))
        return s
    k = case["numel"]
    st, br = _DT[case["stream"]], _DT[case["branch"]]
    s["rng"] = torch.tensor([seed * 0x9E3779B97F4A7C15 % (1 << 62), seed + (1 << 33)],
                            dtype=torch.int64, device="cuda")
    if case["dir"] == "fwd":
        s["y"] = randn(k, dt=br)
        s["x"] = randn(k, dt=st) if case["x"] else None
        s["out"] = torch.empty(k, dtype=st, device="cuda")
    else:
        s["d_out"] = randn(k, sd=0.02, dt=st)
        s["dx"] = torch.empty(k, dtype=st, device="cuda") if case["x"] else None
        s["dy"] = torch.empty(k, dtype=br, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms

def _act(z, kind):
    """(act(z), act'(z))."""
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return z * s, s * (1.0 + z * (1.0 - s))
    if kind == "gelu":
        c = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * c, c + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if kind == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * z * (1.0 + t), (0.5 * (1.0 + t)
                                     + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * z * z))
    on = (z > 0).to(z.dtype)
    return z * on, on


def _plain_ffn(st):
    c, x = st["case"], st["x"].float()
    ag, au = x @ st["w_gate"].float(), x @ st["w_up"].float()
    y = (_act(ag, c["act"])[0] * au) @ st["w_down"].float()
    if st["add"] is not None:
        y = y + st["add"].float()
    got = dict(y=y.to(torch.bfloat16))
    if c["save"]:
        got["a_gate"], got["a_up"] = ag.to(torch.bfloat16), au.to(torch.bfloat16)
    return got


def _plain_ffn_grad(st):
    dy, x = st["dy"].float(), st["x"].float()
    ag, au = st["a_gate"].float(), st["a_up"].float()
    f, df = _act(ag, st["case"]["act"])
    dh = dy @ st["w_down"].float().t()
    dg, du = dh * au * df, dh * f
    dx = dg @ st["w_gate"].float().t() + du @ st["w_up"].float().t()
    if st["add"] is not None:
        dx = dx + st["add"].float()
    got = dict(dx=dx, dw_gate=x.t() @ dg, dw_up=x.t() @ du, dw_down=(f * au).t() @ dy)
    return {key: t.to(torch.bfloat16) for key, t in got.items()}


def _own_rows(ids, n, r):
    """[T, n * r]: 1 in the r columns of each row's own adapter, 0 elsewhere."""
    one = ids.long()[:, None] == torch.arange(n, device=ids.device)[None, :]
    return one.float().repeat_interleave(r, dim=1)


def _plain_shrink(x, a, ids):
    """v [T, r]: every adapter's products, of which each row keeps its own's."""
    n, r, H = a.shape
    v = (x.float() @ a.reshape(n * r, H).float().t()) * _own_rows(ids, n, r)
    return v.view(-1, n, r).sum(dim=1)


def _wide(v, ids, n, scales):
    """v [T, r] in the columns of the row's own adapter of [T, n * r], times its scale."""
    w = v.repeat(1, n) * _own_rows(ids, n, v.shape[1])
    return w if scales is None else w * scales.repeat_interleave(v.shape[1])


def _plain_lora(st):
    a, b = st["a"], st["b"]
    n, r, N = b.shape
    v = _plain_shrink(st["x"], a, st["ids"])
    out = _wide(v, st["ids"], n, st["scales"]) @ b.reshape(n * r, N).float()
    if st["base"] is not None:
        out = out + st["base"].float()
    return dict(out=out.to(torch.bfloat16), v=v)


def _plain_lora_grad(st):
    a, b, ids = st["a"], st["b"], st["ids"]
    n, r, H = a.shape
    dy, x = st["dy"].float(), st["x"].float()
    w = _wide(_plain_shrink(st["dy"], b, ids), ids, n, st["scales"])
    dx = w @ a.reshape(n * r, H).float()
    if st["base"] is not None:
        dx = dx + st["base"].float()
    return dict(dx=dx.to(torch.bfloat16), da=(w.t() @ x).view(n, r, H),
                db=(_wide(st["v"], ids, n, st["scales"]).t() @ dy).view(n, r, -1))


_MUL = (0xD2511F53, 0xCD9E8D57)
_KEY = (0x9E3779B9, 0xBB67AE85)
_LOW = 0xFFFFFFFF


def _words(numel, rng):
    """The 16-bit number of each of numel elements: Philox 4x32 of ten rounds at
    counter (element / 8, draw) under the key seed, eight numbers a block."""
    seed, at = rng[0], rng[1]
    c = torch.arange((numel + 7) // 8, device=rng.device)
    c0, c1 = c & _LOW, c >> 32
    c2, c3 = (at & _LOW).expand_as(c), ((at >> 32) & _LOW).expand_as(c)
    k0, k1 = seed & _LOW, (seed >> 32) & _LOW
    for _ in range(10):
        p, q = c0 * _MUL[0], c2 * _MUL[1]
        c0, c1, c2, c3 = (((q >> 32) & _LOW) ^ c1 ^ k0, q & _LOW,
                          ((p >> 32) & _LOW) ^ c3 ^ k1, p & _LOW)
        k0, k1 = (k0 + _KEY[0]) & _LOW, (k1 + _KEY[1]) & _LOW
    w = torch.stack([c0, c1, c2, c3], dim=1)
    return torch.stack([w & 0xFFFF, w >> 16], dim=2).reshape(-1)[:numel]


def _threshold(p):
    return min(65535, int(round(p * 65536)))


def _plain_drop(st):
    c = st["case"]
    keep = _words(c["numel"], st["rng"]) >= _threshold(c["p"])
    f = c["b"] / (1.0 - _threshold(c["p"]) / 65536)
    if c["dir"] == "fwd":
        out = torch.where(keep, st["y"].float() * f, 0.0)
        if st["x"] is not None:
            out = out + c["a"] * st["x"].float()
        return dict(out=out.to(_DT[c["stream"]]))
    d = st["d_out"].float()
    got = dict(dy=torch.where(keep, d * f, 0.0).to(_DT[c["branch"]]))
    if c["x"]:
        got["dx"] = (c["a"] * d).to(_DT[c["stream"]])
    return got


# ------------------------------------------------------------------ one pass

def run(state):
    c = state["case"]
    back = c["dir"] == "bwd"
    if not own:
        if c["op"] == "ffn":
            return _plain_ffn_grad(state) if back else _plain_ffn(state)
        if c["op"] == "lora":
            return _plain_lora_grad(state) if back else _plain_lora(state)
        return _plain_drop(state)
    import moe_expert_dispatch_gb300 as m
    if c["op"] == "ffn":
        weights = (state["w_gate"], state["w_up"], state["w_down"])
        if back:
            return m.moe_gated_ffn_backward(state["dy"], state["x"], *weights, state["a_gate"],
                                            state["a_up"], act=c["act"], add=state["add"],
                                            **state["outs"])
        got = m.moe_gated_ffn(state["x"], *weights, act=c["act"], add=state["add"],
                              save_for_backward=c["save"], **state["outs"])
        return {key: t for key, t in got.items() if t is not None}
    if c["op"] == "lora":
        how = dict(scales=state["scales"], base=state["base"], plan=state["plan"])
        if back:
            return m.moe_lora_backward(state["dy"], state["x"], state["v"], state["a"], state["b"],
                                       state["ids"], dx=state["out"], da=state["da"],
                                       db=state["db"], **how)
        return m.moe_lora(state["x"], state["a"], state["b"], state["ids"], out=state["out"],
                          **how)
    how = dict(residual_scale=c["a"], branch_scale=c["b"])
    if back:
        got = m.moe_dropout_residual_backward(state["d_out"], state["rng"], c["p"],
                                              residual=c["x"], dx=state["dx"], dy=state["dy"],
                                              **how)
        return {key: t for key, t in got.items() if t is not None}
    return dict(out=m.moe_dropout_residual(state["y"], state["rng"], c["p"], x=state["x"],
                                           out=state["out"], **how))


# ------------------------------------------------------------------ work and the answers in 64 bits

def work(case):
    if case["op"] == "ffn":
        T, H, F = case["T"], case["H"], case["F"]
        rows = 2 * T * H * (3 if case["add"] else 2)
        if case["dir"] == "fwd":
            kept = 4 * T * F if case["save"] else 0
            return dict(bytes=6 * H * F + rows + kept, flops=6 * T * H * F)
        return dict(bytes=12 * H * F + rows + 2 * T * H + 4 * T * F, flops=12 * T * H * F)
    if case["op"] == "lora":
        T, H, N, r, k = case["T"], case["H"], case["N"], case["r"], _used(case)
        if case["dir"] == "fwd":
            return dict(bytes=2 * T * (H + N * (2 if case["base"] else 1)) + 4 * T * r
                        + 2 * k * r * (H + N), flops=2 * T * r * (H + N))
        return dict(bytes=2 * T * (N + H * (3 if case["base"] else 2)) + 4 * T * r
                    + 2 * k * r * (H + N) + 4 * case["n"] * r * (H + N),
                    flops=4 * T * r * (H + N))
    z, b, k = _SZ[case["stream"]], _SZ[case["branch"]], case["numel"]
    return dict(bytes=k * (z + b + (z if case["x"] else 0)), flops=3 * k)


def _exact_act(z, kind):
    if kind == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    if kind == "gelu":
        c = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        # 0.5 (1 + tanh u) = sigmoid(2 u)
        u = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        s = torch.sigmoid(u)
        return z * s, s + z * s * (1 - s) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z * z)
    return z.clamp(min=0), torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))


def _exact_ffn(st):
    c = st["case"]
    d = {key: t.double() for key, t in st.items() if isinstance(t, torch.Tensor)}
    if c["dir"] == "fwd":
        ag, au = torch.mm(d["x"], d["w_gate"]), torch.mm(d["x"], d["w_up"])
        y = torch.mm(_exact_act(ag, c["act"])[0] * au, d["w_down"])
        got = dict(y=y if "add" not in d else d["add"] + y)
        if c["save"]:
            got["a_gate"], got["a_up"] = ag, au
        return got
    f, df = _exact_act(d["a_gate"], c["act"])
    dh = torch.mm(d["dy"], d["w_down"].T)
    both = torch.cat([dh * d["a_up"] * df, dh * f], dim=1)
    dx = torch.mm(both, torch.cat([d["w_gate"], d["w_up"]], dim=1).T)
    dw = torch.mm(d["x"].T, both)
    return dict(dx=dx if "add" not in d else d["add"] + dx, dw_gate=dw[:, :c["F"]],
                dw_up=dw[:, c["F"]:], dw_down=torch.mm((f * d["a_up"]).T, d["dy"]))


def _exact_lora(st):
    """Adapter by adapter, on its own rows alone."""
    c = st["case"]
    T, r, back = c["T"], c["r"], c["dir"] == "bwd"
    x, a, b = st["x"].double(), st["a"].double(), st["b"].double()
    s = st["scales"]
    if back:
        dy, kept = st["dy"].double(), st["v"].double()
        out = torch.zeros_like(x)
        da, db = torch.zeros_like(a), torch.zeros_like(b)
    else:
        out = torch.zeros(T, c["N"], dtype=torch.float64, device=x.device)
        v = torch.zeros(T, r, dtype=torch.float64, device=x.device)
    for i in range(c["n"]):
        at = torch.nonzero(st["ids"] == i).flatten()
        f = 1.0 if s is None else float(s[i])
        if back:
            dv = f * torch.einsum("tn,rn->tr", dy[at], b[i])
            out[at] = torch.einsum("tr,rh->th", dv, a[i])
            da[i] = torch.einsum("tr,th->rh", dv, x[at])
            db[i] = f * torch.einsum("tr,tn->rn", kept[at], dy[at])
        else:
            v[at] = torch.einsum("th,rh->tr", x[at], a[i])
            out[at] = f * torch.einsum("tr,rn->tn", v[at], b[i])
    if st["base"] is not None:
        out += st["base"].double()
    return dict(dx=out, da=da, db=db) if back else dict(out=out, v=v)


def _exact_kept(numel, seed, at, threshold):
    """Which elements stay, with the generator in unsigned numpy arithmetic."""
    u = np.uint64
    mask, half = u(0xFFFFFFFF), u(32)
    n = (numel + 7) // 8
    ctr = np.zeros((4, n), dtype=np.uint64)
    ctr[0] = np.arange(n, dtype=np.uint64) & mask
    ctr[1] = np.arange(n, dtype=np.uint64) >> half
    ctr[2], ctr[3] = u(at) & mask, u(at) >> half
    for i in range(10):
        k0 = u((seed + i * _KEY[0]) & _LOW)
        k1 = u(((seed >> 32) + i * _KEY[1]) & _LOW)
        p, q = ctr[0] * u(_MUL[0]), ctr[2] * u(_MUL[1])
        ctr = np.stack([(q >> half) ^ ctr[1] ^ k0, q & mask, (p >> half) ^ ctr[3] ^ k1, p & mask])
    parts = np.stack([ctr & u(0xFFFF), ctr >> u(16)], axis=1)      # word, half, block
    return parts.transpose(2, 0, 1).reshape(-1)[:numel] >= threshold


def _exact_drop(st):
    c = st["case"]
    t = _threshold(c["p"])
    seed, at = (int(v) for v in st["rng"].tolist())
    keep = torch.from_numpy(_exact_kept(c["numel"], seed, at, t)).cuda()
    f = c["b"] * 65536 / (65536 - t)
    if c["dir"] == "fwd":
        out = f * st["y"].double() * keep
        return dict(out=out if st["x"] is None else out + c["a"] * st["x"].double())
    d = st["d_out"].double()
    got = dict(dy=f * d * keep)
    if c["x"]:
        got["dx"] = c["a"] * d
    return got


def exact(case, seed):
    st = prepare(case, seed)
    return {"ffn": _exact_ffn, "lora": _exact_lora, "drop": _exact_drop}[case["op"]](st)
