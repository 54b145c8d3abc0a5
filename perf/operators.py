"""Cases of the operators around the expert block: the balanced gate, the
norms before and after the block, and the clip of all gradients by one norm.

With own false, run() computes the plain forms in elementary torch
operations; with own true it calls the library."""
import math

import numpy as np
import torch

own = False

F32MAX = 3.4028234663852886e38


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoding step of 32 sequences through a fine-grained gate: latency
        dict(name="gate_step", op="gate", dir="fwd", T=32, E=256, k=8, dtype="f32", score="sigmoid",
             bias=True, n_group=8, topk_group=4, group_topk=2, renorm=True, scale=2.5),
        # the prefill of the skewed workload, logits as a bf16 projection leaves them
        dict(name="gate_prefill", op="gate", dir="fwd", T=8192, E=128, k=8, dtype="bf16",
             score="softmax", bias=False, n_group=1, topk_group=1, group_topk=1, renorm=True,
             scale=1.0),
        # a large training batch on a fine-grained gate with groups and a balance bias
        dict(name="gate_train", op="gate", dir="fwd", T=65536, E=256, k=8, dtype="f32",
             score="sigmoid", bias=True, n_group=8, topk_group=4, group_topk=2, renorm=True,
             scale=2.5),
        # the gradient of softmax weights that are not renormalised: dense over the experts
        dict(name="gate_grad", op="gate", dir="bwd", T=16384, E=64, k=6, dtype="f32",
             score="softmax", bias=True, n_group=1, topk_group=1, group_topk=1, renorm=False,
             scale=1.0),
        # one token of one sequence between two blocks: latency
        dict(name="norm_step", op="norm", dir="fwd", T=1, H=7168, stream="bf16", weights="bf16",
             post=True, gates=0, nxt=True, a=1.0, b=1.0),
        # the prefill of the Mixtral-shaped workload with a gate for each channel
        dict(name="norm_prefill", op="norm", dir="fwd", T=4096, H=4096, stream="bf16",
             weights="bf16", post=True, gates=1, nxt=True, a=1.0, b=1.0),
        # three sequences of odd length, a gate row each, scaled residual
        dict(name="norm_ragged_grad", op="norm", dir="bwd", T=4083, H=2048, stream="bf16",
             weights="f32", post=True, gates=3, nxt=True, a=0.5, b=2.0),
        # the training step of the widest workload with a float residual stream
        dict(name="norm_train_grad", op="norm", dir="bwd", T=16384, H=7168, stream="f32",
             weights="f32", post=True, gates=1, nxt=True, a=1.0, b=1.0),
        # the router's and the norms' gradients alone (experts frozen): latency
        dict(name="clip_router", op="clip", sizes="given", n0=4096, n1=4096, n2=32768, n3=4096,
             dtype="f32", kind="l2", max_norm=1.0),
        # the tiny block's three weight gradients
        dict(name="clip_tiny", op="clip", sizes="given", n0=4194304, n1=4194304, n2=4194304, n3=0,
             dtype="f32", kind="l2", max_norm=1.0),
        # a flat bf16 bucket of 300 parameters of any size, packed without padding
        dict(name="clip_bucket", op="clip", sizes="ragged", count=300, total=50331653,
             dtype="bf16", kind="l2", max_norm=1.0),
        # the Mixtral-shaped training step's weight gradients, 5.6 GB
        dict(name="clip_train", op="clip", sizes="given", n0=469762048, n1=469762048,
             n2=469762048, n3=32768, dtype="f32", kind="l2", max_norm=1.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gate", "gate", "norm", "norm", "clip"])
    if op == "gate":
        E = rng.choice([8, 16, 24, 40, 60, 64, 72, 128, 160, 256, 384])
        k = rng.randint(1, min(8, E))
        n_group = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0 and E // g >= 2])
        need = -(-k // (E // n_group))
        return dict(op="gate", dir=rng.choice(["fwd", "fwd", "bwd"]),
                    T=_log_int(rng, 1, 65536 * 256 // max(E, 256)), E=E, k=k,
                    dtype=rng.choice(["f32", "bf16"]), score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.6, n_group=n_group,
                    topk_group=rng.randint(need, n_group), group_topk=rng.choice([1, 2]),
                    renorm=rng.random() < 0.6, scale=rng.choice([1.0, 1.0, 2.5, 16.0]))
    if op == "norm":
        H = rng.choice([512, 1024, 2048, 2560, 4096, 5120, 7168, 1000, 333])
        post = rng.random() < 0.7
        T = _log_int(rng, 1, 16384)
        gates = rng.choice([0, 1, 1, rng.choice([d for d in range(1, 65) if T % d == 0])])
        return dict(op="norm", dir=rng.choice(["fwd", "bwd"]), T=T, H=H,
                    stream=rng.choice(["bf16", "f32"]), weights=rng.choice(["bf16", "f32"]),
                    post=post, gates=gates, nxt=rng.random() < 0.8,
                    a=rng.choice([1.0, 1.0, 0.5, 1.25]), b=rng.choice([1.0, 1.0, 0.7]))
    return dict(op="clip", sizes="ragged", count=_log_int(rng, 1, 400),
                total=_log_int(rng, 5000, 300000000), dtype=rng.choice(["f32", "bf16"]),
                kind=rng.choice(["l2", "l2", "inf"]), max_norm=rng.choice([1.0, 0.25]))


_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SZ = {"f32": 4, "bf16": 2}


def _numels(case):
    """Element counts of the tensors of a clip case."""
    if case["sizes"] == "given":
        return [case[key] for key in ("n0", "n1", "n2", "n3") if case[key]]
    r = np.random.RandomState(case["count"] + 7)
    cuts = np.exp(r.uniform(0.0, math.log(1000.0), case["count"]))
    n = np.maximum(1, np.floor(cuts / cuts.sum() * (case["total"] - case["count"]))).astype(np.int64)
    n[-1] += max(0, case["total"] - int(n.sum()))
    return [int(v) for v in n]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, sd=1.0, mean=0.0, dt=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * sd + mean).to(dt)

    s = dict(case=case)
    if case["op"] == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        # some experts are more popular than others, as in training; the bias leans against it
        lean = randn(E, sd=0.5)
        s["logits"] = (randn(T, E) + lean).to(_DT[case["dtype"]])
        s["bias"] = (-0.1 * lean + randn(E, sd=0.02)) if case["bias"] else None
        if case["dir"] == "bwd":
            # the choice that the forward made on these logits, and the block's gradient
            s["ids"] = _plain_gate(s)[0]
            s["dprobs"] = randn(T, k, sd=0.02)
            s["dlogits"] = torch.empty_like(s["logits"])
        else:
            s["ids_out"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
            s["probs_out"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
            s["counts_out"] = torch.empty(E, dtype=torch.int32, device="cuda")
            s["offsets_out"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        return s
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        st, wt = _DT[case["stream"]], _DT[case["weights"]]
        s["x"] = randn(T, H, dt=st)
        s["y"] = randn(T, H, sd=0.4, dt=torch.bfloat16)
        s["w_post"] = randn(H, sd=0.1, mean=1.0, dt=wt) if case["post"] else None
        s["gate"] = randn(case["gates"], H, sd=0.2, mean=0.5, dt=wt) if case["gates"] else None
        s["w_next"] = randn(H, sd=0.1, mean=1.0, dt=wt) if case["nxt"] else None
        if case["dir"] == "bwd":
            # what the forward kept, and the gradients that reach its two results
            f = _plain_norm(s)
            s["out"], s["rstd_y"], s["rstd_out"] = f["out"], f.get("rstd_y"), f.get("rstd_out")
            s["d_out"] = randn(T, H, sd=0.01, dt=st)
            s["d_n"] = randn(T, H, sd=0.01, dt=torch.bfloat16) if case["nxt"] else None
            s["x"] = None
            s["dx"], s["dy"] = torch.empty_like(s["d_out"]), torch.empty_like(s["y"])
        else:
            s["out_out"] = torch.empty_like(s["x"])
            s["n_out"] = torch.empty_like(s["y"]) if case["nxt"] else None
        return s
    numels = _numels(case)
    dt = _DT[case["dtype"]]
    # gradients of different size from tensor to tensor, as layers have them
    flat = torch.empty(sum(numels), dtype=dt, device="cuda")
    out = torch.empty_like(flat)
    scale = torch.exp(torch.randn(len(numels), generator=g, device="cuda") - 4.0).tolist()
    at, s["grads"], s["outs"] = 0, [], []
    for n, sd in zip(numels, scale):
        flat[at:at + n].normal_(0.0, sd, generator=g)
        s["grads"].append(flat[at:at + n])
        s["outs"].append(out[at:at + n])
        at += n
    s["out_flat"] = out
    return s


# ------------------------------------------------------------------ plain forms

def _plain_scores(logits, score):
    """(logits as ranked, scores), both in 64 bits: two scores may lie next to each other."""
    l = logits.double()
    l = torch.where(torch.isnan(l), torch.full_like(l, -math.inf), l).clamp(max=F32MAX)
    if score == "sigmoid":
        return l, 1.0 / (1.0 + torch.exp(-l))
    m = l.max(dim=1, keepdim=True).values
    e = torch.exp(l - torch.where(m == -math.inf, torch.zeros_like(m), m))
    t = e.sum(dim=1, keepdim=True)
    return l, e / torch.where(t > 0, t, torch.ones_like(t))


def _plain_weights(l, s, case, ids, bias):
    """The chosen experts' scores and weights before the scale; bias: the chosen experts' or None."""
    sj, lj = s.gather(1, ids), l.gather(1, ids)
    ok = lj > -math.inf
    if bias is not None:
        ok = ok & (bias > -math.inf)
    sj = torch.where(ok, sj, torch.zeros_like(sj))
    if not case["renorm"]:
        return sj, sj
    if case["score"] == "softmax":
        lj = torch.where(ok, lj, torch.full_like(lj, -math.inf))
        m = lj.max(dim=1, keepdim=True).values
        w = torch.exp(lj - torch.where(m == -math.inf, torch.zeros_like(m), m))
    else:
        w = sj
    t = w.sum(dim=1, keepdim=True)
    return sj, w / torch.where(t > 0, t, torch.ones_like(t))


def _plain_gate(st):
    c = st["case"]
    T, E, k = c["T"], c["E"], c["k"]
    l, s = _plain_scores(st["logits"], c["score"])
    bias = st["bias"]
    v = s if bias is None else s + bias.double()
    v = v.masked_fill(l == -math.inf, -math.inf)
    rank = l if bias is None else v
    if c["n_group"] > 1:
        size = E // c["n_group"]
        best = v.view(T, c["n_group"], size).sort(dim=2, descending=True).values
        groups = best[:, :, :c["group_topk"]].clone()
        groups[:, :, 1:].masked_fill_(groups[:, :, 1:] == -math.inf, 0.0)
        groups = groups.sum(dim=2)
        kept = groups.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        keep = torch.zeros((T, c["n_group"]), dtype=torch.bool, device=l.device)
        keep.scatter_(1, kept, True)
        # what is masked ranks last, and before what its group excludes
        rank = rank.masked_fill(rank == -math.inf, -1e308)
        rank = rank.masked_fill(~keep.repeat_interleave(size, dim=1), -math.inf)
    ids = rank.sort(dim=1, descending=True, stable=True).indices[:, :k]
    _, w = _plain_weights(l, s, c, ids, None if bias is None else bias[ids])
    counts = torch.bincount(ids.reshape(-1), minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return (ids.to(torch.int32), (c["scale"] * w).float(), counts.to(torch.int32),
            offsets.to(torch.int32))


def _plain_gate_grad(st):
    c = st["case"]
    ids, dp = st["ids"].long(), st["dprobs"].double()
    l, s = _plain_scores(st["logits"], c["score"])
    sj, w = _plain_weights(l, s, c, ids, None if st["bias"] is None else st["bias"][ids])
    d = (dp * w).sum(dim=1, keepdim=True)
    if c["score"] == "sigmoid":
        far = 1.0 / (1.0 + torch.exp(l.gather(1, ids)))
        gj = w * far * (dp - d) if c["renorm"] else sj * far * dp
        grad = torch.zeros_like(l).scatter_(1, ids, gj)
    elif c["renorm"]:
        grad = torch.zeros_like(l).scatter_(1, ids, w * (dp - d))
    else:
        grad = (-s * d).scatter_add(1, ids, sj * dp)
    return (c["scale"] * grad).to(st["logits"].dtype)


EPS = 1e-6


def _rows(gate, T):
    """The gate of every token, or 1."""
    return 1.0 if gate is None else gate.float().repeat_interleave(T // gate.shape[0], dim=0)


def _plain_norm(st):
    c, x, y = st["case"], st["x"].float(), st["y"].float()
    got = {}
    z = y
    if st["w_post"] is not None:
        ry = torch.rsqrt(y.square().mean(dim=1) + EPS)
        z = y * ry[:, None] * st["w_post"].float()
        got["rstd_y"] = ry
    out = c["a"] * x + c["b"] * _rows(st["gate"], c["T"]) * z
    got["out"] = out.to(st["x"].dtype)
    if st["w_next"] is not None:
        ro = torch.rsqrt(out.square().mean(dim=1) + EPS)
        got["n"] = (out * ro[:, None] * st["w_next"].float()).to(torch.bfloat16)
        got["rstd_out"] = ro
    return got


def _plain_norm_grad(st):
    c = st["case"]
    T, H = c["T"], c["H"]
    D, y = st["d_out"].float(), st["y"].float()
    got = {}
    if st["w_next"] is not None:
        dn, oh = st["d_n"].float(), st["out"].float() * st["rstd_out"][:, None]
        q = dn * st["w_next"].float()
        D = D + st["rstd_out"][:, None] * (q - oh * (q * oh).mean(dim=1, keepdim=True))
        got["dw_next"] = (dn * oh).sum(dim=0)
    got["dx"] = (c["a"] * D).to(st["d_out"].dtype)
    yh = y if st["w_post"] is None else y * st["rstd_y"][:, None]
    w = 1.0 if st["w_post"] is None else st["w_post"].float()
    if st["gate"] is not None:
        G = st["gate"].shape[0]
        got["dgate"] = (c["b"] * D * yh * w).view(G, T // G, H).sum(dim=1)
    q = c["b"] * D * _rows(st["gate"], T)
    if st["w_post"] is not None:
        got["dw_post"] = (q * yh).sum(dim=0)
        q = q * w
        q = st["rstd_y"][:, None] * (q - yh * (q * yh).mean(dim=1, keepdim=True))
    got["dy"] = q.to(torch.bfloat16)
    return got


def _plain_clip(st):
    c = st["case"]
    if c["kind"] == "inf":
        norm = torch.stack([g.float().abs().max() for g in st["grads"]]).max().double()
    else:
        norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in st["grads"]]).sum().sqrt()
    coef = (c["max_norm"] / (norm + EPS)).clamp(max=1.0)
    outs = [(g.float() * coef.float()).to(g.dtype) for g in st["grads"]]
    return dict(norm=norm.float().reshape(1), coef=coef.float().reshape(1), out=torch.cat(outs))


# ------------------------------------------------------------------ one pass

def run(state):
    c = state["case"]
    if not own:
        if c["op"] == "gate":
            return _plain_gate(state) if c["dir"] == "fwd" else [_plain_gate_grad(state)]
        if c["op"] == "norm":
            return _plain_norm(state) if c["dir"] == "fwd" else _plain_norm_grad(state)
        return _plain_clip(state)
    import moe_expert_dispatch_gb300 as m
    if c["op"] == "gate":
        how = dict(bias=state["bias"], score=c["score"], renormalise=c["renorm"],
                   scale=c["scale"])
        if c["dir"] == "bwd":
            return [m.moe_route_gate_backward(state["dprobs"], state["logits"], state["ids"],
                                              dlogits=state["dlogits"], **how)]
        return m.moe_route_gate(state["logits"], c["k"], n_group=c["n_group"],
                                topk_group=c["topk_group"], group_topk=c["group_topk"],
                                expert_ids=state["ids_out"], probs=state["probs_out"],
                                counts=state["counts_out"], offsets=state["offsets_out"], **how)
    if c["op"] == "norm":
        how = dict(w_post=state["w_post"], gate=state["gate"], w_next=state["w_next"], eps=EPS,
                   residual_scale=c["a"], branch_scale=c["b"])
        if c["dir"] == "fwd":
            got = m.moe_norm_residual(state["x"], state["y"], out=state["out_out"],
                                      n=state["n_out"], **how)
        else:
            got = m.moe_norm_residual_backward(state["d_out"], state["d_n"], state["out"],
                                               state["y"], rstd_y=state["rstd_y"],
                                               rstd_out=state["rstd_out"], dx=state["dx"],
                                               dy=state["dy"], **how)
        return {key: t for key, t in got.items() if t is not None}
    norm, coef = m.moe_clip_grad_norm(state["grads"], c["max_norm"], out=state["outs"],
                                      norm_type=2.0 if c["kind"] == "l2" else math.inf, eps=EPS)
    return dict(norm=norm, coef=coef, out=state["out_flat"])


# ------------------------------------------------------------------ work and the answers in 64 bits

def work(case):
    if case["op"] == "gate":
        T, E, k, z = case["T"], case["E"], case["k"], _SZ[case["dtype"]]
        if case["dir"] == "bwd":
            return dict(bytes=2 * T * E * z + T * k * 8 + (E * 4 if case["bias"] else 0),
                        flops=8 * T * E)
        return dict(bytes=T * E * z + T * k * 8 + E * 8 + 4 + (E * 4 if case["bias"] else 0),
                    flops=8 * T * E)
    if case["op"] == "norm":
        T, H, z, wz = case["T"], case["H"], _SZ[case["stream"]], _SZ[case["weights"]]
        params = (int(case["post"]) + int(case["nxt"]) + case["gates"]) * H
        stats = 4 * T * (int(case["post"]) + int(case["nxt"]))
        if case["dir"] == "fwd":
            per = 2 * z + 2 + (2 if case["nxt"] else 0)
            return dict(bytes=T * H * per + params * wz + stats, flops=8 * T * H)
        per = 2 * z + 4 + ((z + 2) if case["nxt"] else 0)
        return dict(bytes=T * H * per + params * (wz + 4) + stats, flops=20 * T * H)
    n = sum(_numels(case))
    return dict(bytes=2 * n * _SZ[case["dtype"]], flops=3 * n)


def _exact_gate(st):
    """From the definition, by rounds of the largest remaining value."""
    c = st["case"]
    T, E, k = c["T"], c["E"], c["k"]
    l = st["logits"].double().cpu().numpy().copy()
    l[np.isnan(l)] = -np.inf
    l = np.minimum(l, F32MAX)
    with np.errstate(over="ignore"):
        if c["score"] == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-l))
        else:
            s = np.exp(l - l.max(axis=1, keepdims=True))
            s /= s.sum(axis=1, keepdims=True)
    b = None if st["bias"] is None else st["bias"].double().cpu().numpy()
    rows = np.arange(T)
    if c["dir"] == "bwd":
        ids = st["ids"].cpu().numpy().astype(np.int64)
    else:
        v = s if b is None else s + b[None, :]
        rank = (l if b is None else v).copy()
        if c["n_group"] > 1:
            size = E // c["n_group"]
            vg = v.reshape(T, c["n_group"], size).copy()
            score = np.zeros((T, c["n_group"]))
            for _ in range(c["group_topk"]):
                at = vg.argmax(axis=2)
                score += np.take_along_axis(vg, at[:, :, None], 2)[:, :, 0]
                np.put_along_axis(vg, at[:, :, None], -np.inf, 2)
            out = np.ones((T, c["n_group"]), dtype=bool)
            for _ in range(c["topk_group"]):
                at = score.argmax(axis=1)
                out[rows, at] = False
                score[rows, at] = -np.inf
            rank[np.repeat(out, size, axis=1)] = -np.inf
        ids = np.empty((T, k), dtype=np.int64)
        for j in range(k):
            ids[:, j] = rank.argmax(axis=1)
            rank[rows, ids[:, j]] = -np.inf
    sj = np.take_along_axis(s, ids, 1)
    w = sj / sj.sum(axis=1, keepdims=True) if c["renorm"] else sj
    if c["dir"] == "fwd":
        counts = np.bincount(ids.reshape(-1), minlength=E)
        return [ids.astype(np.int32), c["scale"] * w, counts.astype(np.int32),
                np.concatenate([[0], counts.cumsum()]).astype(np.int32)]
    # d(weights)/d(scores), then d(scores)/d(logits)
    dp = st["dprobs"].double().cpu().numpy() * c["scale"]
    ds = dp
    if c["renorm"]:
        ds = (dp - (dp * w).sum(axis=1, keepdims=True)) / sj.sum(axis=1, keepdims=True)
    dense = np.zeros((T, E))
    np.put_along_axis(dense, ids, ds, 1)
    if c["score"] == "sigmoid":
        return [dense * s * (1.0 - s)]
    return [s * (dense - (dense * s).sum(axis=1, keepdims=True))]


def _exact_norm(st):
    c = st["case"]
    T, H = c["T"], c["H"]
    d = lambda t: None if t is None else t.double()  # noqa: E731
    y, wp, wn = d(st["y"]), d(st["w_post"]), d(st["w_next"])
    g = None if st["gate"] is None else d(st["gate"])[torch.arange(T, device=y.device)
                                                      // (T // st["gate"].shape[0])]
    got = {}
    if c["dir"] == "fwd":
        z = y
        if wp is not None:
            got["rstd_y"] = 1.0 / torch.sqrt((y * y).mean(dim=1) + EPS)
            z = wp * (y * got["rstd_y"].unsqueeze(1))
        if g is not None:
            z = z * g
        out = c["a"] * d(st["x"]) + c["b"] * z
        got["out"] = out
        if wn is not None:
            got["rstd_out"] = 1.0 / torch.sqrt((out * out).mean(dim=1) + EPS)
            got["n"] = wn * (out * got["rstd_out"].unsqueeze(1))
        return got
    D = d(st["d_out"])
    if wn is not None:
        r = d(st["rstd_out"]).unsqueeze(1)
        o, dn = d(st["out"]), d(st["d_n"])
        t = ((dn * wn) * o).sum(dim=1, keepdim=True)
        D = D + r * dn * wn - o * (r ** 3) * t / H
        got["dw_next"] = (dn * o * r).sum(dim=0)
    got["dx"] = c["a"] * D
    D = c["b"] * D
    r = 1.0 if wp is None else d(st["rstd_y"]).unsqueeze(1)
    u = y * r if wp is None else wp * y * r
    if g is not None:
        G = c["gates"]
        got["dgate"] = torch.stack([p.sum(dim=0) for p in (D * u).split(T // G)])
        D = D * g
    if wp is None:
        got["dy"] = D
    else:
        got["dw_post"] = (D * y * r).sum(dim=0)
        t = ((D * wp) * y).sum(dim=1, keepdim=True)
        got["dy"] = r * D * wp - y * (r ** 3) * t / H
    return got


def _exact_clip(st):
    c = st["case"]
    if c["kind"] == "inf":
        norm = max(float(g.abs().max().double()) for g in st["grads"])
    else:
        norm = math.sqrt(math.fsum(float((g.double() ** 2).sum()) for g in st["grads"]))
    coef = min(1.0, c["max_norm"] / (norm + EPS))
    out = torch.cat([g.double() * coef for g in st["grads"]])
    return dict(norm=np.array([norm]), coef=np.array([coef]), out=out)


def exact(case, seed):
    st = prepare(case, seed)
    return {"gate": _exact_gate, "norm": _exact_norm, "clip": _exact_clip}[case["op"]](st)
