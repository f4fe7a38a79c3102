"""The operators that train a DeepSeekMoE layer, as measured cases: the grouped
gated feed-forward block that keeps its pre-activations and its backward pass,
the router's backward pass, and the global gradient norm with clipping.

Each case is one call sequence of a training step on one GPU. With `own` set,
run() makes the package's calls; otherwise it computes the same from elementary
torch operations in 32 bits (64 for the norm's long sum), rounded once."""
import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"
_T = {BF16: torch.bfloat16, F32: torch.float32}


def listed():
    return [
        # one of 8 expert-parallel ranks of the V3-shaped layer: 32 experts, 4096 tokens' share of the rows twice over
        dict(name="fwd_v3_ep8", op="fwd", E=32, rows=8192, d=7168, F=2048, dtype=BF16, skew=0.3),
        # the 2B-scale layer on one GPU: 8192 tokens, 7 of 63 experts each
        dict(name="fwd_2b", op="fwd", E=63, rows=57344, d=1280, F=896, dtype=BF16, skew=0.3),
        dict(name="bwd_v3_ep8", op="bwd", E=32, rows=8192, d=7168, F=2048, dtype=BF16, skew=0.3),
        dict(name="bwd_2b", op="bwd", E=63, rows=57344, d=1280, F=896, dtype=BF16, skew=0.3),
        # the V3-shaped layer's shared expert: one dense block over all 4096 tokens, no gate
        dict(name="bwd_shared_v3", op="bwd", E=1, rows=4096, d=7168, F=2048, dtype=BF16, skew=0.0),
        # a handful of rows spread over 16 experts, most of them empty: launch latency and weight traffic
        dict(name="bwd_few_rows", op="bwd", E=16, rows=37, d=1280, F=896, dtype=BF16, skew=1.5),
        # the GShard toy layer in fp32: 256 tokens, 2 of 16 experts each
        dict(name="bwd_toy_f32", op="bwd", E=16, rows=512, d=256, F=512, dtype=F32, skew=0.3),
        # the V3-shaped router: sigmoid scores, gates normalised over the selection
        dict(name="route_v3", op="route", T=4096, N=256, k=8, d=7168, score="sigmoid", normalize=True, scale=2.5,
             dtype=BF16),
        # the 2B-scale router: plain softmax gates, so every logit has a gradient; N is odd
        dict(name="route_2b", op="route", T=8192, N=63, k=7, d=1280, score="softmax", normalize=False, scale=1.0,
             dtype=BF16),
        # clipping the bf16 gradients of 32 V3 experts into the optimizer's buffers
        dict(name="clip_v3_ep8", op="clip", tensors=96, total=32 * 3 * 7168 * 2048, spread=0.0, dtype=BF16,
             inplace=False, ratio=0.3),
        # the 2B-scale layer's fp32 gradients in place, the norm below the limit: nothing is rewritten
        dict(name="clip_2b_f32", op="clip", tensors=190, total=63 * 3 * 1280 * 896, spread=0.0, dtype=F32,
             inplace=True, ratio=4.0),
        # many small tensors of uneven sizes at odd offsets of one bucket
        dict(name="clip_small", op="clip", tensors=300, total=2_000_003, spread=2.0, dtype=F32, inplace=False,
             ratio=0.5),
    ]


def _log(rng, lo, hi, mult=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(mult, int(round(v / mult)) * mult)


def draw(rng):
    op = rng.choice(["fwd", "bwd", "bwd", "route", "clip"])
    if op in ("fwd", "bwd"):
        dtype = BF16 if rng.random() < 0.8 else F32
        E = _log(rng, 1, 64)
        d, F = _log(rng, 64, 7168, 8), _log(rng, 64, 4096, 8)
        rows = _log(rng, 1, 57344)
        # no dearer than the largest listed cases: weights, rows and products
        E = max(1, min(E, 32 * 7168 * 2048 // (d * F)))
        top = 8192 * 7168 * 2048 if dtype == BF16 else 1 << 32
        rows = max(1, min(rows, top // (d * F), 57344 * 1280 // max(d, F)))
        return dict(op=op, E=E, rows=rows, d=d, F=F, dtype=dtype, skew=round(rng.uniform(0, 0.8), 3))
    if op == "route":
        N = _log(rng, 4, 512)
        d = _log(rng, 64, 7168, 8)
        T = max(1, min(_log(rng, 1, 16384), 4096 * 7168 * 256 // (d * N), 4096 * 7168 // d))
        dtype = BF16 if rng.random() < 0.8 else F32
        if dtype == F32:
            T = max(1, min(T, (1 << 31) // (d * N)))
        return dict(op=op, T=T, N=N, k=rng.randint(2, min(16, N)), d=d, score=rng.choice(["sigmoid", "softmax"]),
                    normalize=rng.random() < 0.5, scale=round(rng.uniform(0.5, 3.0), 3), dtype=dtype)
    return dict(op=op, tensors=_log(rng, 1, 400), total=_log(rng, 1000, 32 * 3 * 7168 * 1024),
                spread=round(rng.uniform(0, 2.5), 3), dtype=rng.choice([BF16, F32]), inplace=rng.random() < 0.3,
                ratio=round(math.exp(rng.uniform(math.log(0.05), math.log(5.0))), 4))


# ------------------------------------------------------------------- inputs --


def _normal(gen, shape, std, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _counts(gen, E, rows, skew):
    """Rows of each group: a draw of every row's group from uneven loads."""
    p = torch.exp(skew * torch.randn(E, generator=gen, device="cuda", dtype=torch.float64))
    pick = torch.multinomial((p / p.sum()).float(), rows, replacement=True, generator=gen)
    return torch.bincount(pick, minlength=E).to(torch.int32)


def _sizes(case):
    """The tensors' sizes, all positive: even, or uneven by `spread`. They belong to the model, not to the inputs."""
    rng = random.Random("%(tensors)d %(total)d" % case)
    w = [math.exp(case["spread"] * rng.gauss(0, 1)) for _ in range(case["tensors"])]
    return [max(1, int(v / sum(w) * case["total"])) for v in w]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _T[case["dtype"]]
    st = {"case": case}
    if case["op"] in ("fwd", "bwd"):
        E, R, d, F = case["E"], case["rows"], case["d"], case["F"]
        st["counts"] = _counts(gen, E, R, case["skew"])
        st["x"] = _normal(gen, (R, d), 1.0, dt)
        st["W1"] = _normal(gen, (E, F, d), d ** -0.5, dt)
        st["W3"] = _normal(gen, (E, F, d), d ** -0.5, dt)
        st["W2"] = _normal(gen, (E, d, F), F ** -0.5, dt)
        # a dense block has no gate; routed rows carry theirs
        st["gate"] = None if E == 1 else torch.rand(R, generator=gen, device="cuda") * 0.6 + 0.02
        if case["op"] == "bwd":
            st["gu"] = _normal(gen, (R, 2 * F), 1.0, dt)  # unit pre-activations, as x and W give them
            st["dy"] = _normal(gen, (R, d), 1e-3, dt)
    elif case["op"] == "route":
        T, N, k, d = case["T"], case["N"], case["k"], case["d"]
        st["x"] = _normal(gen, (T, d), 1.0, dt)
        st["W_r"] = _normal(gen, (N, d), d ** -0.5, dt)
        st["logits"] = _normal(gen, (T, N), 1.0, torch.float32)
        st["idx"] = torch.topk(st["logits"], k, dim=1).indices.to(torch.int32)
        st["dgates"] = _normal(gen, (T, k), 1e-2, torch.float32)
    else:
        sizes = _sizes(case)
        n = sum(sizes)
        st["flat"] = _normal(gen, (n,), 1e-3, dt)
        st["src"] = list(torch.split(st["flat"], sizes))
        if case["inplace"] and case["ratio"] < 1.5:
            # a clip in place changes its input: such a case writes to other buffers
            st["out"] = torch.empty_like(st["flat"])
        else:
            st["out"] = st["flat"] if case["inplace"] else torch.empty_like(st["flat"])
        st["dst"] = list(torch.split(st["out"], sizes))
        st["max_norm"] = case["ratio"] * 1e-3 * math.sqrt(n)
    return st


# ------------------------------------------------------------- plain forms --


def _groups(st):
    """(index of each row in the padded groups, E, rows of the largest group)."""
    E, R = st["case"]["E"], st["case"]["rows"]
    c = st["counts"].long()
    start = torch.cumsum(c, 0) - c
    g = torch.repeat_interleave(torch.arange(E, device=c.device), c, output_size=R)
    m = int(c.max())
    return g * m + (torch.arange(R, device=c.device) - start[g]), E, m


def _pad(rows, at, E, m):
    out = torch.zeros((E * m, rows.shape[1]), dtype=torch.float32, device=rows.device)
    out[at] = rows.float()
    return out.view(E, m, rows.shape[1])


def _plain_fwd(st):
    dt = st["x"].dtype
    at, E, m = _groups(st)
    xp = _pad(st["x"], at, E, m)
    g = torch.bmm(xp, st["W1"].float().transpose(1, 2))
    u = torch.bmm(xp, st["W3"].float().transpose(1, 2))
    h = g * (1.0 / (1.0 + torch.exp(-g))) * u
    y = torch.bmm(h, st["W2"].float().transpose(1, 2)).flatten(0, 1)[at]
    if st["gate"] is not None:
        y = y * st["gate"][:, None]
    gu = torch.cat([g.flatten(0, 1)[at], u.flatten(0, 1)[at]], dim=1)
    return {"y": y.to(dt), "gu": gu.to(dt)}


def _plain_bwd(st):
    dt, F = st["x"].dtype, st["case"]["F"]
    at, E, m = _groups(st)
    dyp = _pad(st["dy"], at, E, m)
    q = torch.bmm(dyp, st["W2"].float()).flatten(0, 1)[at]
    g, u = st["gu"][:, :F].float(), st["gu"][:, F:].float()
    s = 1.0 / (1.0 + torch.exp(-g))
    h = g * s * u
    gate = 1.0 if st["gate"] is None else st["gate"][:, None]
    dh = q * gate
    dgp = _pad(dh * u * s * (1.0 + g * (1.0 - s)), at, E, m)
    dup = _pad(dh * (g * s), at, E, m)
    xp = _pad(st["x"], at, E, m)
    dx = (torch.bmm(dgp, st["W1"].float()) + torch.bmm(dup, st["W3"].float())).flatten(0, 1)[at]
    out = {"dx": dx.to(dt)}
    out["dW1"] = torch.bmm(dgp.transpose(1, 2), xp).to(dt)
    out["dW3"] = torch.bmm(dup.transpose(1, 2), xp).to(dt)
    out["dW2"] = torch.bmm(dyp.transpose(1, 2), _pad(h * gate, at, E, m)).to(dt)
    if st["gate"] is not None:
        out["dgate"] = (q * h).sum(dim=1)
    return out


def _plain_route(st):
    c, dt, z, idx = st["case"], st["x"].dtype, st["logits"], st["idx"].long()
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-z))
    else:
        p = torch.exp(z - z.max(dim=1, keepdim=True).values)
        s = p / p.sum(dim=1, keepdim=True)
    dG, sel = st["dgates"], s.gather(1, idx)
    if c["normalize"]:
        Z = sel.sum(dim=1, keepdim=True)
        dsel = c["scale"] / Z * (dG - (dG * sel).sum(dim=1, keepdim=True) / Z)
    else:
        dsel = c["scale"] * dG
    ds = torch.zeros_like(s).scatter_(1, idx, dsel)
    if c["score"] == "sigmoid":
        dz = ds * s * (1.0 - s)
    else:
        dz = s * (ds - (ds * s).sum(dim=1, keepdim=True))
    return {"dx": (dz @ st["W_r"].float()).to(dt), "dW_r": (dz.t() @ st["x"].float()).to(dt)}


def _plain_clip(st):
    g = torch.cat(st["src"])
    norm = torch.sqrt(g.double().square().sum())
    coef = torch.clamp(st["max_norm"] / norm, max=1.0)
    return {"norm": norm.float(), "grads": (g.float() * coef.float()).to(g.dtype)}


# --------------------------------------------------------- the framework's --


def _own_experts(st):
    import mixture_experts_layer_group_b200 as moe
    c, x = st["case"], st["x"]
    E, R, d, F = c["E"], c["rows"], c["d"], c["F"]
    if "cfg" not in st:  # what a program keeps between its steps: the configuration, the workspace and the outputs
        st["cfg"] = moe.make_cfg(d, F, E, 0, 1, dtype=c["dtype"])
        n = (moe.experts_workspace_size if c["op"] == "fwd" else moe.experts_backward_workspace_size)(st["cfg"], R)
        st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        if c["op"] == "fwd":
            st["res"] = {"y": torch.empty_like(x), "gu": torch.empty((R, 2 * F), dtype=x.dtype, device="cuda")}
        else:
            st["res"] = {"dx": torch.empty_like(x), "dW1": torch.empty_like(st["W1"]),
                         "dW3": torch.empty_like(st["W3"]), "dW2": torch.empty_like(st["W2"])}
            if st["gate"] is not None:
                st["res"]["dgate"] = torch.empty_like(st["gate"])
    r = st["res"]
    if c["op"] == "fwd":
        moe.experts_train(st["cfg"], R, st["counts"], x, st["gate"], st["W1"], st["W3"], st["W2"], r["y"], r["gu"],
                          st["ws"])
    else:
        moe.experts_backward(st["cfg"], R, st["counts"], x, st["gate"], st["W1"], st["W3"], st["W2"], st["gu"],
                             st["dy"], r["dx"], r.get("dgate"), r["dW1"], r["dW3"], r["dW2"], st["ws"])
    return r


def _own_route(st):
    import mixture_experts_layer_group_b200 as moe
    c = st["case"]
    if "cfg" not in st:
        st["cfg"] = moe.make_cfg(c["d"], 8, c["N"], 0, c["k"], score=c["score"], normalize=c["normalize"],
                                 route_scale=c["scale"], dtype=c["dtype"])
        st["ws"] = torch.empty(moe.route_backward_workspace_size(st["cfg"], c["T"]), dtype=torch.uint8, device="cuda")
        st["res"] = {"dx": torch.empty_like(st["x"]), "dW_r": torch.empty_like(st["W_r"])}
    r = st["res"]
    moe.route_backward(st["cfg"], c["T"], st["x"], st["W_r"], st["logits"], st["idx"], st["dgates"], None, r["dx"],
                       r["dW_r"], st["ws"])
    return r


def _own_clip(st):
    import mixture_experts_layer_group_b200 as moe
    if "list" not in st:
        st["list"] = moe.GradList(st["src"], st["dst"])
        st["ws"] = torch.empty(moe.grad_norm_workspace_size(st["list"]), dtype=torch.uint8, device="cuda")
        st["sumsq"] = torch.empty(1, dtype=torch.float64, device="cuda")
        st["norm"] = torch.empty(1, dtype=torch.float32, device="cuda")
    moe.grad_norm(st["list"], st["sumsq"], st["ws"])
    moe.grad_clip(st["list"], st["sumsq"], st["max_norm"], st["norm"])
    return {"norm": st["norm"][0], "grads": st["out"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return _own_experts(state) if op in ("fwd", "bwd") else _own_route(state) if op == "route" else _own_clip(state)
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "route": _plain_route, "clip": _plain_clip}[op](state)


# -------------------------------------------------------------- accounting --


def work(case):
    b = 2 if case["dtype"] == BF16 else 4
    if case["op"] in ("fwd", "bwd"):
        E, R, d, F = case["E"], case["rows"], case["d"], case["F"]
        w = 3 * min(E, R) * d * F * b
        if case["op"] == "fwd":
            return {"bytes": w + R * (2 * d + 2 * F) * b + 4 * R, "flops": 6 * R * d * F}
        return {"bytes": w + 3 * E * d * F * b + R * (3 * d + 2 * F) * b + 8 * R, "flops": 12 * R * d * F}
    if case["op"] == "route":
        T, N, k, d = case["T"], case["N"], case["k"], case["d"]
        return {"bytes": 2 * (T + N) * d * b + 4 * T * N + 8 * T * k, "flops": 4 * T * N * d}
    n = case["total"]
    return {"bytes": n * b * (1 if case["inplace"] and case["ratio"] >= 1.5 else 2), "flops": 3 * n}


# ------------------------------------------------------------------- exact --


def _exact_experts(case, st):
    """Each group by itself, in 64 bits."""
    E, R, d, F = case["E"], case["rows"], case["d"], case["F"]
    f = torch.float64
    new = lambda *shape: torch.zeros(shape, dtype=f, device="cuda")  # noqa: E731
    bwd = case["op"] == "bwd"
    out = {"dx": new(R, d), "dW1": new(E, F, d), "dW3": new(E, F, d), "dW2": new(E, d, F)} if bwd else \
        {"y": new(R, d), "gu": new(R, 2 * F)}
    if bwd and st["gate"] is not None:
        out["dgate"] = new(R)
    lo = 0
    for e, n in enumerate(st["counts"].tolist()):
        if n == 0:
            continue
        r = slice(lo, lo + n)
        lo += n
        x, A, B, C = st["x"][r].to(f), st["W1"][e].to(f), st["W3"][e].to(f), st["W2"][e].to(f)
        gate = torch.ones(n, 1, dtype=f, device="cuda") if st["gate"] is None else st["gate"][r].to(f)[:, None]
        if not bwd:
            g, u = x @ A.T, x @ B.T
            out["gu"][r] = torch.cat([g, u], 1)
            out["y"][r] = gate * ((g * torch.sigmoid(g) * u) @ C.T)
            continue
        g, u = st["gu"][r, :F].to(f), st["gu"][r, F:].to(f)
        dy = st["dy"][r].to(f)
        sg = torch.sigmoid(g)
        act = g * sg
        q = dy @ C
        if "dgate" in out:
            out["dgate"][r] = torch.einsum("rf,rf->r", q, act * u)
        dg = gate * q * u * (sg + act - act * sg)
        du = gate * q * act
        out["dx"][r] = dg @ A + du @ B
        out["dW1"][e], out["dW3"][e] = dg.T @ x, du.T @ x
        out["dW2"][e] = (gate * dy).T @ (act * u)
    return out


def _exact_route(case, st):
    """The gradient by the Jacobian of the gates with respect to each token's logits."""
    z, idx, dG = st["logits"].double(), st["idx"].long(), st["dgates"].double()
    T, N, k = case["T"], case["N"], case["k"]
    lead = torch.zeros(T, N, dtype=torch.float64, device="cuda").scatter_(1, idx, dG * case["scale"])
    chosen = torch.zeros(T, N, dtype=torch.bool, device="cuda").scatter_(1, idx, True)
    if case["score"] == "sigmoid":
        s = torch.sigmoid(z)
        slope = s * torch.sigmoid(-z)
    else:
        # normalised over the selection, a softmax gate is the softmax of the chosen logits alone
        s = torch.softmax(torch.where(chosen, z, -math.inf) if case["normalize"] else z, dim=1)
    if case["score"] == "softmax":
        dz = s * lead - s * torch.einsum("tn,tn->t", s, lead)[:, None]
    elif case["normalize"]:
        Z = torch.einsum("tn,tn->t", s, chosen.double())[:, None]
        mean = torch.einsum("tn,tn->t", s, lead)[:, None] / Z
        dz = torch.where(chosen, slope * (lead - mean) / Z, 0.0)
    else:
        dz = slope * lead
    return {"dx": dz @ st["W_r"].double(), "dW_r": dz.T @ st["x"].double()}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("fwd", "bwd"):
        return _exact_experts(case, st)
    if case["op"] == "route":
        return _exact_route(case, st)
    norm = torch.linalg.vector_norm(st["flat"], dtype=torch.float64)
    return {"norm": norm, "grads": st["flat"].double() * min(1.0, st["max_norm"] / float(norm))}
