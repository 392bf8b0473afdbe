"""Cases of the router's and the adapters' operators: their inputs, their plain forms in
elementary torch operations, the framework's calls, and what each cannot do without.

Three operators stand beside the layer's own products:

  route    scored routing: softmax or sigmoid scores, a selection bias, expert groups,
           top-k, renormalised and scaled weights; with its gradient
  router   the bf16 router projection, logits = x W^T, with dW and the term of dx
  lora     low-rank adapters of many requests beside a projection of T tokens,
           y = base + scale_a (x A_a^T) B_a^T, with dA, dB and the term of dx

A case's "pass" is "forward" (serving) or "train" (the forward and its gradients).
"""
import math

import numpy as np
import torch

own = False  # False: the plain forms; True: the framework's entry points


# ------------------------------------------------------------------------- cases
def _route(name, T, E, k, score, groups, keep, top, renorm, bias, scale, pas):
    return {"name": name, "op": "route", "pass": pas, "T": T, "E": E, "k": k, "score": score,
            "groups": groups, "keep": keep, "top": top, "renorm": renorm, "bias": bias,
            "scale": scale}


def _router(name, T, H, E, pas):
    return {"name": name, "op": "router", "pass": pas, "T": T, "H": H, "E": E}


def _lora(name, T, H_in, H_out, n, r, requests, free, pas):
    return {"name": name, "op": "lora", "pass": pas, "T": T, "H_in": H_in, "H_out": H_out, "n": n,
            "r": r, "requests": requests, "free": free}


def listed():
    return [
        # one generated token of the 256-expert layer: launch latency
        _route("route_token", 1, 256, 8, "sigmoid", 8, 4, 2, True, True, 2.5, "forward"),
        # the routing of a full batch of prompt tokens, groups and balance bias
        _route("route_prompt", 8192, 256, 8, "sigmoid", 8, 4, 2, True, True, 2.5, "forward"),
        # a ragged batch of the 64-expert layer: plain softmax gates, whose gradient is dense
        _route("route_softmax_train", 1003, 64, 6, "softmax", 1, 1, 1, False, False, 1.0, "train"),
        # the training step's routing at the 256-expert layer
        _route("route_train", 8192, 256, 8, "sigmoid", 8, 4, 2, True, True, 2.5, "train"),
        # one generated token: the router's weights are read once
        _router("router_token", 1, 7168, 256, "forward"),
        # a full batch of prompt tokens
        _router("router_prompt", 8192, 7168, 256, "forward"),
        # a ragged batch and an expert count that ends inside a tile
        _router("router_train_odd", 777, 2048, 60, "train"),
        # the training step's router at the 256-expert layer
        _router("router_train", 4096, 7168, 256, "train"),
        # one request, one token
        _lora("lora_token", 1, 7168, 7168, 8, 16, 1, 0.0, "forward"),
        # a decode batch: every token is a request's next one, 32 adapters, some without
        _lora("lora_decode", 96, 7168, 2048, 32, 16, 96, 0.1, "forward"),
        # a few ragged requests into a wider projection
        _lora("lora_train_odd", 1029, 2048, 7168, 5, 8, 7, 0.25, "train"),
        # fine-tuning eight adapters at once at the layer's width
        _lora("lora_train", 8192, 7168, 7168, 8, 64, 24, 0.05, "train"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _drawn(rng):
    op = rng.choice(["route", "router", "lora"])
    pas = rng.choice(["forward", "train"])
    T = _log_int(rng, 1, 8192)
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        per = max(2, _log_int(rng, 8, 512) // groups)
        E = groups * per
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(16, keep * per))
        return _route("", T, E, k, rng.choice(["softmax", "sigmoid"]), groups, keep,
                      rng.choice([1, 2]), rng.random() < 0.6, rng.random() < 0.6,
                      rng.choice([1.0, 2.5]), pas)
    if op == "router":
        return _router("", T, 128 * _log_int(rng, 1, 56), _log_int(rng, 4, 384), pas)
    return _lora("", T, 8 * _log_int(rng, 16, 896), 8 * _log_int(rng, 16, 896),
                 _log_int(rng, 1, 48), 8 * _log_int(rng, 1, 8), min(T, _log_int(rng, 1, 128)),
                 rng.choice([0.0, 0.0, 0.2]), pas)


def draw(rng):
    most = [work(c) for c in listed()]
    case = _drawn(rng)
    while any(work(case)[q] > max(w[q] for w in most) for q in ("bytes", "flops")):
        case = _drawn(rng)
    case.pop("name")
    return case


def work(case):
    c = case
    train = c["pass"] == "train"
    T = c["T"]
    if c["op"] == "route":
        n, sel = T * c["E"], T * c["k"]
        by = 4 * n + 8 * sel + (4 * c["E"] if c["bias"] else 0)
        fl = 6 * n + 8 * sel
        if train:  # d_topk_w in, d_logits out
            by += 4 * sel + 4 * n
            fl += 3 * n + 6 * sel
        return {"bytes": by, "flops": fl}
    if c["op"] == "router":
        x, w, L = 2 * T * c["H"], 2 * c["E"] * c["H"], 4 * T * c["E"]
        by, fl = x + w + L, 2 * T * c["H"] * c["E"]
        if train:  # d_logits, dx_in in; dw, dx out
            by += L + 2 * x + w
            fl *= 3
        return {"bytes": by, "flops": fl}
    rows = T * (1.0 - c["free"])
    used = min(c["n"], c["requests"])
    ab = 2 * used * c["r"] * (c["H_in"] + c["H_out"])
    by = 2 * rows * c["H_in"] + 4 * T * c["H_out"] + ab
    fl = 2 * rows * c["r"] * (c["H_in"] + c["H_out"])
    if train:  # dy, dx_in in; dx, dA, dB out
        by += 2 * rows * c["H_out"] + 4 * T * c["H_in"] + 2 * c["n"] * c["r"] * (c["H_in"] + c["H_out"])
        fl *= 3
    return {"bytes": int(by), "flops": int(fl)}


# ------------------------------------------------------------------------ inputs
def _inputs(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = c["T"]

    def randn(*shape, std=1.0, dtype=torch.float32):
        t = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
        return (t if std == 1.0 else t.mul_(std)).to(dtype)

    if c["op"] == "route":
        # noise plus a popularity of the experts that falls like a power of their rank
        rank = torch.randperm(c["E"], generator=g, device="cuda").to(torch.float32) + 1.0
        d = {"logits": randn(T, c["E"]) - 0.6 * torch.log(rank)[None, :]}
        d["bias"] = randn(c["E"], std=0.05) if c["bias"] else None
        if c["pass"] == "train":
            d["dw"] = randn(T, c["k"])
        return d
    if c["op"] == "router":
        d = {"x": randn(T, c["H"], dtype=torch.bfloat16),
             "w": randn(c["E"], c["H"], std=0.02, dtype=torch.bfloat16)}
        if c["pass"] == "train":
            d["dL"] = randn(T, c["E"], std=0.05)
            d["dx_in"] = randn(T, c["H"], dtype=torch.bfloat16)
        return d
    n, r = c["n"], c["r"]
    # the tokens of one request are neighbours; a request has one adapter or none (-1)
    req = torch.randint(0, n, (c["requests"],), generator=g, device="cuda")
    none = torch.rand((c["requests"],), generator=g, device="cuda") < c["free"]
    req = torch.where(none, torch.full_like(req, -1), req)
    at = torch.arange(T, device="cuda") * c["requests"] // T
    d = {"idx": req[at].to(torch.int32),
         "x": randn(T, c["H_in"], dtype=torch.bfloat16),
         "base": randn(T, c["H_out"], dtype=torch.bfloat16),
         "a": randn(n, r, c["H_in"], std=c["H_in"] ** -0.5, dtype=torch.bfloat16),
         "b": randn(n, c["H_out"], r, std=0.5 * r ** -0.5, dtype=torch.bfloat16),
         "scale": 0.5 + torch.rand((n,), generator=g, device="cuda", dtype=torch.float32)}
    if c["pass"] == "train":
        d["dy"] = randn(T, c["H_out"], dtype=torch.bfloat16)
        d["dx_in"] = randn(T, c["H_in"], dtype=torch.bfloat16)
    return d


def prepare(case, seed):
    """The inputs, and for the framework's calls the buffers that its user allocates once:
    outputs, workspaces, and the plan of the batch's adapters (one per batch of requests)."""
    d = _inputs(case, seed)
    st = {"case": case, "in": d}
    if own:
        from mixture_experts_layer_plan_amd import binding as B
        c = case
        dev = dict(device="cuda")
        T = c["T"]
        st["B"] = B
        if c["op"] == "route":
            s = st["s"] = B.shape(T, 128, 128, c["E"], c["k"])
            st["sc"] = B.scoring(score=c["score"], n_groups=c["groups"], topk_groups=c["keep"],
                                 group_top=c["top"], renormalise=c["renorm"], scale=c["scale"])
            st["idx"] = torch.empty((T, c["k"]), dtype=torch.int32, **dev)
            st["w"] = torch.empty((T, c["k"]), dtype=torch.float32, **dev)
            st["dL"] = torch.empty((T, c["E"]), dtype=torch.float32, **dev)
        elif c["op"] == "router":
            s = st["s"] = B.shape(T, c["H"], 128, c["E"], 1)
            st["logits"] = torch.empty((T, c["E"]), dtype=torch.float32, **dev)
            st["dw"] = torch.empty_like(d["w"])
            st["dx"] = torch.empty_like(d["x"])
            st["ws"] = torch.empty(B.moe_router_workspace_bytes(s, False), dtype=torch.uint8, **dev)
            st["ws_b"] = torch.empty(B.moe_router_workspace_bytes(s, True), dtype=torch.uint8, **dev)
        else:
            s = st["s"] = B.lora_shape(T, c["H_in"], c["H_out"], c["n"], c["r"])
            train = c["pass"] == "train"
            st["plan"] = torch.empty(B.moe_lora_plan_bytes(s), dtype=torch.uint8, **dev)
            B.moe_lora_plan(s, d["idx"], st["plan"])
            st["saved"] = torch.empty(B.moe_lora_saved_bytes(s), dtype=torch.uint8, **dev) if train else None
            st["y"] = torch.empty_like(d["base"])
            st["ws"] = torch.empty(B.moe_lora_workspace_bytes(s, train), dtype=torch.uint8, **dev)
            if train:
                st["dx"] = torch.empty_like(d["x"])
                st["da"] = torch.empty_like(d["a"])
                st["db"] = torch.empty_like(d["b"])
    return st


# ------------------------------------------------------------------- plain forms
def _plain_route(c, d):
    L = d["logits"]
    T, E, k = c["T"], c["E"], c["k"]
    # the choice is made in 64 bits: a score next to the border of the top k decides
    L64 = L.double()
    if c["score"] == "softmax":
        e64 = torch.exp(L64 - L64.amax(1, keepdim=True))
        choice = e64 / e64.sum(1, keepdim=True)
        e32 = torch.exp(L - L.amax(1, keepdim=True))
        s = e32 / e32.sum(1, keepdim=True)
    else:
        choice = 1.0 / (1.0 + torch.exp(-L64))
        s = 1.0 / (1.0 + torch.exp(-L))
    if d["bias"] is not None:
        choice = choice + d["bias"].double()
    if c["groups"] > 1:
        best = torch.sort(choice.view(T, c["groups"], -1), dim=2, descending=True)[0]
        rank = best[:, :, :c["top"]].sum(2)
        kept = torch.sort(rank, dim=1, descending=True, stable=True)[1][:, :c["keep"]]
        in_kept = torch.zeros((T, c["groups"]), dtype=torch.bool, device=L.device).scatter_(1, kept, True)
        choice = torch.where(in_kept.repeat_interleave(E // c["groups"], 1), choice, -math.inf)
    idx = torch.sort(choice, dim=1, descending=True, stable=True)[1][:, :k]
    sel = torch.gather(s, 1, idx)
    total = sel.sum(1, keepdim=True) if c["renorm"] else torch.ones_like(sel[:, :1])
    w = c["scale"] * sel / total
    if c["pass"] == "forward":
        return {"idx": idx.to(torch.int32), "w": w}
    # ds of the selected scores, then through the score function
    dw = d["dw"]
    ds = c["scale"] * dw / total
    if c["renorm"]:
        ds = ds - (dw * w).sum(1, keepdim=True) / total
    g = torch.zeros_like(L).scatter_(1, idx, ds)
    if c["score"] == "softmax":
        dL = s * (g - (g * s).sum(1, keepdim=True))
    else:
        dL = g * s * (1.0 - s)
    return {"idx": idx.to(torch.int32), "w": w, "d_logits": dL}


def _plain_router(c, d):
    x, w = d["x"].float(), d["w"].float()
    out = {"logits": x @ w.t()}
    if c["pass"] == "train":
        out["dw"] = (d["dL"].t() @ x).to(torch.bfloat16)
        out["dx"] = (d["dx_in"].float() + d["dL"] @ w).to(torch.bfloat16)
    return out


def _plain_lora(c, d):
    # every adapter's products for every token, and a mask that keeps each token's own
    n, r = c["n"], c["r"]
    a = d["a"].float().reshape(n * r, -1)
    b = d["b"].float().permute(0, 2, 1).reshape(n * r, -1)
    hot = d["idx"][:, None] == torch.arange(n, device="cuda", dtype=torch.int32)[None, :]
    mask = (hot * d["scale"][None, :]).repeat_interleave(r, 1)
    x = d["x"].float()
    u = (x @ a.t()) * mask
    out = {"y": (d["base"].float() + u @ b).to(torch.bfloat16)}
    if c["pass"] == "train":
        dy = d["dy"].float()
        v = (dy @ b.t()) * mask
        out["dx"] = (d["dx_in"].float() + v @ a).to(torch.bfloat16)
        out["da"] = (v.t() @ x).reshape(n, r, -1).to(torch.bfloat16)
        out["db"] = (dy.t() @ u).reshape(-1, n, r).permute(1, 0, 2).contiguous().to(torch.bfloat16)
    return out


# --------------------------------------------------------------- framework calls
def _own(st):
    c, d, B, s = st["case"], st["in"], st["B"], st["s"]
    train = c["pass"] == "train"
    if c["op"] == "route":
        B.moe_route_scored(s, st["sc"], d["logits"], d["bias"], st["idx"], st["w"])
        out = {"idx": st["idx"], "w": st["w"]}
        if train:
            B.moe_route_scored_backward(s, st["sc"], d["logits"], st["idx"], d["dw"], st["dL"])
            out["d_logits"] = st["dL"]
        return out
    if c["op"] == "router":
        B.moe_router_logits_bf16(s, d["x"], d["w"], st["logits"], st["ws"])
        out = {"logits": st["logits"]}
        if train:
            B.moe_router_backward_bf16(s, d["x"], d["w"], d["dL"], d["dx_in"], st["dw"], st["dx"], st["ws_b"])
            out["dw"], out["dx"] = st["dw"], st["dx"]
        return out
    B.moe_lora_bf16(s, st["plan"], d["x"], d["a"], d["b"], d["scale"], d["base"], st["y"],
                    st["saved"], st["ws"])
    out = {"y": st["y"]}
    if train:
        B.moe_lora_backward_bf16(s, st["plan"], d["x"], d["a"], d["b"], d["scale"], st["saved"],
                                 d["dy"], d["dx_in"], st["dx"], st["da"], st["db"], st["ws"])
        out["dx"], out["da"], out["db"] = st["dx"], st["da"], st["db"]
    return out


def run(state):
    if own:
        return _own(state)
    c, d = state["case"], state["in"]
    return {"route": _plain_route, "router": _plain_router, "lora": _plain_lora}[c["op"]](c, d)


# ------------------------------------------------------------------ 64-bit values
def _exact_route(c, d):
    """Row by row from the definition, on the host."""
    L = d["logits"].double().cpu().numpy()
    bias = np.zeros(c["E"]) if d["bias"] is None else d["bias"].double().cpu().numpy()
    E, k, G = c["E"], c["k"], c["groups"]
    per = E // G
    idx = np.empty((c["T"], k), np.int32)
    w = np.empty((c["T"], k))
    dL = np.zeros_like(L)
    dw = d["dw"].double().cpu().numpy() if c["pass"] == "train" else None
    for t in range(c["T"]):
        row = L[t]
        if c["score"] == "softmax":
            z = np.exp(row - row.max())
            s = z / z.sum()
        else:
            s = 1.0 / (1.0 + np.exp(-row))
        choice = s + bias
        if G > 1:
            by = np.sort(choice.reshape(G, per), axis=1)[:, ::-1]
            rank = by[:, :c["top"]].sum(1)
            kept = np.argsort(-rank, kind="stable")[:c["keep"]]
            away = np.ones(G, bool)
            away[kept] = False
            choice[np.repeat(away, per)] = -np.inf
        i = np.argsort(-choice, kind="stable")[:k]
        total = s[i].sum() if c["renorm"] else 1.0
        idx[t], w[t] = i, c["scale"] * s[i] / total
        if dw is not None:
            g = c["scale"] * dw[t] / total
            if c["renorm"]:
                g = g - (dw[t] * w[t]).sum() / total
            if c["score"] == "softmax":
                dL[t] = -s * (g * s[i]).sum()
                dL[t, i] += s[i] * g
            else:
                dL[t, i] = g * s[i] * (1.0 - s[i])
    out = {"idx": torch.from_numpy(idx), "w": torch.from_numpy(w)}
    if dw is not None:
        out["d_logits"] = torch.from_numpy(dL)
    return out


def _exact_router(c, d):
    x, w = d["x"].double(), d["w"].double()
    out = {"logits": torch.mm(x, w.t())}
    if c["pass"] == "train":
        dL = d["dL"].double()
        out["dw"] = torch.mm(dL.t(), x)
        out["dx"] = torch.addmm(d["dx_in"].double(), dL, w)
    return out


def _exact_lora(c, d):
    """Adapter by adapter, over its own tokens only."""
    x, y = d["x"].double(), d["base"].double()
    a, b, sc = d["a"].double(), d["b"].double(), d["scale"].double()
    train = c["pass"] == "train"
    if train:
        dy, dx = d["dy"].double(), d["dx_in"].double()
        da, db = torch.zeros_like(a), torch.zeros_like(b)
    for i in range(c["n"]):
        at = torch.nonzero(d["idx"] == i).flatten()
        if not at.numel():
            continue
        u = sc[i] * torch.mm(x[at], a[i].t())
        y[at] += torch.mm(u, b[i].t())
        if train:
            v = sc[i] * torch.mm(dy[at], b[i])
            dx[at] += torch.mm(v, a[i])
            da[i] = torch.mm(v.t(), x[at])
            db[i] = torch.mm(dy[at].t(), u)
    return {"y": y, "dx": dx, "da": da, "db": db} if train else {"y": y}


def exact(case, seed):
    d = _inputs(case, seed)
    return {"route": _exact_route, "router": _exact_router, "lora": _exact_lora}[case["op"]](case, d)
