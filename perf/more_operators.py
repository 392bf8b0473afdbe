"""Cases of the training step's operators around the layer: their inputs, their plain forms
in elementary torch operations, the framework's calls, and what each cannot do without.

Three operators stand around the layer's own passes:

  norm     the norm in front of the layer, joined with the residual stream; with its gradient
  balance  the balance loss of the router's scores and the experts' counts, per sequence;
           with its gradient into the logits
  adamw    one AdamW step over all of the layer's tensors, states in 32 or in 8 bits

A case's "pass" is "forward" or "train" (the forward and its gradients).
"""
import math

import torch

own = False  # False: the plain forms; True: the framework's entry points


# ------------------------------------------------------------------------- cases
def _norm(name, T, H, kind, dtype, residual, bias, pas):
    return {"name": name, "op": "norm", "pass": pas, "T": T, "H": H, "kind": kind, "dtype": dtype,
            "residual": residual, "bias": bias}


def _balance(name, T, E, k, score, n_seq, free, tail, join, pas):
    return {"name": name, "op": "balance", "pass": pas, "T": T, "E": E, "k": k, "score": score,
            "n_seq": n_seq, "free": free, "tail": tail, "join": join}


def _adamw(name, sizes, p, g, master, bits, step):
    return {"name": name, "op": "adamw", "pass": "train", "sizes": sizes, "p": p, "g": g,
            "master": master, "bits": bits, "step": step}


def listed():
    # the tensors of one GPU's share of four experts (w_gate, w_up, w_down), the shared
    # expert, the router of 256 experts and two norms, at H = 7168 and I = 2048
    share = "58720256*3+14680064*3+1835008*1+7168*2"
    return [
        # one generated token in front of the layer: launch latency
        _norm("norm_token", 1, 7168, "rms", "bf16", True, False, "forward"),
        # a full batch of prompt tokens, joined with the residual stream
        _norm("norm_prompt", 8192, 7168, "rms", "bf16", True, False, "forward"),
        # a ragged batch of the fp32 layer at a width that ends inside a tile, with a bias
        _norm("norm_train_odd", 1003, 2040, "layer", "f32", False, True, "train"),
        # the training step at the layer's width, with a bias and the residual's gradient
        _norm("norm_train", 8192, 7168, "layer", "bf16", True, True, "train"),
        # the load of a small batch of the 64-expert layer: counts and loss alone
        _balance("balance_small", 96, 64, 6, "softmax", 1, 0.0, 0.0, False, "forward"),
        # seven ragged sequences, padding behind the last one, an odd number of experts
        _balance("balance_train_odd", 1003, 60, 6, "softmax", 7, 0.1, 0.1, False, "train"),
        # the training step's batch at the 256-expert layer: four packed sequences
        _balance("balance_train", 8192, 256, 8, "sigmoid", 4, 0.0, 0.0, True, "train"),
        # one balance over the tokens of a whole accumulated batch, some of them left out
        _balance("balance_long", 32768, 256, 8, "sigmoid", 1, 0.02, 0.0, False, "train"),
        # the tensors of the tiny fp32 layer
        _adamw("adamw_tiny", "262144*3+2048*1+256*2", "f32", "f32", False, 32, 1),
        # adapters of many requests: small ragged tensors, states in 8 bits
        _adamw("adamw_ragged", "130051*40+1001*40+77*40", "bf16", "bf16", False, 8, 100),
        # one GPU's share of the layer: bf16 weights with fp32 masters and states
        _adamw("adamw_share", share, "bf16", "bf16", True, 32, 1000),
        # the same in a quarter of the memory: no masters, states in 8 bits
        _adamw("adamw_share_8bit", share, "bf16", "bf16", False, 8, 1000),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _drawn(rng):
    op = rng.choice(["norm", "balance", "adamw"])
    if op == "norm":
        return _norm("", _log_int(rng, 1, 16384), 8 * _log_int(rng, 1, 2048),
                     rng.choice(["layer", "rms"]), rng.choice(["bf16", "bf16", "f32"]),
                     rng.random() < 0.5, rng.random() < 0.5, rng.choice(["forward", "train"]))
    if op == "balance":
        T, E = _log_int(rng, 1, 32768), _log_int(rng, 2, 512)
        return _balance("", T, E, rng.randint(1, min(16, E)), rng.choice(["softmax", "sigmoid"]),
                        rng.choice([1, 1, _log_int(rng, 2, 64)]), rng.choice([0.0, 0.0, 0.1]),
                        rng.choice([0.0, 0.2]), rng.random() < 0.5,
                        rng.choice(["forward", "train"]))
    kinds = [("%d*%d" % (_log_int(rng, 1, 1 << 25), _log_int(rng, 1, 64))) for _ in range(rng.randint(1, 3))]
    p = rng.choice(["bf16", "bf16", "f32"])
    return _adamw("", "+".join(kinds), p, rng.choice(["bf16", "bf16", "f32"]),
                  p == "bf16" and rng.random() < 0.5, rng.choice([32, 8]), rng.choice([1, 10, 1000]))


def draw(rng):
    most = [work(c) for c in listed()]
    case = _drawn(rng)
    while any(work(case)[q] > max(w[q] for w in most) for q in ("bytes", "flops")):
        case = _drawn(rng)
    case.pop("name")
    return case


_BYTES = {"bf16": 2, "f32": 4}


def _sizes(c):
    out = []
    for part in c["sizes"].split("+"):
        n, times = part.split("*")
        out += [int(n)] * int(times)
    return out


def work(case):
    c = case
    train = c["pass"] == "train"
    if c["op"] == "norm":
        es, n, H = _BYTES[c["dtype"]], c["T"] * c["H"], c["H"]
        rows = 4 if c["residual"] else 2            # x (and residual) in, y (and h) out
        by, fl = es * (rows * n + (2 if c["bias"] else 1) * H), 8 * n
        if train:                                   # h, dy (and dh_in) in, dx, dw, db out
            by += es * ((4 if c["residual"] else 3) * n + 2 * (2 if c["bias"] else 1) * H)
            fl += 12 * n
        return {"bytes": by, "flops": fl}
    if c["op"] == "balance":
        n = c["T"] * c["E"]
        by, fl = 4 * n + 4 * c["T"] * c["k"] + 4 * c["n_seq"] * c["E"], 8 * n
        if train:                                   # d_in in, d_logits out
            by += 4 * n + (4 * n if c["join"] else 0)
            fl += 8 * n
        return {"bytes": by, "flops": fl}
    n = sum(_sizes(c))
    p, g = _BYTES[c["p"]], _BYTES[c["g"]]
    each = g + 2 * p if not c["master"] else g + p + 8
    if c["bits"] == 32:
        return {"bytes": (each + 16) * n, "flops": 16 * n}
    # codes and scales in and out; the values that the codes stand for, out
    return {"bytes": int((each + 4 + 4 / 32 + 4) * n), "flops": 24 * n}


# ------------------------------------------------------------------------ inputs
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ALIGN = 512        # elements: every tensor of an arena, and its scales, start at 16 bytes
_KEYS = (0x5BE0CD19, 0xBB67AE85, 0x3C6EF373)  # of the random bits: fractions of square roots
_BETAS, _EPS, _LR = (0.9, 0.95), 1e-8, 3e-4


def _hyper(case, seed):
    """The step's scalars as the operator takes them, in fp32, and its random seed."""
    b1, b2 = _BETAS
    t = case["step"]
    vals = {"lr": _LR, "b1": b1, "a1": 1 - b1, "b2": b2, "a2": 1 - b2, "eps": _EPS,
            "r1": 1 / (1 - b1 ** t), "r2": 1 / (1 - b2 ** t), "gs": 0.75}
    h = {k: float(torch.tensor(v, dtype=torch.float32)) for k, v in vals.items()}
    h["seed"] = (seed * 2654435761 + 12345) % (1 << 32)
    return h


def _arena(case):
    """(sizes, offsets, elements): the layer's tensors one after another in one buffer."""
    sizes = _sizes(case)
    offsets, at = [], 0
    for n in sizes:
        offsets.append(at)
        at += -(-n // _ALIGN) * _ALIGN
    return sizes, offsets, at


def _decay(i):
    """Every third tensor (norms, biases) has no weight decay."""
    return 0.0 if i % 3 == 2 else 0.1


def _inputs(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std=1.0, dtype=torch.float32):
        t = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
        return (t if std == 1.0 else t.mul_(std)).to(dtype)

    if c["op"] == "norm":
        T, H, dt = c["T"], c["H"], _DT[c["dtype"]]
        # a residual stream has rows of different sizes and a few columns that stand out
        d = {"x": (randn(T, H) * (1.0 + 9.0 * torch.rand((1, H), generator=g, device="cuda") ** 8)
                   + 0.25).to(dt),
             "w": (1.0 + randn(H, std=0.1)).to(dt)}
        d["b"] = randn(H, std=0.1, dtype=dt) if c["bias"] else None
        d["res"] = randn(T, H, std=3.0, dtype=dt) if c["residual"] else None
        if c["pass"] == "train":
            d["dy"] = randn(T, H, dtype=dt)
            d["dh"] = randn(T, H, dtype=dt) if c["residual"] else None
        return d
    if c["op"] == "balance":
        T, E, k = c["T"], c["E"], c["k"]
        rank = torch.randperm(E, generator=g, device="cuda").to(torch.float32) + 1.0
        L = randn(T, E) - 0.6 * torch.log(rank)[None, :]
        idx = torch.topk(L, k, dim=1)[1].to(torch.int32)
        idx[torch.rand((T,), generator=g, device="cuda") < c["free"]] = -1   # tokens left out
        end = T - int(c["tail"] * T)                                         # padding behind
        cuts = torch.randint(0, end + 1, (c["n_seq"] - 1,), generator=g, device="cuda")
        edge = torch.tensor([0, end], device="cuda")
        start = torch.sort(torch.cat([cuts, edge]))[0].to(torch.int32)
        d = {"L": L, "idx": idx, "start": start}
        if c["pass"] == "train":
            d["d_loss"] = torch.ones((1,), device="cuda")
            d["d_in"] = randn(T, E, std=1e-4 / T) if c["join"] else None
        return d
    sizes, offsets, n = _arena(c)
    keep = torch.zeros((n,), dtype=torch.bool, device="cuda")
    for s, o in zip(sizes, offsets):
        keep[o:o + s] = True
    size = 1e-3 * torch.exp2(2.0 * randn(n)) * keep      # gradients span orders of magnitude
    d = {"g": (randn(n) * size).to(_DT[c["g"]])}
    p = randn(n, std=0.02) * keep
    d["p"] = p.to(_DT[c["p"]])
    d["master"] = p if c["master"] else None
    m = randn(n).mul_(0.3).mul_(size)
    v = (0.5 + torch.rand((n,), generator=g, device="cuda")).mul_(size).mul_(size)
    if c["bits"] == 32:
        d["m"], d["v"] = m, v
    else:
        half = torch.full((n,), 1 << 15, dtype=torch.int32, device="cuda")
        d["m"], d["ms"], _ = _encode_m(m, half)
        d["v"], d["vs"], _ = _encode_v(v, half)
    return d


def prepare(case, seed):
    """The inputs, and for the framework's calls the buffers that its user allocates once:
    outputs, workspaces, and the table of the tensors of an optimiser step."""
    d = _inputs(case, seed)
    st = {"case": case, "in": d}
    c = case
    if c["op"] == "adamw":
        st["hyper"] = _hyper(c, seed)
    if own:
        from mixture_experts_layer_plan_amd import binding as B
        dev = dict(device="cuda")
        st["B"] = B
        if c["op"] == "norm":
            s = st["s"] = B.norm_shape(c["T"], c["H"], c["kind"], 1e-5)
            st["y"] = torch.empty_like(d["x"])
            st["h"] = torch.empty_like(d["x"]) if c["residual"] else None
            st["stats"] = torch.empty((c["T"], 2), dtype=torch.float32, **dev)
            if c["pass"] == "train":
                st["dx"] = torch.empty_like(d["x"])
                st["dw"] = torch.empty_like(d["w"])
                st["db"] = torch.empty_like(d["w"]) if c["bias"] else None
                st["ws"] = torch.empty(B.moe_norm_workspace_bytes(s), dtype=torch.uint8, **dev)
        elif c["op"] == "balance":
            s = st["s"] = B.shape(c["T"], 128, 128, c["E"], c["k"])
            ba = st["ba"] = B.balance(c["score"], 0.01, c["n_seq"])
            st["loss"] = torch.empty((1,), dtype=torch.float32, **dev)
            st["counts"] = torch.empty((c["n_seq"], c["E"]), dtype=torch.int32, **dev)
            st["scales"] = torch.empty((c["n_seq"],), dtype=torch.float32, **dev)
            st["ws"] = torch.empty(B.moe_balance_workspace_bytes(s, ba), dtype=torch.uint8, **dev)
            if c["pass"] == "train":
                st["dL"] = torch.empty_like(d["L"])
        else:
            sizes, offsets, _ = _arena(c)
            names = ["p", "m", "v"] + (["master"] if c["master"] else []) + (["ms", "vs"] if c["bits"] == 8 else [])
            st["out"] = o = {k: torch.zeros_like(d[k]) for k in names}
            long = {"p": "param", "ms": "m_scale", "vs": "v_scale"}
            tensors = []
            for i, (n, at) in enumerate(zip(sizes, offsets)):
                t = {"grad": d["g"][at:at + n], "weight_decay": _decay(i)}
                for k in names:
                    lo, hi = (at // 32, at // 32 + -(-n // 32)) if k in ("ms", "vs") else (at, at + n)
                    t[long.get(k, k)] = d[k][lo:hi]
                    t[long.get(k, k) + "_out"] = o[k][lo:hi]
                tensors.append(t)
            s = st["s"] = B.adamw_shape(sum(sizes), len(sizes), c["p"], c["g"], c["master"], c["bits"])
            st["table"] = torch.empty(B.moe_adamw_table_bytes(s), dtype=torch.uint8, **dev)
            B.moe_adamw_table(s, tensors, st["table"])
            b1, b2 = _BETAS
            st["hyper"] = B.adamw_hyper(_LR, b1, b2, _EPS, c["step"], 0.75, st["hyper"]["seed"])
            if c["bits"] == 8:
                st["values"] = [torch.zeros(d["m"].shape, dtype=torch.bfloat16, **dev) for _ in range(2)]
    return st


# ------------------------------------------------------------------- plain forms
def _plain_norm(c, d):
    x = d["x"].float()
    out = {}
    if c["residual"]:
        out["h"] = (x + d["res"].float()).to(d["x"].dtype)
        x = out["h"].float()
    mu = x.mean(1, keepdim=True) if c["kind"] == "layer" else 0.0
    rstd = 1.0 / torch.sqrt(((x - mu) ** 2).mean(1, keepdim=True) + 1e-5)
    xh = (x - mu) * rstd
    w = d["w"].float()
    y = xh * w
    if c["bias"]:
        y = y + d["b"].float()
    out["y"] = y.to(d["x"].dtype)
    if c["pass"] == "forward":
        return out
    dy = d["dy"].float()
    g = dy * w
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if c["kind"] == "layer":
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * rstd
    if c["residual"]:
        dx = dx + d["dh"].float()
    out["dx"] = dx.to(d["x"].dtype)
    out["dw"] = (dy * xh).sum(0).to(d["x"].dtype)
    if c["bias"]:
        out["db"] = dy.sum(0).to(d["x"].dtype)
    return out


def _plain_balance(c, d):
    L, idx = d["L"], d["idx"]
    T, E, k, n_seq = c["T"], c["E"], c["k"], c["n_seq"]
    t = torch.arange(T, device=L.device)
    seq = (d["start"][None, :] <= t[:, None]).sum(1) - 1          # n_seq: behind the last one
    used = (idx >= 0).any(1) & (seq < n_seq)
    seq = torch.where(used, seq, n_seq)
    if c["score"] == "softmax":
        e = torch.exp(L - L.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-L))
        p = s / s.sum(1, keepdim=True)
    zero = torch.zeros((n_seq + 1, E), device=L.device)
    psum = zero.index_add(0, seq, p)[:n_seq]
    hits = torch.zeros((T, E + 1), device=L.device).scatter_add_(
        1, torch.where(idx >= 0, idx, E).long(), torch.ones_like(idx, dtype=torch.float32))[:, :E]
    counts = zero.index_add(0, seq, hits)[:n_seq]
    N = torch.zeros((n_seq + 1,), device=L.device).index_add(0, seq, torch.ones((T,), device=L.device))[:n_seq]
    n = (N > 0).sum()
    scale = torch.where(N > 0, 0.01 * E / (k * N * N * n), 0.0)
    loss = (scale * (counts * psum).sum(1)).sum().reshape(1)
    out = {"loss": loss, "counts": counts.to(torch.int32)}
    if c["pass"] == "train":
        pad = lambda v: torch.cat([v, torch.zeros_like(v[:1])])    # noqa: E731
        ct = pad(counts)[seq]
        dl = p * (ct - (p * ct).sum(1, keepdim=True)) * (pad(scale)[seq] * d["d_loss"])[:, None]
        if c["score"] == "sigmoid":
            dl = dl * (1.0 - s)
        out["d_logits"] = dl if d["d_in"] is None else d["d_in"] + dl
    return out


def _bits(x):
    return x.view(torch.int32)


def _float(i):
    return i.to(torch.int32).view(torch.float32)


def _amax(x):
    return x.abs().view(-1, 32).amax(1)


def _encode_m(m, r16):
    """Codes (one sign, 4 exponent and 3 mantissa bits), scale bytes and the values: the
    smallest power of two that brings a block of 32 under 448, and 16 random bits that
    decide between the two neighbouring codes."""
    e = ((_bits(_amax(m)) + 0x1FFFFF) >> 23) - 8
    e = e.clamp(min=1)
    inv = _float((254 - e) << 23).repeat_interleave(32)
    y = m.abs() * inv
    low = y < 2.0 ** -6                        # below the normal codes: steps of 2^-9
    z = torch.where(low, y + 2.0 ** -6, y)
    code = ((_bits(z) + ((r16 << 4) | 8)) >> 20) - 960 - 8 * low.to(torch.int32)
    mag = torch.where(code < 8, code.float() * 2.0 ** -9, _float((code.clamp(min=8) + 960) << 20))
    neg = torch.signbit(m)
    val = torch.where(neg, -mag, mag) * _float(e << 23).repeat_interleave(32)
    return (code | (neg.to(torch.int32) << 7)).to(torch.uint8), e.to(torch.uint8), val


def _encode_v(v, r16):
    """The same for v >= 0: 5 exponent and 3 mantissa bits up to 1.875, never zero for a
    value that is not."""
    e = ((_bits(_amax(v)) + 0x0FFFFF) >> 23).clamp(min=1)
    inv = _float((254 - e) << 23).repeat_interleave(32)
    y = v * inv
    top = ((_bits(y) + ((r16 << 4) | 8)) >> 20).clamp(min=769)
    code = torch.where(v > 0, top - 768, 0)
    val = torch.where(v > 0, _float(top << 20), 0.0) * _float(e << 23).repeat_interleave(32)
    return code.to(torch.uint8), e.to(torch.uint8), val


def _decode_m(code, e):
    c = code.to(torch.int32)
    mag = c & 127
    val = torch.where(mag < 8, mag.float() * 2.0 ** -9, _float((mag.clamp(min=8) + 960) << 20))
    return torch.where(c > 127, -val, val) * _float(e.to(torch.int32) << 23).repeat_interleave(32)


def _decode_v(code, e):
    c = code.to(torch.int32)
    val = torch.where(c > 0, _float((c + 768) << 20), 0.0)
    return val * _float(e.to(torch.int32) << 23).repeat_interleave(32)


def _mix(x):
    """A 32-bit number's bits, mixed (in 64-bit whole numbers, whose products wrap)."""
    x = x ^ (x >> 16)
    x = (x * _KEYS[0]) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * _KEYS[1]) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random(case, seed, n):
    """32 random bits for each element of the arena, from the step's seed, the tensor's
    place in the table and the element's place in the tensor (all below 2^32 here)."""
    sizes, offsets, _ = _arena(case)
    pads = torch.tensor(offsets + [n], device="cuda").diff()
    start = torch.tensor(offsets, device="cuda")
    key = _mix((_mix(torch.arange(1, len(sizes) + 1, device="cuda")) + seed) & 0xFFFFFFFF)
    local = torch.arange(n, device="cuda") - start.repeat_interleave(pads)
    return _mix(local ^ key.repeat_interleave(pads)).to(torch.int64)


def _plain_adamw(c, d, h):
    sizes, offsets, n = _arena(c)
    pads = torch.tensor(offsets + [n], device="cuda").diff()
    wd = torch.tensor([_decay(i) for i in range(len(sizes))], device="cuda").repeat_interleave(pads)
    p = d["master"] if c["master"] else d["p"].float()
    eight = c["bits"] == 8
    m = _decode_m(d["m"], d["ms"]) if eight else d["m"]
    v = _decode_v(d["v"], d["vs"]) if eight else d["v"]
    g = d["g"].float() * h["gs"]
    m = m * h["b1"] + g * h["a1"]
    v = v * h["b2"] + (g * h["a2"]) * g
    u = (m * h["r1"]) / (torch.sqrt(v * h["r2"]) + h["eps"])
    p = p - h["lr"] * (u + wd * p)
    r = _random(c, h["seed"], n) if eight or (c["p"] == "bf16" and not c["master"]) else None
    out = {}
    if c["master"]:
        out["master"], out["p"] = p, p.to(torch.bfloat16)
    elif c["p"] == "bf16":      # between the two neighbours, by 16 random bits
        up = (_bits(p) + ((r ^ (r >> 16)) & 0xFFFF).to(torch.int32)) & -65536
        out["p"] = _float(up).to(torch.bfloat16)
    else:
        out["p"] = p
    if eight:
        m = _encode_m(m, (r & 0xFFFF).to(torch.int32))[2].to(torch.bfloat16)
        v = _encode_v(v, (r >> 16).to(torch.int32))[2].to(torch.bfloat16)
    out["m"], out["v"] = m, v
    return out


# --------------------------------------------------------------- framework calls
def _own(st):
    c, d, B, s = st["case"], st["in"], st["B"], st["s"]
    train = c["pass"] == "train"
    if c["op"] == "norm":
        f, b = ((B.moe_norm_bf16, B.moe_norm_backward_bf16) if c["dtype"] == "bf16"
                else (B.moe_norm_f32, B.moe_norm_backward_f32))
        f(s, d["x"], d["res"], d["w"], d["b"], st["h"], st["y"], st["stats"])
        out = {"y": st["y"]}
        if c["residual"]:
            out["h"] = st["h"]
        if train:
            b(s, st["h"] if c["residual"] else d["x"], d["w"], st["stats"], d["dy"], d["dh"],
              st["dx"], st["dw"], st["db"], st["ws"])
            out["dx"], out["dw"] = st["dx"], st["dw"]
            if c["bias"]:
                out["db"] = st["db"]
        return out
    if c["op"] == "balance":
        ba = st["ba"]
        B.moe_balance_loss(s, ba, d["L"], d["idx"], d["start"], st["loss"], st["counts"],
                           st["scales"], st["ws"])
        out = {"loss": st["loss"], "counts": st["counts"]}
        if train:
            B.moe_balance_loss_backward(s, ba, d["L"], d["idx"], d["start"], st["counts"],
                                        st["scales"], d["d_loss"], d["d_in"], st["dL"])
            out["d_logits"] = st["dL"]
        return out
    o = st["out"]
    B.moe_adamw_step(s, st["table"], st["hyper"])
    out = {"p": o["p"], "m": o["m"], "v": o["v"]}
    if c["master"]:
        out["master"] = o["master"]
    if c["bits"] == 8:
        out["m"], out["v"] = st["values"]
        B.moe_adamw_values("m", o["m"], o["ms"], out["m"])
        B.moe_adamw_values("v", o["v"], o["vs"], out["v"])
    return out


def run(state):
    if own:
        return _own(state)
    c, d = state["case"], state["in"]
    if c["op"] == "adamw":
        return _plain_adamw(c, d, state["hyper"])
    return {"norm": _plain_norm, "balance": _plain_balance}[c["op"]](c, d)


# ------------------------------------------------------------------ 64-bit values
def _exact_norm(c, d):
    x = d["x"].double()
    out = {}
    if c["residual"]:       # the norm is that of the sum as it is kept
        out["h"] = x = (x + d["res"].double()).to(d["x"].dtype).double()
    centred = x - x.mean(1, keepdim=True) if c["kind"] == "layer" else x
    rstd = (centred.square().sum(1, keepdim=True) / c["H"] + 1e-5).rsqrt()
    w = d["w"].double()
    out["y"] = centred * rstd * w + (d["b"].double() if c["bias"] else 0.0)
    if c["pass"] == "train":
        dy = d["dy"].double()
        xh = centred * rstd
        g = dy * w
        dot = (g * xh).sum(1, keepdim=True) / c["H"]
        dx = rstd * (g - xh * dot)
        if c["kind"] == "layer":
            dx -= rstd * g.sum(1, keepdim=True) / c["H"]
        out["dx"] = dx + d["dh"].double() if c["residual"] else dx
        out["dw"] = (dy * xh).sum(0)
        if c["bias"]:
            out["db"] = dy.sum(0)
    return out


def _exact_balance(c, d):
    """Sequence by sequence, over its own tokens."""
    L, idx = d["L"].double(), d["idx"]
    E, k = c["E"], c["k"]
    start = d["start"].tolist()
    spans = [torch.arange(a, b, device="cuda") for a, b in zip(start, start[1:])]
    spans = [s[(idx[s] >= 0).any(1)] for s in spans]
    n = sum(1 for s in spans if s.numel())
    loss = torch.zeros((1,), dtype=torch.float64, device="cuda")
    counts = torch.zeros((c["n_seq"], E), dtype=torch.int32, device="cuda")
    dL = torch.zeros_like(L)
    for i, s in enumerate(spans):
        if not s.numel():
            continue
        own_idx = idx[s].flatten().long()
        counts[i] = torch.bincount(own_idx[own_idx >= 0], minlength=E).to(torch.int32)
        cnt = counts[i].double()
        if c["score"] == "softmax":
            p, more = torch.softmax(L[s], 1), 1.0
        else:
            sg = torch.sigmoid(L[s])
            p, more = sg / sg.sum(1, keepdim=True), torch.sigmoid(-L[s])
        scale = 0.01 * E / (k * s.numel() ** 2 * n)
        loss += scale * (p.sum(0) * cnt).sum()
        dL[s] = scale * p * (cnt - (p @ cnt)[:, None]) * more
    out = {"loss": loss, "counts": counts}
    if c["pass"] == "train":
        out["d_logits"] = dL if d["d_in"] is None else dL + d["d_in"].double()
    return out


def _exact_codes(x, r16, top, low):
    """x (64 bits) as the neighbouring code value, below or above, that the random bits say:
    codes of 3 mantissa bits up to `top`, with a fixed step below `low`, scaled by block."""
    a = x.abs()
    big = a.view(-1, 32).amax(1)
    scale = torch.exp2(torch.ceil(torch.log2(big / top)).clamp(min=-126.0))
    scale = torch.where(big > 0, scale, 1.0).repeat_interleave(32)
    y = a / scale
    step = torch.exp2(torch.floor(torch.log2(y.clamp(min=low))) - 3.0)
    q = torch.floor(y / step + (r16.double() * 16 + 8) / (1 << 20)) * step
    return torch.copysign(q * scale, x), scale


def _exact_adamw(c, d, h):
    n = d["g"].numel()
    sizes, offsets, _ = _arena(c)
    p = (d["master"] if c["master"] else d["p"]).double()
    wd = torch.zeros((n,), dtype=torch.float64, device="cuda")
    for i, (s, o) in enumerate(zip(sizes, offsets)):
        wd[o:o + s] = float(torch.tensor(_decay(i)))
    eight = c["bits"] == 8
    if eight:
        pow2 = lambda e: torch.exp2(e.double() - 127.0).repeat_interleave(32)    # noqa: E731
        m = d["m"].view(torch.float8_e4m3fn).double() * pow2(d["ms"])
        e, f = d["v"] >> 3, d["v"] & 7
        v = torch.exp2(e.double() - 31.0) * (1.0 + f.double() / 8.0) * (d["v"] > 0) * pow2(d["vs"])
    else:
        m, v = d["m"].double(), d["v"].double()
    g = d["g"].double() * h["gs"]
    m = h["b1"] * m + h["a1"] * g
    v = h["b2"] * v + h["a2"] * g * g
    out = {"m": m, "v": v}
    p = p * (1.0 - h["lr"] * wd) - h["lr"] * (h["r1"] * m) / ((h["r2"] * v).sqrt() + h["eps"])
    out["p"] = p
    if c["master"]:
        out["master"] = p
    if eight:
        r = _random(c, h["seed"], n)
        out["m"] = _exact_codes(m, r & 0xFFFF, 448.0, 2.0 ** -6)[0]
        q, scale = _exact_codes(v, r >> 16, 1.875, 2.0 ** -40)
        out["v"] = torch.where(v > 0, torch.maximum(q, 1.125 * 2.0 ** -31 * scale), 0.0)
    return out


def exact(case, seed):
    d = _inputs(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(case, d, _hyper(case, seed))
    return {"norm": _exact_norm, "balance": _exact_balance}[case["op"]](case, d)
