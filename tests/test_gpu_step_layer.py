"""The norm, the router with its balance loss, the experts and the adapters as one layer, and
the AdamW step over its weights: through LayerBuffers, AdamW and run_layer, against the same
layer in fp64 by autograd.

Tolerances of the layer are its own (bf16: normwise relative 1e-2), as in the other layer
tests; those of the norm, the loss and the step have tests of their own."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import digest, np_, say, to_dev
from step_tol import f64
from test_gpu_adamw import as_dict, verify
from test_gpu_adapted_layer import inputs as adapted_inputs

pytestmark = pytest.mark.gpu
H, E, K = 256, 16, 4


def inputs(T, dtype="bf16", seed=0):
    shape, inp = adapted_inputs(T, dtype, seed)
    g = torch.Generator().manual_seed(seed + 7)
    r = lambda *s: torch.randn(*s, generator=g)    # noqa: E731
    # a residual stream several times the norm's unit, and a gradient on it
    inp["x"] = (3 * r(T, H)).bfloat16()
    inp["residual"], inp["dh"] = (5 * r(T, H) + 1).bfloat16(), r(T, H).bfloat16()
    inp["norm_w"], inp["norm_b"] = (1 + 0.2 * r(H)).bfloat16(), (0.2 * r(H)).bfloat16()
    inp["seq_start"] = torch.tensor([0, T // 3, T // 3, T - T // 8], dtype=torch.int32)
    inp["d_loss"] = torch.tensor([2.0])
    return inp


def buffers(T, dtype, kind="layer", coef=0.5, **kw):
    from mixture_experts_layer_plan_amd import LayerBuffers, binding as B
    sc = B.scoring("sigmoid", n_groups=4, topk_groups=2, group_top=2, renormalise=True, scale=2.5)
    args = dict(scoring=sc, router_proj=True, adapters=(3, 16), norm=(kind, 1e-5),
                balance=B.balance("sigmoid", coef, 3))
    args.update(kw)
    return LayerBuffers(T, H, 256, E, K, 128, dtype, backward=True, **args)


def reference(inp, idx, kind, coef):
    """fp64 autograd with the choice held fixed; the loss of y, h and the balance together"""
    p = {k: v.double().requires_grad_(True) for k, v in inp.items() if v.is_floating_point()
         and k not in ("lora_scale", "router_bias", "dy", "dh", "d_loss")}
    # h as it is kept: the sum rounded once, its gradient that of the sum
    h = p["x"] + p["residual"]
    h = h + ((inp["x"].float() + inp["residual"].float()).bfloat16().double() - h).detach()
    c = h - h.mean(1, keepdim=True) if kind == "layer" else h
    x = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * p["norm_w"] + p["norm_b"]
    logits = x @ p["w_router"].T
    logits.retain_grad()
    sg = torch.sigmoid(logits)
    w = torch.gather(sg, 1, idx)
    w = 2.5 * w / w.sum(1, keepdim=True)

    def ffn(v, g, u, d):
        return (torch.nn.functional.silu(v @ g.T) * (v @ u.T)) @ d.T
    rows = []
    for t in range(x.shape[0]):
        y = ffn(x[t], p["s_gate"], p["s_up"], p["s_down"])
        for j, e in enumerate(idx[t].tolist()):
            y = y + w[t, j] * ffn(x[t], p["w_gate"][e], p["w_up"][e], p["w_down"][e])
        a = int(inp["adapter_idx"][t])
        if a >= 0:
            y = y + inp["lora_scale"][a].double() * (p["lora_b"][a] @ (p["lora_a"][a] @ x[t]))
        rows.append(y)
    y = torch.stack(rows)
    share = sg / sg.sum(1, keepdim=True)
    start = inp["seq_start"].tolist()
    spans = [(a, b) for a, b in zip(start, start[1:]) if b > a]
    loss = 0.0
    for a, b in spans:
        cnt = torch.bincount(idx[a:b].flatten(), minlength=E).double()
        loss = loss + coef / len(spans) * E / (K * (b - a) ** 2) * (cnt * share[a:b].sum(0)).sum()
    total = (y * inp["dy"].double()).sum() + (h * inp["dh"].double()).sum() + float(inp["d_loss"]) * loss
    total.backward()
    return y.detach(), float(loss.detach()), {k: v.grad for k, v in p.items()}, logits.grad


GRADS = [("dx", "x"), ("d_norm_w", "norm_w"), ("d_norm_b", "norm_b"), ("dw_router", "w_router"),
         ("dw_gate", "w_gate"), ("dw_up", "w_up"), ("dw_down", "w_down"), ("ds_down", "s_down"),
         ("d_lora_a", "lora_a"), ("d_lora_b", "lora_b")]


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("T", [24, 150])
def test_training_step_of_the_layer(T, kind):
    say(f"step layer bf16 T={T} {kind}")
    from mixture_experts_layer_plan_amd import run_layer
    coef = 50.0       # large enough that its part of the gradients shows
    inp = inputs(T, seed=T)
    b, dev = buffers(T, "bf16", kind, coef), to_dev(inp)
    run_layer(b, dev, backward=True)
    torch.cuda.synchronize()
    idx = b.topk_idx.cpu().long()
    ridx, _ = oracle.route_scored(b.logits, K, "sigmoid", inp["router_bias"], 4, 2, 2, True, 2.5)
    np.testing.assert_array_equal(np_(b.topk_idx), ridx)
    y, loss, g, dL = reference(inp, idx, kind, coef)

    def rel(got, ref, name):
        e = (got.detach().cpu().double() - ref).norm() / ref.norm()
        assert e <= 1e-2, (name, float(e))
    rel(b.y, y, "y")
    assert torch.equal(b.h.cpu(), (inp["x"].float() + inp["residual"].float()).bfloat16())
    assert abs(float(b.loss) - loss) <= 1e-2 * loss
    np.testing.assert_array_equal(np_(b.counts), oracle.balance(b.logits.cpu(), idx, "sigmoid", coef,
                                                                inp["seq_start"])[1])
    rel(b.d_logits, dL, "d_logits")
    for name, of in GRADS:
        rel(getattr(b, name), g[of], name)


@pytest.mark.parametrize("dtype,kw", [("bf16", {}), ("mxfp8", dict(T_minibatch=64)), ("mxfp8", {})])
def test_options_are_the_calls_around_the_layer(dtype, kw):
    """Bit for bit the layer without them, run on the norm's output."""
    say(f"step layer against its parts, {dtype} {kw}")
    from mixture_experts_layer_plan_amd import binding as B, run_layer
    T = 150
    inp = inputs(T, dtype, seed=5)
    b, dev = buffers(T, dtype, coef=0.0, **kw), to_dev(inp)
    run_layer(b, dev, backward=True)
    plain = buffers(T, dtype, norm=None, balance=None, **kw)
    run_layer(plain, dict(dev, x=b.xn), backward=True)
    torch.cuda.synchronize()
    for n in ("y", "topk_idx", "topk_w", "d_logits", "dw_router", "dw_gate", "dw_down", "d_lora_a"):
        assert torch.equal(getattr(b, n), getattr(plain, n)), n
    s = B.norm_shape(T, H, "layer", 1e-5)
    ws = torch.empty(B.moe_norm_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    dx, dw, db = torch.empty_like(plain.dx), torch.empty_like(b.d_norm_w), torch.empty_like(b.d_norm_b)
    B.moe_norm_backward_bf16(s, b.h, dev["norm_w"], b.norm_stats, plain.dx, dev["dh"], dx, dw, db, ws)
    torch.cuda.synchronize()
    assert torch.equal(dx, b.dx) and torch.equal(dw, b.d_norm_w) and torch.equal(db, b.d_norm_b)


def test_the_fp32_layer_with_norm_balance_and_step():
    say("step layer f32")
    from mixture_experts_layer_plan_amd import AdamW, LayerBuffers, binding as B, run_layer
    T = 40
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g) * 0.1    # noqa: E731
    inp = dict(x=10 * r(T, H), w_router=r(E, H), w_gate=r(E, 128, H), w_up=r(E, 128, H),
               w_down=r(E, H, 128), dy=r(T, H), norm_w=1 + r(H))
    b = LayerBuffers(T, H, 128, E, K, 0, "f32", router_gemm=True, norm=("rms", 1e-6),
                     balance=B.balance("softmax", 1.0))
    dev = to_dev(inp)
    opt = AdamW(b, dev)
    run_layer(b, dev, adamw=opt, hyper=B.adamw_hyper(1e-2, step=1))
    torch.cuda.synchronize()
    p = {k: v.double().requires_grad_(True) for k, v in inp.items() if k != "dy"}
    x = p["x"] / torch.sqrt((p["x"] ** 2).mean(1, keepdim=True) + 1e-6) * p["norm_w"]
    logits = x @ p["w_router"].T
    idx = b.topk_idx.cpu().long()
    w = torch.softmax(torch.gather(logits, 1, idx), 1)
    y = torch.zeros(T, H, dtype=torch.float64)
    rows = []
    for t in range(T):
        rows.append(sum(w[t, j] * ((torch.nn.functional.silu(x[t] @ p["w_gate"][e].T) * (x[t] @ p["w_up"][e].T))
                                   @ p["w_down"][e].T) for j, e in enumerate(idx[t].tolist())))
    y = torch.stack(rows)
    cnt = torch.bincount(idx.flatten(), minlength=E).double()
    loss = E / (K * T * T) * (cnt * torch.softmax(logits, 1).sum(0)).sum()
    ((y * inp["dy"].double()).sum() + loss).backward()
    # fp32 sums over at most 256 values and products of three: 1e-5 of the norm
    for got, ref in ((b.y, y.detach()), (b.dx, p["x"].grad), (b.dw_router, p["w_router"].grad),
                     (b.d_norm_w, p["norm_w"].grad), (b.dw_gate, p["w_gate"].grad)):
        assert (got.cpu().double() - ref).norm() <= 1e-5 * ref.norm()
    assert set(opt.state) == {"w_gate", "w_up", "w_down", "w_router", "norm_w"}
    # a first step moves every weight by lr against its gradient's sign (and decays it)
    moved = (dev["norm_w"].cpu() - inp["norm_w"]) / 1e-2
    big = b.d_norm_w.cpu().abs() > 1e-4
    assert torch.allclose(moved[big], -b.d_norm_w.cpu().sign()[big], atol=1e-2)


@pytest.mark.parametrize("bits,master", [(32, True), (8, False), (8, True)])
def test_steps_of_the_optimiser(bits, master):
    say(f"step layer with AdamW bits={bits} master={master}")
    from mixture_experts_layer_plan_amd import AdamW, binding as B, run_layer
    T = 64
    inp = inputs(T, seed=9)
    b, dev = buffers(T, "bf16"), to_dev(inp)
    opt = AdamW(b, dev, bits, master, weight_decay=0.1)
    names = list(opt.state)
    assert names == ["w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down", "w_router", "lora_a", "lora_b",
                     "norm_w", "norm_b"]
    for step in (1, 2):
        before = {n: dict({k: v.cpu().clone() for k, v in opt.state[n].items()}, param=dev[n].cpu().clone())
                  for n in names}
        h = B.adamw_hyper(1e-2, step=step, grad_scale=0.5, seed=step)
        run_layer(b, dev, adamw=opt, hyper=h)
        torch.cuda.synchronize()
        for j, n in enumerate(names):
            if n in ("w_gate", "w_up", "w_down"):   # (a million values each: the others say it)
                continue
            grad = b.__dict__[dict((a, g) for a, g, _ in _weights())[n]]
            flat = lambda d: {k: v.flatten() for k, v in d.items()}    # noqa: E731
            host = dict(flat(before[n]), grad=grad.cpu().flatten(),
                        weight_decay=0.0 if n.startswith("norm") else 0.1)
            verify([host], [dict(flat(opt.state[n]), param=dev[n].flatten())], "bf16", master, bits,
                   as_dict(h), tensor0=j)


def _weights():
    from mixture_experts_layer_plan_amd import layer
    return layer._WEIGHTS


def test_steps_in_a_graph():
    """Forward, backward and step captured once: replays follow the eager run bit for bit,
    each with its own scalars."""
    say("step layer in a graph")
    from mixture_experts_layer_plan_amd import AdamW, binding as B, run_layer
    T = 96
    names = ("y", "dx", "loss", "counts", "d_logits", "dw_gate", "d_norm_w")

    def put(t, h):
        t.copy_(torch.frombuffer(bytearray(bytes(h)), dtype=torch.uint8))
    runs = []
    for graph in (False, True):
        inp = inputs(T, seed=3)
        b, dev = buffers(T, "bf16"), to_dev(inp)
        start = {k: v.clone() for k, v in dev.items()}
        opt = AdamW(b, dev, 8)
        hd = torch.zeros(40, dtype=torch.uint8, device="cuda")
        put(hd, B.adamw_hyper(1e-2, step=1))
        if graph:
            run_layer(b, dev, adamw=opt, hyper=hd)    # an eager pass first: the side stream exists
            torch.cuda.synchronize()
            for k, v in start.items():
                dev[k].copy_(v)
            for st in opt.state.values():
                for v in st.values():
                    v.zero_()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                run_layer(b, dev, adamw=opt, hyper=hd)
        got = []
        for step in (1, 2, 3):
            put(hd, B.adamw_hyper(1e-2 / step, step=step, seed=step))
            if graph:
                g.replay()
            else:
                run_layer(b, dev, adamw=opt, hyper=hd)
            torch.cuda.synchronize()
            got.append(digest(*[getattr(b, n) for n in names], *[dev[n] for n in opt.state],
                              *[v for st in opt.state.values() for v in st.values()]))
        runs.append(got)
    assert runs[0] == runs[1] and len(set(runs[0])) == 3


def test_options_that_do_not_fit():
    from mixture_experts_layer_plan_amd import AdamW, LayerBuffers, binding as B, run_layer
    say("step layer refusals")
    inp = to_dev(inputs(16, seed=1))
    b = buffers(16, "bf16")
    with pytest.raises(ValueError):
        run_layer(b, inp, hyper=B.adamw_hyper(1e-3))
    opt = AdamW(b, inp)
    with pytest.raises(ValueError):
        run_layer(b, inp, adamw=opt)
    with pytest.raises(ValueError):
        run_layer(b, inp, backward=False, adamw=opt, hyper=B.adamw_hyper(1e-3))
    with pytest.raises(ValueError):
        AdamW(LayerBuffers(16, H, 256, E, K, 128, "bf16", backward=False), inp)
    with pytest.raises(ValueError):
        LayerBuffers(16, H, 256, E, K, norm=("batch", 1e-5))
