"""The router projection, scored routing, the experts and the adapters as one layer: forward
and backward through LayerBuffers / run_layer, against the same layer in fp64 by autograd.

Tolerances are the layer's own (bf16: normwise relative 1e-2), as in the other layer
tests; the adapters' and the router's own roundings are bounded in their own tests."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import digest, np_, say, to_dev
from synth import Shape, make_inputs

pytestmark = pytest.mark.gpu


def inputs(T, dtype, seed=0, E=16, n=3, r=16, H=256):
    shape = Shape(T=T, H=H, I=256, E=E, k=4, I_shared=128, dtype=dtype)
    inp = make_inputs(shape, seed=seed, device="cpu", with_dy=True)
    g = torch.Generator().manual_seed(seed + 99)

    def rand(*s, std, dt=torch.bfloat16):
        return (torch.randn(*s, generator=g) * std).to(dt)
    del inp["logits"]
    inp["w_router"] = rand(E, H, std=0.06)
    inp["router_bias"] = rand(E, std=0.05, dt=torch.float32)
    inp["lora_a"] = rand(n, r, H, std=H ** -0.5)
    inp["lora_b"] = rand(n, H, r, std=0.1)
    inp["lora_scale"] = torch.tensor([0.5, 1.0, 2.0])
    inp["adapter_idx"] = torch.randint(-1, n, (T,), generator=g).to(torch.int32)
    return shape, inp


def layer(T, inp, dtype, **kw):
    from mixture_experts_layer_plan_amd import LayerBuffers, binding as B, run_layer
    sc = B.scoring("sigmoid", n_groups=4, topk_groups=2, group_top=2, renormalise=True, scale=2.5)
    args = dict(scoring=sc, router_proj=True, adapters=(3, 16))
    args.update(kw)
    b = LayerBuffers(T, 256, 256, 16, 4, 128, dtype, backward=True, **args)
    dev = to_dev(inp)
    run_layer(b, dev, backward=True)
    torch.cuda.synchronize()
    return b, dev


def reference(inp, idx):
    """fp64 autograd of the whole layer with the choice held fixed"""
    p = {k: v.double().requires_grad_(True) for k, v in inp.items()
         if k not in ("adapter_idx", "lora_scale", "router_bias", "dy")}
    x = p["x"]
    logits = x @ p["w_router"].T
    logits.retain_grad()
    s = torch.gather(torch.sigmoid(logits), 1, idx)
    w = 2.5 * s / s.sum(1, keepdim=True)

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
    (y * inp["dy"].double()).sum().backward()
    return y.detach(), {k: v.grad for k, v in p.items()}, logits.grad


@pytest.mark.parametrize("T", [1, 37, 200])
def test_layer_with_router_and_adapters(T):
    say(f"adapted layer bf16 T={T}")
    shape, inp = inputs(T, "bf16", seed=T)
    b, _ = layer(T, inp, "bf16")
    ridx, rw = oracle.route_scored(b.logits, 4, "sigmoid", inp["router_bias"], 4, 2, 2, True, 2.5)
    np.testing.assert_array_equal(np_(b.topk_idx), ridx)
    np.testing.assert_allclose(np_(b.topk_w), rw, rtol=3e-6)
    y, g, dL = reference(inp, b.topk_idx.cpu().long())

    def rel(got, ref, name):
        e = (got.detach().cpu().double() - ref).norm() / ref.norm()
        assert e <= 1e-2, (name, float(e))
    rel(b.y, y, "y")
    rel(b.dx, g["x"], "dx")
    rel(b.d_logits, dL, "d_logits")
    rel(b.dw_router, g["w_router"], "dw_router")
    rel(b.dw_gate, g["w_gate"], "dw_gate")
    rel(b.dw_down, g["w_down"], "dw_down")
    rel(b.ds_up, g["s_up"], "ds_up")
    if (inp["adapter_idx"] >= 0).any():
        rel(b.d_lora_a, g["lora_a"], "d_lora_a")
        rel(b.d_lora_b, g["lora_b"], "d_lora_b")
    again, _ = layer(T, inp, "bf16")
    names = ("y", "dx", "d_logits", "dw_router", "dw_gate", "d_lora_a", "d_lora_b")
    assert digest(*[getattr(b, n) for n in names]) == digest(*[getattr(again, n) for n in names])


@pytest.mark.parametrize("dtype,kw", [("bf16", {}), ("bf16", dict(fused_forward=True)),
                                      ("mxfp8", dict(T_minibatch=64)), ("mxfp8", {})])
def test_options_are_the_calls_after_the_layer(dtype, kw):
    """The adapters and the router's gradient join a layer that is otherwise the same, bit
    for bit, as the one without them."""
    say(f"adapted layer against its parts, {dtype} {kw}")
    from mixture_experts_layer_plan_amd import binding as B
    T = 150
    shape, inp = inputs(T, dtype, seed=5)
    b, dev = layer(T, inp, dtype, **kw)
    plain, _ = layer(T, {k: v for k, v in inp.items()}, dtype, adapters=None, **kw)
    s = B.lora_shape(T, 256, 256, 3, 16)
    u8 = dict(dtype=torch.uint8, device="cuda")
    plan, saved = torch.empty(B.moe_lora_plan_bytes(s), **u8), torch.empty(B.moe_lora_saved_bytes(s), **u8)
    ws = torch.empty(B.moe_lora_workspace_bytes(s, True), **u8)
    y = torch.empty_like(plain.y)
    B.moe_lora_plan(s, dev["adapter_idx"], plan)
    B.moe_lora_bf16(s, plan, dev["x"], dev["lora_a"], dev["lora_b"], dev["lora_scale"], plain.y, y, saved, ws)
    torch.cuda.synchronize()
    assert torch.equal(y, b.y)
    for n in ("topk_idx", "topk_w", "d_logits", "dw_router", "dw_gate", "dw_up", "dw_down", "ds_gate"):
        assert torch.equal(getattr(b, n), getattr(plain, n)), n
    none = dict(inp, adapter_idx=torch.full((T,), -1, dtype=torch.int32))
    c, _ = layer(T, none, dtype, **kw)
    assert torch.equal(c.y, plain.y) and torch.equal(c.dx, plain.dx)
    assert not c.d_lora_a.any() and not c.d_lora_b.any()


def test_pairs_without_an_expert():
    """A token whose logits are all -inf reaches no expert: y is the shared expert's and
    the adapter's part, and its routing gives no gradient."""
    say("adapted layer with a masked token")
    from mixture_experts_layer_plan_amd import LayerBuffers, binding as B, run_layer
    T = 40
    shape, inp = inputs(T, "bf16", seed=7)
    del inp["w_router"]
    inp["logits"] = torch.randn(T, 16, generator=torch.Generator().manual_seed(1))
    inp["logits"][9] = float("-inf")
    sc = B.scoring("sigmoid", n_groups=4, topk_groups=2, group_top=2)
    b = LayerBuffers(T, 256, 256, 16, 4, 128, "bf16", backward=True, scoring=sc)
    dev = to_dev(inp)
    run_layer(b, dev, backward=True)
    torch.cuda.synchronize()
    v = b.plan_views()
    assert int(v["err_flag"][0]) == 1 and (v["pos"][9] == -1).all()
    assert (b.topk_idx[9] == -1).all() and not b.topk_w[9].any() and not b.d_logits[9].any()
    x = inp["x"][9].double()
    ref = (torch.nn.functional.silu(inp["s_gate"].double() @ x) * (inp["s_up"].double() @ x))
    ref = inp["s_down"].double() @ ref
    assert (b.y[9].cpu().double() - ref).norm() <= 1e-2 * ref.norm()
    assert torch.isfinite(b.y).all() and torch.isfinite(b.dx).all()


def test_the_layer_in_a_graph():
    say("adapted layer in a captured graph")
    from mixture_experts_layer_plan_amd import run_layer
    T = 96
    shape, inp = inputs(T, "bf16", seed=3)
    b, dev = layer(T, inp, "bf16")        # an eager pass first: the side stream exists
    names = ("y", "dx", "d_logits", "dw_router", "dw_gate", "d_lora_a", "d_lora_b")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run_layer(b, dev, backward=True)
    for seed in (11, 12, 13):
        _, other = inputs(T, "bf16", seed=seed)
        for k in ("x", "dy", "adapter_idx"):
            dev[k].copy_(other[k])
        g.replay()
        torch.cuda.synchronize()
        got = digest(*[getattr(b, n) for n in names])
        c, _ = layer(T, {k: v.cpu() for k, v in dev.items()}, "bf16")
        assert got == digest(*[getattr(c, n) for n in names]), seed
