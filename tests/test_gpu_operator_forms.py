"""The forms of the adapters' and the router's kernels that sizes choose between, each at
sizes that reach it: against fp64, after a launch that left infinities in LDS, and with a
token that holds an infinity."""
import pytest
import torch

import oracle
import test_gpu_router_bf16 as router
from gpu_util import digest, say
from operator_tol import UB, abs64, bf16_of, check, depth, dot_bound
from test_gpu_lora import case, run, verify

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_plan_amd import binding
    return binding


def leave_infinities_in_lds(B):
    """Rank 128 with infinite weights: its stages of 32 KiB fill with them on every CU."""
    T, hi, ho, n = 2048, 64, 7168, 1
    s = B.lora_shape(T, hi, ho, n, 128)
    u8 = dict(dtype=torch.uint8, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    plan = torch.empty(B.moe_lora_plan_bytes(s), **u8)
    B.moe_lora_plan(s, torch.zeros(T, dtype=torch.int32, device="cuda"), plan)
    y = torch.zeros(T, ho, **bf)
    B.moe_lora_bf16(s, plan, torch.ones(T, hi, **bf), torch.ones(n, 128, hi, **bf),
                    torch.full((n, ho, 128), float("inf"), **bf), torch.ones(n, device="cuda"), y, y,
                    None, torch.empty(B.moe_lora_workspace_bytes(s, False), **u8))


# 64-row tiles of two column blocks a workgroup, then 128-row tiles, of y and of dx
@pytest.mark.parametrize("T,hi,ho,n,r", [(600, 64, 7168, 4, 96), (600, 7168, 64, 4, 96), (1000, 64, 7168, 8, 96),
                                         (600, 64, 7168, 4, 72), (600, 64, 7168, 4, 120), (1100, 64, 6656, 1, 96),
                                         (1100, 6656, 64, 1, 96), (1100, 64, 6656, 1, 88), (1100, 6656, 64, 1, 128)])
def test_ranks_past_64(B, T, hi, ho, n, r):
    say(f"lora forms T={T} {hi}->{ho} n={n} r={r}")
    c = case(T, hi, ho, n, r, "all")
    leave_infinities_in_lds(B)
    got = run(B, c)
    verify(c, got)
    assert digest(*run(B, c, base="inplace", fill=0)) == digest(*got)


@pytest.mark.parametrize("T,hi,ho,n,r", [(1100, 64, 6656, 1, 72), (1100, 64, 6656, 1, 96), (1100, 64, 6656, 1, 128),
                                         (1100, 6656, 64, 1, 96), (2300, 64, 6912, 1, 64), (2300, 13824, 64, 1, 16),
                                         (1000, 64, 7168, 8, 16), (1000, 64, 7168, 8, 64), (1000, 64, 7168, 8, 96),
                                         (1000, 7168, 64, 8, 96), (96, 264, 520, 32, 24), (50, 72, 264, 20, 16)])
def test_an_infinite_token_spoils_its_own_rows(B, T, hi, ho, n, r):
    """A token's infinity reaches its own y (dx) and the gradients it enters, nothing else,
    wherever the token lies in its tile."""
    say(f"lora with inf T={T} {hi}->{ho} n={n} r={r}")
    c = case(T, hi, ho, n, r, "all")
    clean = run(B, c)
    group = [t for t in range(T) if c["idx"][t] == c["idx"][0]]
    a = int(c["idx"][0])
    others = [i for i in range(n) if i != a]
    for t in {group[min(100, len(group) - 1)], group[-1]}:
        rows = torch.arange(T, device="cuda") != t
        cols = torch.arange(hi, device="cuda") != 9
        cx = dict(c, x=c["x"].clone())
        cx["x"][t, 9] = float("inf")
        y, dx, da, db = run(B, cx)
        assert torch.equal(y[rows], clean[0][rows]) and not torch.isfinite(y[t]).any()
        assert torch.equal(dx, clean[1]) and torch.equal(da[:, :, cols], clean[2][:, :, cols])
        assert torch.equal(da[others], clean[2][others]) and torch.equal(db[others], clean[3][others])
        cy = dict(c, dy=c["dy"].clone())
        cy["dy"][t, 9] = float("-inf")
        y, dx, da, db = run(B, cy)
        assert torch.equal(dx[rows], clean[1][rows]) and not torch.isfinite(dx[t]).any()
        keep = torch.arange(ho, device="cuda") != 9
        assert torch.equal(y, clean[0]) and torch.equal(db[:, keep], clean[3][:, keep])
        assert torch.equal(da[others], clean[2][others]) and torch.equal(db[others], clean[3][others])


def test_one_workspace_for_both_passes(B):
    """A long H_in and a short H_out: the forward needs the larger workspace."""
    say("lora 97 tokens with the backward's workspace")
    T, hi, ho, n, r = 97, 4992, 272, 3, 64
    c = {k: v.cuda() for k, v in case(T, hi, ho, n, r).items()}
    s = B.lora_shape(T, hi, ho, n, r)
    u8 = dict(dtype=torch.uint8, device="cuda")
    plan, saved = (torch.empty(f(s), **u8) for f in (B.moe_lora_plan_bytes, B.moe_lora_saved_bytes))
    size = B.moe_lora_workspace_bytes(s, True)
    ws = torch.full((size + 4096,), 255, **u8)
    outs = [torch.empty_like(c[k]) for k in ("base", "x", "a", "b")]
    B.moe_lora_plan(s, c["idx"], plan)
    B.moe_lora_bf16(s, plan, c["x"], c["a"], c["b"], c["scale"], c["base"], outs[0], saved, ws[:size])
    B.moe_lora_backward_bf16(s, plan, c["x"], c["a"], c["b"], c["scale"], saved, c["dy"], c["dx_in"],
                             outs[1], outs[2], outs[3], ws[:size])
    assert bool((ws[size:] == 255).all())
    assert digest(*outs) == digest(*run(B, {k: v.cpu() for k, v in c.items()}))


# the logits of few tokens; dx in 128-row tiles of one, two and four K steps
@pytest.mark.parametrize("T,H,E", [(7, 384, 33), (20, 128, 9), (31, 256, 30), (4100, 8192, 24), (4100, 4224, 60),
                                   (4100, 4224, 100), (4100, 4224, 128)])
def test_router_projection(B, T, H, E):
    say(f"router forms T={T} H={H} E={E}")
    g = torch.Generator().manual_seed(T * 7 + E)
    x, w = router.rand(g, T, H), router.rand(g, E, H, std=0.05)
    dL, dx_in = router.rand(g, T, E, std=0.3, dtype=torch.float32), router.rand(g, T, H)
    leave_infinities_in_lds(B)
    logits, dw, dx = clean = router.run(B, x, w, dL, dx_in)
    check(logits, oracle.router_logits(x, w), dot_bound(x, w), "logits")
    rdw, rdx = oracle.router_backward(x, w, dL, dx_in)
    ew = (depth(2 * T) + UB * UB) * (abs64(dL).T @ abs64(x))
    check(dw, rdw, bf16_of(rdw, ew), "dw")
    full = abs64(dL) @ abs64(w)
    ex = (depth(2 * E) + UB * UB) * full + 2.0 ** -24 * (full + abs64(dx_in))
    check(dx, rdx, bf16_of(rdx, ex), "dx")
    assert digest(*router.run(B, x, w, dL, dx_in, in_place=True)) == digest(*clean)
    # an infinite token, an infinite gradient: their rows, and the gradients they enter
    t = min(100, T - 1)
    rows = torch.arange(T, device="cuda") != t
    cols = torch.arange(H, device="cuda") != 9
    x2 = x.clone()
    x2[t, 9] = float("inf")
    logits, dw, dx = router.run(B, x2, w, dL, dx_in)
    assert torch.equal(logits[rows], clean[0][rows]) and not torch.isfinite(logits[t]).any()
    assert torch.equal(dx, clean[2]) and torch.equal(dw[:, cols], clean[1][:, cols])
    dL2 = dL.clone()
    dL2[t, 3] = float("inf")
    _, dw, dx = router.run(B, x, w, dL2, dx_in)
    keep = torch.arange(E, device="cuda") != 3
    assert torch.equal(dx[rows], clean[2][rows]) and not torch.isfinite(dx[t]).any()
    assert torch.equal(dw[keep], clean[1][keep])
