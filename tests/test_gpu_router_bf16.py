"""GPU parity of the bf16 router projection and its backward against fp64."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import digest, say
from operator_tol import UB, abs64, bf16_of, check, depth, dot_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_plan_amd import binding
    return binding


def rand(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def rows_guarded(T, n, dtype):
    buf = torch.full(((T + 2) * n + 64,), 33, dtype=dtype, device="cuda")
    lo = -(-n // 32) * 32          # keeps the slice 16-byte aligned
    v = buf[lo:lo + T * n].view(T, n)

    def ok():
        assert bool((buf[:lo] == 33).all()) and bool((buf[lo + T * n:] == 33).all())
    return v, ok


def run(B, x, w, dL, dx_in, in_place=False):
    T, H = x.shape
    E = w.shape[0]
    s = B.shape(T, H, 128, E, 1)
    xd, wd, dLd = x.cuda(), w.cuda(), dL.cuda()
    ws = torch.full((max(B.moe_router_workspace_bytes(s, False), B.moe_router_workspace_bytes(s, True)),),
                    255, dtype=torch.uint8, device="cuda")
    logits, ok1 = rows_guarded(T, E, torch.float32)
    dw, ok2 = rows_guarded(E, H, torch.bfloat16)
    dx, ok3 = rows_guarded(T, H, torch.bfloat16)
    B.moe_router_logits_bf16(s, xd, wd, logits, ws)
    if in_place:
        dx.copy_(dx_in)
        base = dx
    else:
        base = None if dx_in is None else dx_in.cuda()
    ws.fill_(255)
    B.moe_router_backward_bf16(s, xd, wd, dLd, base, dw, dx, ws)
    torch.cuda.synchronize()
    ok1(), ok2(), ok3()
    return logits, dw, dx


SHAPES = [(1, 128, 1), (1, 256, 8), (2, 384, 3), (15, 128, 16), (16, 256, 17), (17, 1152, 60),
          (31, 128, 64), (33, 256, 65), (64, 512, 128), (65, 256, 130), (129, 2048, 256),
          (300, 256, 257), (47, 384, 511), (40, 256, 1000), (70, 128, 1024), (1025, 256, 33),
          (2100, 128, 8), (1500, 384, 300)]


@pytest.mark.parametrize("T,H,E", SHAPES)
def test_projection_and_backward(B, T, H, E):
    say(f"router bf16 T={T} H={H} E={E}")
    g = torch.Generator().manual_seed(T * 7 + E)
    x, w = rand(g, T, H), rand(g, E, H, std=0.05)
    dL, dx_in = rand(g, T, E, std=0.3, dtype=torch.float32), rand(g, T, H)
    logits, dw, dx = run(B, x, w, dL, dx_in)
    check(logits, oracle.router_logits(x, w), dot_bound(x, w), "logits")
    rdw, rdx = oracle.router_backward(x, w, dL, dx_in)
    ew = (depth(2 * T) + UB * UB) * (abs64(dL).T @ abs64(x))
    check(dw, rdw, bf16_of(rdw, ew), "dw")
    full = abs64(dL) @ abs64(w)
    ex = (depth(2 * E) + UB * UB) * full + 2.0 ** -24 * (full + abs64(dx_in))
    check(dx, rdx, bf16_of(rdx, ex), "dx")
    for kw in (dict(in_place=True),):
        again = run(B, x, w, dL, dx_in, **kw)
        assert digest(*again) == digest(logits, dw, dx)
    nob = run(B, x, w, dL, None)
    ref = rdx - dx_in.double().numpy()
    check(nob[2], ref, bf16_of(ref, ex), "dx without dx_in")


def test_no_tokens(B):
    say("router bf16 T=0")
    E, H = 24, 256
    s = B.shape(0, H, 128, E, 1)
    w = torch.ones((E, H), dtype=torch.bfloat16, device="cuda")
    dw = torch.full((E, H), 5, dtype=torch.bfloat16, device="cuda")
    e = torch.empty((0, H), dtype=torch.bfloat16, device="cuda")
    f = torch.empty((0, E), device="cuda")
    ws = torch.empty(B.moe_router_workspace_bytes(s, True), dtype=torch.uint8, device="cuda")
    B.moe_router_logits_bf16(s, e, w, f, ws)
    B.moe_router_backward_bf16(s, e, w, f, None, dw, e, ws)
    torch.cuda.synchronize()
    assert not dw.any()


def test_infinities_stay_in_their_rows(B):
    """A row with an infinity spoils its own logits and dx, and the gradient columns it
    enters, nothing else.  There the results are not finite, infinities or NaN: d_logits
    enters as two halves, and inf * lo is NaN where lo = 0 and the other infinity where the
    halves' signs differ, so that no sign is left to promise."""
    say("router bf16 with inf")
    g = torch.Generator().manual_seed(3)
    T, H, E = 50, 256, 20
    x, w = rand(g, T, H), rand(g, E, H)
    dL, dx_in = rand(g, T, E, dtype=torch.float32), rand(g, T, H)
    clean = run(B, x, w, dL, dx_in)
    x2 = x.clone()
    x2[49, 7] = float("inf")
    logits, dw, dx = run(B, x2, w, dL, dx_in)
    assert torch.equal(logits[:49], clean[0][:49]) and torch.equal(dx, clean[2])
    cols = torch.arange(H, device="cuda") != 7
    assert torch.equal(dw[:, cols], clean[1][:, cols]) and not torch.isfinite(dw[:, 7]).any()
    dL2 = dL.clone()
    dL2[11, 3] = float("inf")
    _, dw, dx = run(B, x, w, dL2, dx_in)
    rows = torch.arange(T, device="cuda") != 11
    assert torch.equal(dx[rows], clean[2][rows]) and not torch.isfinite(dx[11]).any()
    keep = torch.arange(E, device="cuda") != 3
    assert torch.equal(dw[keep], clean[1][keep])


def test_graph_replay(B):
    say("router bf16 in a captured graph")
    g0 = torch.Generator().manual_seed(4)
    T, H, E = 1100, 256, 40
    s = B.shape(T, H, 128, E, 1)
    w = rand(g0, E, H).cuda()
    x, dxi = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda"), rand(g0, T, H).cuda()
    logits, dw, dx = torch.empty((T, E), device="cuda"), torch.empty_like(w), torch.empty_like(x)
    ws = torch.empty(max(B.moe_router_workspace_bytes(s, False), B.moe_router_workspace_bytes(s, True)),
                     dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.moe_router_logits_bf16(s, x, w, logits, ws)
        B.moe_router_backward_bf16(s, x, w, logits, dxi, dw, dx, ws)
    for _ in range(3):
        v = rand(g0, T, H).cuda()
        x.copy_(v)
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        l2, dw2, dx2 = torch.empty_like(logits), torch.empty_like(dw), torch.empty_like(dx)
        ws.fill_(255)
        B.moe_router_logits_bf16(s, v, w, l2, ws)
        B.moe_router_backward_bf16(s, v, w, l2, dxi, dw2, dx2, ws)
        torch.cuda.synchronize()
        assert digest(logits, dw, dx) == digest(l2, dw2, dx2)


def test_binding_refuses(B):
    s = B.shape(4, 128, 128, 8, 1)
    x, w = torch.zeros((4, 128), dtype=torch.bfloat16), torch.zeros((8, 128), dtype=torch.bfloat16)
    out = torch.zeros((4, 8), device="cuda")
    with pytest.raises(ValueError):
        B.moe_router_logits_bf16(s, x, w.cuda(), out, None)               # host tensor
    with pytest.raises(ValueError):
        B.moe_router_logits_bf16(s, x.cuda().float(), w.cuda(), out, None)
    with pytest.raises(ValueError):
        B.moe_router_logits_bf16(s, x.cuda()[:2], w.cuda(), out, None)
    with pytest.raises(ValueError):
        B.moe_router_logits_bf16(s, x.cuda().t().contiguous().t(), w.cuda(), out, None)


def test_many_rows_of_many_values(B):
    """T * H past 2^25 at E <= 64: 128-row tiles, a ragged last one."""
    T, H, E = 6100, 5632, 60
    say(f"router bf16 T={T} H={H} E={E}")
    g = torch.Generator().manual_seed(5)
    x, w = rand(g, T, H), rand(g, E, H, std=0.05)
    s = B.shape(T, H, 128, E, 1)
    logits, ok = rows_guarded(T, E, torch.float32)
    ws = torch.full((B.moe_router_workspace_bytes(s, False),), 255, dtype=torch.uint8, device="cuda")
    B.moe_router_logits_bf16(s, x.cuda(), w.cuda(), logits, ws)
    ok()
    check(logits, oracle.router_logits(x, w), dot_bound(x, w), "logits")
