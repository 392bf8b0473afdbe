"""The operators where byte and element offsets pass 2^31: the first and last rows and the
last group, the only ones that are not zero, against fp64."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import say
from operator_tol import UB, abs64, bf16_of, check, depth, dot_bound, lora_bounds, outer_bound

pytestmark = pytest.mark.gpu
N = 40                                            # rows that hold something at each end


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_plan_amd import binding
    yield binding
    torch.cuda.empty_cache()


def rand(*shape, std=1.0, dtype=torch.bfloat16, seed=0):
    g = torch.Generator().manual_seed(seed + sum(shape))
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def ends(T, rows):
    """[T, n] on the GPU with the first and last N rows of ``rows``, zero between."""
    t = torch.zeros((T, rows.shape[1]), dtype=rows.dtype, device="cuda")
    t[:N], t[T - N:] = rows[:N].cuda(), rows[N:].cuda()
    return t


def both(t):
    return torch.cat([t[:N], t[t.shape[0] - N:]]).cpu()


def test_router_projection(B):
    T, H, E = 7_900_000, 256, 136                 # x: 4.04e9 bytes, logits 4.3e9
    say(f"router bf16 T={T} H={H} E={E}")
    s = B.shape(T, H, 128, E, 1)
    x, w = rand(2 * N, H), rand(E, H, std=0.05, seed=1)
    dL, dxi = rand(2 * N, E, dtype=torch.float32, seed=2), rand(2 * N, H, seed=3)
    xd, dLd, dx = ends(T, x), ends(T, dL), ends(T, dxi)
    ws = torch.empty(max(B.moe_router_workspace_bytes(s, v) for v in (False, True)),
                     dtype=torch.uint8, device="cuda")
    logits = torch.empty((T, E), device="cuda")
    dw = torch.empty((E, H), dtype=torch.bfloat16, device="cuda")
    B.moe_router_logits_bf16(s, xd, w.cuda(), logits, ws)
    check(both(logits), oracle.router_logits(x, w), dot_bound(x, w), "logits")
    assert not logits[N:T - N].any()
    del logits
    B.moe_router_backward_bf16(s, xd, w.cuda(), dLd, dx, dw, dx, ws)
    rdw, rdx = oracle.router_backward(x, w, dL, dxi)
    # zeros add nothing and round to nothing; the parts of 1024 rows are joined one by one
    ew = (depth(2 * 2 * N) + T / 1024 * 2.0 ** -24 + UB * UB) * (abs64(dL).T @ abs64(x))
    check(dw, rdw, bf16_of(rdw, ew), "dw")
    full = abs64(dL) @ abs64(w)
    check(both(dx), rdx, bf16_of(rdx, (depth(2 * E) + UB * UB) * full
                                 + 2.0 ** -24 * (full + abs64(dxi))), "dx")
    assert not dx[N:T - N].any()


@pytest.mark.parametrize("T,hi,ho", [(520_000, 4096, 72), (520_000, 72, 4096)])
def test_adapters_of_many_tokens(B, T, hi, ho):
    say(f"lora T={T} {hi}->{ho}")
    n, r = 3, 16
    s = B.lora_shape(T, hi, ho, n, r)
    c = dict(x=rand(2 * N, hi), a=rand(n, r, hi, std=hi ** -0.5), b=rand(n, ho, r, std=0.25),
             scale=torch.tensor([0.5, 1.0, 2.0]), base=rand(2 * N, ho, seed=4),
             dy=rand(2 * N, ho, seed=5), dx_in=rand(2 * N, hi, seed=6))
    few = torch.cat([torch.arange(N) % n, 2 - torch.arange(N) % n]).to(torch.int32)
    idx = torch.full((T,), 1, dtype=torch.int32, device="cuda")
    idx[:N], idx[T - N:] = few[:N].cuda(), few[N:].cuda()
    x, dy, y, dx = (ends(T, c[k]) for k in ("x", "dy", "base", "dx_in"))
    a, b, sc = c["a"].cuda(), c["b"].cuda(), c["scale"].cuda()
    u8 = dict(dtype=torch.uint8, device="cuda")
    plan, saved = (torch.empty(f(s), **u8) for f in (B.moe_lora_plan_bytes, B.moe_lora_saved_bytes))
    ws = torch.empty(max(B.moe_lora_workspace_bytes(s, v) for v in (False, True)), **u8)
    da, db = torch.empty_like(a), torch.empty_like(b)
    B.moe_lora_plan(s, idx, plan)
    B.moe_lora_bf16(s, plan, x, a, b, sc, y, y, saved, ws)
    B.moe_lora_backward_bf16(s, plan, x, a, b, sc, saved, dy, dx, dx, da, db, ws)
    i = few.numpy()
    u, uerr, yerr = lora_bounds(i, c["x"], c["a"], c["b"], c["scale"], c["base"])
    ref = oracle.lora(i, c["x"], c["a"], c["b"], c["scale"], c["base"])
    check(both(y), ref, bf16_of(ref, yerr), "y")
    assert not y[N:T - N].any() and not dx[N:T - N].any()
    v, verr, xerr = lora_bounds(i, c["dy"], c["b"].transpose(1, 2), c["a"].transpose(1, 2), c["scale"],
                                c["dx_in"])
    rdx, rda, rdb = oracle.lora_backward(i, c["x"], c["a"], c["b"], c["scale"], c["dy"], c["dx_in"])
    check(both(dx), rdx, bf16_of(rdx, xerr), "dx")
    more = T / 1024 * 2.0 ** -24                  # the parts, joined one by one

    def bound(p, perr, q):
        e = outer_bound(i, n, p, perr, q)
        for k in range(n):
            at = i == k
            e[k] += more * ((p[at] + perr[at]).T @ abs64(q)[at])
        return e
    check(da, rda, bf16_of(rda, bound(v, verr, c["x"])), "da")
    check(db, rdb, bf16_of(rdb, bound(u, uerr, c["dy"]).transpose(0, 2, 1)), "db")


def test_many_large_adapters(B):
    T, H, n, r = 40, 16512, 1024, 128             # A and B: 4.3e9 bytes, 2.2e9 values each
    say(f"lora T={T} H={H} n={n} r={r}")
    s = B.lora_shape(T, H, H, n, r)
    few = torch.tensor([0, 511, n - 1])
    idx = few.repeat(T)[:T].to(torch.int32)
    c = dict(x=rand(T, H), a=rand(3, r, H, std=H ** -0.5), b=rand(3, H, r, std=0.1),
             scale=torch.tensor([0.5, 1.0, 2.0]), base=rand(T, H, seed=4), dy=rand(T, H, seed=5))
    A, Bm = (torch.zeros(z, dtype=torch.bfloat16, device="cuda") for z in ((n, r, H), (n, H, r)))
    sc = torch.ones(n, device="cuda")
    for j, k in enumerate(few.tolist()):
        A[k], Bm[k], sc[k] = c["a"][j].cuda(), c["b"][j].cuda(), c["scale"][j].cuda()
    u8 = dict(dtype=torch.uint8, device="cuda")
    plan, saved = (torch.empty(f(s), **u8) for f in (B.moe_lora_plan_bytes, B.moe_lora_saved_bytes))
    ws = torch.empty(max(B.moe_lora_workspace_bytes(s, v) for v in (False, True)), **u8)
    x, dy, base = c["x"].cuda(), c["dy"].cuda(), c["base"].cuda()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dA, dB = torch.full_like(A, 9), torch.full_like(Bm, 9)
    B.moe_lora_plan(s, idx.cuda(), plan)
    B.moe_lora_bf16(s, plan, x, A, Bm, sc, base, y, saved, ws)
    B.moe_lora_backward_bf16(s, plan, x, A, Bm, sc, saved, dy, None, dx, dA, dB, ws)
    i = np.arange(T) % 3
    u, uerr, yerr = lora_bounds(i, c["x"], c["a"], c["b"], c["scale"], c["base"])
    ref = oracle.lora(i, c["x"], c["a"], c["b"], c["scale"], c["base"])
    check(y, ref, bf16_of(ref, yerr), "y")
    v, verr, xerr = lora_bounds(i, c["dy"], c["b"].transpose(1, 2), c["a"].transpose(1, 2), c["scale"], None)
    rdx, rda, rdb = oracle.lora_backward(i, c["x"], c["a"], c["b"], c["scale"], c["dy"], None)
    check(dx, rdx, bf16_of(rdx, xerr), "dx")
    check(dA[few.cuda()], rda, bf16_of(rda, outer_bound(i, 3, v, verr, c["x"])), "da")
    check(dB[few.cuda()], rdb, bf16_of(rdb, outer_bound(i, 3, u, uerr, c["dy"]).transpose(0, 2, 1)), "db")
    dA[few.cuda()] = 0
    dB[few.cuda()] = 0
    assert not dA.any() and not dB.any()


def test_base_of_more_tokens_than_one_launch_has_wavefronts(B):
    """Close to 2^26 tokens, all but the ends without an adapter: their base is copied."""
    T, hi, ho, n, r = 66_000_000, 8, 16, 2, 8
    say(f"lora T={T} {hi}->{ho}")
    s = B.lora_shape(T, hi, ho, n, r)
    c = dict(x=rand(2 * N, hi), a=rand(n, r, hi, std=hi ** -0.5), b=rand(n, ho, r, std=0.25),
             scale=torch.tensor([0.5, 2.0]), dy=rand(2 * N, ho, seed=5))
    few = (torch.arange(2 * N) % n).to(torch.int32)
    idx = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    idx[:N], idx[T - N:] = few[:N].cuda(), few[N:].cuda()
    g = torch.Generator(device="cuda").manual_seed(6)
    base, dx_in = (torch.randn((T, h), generator=g, device="cuda", dtype=torch.bfloat16) for h in (ho, hi))
    x, dy = ends(T, c["x"]), ends(T, c["dy"])
    y, dx = torch.full_like(base, 7), torch.full_like(dx_in, 7)
    a, b, sc = c["a"].cuda(), c["b"].cuda(), c["scale"].cuda()
    u8 = dict(dtype=torch.uint8, device="cuda")
    plan, saved = (torch.empty(f(s), **u8) for f in (B.moe_lora_plan_bytes, B.moe_lora_saved_bytes))
    ws = torch.empty(B.moe_lora_workspace_bytes(s, True), **u8)
    da, db = torch.empty_like(a), torch.empty_like(b)
    B.moe_lora_plan(s, idx, plan)
    B.moe_lora_bf16(s, plan, x, a, b, sc, base, y, saved, ws)
    B.moe_lora_backward_bf16(s, plan, x, a, b, sc, saved, dy, dx_in, dx, da, db, ws)
    assert torch.equal(y[N:T - N], base[N:T - N]) and torch.equal(dx[N:T - N], dx_in[N:T - N])
    i, yb, xb = few.numpy(), both(base), both(dx_in)
    u, uerr, yerr = lora_bounds(i, c["x"], c["a"], c["b"], c["scale"], yb)
    ref = oracle.lora(i, c["x"], c["a"], c["b"], c["scale"], yb)
    check(both(y), ref, bf16_of(ref, yerr), "y")
    v, verr, xerr = lora_bounds(i, c["dy"], c["b"].transpose(1, 2), c["a"].transpose(1, 2), c["scale"], xb)
    rdx, rda, rdb = oracle.lora_backward(i, c["x"], c["a"], c["b"], c["scale"], c["dy"], xb)
    check(both(dx), rdx, bf16_of(rdx, xerr), "dx")
    check(da, rda, bf16_of(rda, outer_bound(i, n, v, verr, c["x"])), "da")
    check(db, rdb, bf16_of(rdb, outer_bound(i, n, u, uerr, c["dy"]).transpose(0, 2, 1)), "db")
