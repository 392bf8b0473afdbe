"""GPU parity of the low-rank adapters, forward and backward, against the fp64 oracle."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import digest, say
from operator_tol import bf16_of, check, lora_bounds, outer_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_plan_amd import binding
    return binding


def case(T, hi, ho, n, r, kind="mixed", seed=0):
    g = torch.Generator().manual_seed(seed + T * 13 + r)
    def rand(*shape, std=1.0, dt=torch.bfloat16):
        return (torch.randn(*shape, generator=g) * std).to(dt)
    if kind == "none":
        idx = torch.full((T,), -1)
    elif kind == "one":
        idx = torch.full((T,), n - 1)
    elif kind == "all":
        idx = torch.randint(0, n, (T,), generator=g)
    else:                       # some without an adapter, by -1 and by an id past the last
        idx = torch.randint(-1, n + 1, (T,), generator=g)
    return dict(idx=idx.to(torch.int32), x=rand(T, hi), a=rand(n, r, hi, std=hi ** -0.5),
                b=rand(n, ho, r, std=r ** -0.5), scale=0.5 + torch.rand(n, generator=g),
                base=rand(T, ho), dy=rand(T, ho), dx_in=rand(T, hi))


def guarded(ref):
    buf = torch.full((ref.numel() + 256,), 9, dtype=ref.dtype, device="cuda")
    v = buf[128:128 + ref.numel()].view(ref.shape)

    def ok():
        assert bool((buf[:128] == 9).all()) and bool((buf[128 + ref.numel():] == 9).all())
    return v, ok


def run(B, c, base="apart", train=True, fill=255):
    """base: "apart", "inplace" or "none"; returns (y, dx, da, db)"""
    d = {k: v.cuda() for k, v in c.items()}
    T, hi = c["x"].shape
    n, ho, r = c["b"].shape
    s = B.lora_shape(T, hi, ho, n, r)
    u8 = dict(dtype=torch.uint8, device="cuda")
    plan = torch.empty(B.moe_lora_plan_bytes(s), **u8)
    saved = torch.full((B.moe_lora_saved_bytes(s),), fill, **u8) if train else None
    ws = torch.full((max(B.moe_lora_workspace_bytes(s, v) for v in (False, True)),), fill, **u8)
    outs = [guarded(t) for t in (c["base"], c["x"], c["a"], c["b"])]
    (y, _), (dx, _), (da, _), (db, _) = outs
    for t in (y, dx, da, db):
        t.fill_(float("nan"))
    yb, xb = d["base"], d["dx_in"]
    if base == "inplace":
        y.copy_(d["base"])
        dx.copy_(d["dx_in"])
        yb, xb = y, dx
    elif base == "none":
        yb = xb = None
    B.moe_lora_plan(s, d["idx"], plan)
    B.moe_lora_bf16(s, plan, d["x"], d["a"], d["b"], d["scale"], yb, y, saved, ws)
    if train:
        ws.fill_(fill)
        B.moe_lora_backward_bf16(s, plan, d["x"], d["a"], d["b"], d["scale"], saved, d["dy"], xb, dx,
                                 da, db, ws)
    torch.cuda.synchronize()
    for _, ok in outs:
        ok()
    return y, dx, da, db


def verify(c, got, base=True):
    idx = c["idx"].numpy()
    n = c["a"].shape[0]
    yb, xb = (c["base"], c["dx_in"]) if base else (None, None)
    u, uerr, yerr = lora_bounds(idx, c["x"], c["a"], c["b"], c["scale"], yb)
    ref = oracle.lora(idx, c["x"], c["a"], c["b"], c["scale"], yb)
    check(got[0], ref, bf16_of(ref, yerr), "y")
    bt, at = c["b"].transpose(1, 2), c["a"].transpose(1, 2)
    v, verr, xerr = lora_bounds(idx, c["dy"], bt, at, c["scale"], xb)
    rdx, rda, rdb = oracle.lora_backward(idx, c["x"], c["a"], c["b"], c["scale"], c["dy"], xb)
    check(got[1], rdx, bf16_of(rdx, xerr), "dx")
    check(got[2], rda, bf16_of(rda, outer_bound(idx, n, v, verr, c["x"])), "da")
    db = outer_bound(idx, n, u, uerr, c["dy"]).transpose(0, 2, 1)
    check(got[3], rdb, bf16_of(rdb, db), "db")
    out = (idx < 0) | (idx >= n)
    if out.any():               # tokens without an adapter: the base, bit for bit
        y = got[0].cpu()[torch.tensor(out)]
        assert torch.equal(y, c["base"][torch.tensor(out)] if base else torch.zeros_like(y))


SHAPES = [(1, 128, 128, 1, 8), (1, 8, 8, 3, 8), (2, 24, 40, 2, 16), (15, 128, 256, 4, 16),
          (16, 72, 136, 16, 24), (17, 1000, 264, 2, 32), (33, 256, 1000, 1, 40), (63, 320, 32, 5, 64),
          (64, 128, 128, 1, 64), (65, 2048, 512, 1, 72), (129, 264, 392, 3, 128), (96, 512, 512, 32, 16),
          (200, 136, 120, 100, 8), (300, 256, 384, 7, 96), (1030, 128, 256, 1, 16), (1100, 256, 72, 3, 64),
          (2100, 64, 128, 2, 8), (40, 64, 64, 1024, 8), (1500, 136, 200, 70, 32), (2500, 72, 64, 1, 128)]


@pytest.mark.parametrize("T,hi,ho,n,r", SHAPES)
def test_forward_and_backward(B, T, hi, ho, n, r):
    say(f"lora T={T} {hi}->{ho} n={n} r={r}")
    c = case(T, hi, ho, n, r)
    got = run(B, c)
    verify(c, got)
    again = run(B, c, base="inplace", fill=0)
    assert digest(*again) == digest(*got)
    verify(c, run(B, c, base="none"), base=False)
    assert digest(run(B, c, train=False)[0]) == digest(got[0])


@pytest.mark.parametrize("kind", ["none", "one", "all"])
@pytest.mark.parametrize("T,n", [(1, 4), (70, 4), (1300, 5)])
def test_who_has_an_adapter(B, T, n, kind):
    say(f"lora T={T} n={n} {kind}")
    c = case(T, 136, 72, n, 16, kind)
    got = run(B, c)
    verify(c, got)
    if kind != "all":
        empty = n if kind == "none" else n - 1
        assert not got[2][:empty].any() and not got[3][:empty].any()


def test_no_tokens(B):
    say("lora T=0")
    c = case(0, 64, 128, 3, 16)
    _, _, da, db = run(B, c)
    assert not da.any() and not db.any()


def test_infinities_stay_in_their_rows(B):
    say("lora with inf")
    c = case(60, 128, 128, 2, 16, "all")
    c["idx"][:] = torch.arange(60) % 2
    clean = run(B, c)
    c["x"][4, 9] = float("inf")                    # adapter 0
    y, dx, da, db = run(B, c)
    rows = torch.arange(60, device="cuda") != 4
    assert torch.equal(y[rows], clean[0][rows]) and torch.equal(dx, clean[1])
    assert torch.equal(da[1], clean[2][1]) and torch.equal(db[1], clean[3][1])
    cols = torch.arange(128, device="cuda") != 9
    assert torch.equal(da[0][:, cols], clean[2][0][:, cols])
    # a token without an adapter may hold anything
    c = case(60, 128, 128, 2, 16, "all")
    c["idx"][7] = -1
    clean = run(B, c)
    c["x"][7], c["dy"][7] = float("nan"), float("inf")
    for a, b in zip(run(B, c), clean):
        assert torch.equal(a, b)


def test_gradients_against_differences(B):
    """<dy, y> moves by <dy, dy/dp> h when a parameter moves by h: with base none and h a
    power of two that bf16 holds exactly, y is bilinear in (x, A, B), so the central
    difference has no truncation; what is left is the rounding of y (2^-8 of |y| |dy|)
    over the step and of the gradient itself."""
    say("lora gradients against differences")
    c = case(24, 64, 64, 2, 8, "all")
    _, dx, da, db = run(B, c, base="none")
    dy = c["dy"].double()
    for name, grad, at in (("x", dx, (3, 5)), ("a", da, (1, 2, 7)), ("b", db, (0, 9, 3))):
        h = 4.0
        f = []
        for sgn in (1, -1):
            c2 = {k: v.clone() for k, v in c.items()}
            c2[name][at] = (c[name][at].double() + sgn * h).to(torch.bfloat16)
            y = run(B, c2, base="none", train=False)[0].double().cpu()
            f.append(((y * dy).sum().item(), c2[name][at].double().item(), (y * dy).abs().sum().item()))
        num = (f[0][0] - f[1][0]) / (f[0][1] - f[1][1])
        tol = 2.0 ** -8 * (f[0][2] + f[1][2]) / (f[0][1] - f[1][1]) + 2.0 ** -7 * abs(num)
        assert abs(grad[at].double().item() - num) <= tol, name


def test_graph_replay_and_other_stream(B):
    say("lora in a captured graph")
    c = case(1200, 136, 264, 3, 16)
    d = {k: v.cuda() for k, v in c.items()}
    s = B.lora_shape(1200, 136, 264, 3, 16)
    u8 = dict(dtype=torch.uint8, device="cuda")

    def bufs():
        return (torch.empty(B.moe_lora_plan_bytes(s), **u8), torch.empty(B.moe_lora_saved_bytes(s), **u8),
                torch.empty(B.moe_lora_workspace_bytes(s, False), **u8),
                torch.empty(B.moe_lora_workspace_bytes(s, True), **u8),
                torch.empty_like(d["base"]), torch.empty_like(d["x"]), torch.empty_like(d["a"]),
                torch.empty_like(d["b"]))

    def step(b, idx, x, stream=None):
        B.moe_lora_plan(s, idx, b[0], stream)
        B.moe_lora_bf16(s, b[0], x, d["a"], d["b"], d["scale"], d["base"], b[4], b[1], b[2], stream)
        B.moe_lora_backward_bf16(s, b[0], x, d["a"], d["b"], d["scale"], b[1], d["dy"], d["dx_in"], b[5],
                                 b[6], b[7], b[3], stream)
    b1, b2 = bufs(), bufs()
    idx, x = d["idx"].clone(), d["x"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(b1, idx, x)
    for i in range(3):
        c2 = case(1200, 136, 264, 3, 16, ["mixed", "one", "all"][i], seed=i)
        idx.copy_(c2["idx"])
        x.copy_(c2["x"])
        for t in b1[1:4]:
            t.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        step(b2, c2["idx"].cuda(), c2["x"].cuda(), st)
        st.synchronize()
        assert digest(*b1[4:]) == digest(*b2[4:]), i


@pytest.mark.parametrize("T,hi,ho,n,r", [(1, 4104, 1032, 1, 16), (31, 2504, 200, 1, 8), (50, 4104, 264, 20, 16),
                                         (17, 512, 2056, 2, 16), (40, 520, 136, 1024, 8), (900, 72, 600, 100, 16)])
def test_few_rows_of_many_values(B, T, hi, ho, n, r):
    """Both products in one launch: several stages along K, a last one of 8 values, full and
    ragged 16-row tiles, several parts of the columns."""
    say(f"lora few T={T} {hi}->{ho} n={n} r={r}")
    c = case(T, hi, ho, n, r)
    got = run(B, c)
    verify(c, got)
    assert digest(*run(B, c, base="inplace", fill=0)) == digest(*got)
    assert digest(run(B, c, train=False)[0]) == digest(got[0])
    assert digest(*run(B, c, base="none")) == digest(*run(B, c, base="none", fill=0))


@pytest.mark.parametrize("T,hi,ho,n,r", [(9000, 3736, 64, 3, 64), (6000, 64, 5600, 2, 40)])
def test_many_rows_of_many_values(B, T, hi, ho, n, r):
    """T * H past 2^25: the first product in 128-row tiles, ragged ones among them."""
    say(f"lora many T={T} {hi}->{ho} n={n} r={r}")
    c = case(T, hi, ho, n, r)
    got = run(B, c)
    verify(c, got)
    assert digest(*run(B, c, base="inplace", fill=0)) == digest(*got)


@pytest.mark.parametrize("T,hi,ho,n", [(3, 8200, 64, 2), (130, 8200, 72, 130)])
def test_more_values_than_one_workgroup_takes(B, T, hi, ho, n):
    """Past 8192 values a row the products are two launches for few tiles, one for many."""
    say(f"lora long rows T={T} {hi}->{ho} n={n}")
    c = case(T, hi, ho, n, 16)
    got = run(B, c)
    verify(c, got)
    assert digest(run(B, c, train=False)[0]) == digest(got[0])
