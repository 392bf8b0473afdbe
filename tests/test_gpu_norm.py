"""GPU parity of the norm in front of the layer and its gradient against the fp64 oracle;
tolerances: step_tol."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import digest, say
from step_tol import check, f64, norm_back_bounds, norm_bounds, rounded

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_plan_amd import binding
    return binding


def guarded(shape, dtype):
    """A tensor between two guard zones, and a check that they stayed as they were."""
    n = int(np.prod(shape))
    buf = torch.full((n + 128,), 77, dtype=dtype, device="cuda")
    def ok():
        assert bool((buf[:64] == 77).all()) and bool((buf[64 + n:] == 77).all())
    return buf[64:64 + n].view(shape), ok


def inputs(T, H, dtype, residual=False, affine=(True, True), seed=0):
    g = torch.Generator().manual_seed(seed + 1000 * T + H)
    r = lambda *s: torch.randn(*s, generator=g)    # noqa: E731
    dt = DT[dtype]
    return dict(x=(r(T, H) * 2 + 0.5).to(dt), res=r(T, H).to(dt) if residual else None,
                w=(1 + 0.3 * r(H)).to(dt) if affine[0] else None,
                b=r(H).to(dt) if affine[1] else None, dy=r(T, H).to(dt),
                dh=r(T, H).to(dt) if residual else None)


def calls(B, dtype):
    return ((B.moe_norm_bf16, B.moe_norm_backward_bf16) if dtype == "bf16"
            else (B.moe_norm_f32, B.moe_norm_backward_f32))


def run(B, i, dtype, kind="layer", eps=1e-5, grads=(True, True)):
    T, H = i["x"].shape
    d = {k: None if v is None else v.cuda() for k, v in i.items()}
    s = B.norm_shape(T, H, kind, eps)
    f, b = calls(B, dtype)
    oks = []

    def out(shape, dt, want=True):
        if not want:
            return None
        t, ok = guarded(shape, dt)
        oks.append(ok)
        return t
    dt = DT[dtype]
    o = dict(y=out((T, H), dt), h=out((T, H), dt, d["res"] is not None),
             stats=out((T, 2), torch.float32), dx=out((T, H), dt), dw=out((H,), dt, grads[0]),
             db=out((H,), dt, grads[1]))
    ws, ok = guarded((B.moe_norm_workspace_bytes(s),), torch.uint8)
    oks.append(ok)
    f(s, d["x"], d["res"], d["w"], d["b"], o["h"], o["y"], o["stats"])
    h = d["x"] if d["res"] is None else o["h"]
    b(s, h, d["w"], o["stats"], d["dy"], d["dh"], o["dx"], o["dw"], o["db"], ws)
    torch.cuda.synchronize()
    for ok in oks:
        ok()
    return o


def verify(i, o, dtype, kind="layer", eps=1e-5):
    bf = dtype == "bf16"
    h = f64(i["x"])
    if i["res"] is not None:
        h = f64((i["x"].float() + i["res"].float()).to(DT[dtype]))
        check(o["h"], h, 0.0, "h")
    y, xh, rstd = oracle.norm(h, None if i["w"] is None else f64(i["w"]),
                              None if i["b"] is None else f64(i["b"]), kind, eps)
    check(o["y"], y, rounded(y, norm_bounds(h, i["w"], i["b"], xh, rstd, kind), bf), "y")
    w = None if i["w"] is None else f64(i["w"])
    dx, dw, db = oracle.norm_backward(h, w, f64(i["dy"]), None if i["dh"] is None else f64(i["dh"]),
                                      kind, eps)
    ex, ew, eb = norm_back_bounds(h, i["w"], i["dy"], i["dh"], xh, rstd, kind)
    check(o["dx"], dx, rounded(dx, ex, bf), "dx")
    if o["dw"] is not None:
        check(o["dw"], dw, rounded(dw, ew, bf), "dw")
    if o["db"] is not None:
        check(o["db"], db, rounded(db, eb, bf), "db")


SIZES = [(1, 8), (1, 7168), (2, 504), (3, 512), (5, 520), (7, 1016), (4, 1024), (9, 1032), (33, 2040),
         (17, 2056), (6, 4104), (130, 256), (5, 7168), (3, 8192), (2, 8200), (2, 16384), (1003, 264)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("T,H", SIZES)
def test_parity(B, T, H, kind, dtype):
    say(f"norm {kind} {dtype} T={T} H={H}")
    for residual in (False, True):
        i = inputs(T, H, dtype, residual)
        verify(i, run(B, i, dtype, kind), dtype, kind)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("w,b", [(False, False), (True, False), (False, True)])
def test_without_weight_or_bias(B, w, b, dtype):
    say(f"norm {dtype} w={w} b={b}")
    for grads in ((w, b), (True, True), (False, True), (False, False)):
        i = inputs(21, 776, dtype, True, (w, b))
        verify(i, run(B, i, dtype, grads=grads), dtype)


def test_rows_that_are_far_from_zero_or_constant(B):
    """A mean of 300 times the deviation, rows of one value, subnormal rows, the largest finite
    values whose squares still sum."""
    say("norm of offset rows")
    i = inputs(6, 640, "f32")
    i["x"][0] += 700.0
    i["x"][1] = 3.25
    i["x"][2] = 0.0
    i["x"][3] *= 1e-39
    i["x"][4] *= 1e16
    for kind in ("layer", "rms"):
        verify(i, run(B, i, "f32", kind, 1e-3), "f32", kind, 1e-3)


def test_a_row_that_is_not_finite_stays_alone(B):
    say("norm with inf and NaN rows")
    for dtype in ("bf16", "f32"):
        i = inputs(40, 512, dtype, True)
        ref = run(B, i, dtype)
        i["x"][7, 3] = float("inf")
        i["x"][11, 500] = float("nan")
        o = run(B, i, dtype)
        keep = [t for t in range(40) if t not in (7, 11)]
        for k in ("y", "dx"):
            assert torch.equal(o[k][keep], ref[k][keep])
            assert torch.isnan(o[k][[7, 11]]).any(1).all()
        assert torch.isnan(o["dw"]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(255, 104), (256, 1032), (257, 1032), (512, 520), (513, 520), (300, 7168),
                                 (600, 16), (256, 16384), (2100, 2056)])
def test_batches_at_the_borders_of_the_backwards_forms(B, T, H, dtype):
    """Column sums beside the rows, joined by a second launch, and both row lengths."""
    say(f"norm forms {dtype} T={T} H={H}")
    i = inputs(T, H, dtype, True)
    o = run(B, i, dtype)
    verify(i, o, dtype)
    half = run(B, i, dtype, grads=(False, True))
    assert torch.equal(half["db"], o["db"]) and torch.equal(half["dx"], o["dx"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(B, dtype):
    """h over x, y over residual, dx over dy and over dh_in."""
    say("norm in place", dtype)
    for T, H in ((37, 2048), (3000, 64), (200, 256), (700, 1024)):
        i = inputs(T, H, dtype, True)
        ref = run(B, i, dtype)
        f, b = calls(B, dtype)
        s = B.norm_shape(T, H)
        d = {k: v.cuda() for k, v in i.items()}
        stats = torch.empty((T, 2), device="cuda")
        ws = torch.empty(B.moe_norm_workspace_bytes(s), dtype=torch.uint8, device="cuda")
        f(s, d["x"], d["res"], d["w"], d["b"], d["x"], d["res"], stats)
        assert torch.equal(d["x"], ref["h"]) and torch.equal(d["res"], ref["y"])
        dw, db = torch.empty_like(d["w"]), torch.empty_like(d["w"])
        dy, dh = d["dy"].clone(), d["dh"].clone()
        b(s, d["x"], d["w"], stats, dy, d["dh"], dy, dw, db, ws)
        b(s, d["x"], d["w"], stats, d["dy"], dh, dh, None, None, None)
        assert torch.equal(dy, ref["dx"]) and torch.equal(dh, ref["dx"])
        assert torch.equal(dw, ref["dw"]) and torch.equal(db, ref["db"])


def test_no_tokens(B):
    say("norm of no tokens")
    s = B.norm_shape(0, 640)
    ws = torch.empty(max(1, B.moe_norm_workspace_bytes(s)), dtype=torch.uint8, device="cuda")
    e = torch.empty((0, 640), device="cuda")
    w, dw, db = (torch.full((640,), 5.0, device="cuda") for _ in range(3))
    st = torch.empty((0, 2), device="cuda")
    B.moe_norm_f32(s, e, None, w, None, None, e, st)
    B.moe_norm_backward_f32(s, e, w, st, e, None, e, dw, db, ws)
    torch.cuda.synchronize()
    assert not dw.any() and not db.any()


def test_gradient_against_differences(B):
    """The forward's own change along a direction.  A central difference is off by its
    truncation, which the oracle gives (its difference against its gradient), and by the
    rounding of the two forwards over the step."""
    say("norm by differences")
    for kind in ("layer", "rms"):
        i = inputs(4, 256, "f32")
        o = run(B, i, "f32", kind)
        v = torch.randn(4, 256, generator=torch.Generator().manual_seed(5))
        w, b, dy = f64(i["w"]), f64(i["b"]), f64(i["dy"])
        got, exact, noise = [], [], 0.0
        e = 2.0 ** -6
        for sign in (1, -1):
            j = dict(i, x=i["x"] + sign * e * v)
            got.append(f64(run(B, j, "f32", kind)["y"]))
            x = f64(j["x"])
            y, xh, rstd = oracle.norm(x, w, b, kind)
            exact.append(y)
            noise = noise + rounded(y, norm_bounds(x, i["w"], i["b"], xh, rstd, kind), False)
        step = f64(i["x"] + e * v) - f64(i["x"] - e * v)
        ana = (f64(o["dx"]) * step).sum(1)
        rdx = oracle.norm_backward(f64(i["x"]), w, dy, None, kind)[0]
        truncation = np.abs(((exact[0] - exact[1]) * dy).sum(1) - (rdx * step).sum(1))
        num = ((got[0] - got[1]) * dy).sum(1)
        xh, rstd = oracle.norm(f64(i["x"]), w, b, kind)[1:]
        edx = rounded(rdx, norm_back_bounds(f64(i["x"]), i["w"], i["dy"], None, xh, rstd, kind)[0], False)
        bound = truncation + (noise * np.abs(dy)).sum(1) + (edx * np.abs(step)).sum(1)
        assert (np.abs(num - ana) <= bound).all(), (kind, np.abs(num - ana), bound)
        assert (bound < 0.05 * np.abs(step * rdx).sum(1)).all()      # it says something


def test_repeated_calls_other_streams_and_a_graph(B):
    say("norm repeated, streams, graph")
    i = inputs(300, 2048, "bf16", True)
    names = ("y", "h", "dx", "dw", "db")
    ref = run(B, i, "bf16")
    want = digest(*[ref[n] for n in names])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o = run(B, i, "bf16")
    assert digest(*[o[n] for n in names]) == want
    d = {k: v.cuda() for k, v in i.items()}
    s = B.norm_shape(300, 2048)
    o = {n: torch.empty_like(ref[n]) for n in names}
    st = torch.empty((300, 2), device="cuda")
    ws = torch.empty(B.moe_norm_workspace_bytes(s), dtype=torch.uint8, device="cuda")

    def step():
        B.moe_norm_bf16(s, d["x"], d["res"], d["w"], d["b"], o["h"], o["y"], st)
        B.moe_norm_backward_bf16(s, o["h"], d["w"], st, d["dy"], d["dh"], o["dx"], o["dw"], o["db"], ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2, 3):
        j = inputs(300, 2048, "bf16", True, seed=seed)
        for k in d:
            d[k].copy_(j[k])
        graph.replay()
        torch.cuda.synchronize()
        r = run(B, j, "bf16")
        assert digest(*[o[n] for n in names]) == digest(*[r[n] for n in names])


def test_tensors_that_do_not_fit(B):
    say("norm refusals of the binding")
    s = B.norm_shape(4, 64)
    x = torch.zeros((4, 64), device="cuda")
    st = torch.zeros((4, 2), device="cuda")
    for bad in (x.bfloat16(), x[:3], x.t(), x.cpu()):
        with pytest.raises(ValueError):
            B.moe_norm_f32(s, bad, None, None, None, None, x.clone(), st)
    with pytest.raises(B.MoeError):
        B.moe_norm_f32(s, x, None, None, None, None, torch.zeros((8, 64), device="cuda").view(-1)[1:257], st)


def test_offsets_past_32_bits(B):
    """The last rows of a batch whose elements pass 2^31."""
    say("norm of 2^31 elements and more")
    T, H = 140000, 16384
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    i = inputs(3, H, "bf16")
    x[-3:] = i["x"].cuda()
    y = torch.empty_like(x)
    st = torch.empty((T, 2), device="cuda")
    s = B.norm_shape(T, H)
    B.moe_norm_bf16(s, x, None, i["w"].cuda(), i["b"].cuda(), None, y, st)
    dw, db = (torch.empty((H,), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.empty(B.moe_norm_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    dy = torch.zeros_like(x)
    dy[-3:] = i["dy"].cuda()
    B.moe_norm_backward_bf16(s, x, i["w"].cuda(), st, dy, None, dy, dw, db, ws)
    torch.cuda.synchronize()
    verify(i, dict(y=y[-3:], dx=dy[-3:], dw=dw, db=db), "bf16")
    assert torch.equal(y[100], i["b"].cuda()) and not dy[:-3].any()


def test_the_smallest_eps(B):
    """Rows whose squares lie around the smallest normal number, beside an eps of it: below 640
    additions a square is off by 2^-150 beside the sum of 2^-126 and more, 2^-24 of it, which
    the bound has (a row of 640 takes 30 of its 56 roundings at most)."""
    say("norm with eps = 2^-126")
    i = inputs(6, 640, "f32")
    i["x"] *= torch.tensor([1e-23, 1e-21, 1e-20, 1e-19, 1e-18, 1e-10])[:, None]
    i["dy"] *= 1e-20
    for kind in ("layer", "rms"):
        verify(i, run(B, i, "f32", kind, 2.0 ** -126), "f32", kind, 2.0 ** -126)


def test_rows_whose_squares_pass_the_range(B):
    """1 / sqrt(variance + eps) is 0 and y is b; with a mean that passes the range too, NaN."""
    say("norm of rows past 2^64")
    for dtype in ("bf16", "f32"):
        i = inputs(5, 1024, dtype)
        i["x"] *= torch.tensor([1.0, 1e21, 1e30, 1.0, 3e37])[:, None].to(DT[dtype])
        i["x"][4] = i["x"][4].abs()
        for kind in ("layer", "rms"):
            o = run(B, i, dtype, kind)
            assert torch.equal(o["y"][[1, 2]].cpu(), i["b"].expand(2, -1))
            assert not o["stats"][[1, 2, 4], 1].any() and torch.isfinite(o["y"][[0, 3]]).all()
            assert torch.isnan(o["y"][4]).all() if kind == "layer" else torch.equal(o["y"][4].cpu(), i["b"])
