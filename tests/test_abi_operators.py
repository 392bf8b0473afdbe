"""Host-side refusals of scored routing, the bf16 router projection and the low-rank
adapters (the fake pointers are never dereferenced: every call here is refused)."""
import ctypes
import random

import pytest

B = pytest.importorskip("mixture_experts_layer_plan_amd.binding")

F, BAD = 0x10000, 0x10004
OK, NULL, SHAPE, ALIGN, WS, UNSUP = 0, 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def L():
    return B.lib()


def s_(**kw):
    d = dict(T=64, H=256, I=128, E=16, k=2)
    d.update(kw)
    return B.shape(**d)


def route(L, s, sc, logits=F, bias=None, idx=F, w=F):
    return L.moe_route_scored(ctypes.byref(s), sc if sc is None else ctypes.byref(sc), logits, bias,
                              idx, w, None)


def route_b(L, s, sc, logits=F, idx=F, dw=F, dL=F):
    return L.moe_route_scored_backward(ctypes.byref(s), ctypes.byref(sc), logits, idx, dw, dL, None)


@pytest.mark.parametrize("kw", [dict(n_groups=0), dict(n_groups=3), dict(n_groups=65),
                                dict(n_groups=4, topk_groups=5), dict(topk_groups=0),
                                dict(group_top=0), dict(group_top=3), dict(scale=float("nan")),
                                dict(scale=float("inf")), dict(n_groups=16, topk_groups=1)])
def test_scoring_that_does_not_fit(L, kw):
    assert route(L, s_(), B.scoring(**kw)) == SHAPE
    assert route_b(L, s_(), B.scoring(**kw)) == SHAPE


def test_scoring_fields(L):
    sc = B.scoring()
    for name, v in (("score", 2), ("score", -1), ("renormalise", 2)):
        bad = B.scoring()
        setattr(bad, name, v)
        assert route(L, s_(), bad) == SHAPE
    assert route(L, s_(), None) == NULL
    assert route(L, s_(), sc, logits=None) == NULL
    assert route(L, s_(), sc, bias=BAD) == ALIGN
    assert route(L, s_(k=17), sc) == SHAPE
    assert route_b(L, s_(), sc, dw=None) == NULL
    assert route_b(L, s_(), sc, dL=BAD) == ALIGN
    assert route(L, s_(T=0), sc, logits=None, idx=None, w=None) == OK
    with pytest.raises(ValueError):
        B.scoring(score="tanh")


def test_router_projection(L):
    s = s_()
    fwd, bwd = B.moe_router_workspace_bytes(s, False), B.moe_router_workspace_bytes(s, True)
    assert bwd > 0

    def logits(s, x=F, w=F, out=F, ws=F, n=fwd):
        return L.moe_router_logits_bf16(ctypes.byref(s), x, w, out, ws, n, None)

    def back(s, x=F, w=F, dL=F, dxi=F, dw=F, dx=F + 4096, ws=F, n=bwd):
        return L.moe_router_backward_bf16(ctypes.byref(s), x, w, dL, dxi, dw, dx, ws, n, None)

    assert logits(s_(H=200)) == SHAPE and back(s_(H=200)) == SHAPE
    assert logits(s_(E=1025, k=1)) == SHAPE
    assert logits(s, w=None) == NULL and logits(s, x=None) == NULL
    assert logits(s, x=BAD) == ALIGN
    if fwd:
        assert logits(s, n=fwd - 1) == WS and logits(s, ws=None) == NULL
    assert back(s, n=bwd - 1) == WS
    assert back(s, ws=None) == NULL and back(s, dw=None) == NULL and back(s, dL=None) == NULL
    assert back(s, dxi=BAD) == ALIGN
    assert B.moe_router_workspace_bytes(s_(H=100), True) == 0
    # 32-bit byte offsets: T H 2 and E H 2 below 4 GiB
    assert logits(s_(T=1 << 24, H=128, k=1)) == UNSUP
    assert logits(s_(T=1, H=1 << 27, k=1)) == UNSUP
    assert back(s, x=F, dx=F) == UNSUP                                     # dx over x


def lora(L, s, n, plan=F, x=F, a=F, b=F, sc=F, base=F, y=F, saved=None, ws=F):
    return L.moe_lora_bf16(ctypes.byref(s), plan, x, a, b, sc, base, y, saved, ws, n, None)


def lora_b(L, s, n, plan=F, x=F, a=F, b=F, sc=F, saved=F, dy=F + 4096, dxi=F, dx=F + 8192, da=F, db=F,
           ws=F):
    return L.moe_lora_backward_bf16(ctypes.byref(s), plan, x, a, b, sc, saved, dy, dxi, dx, da, db,
                                    ws, n, None)


@pytest.mark.parametrize("args,code", [((-1, 64, 64, 2, 8), SHAPE), ((4, 0, 64, 2, 8), SHAPE),
                                       ((4, 60, 64, 2, 8), SHAPE), ((4, 64, 4, 2, 8), SHAPE),
                                       ((4, 64, 64, 0, 8), SHAPE), ((4, 64, 64, 1025, 8), SHAPE),
                                       ((4, 64, 64, 2, 4), SHAPE), ((4, 64, 64, 2, 12), SHAPE),
                                       ((4, 64, 64, 2, 136), SHAPE),
                                       ((1 << 20, 64, 4096, 2, 8), UNSUP),
                                       ((1, 64, 1 << 28, 2, 8), UNSUP)])
def test_lora_shapes(L, args, code):
    s = B.lora_shape(*args)
    assert lora(L, s, 1 << 40) == code and lora_b(L, s, 1 << 40) == code
    assert L.moe_lora_plan(ctypes.byref(s), F, F, None) == code
    assert B.moe_lora_plan_bytes(s) == B.moe_lora_saved_bytes(s) == 0
    assert B.moe_lora_workspace_bytes(s, True) == 0


def test_lora_pointers_and_workspace(L):
    s = B.lora_shape(70, 64, 128, 3, 16)
    f, b = B.moe_lora_workspace_bytes(s, False), B.moe_lora_workspace_bytes(s, True)
    assert f > 0 and b > f and B.moe_lora_saved_bytes(s) >= 70 * 16 * 4
    for arg in ("plan", "x", "a", "b", "sc", "y", "ws"):
        assert lora(L, s, f, **{arg: None}) == NULL
    for arg in ("plan", "x", "a", "b", "sc", "saved", "dy", "dx", "da", "db", "ws"):
        assert lora_b(L, s, b, **{arg: None}) == NULL
    for arg in ("x", "base", "y", "saved"):
        assert lora(L, s, f, **{arg: BAD}) == ALIGN
    assert lora_b(L, s, b, dxi=BAD) == ALIGN
    assert lora(L, s, f - 1) == WS and lora_b(L, s, b - 1) == WS
    assert lora_b(L, s, b, dx=F) == UNSUP and lora_b(L, s, b, dx=F + 4096) == UNSUP  # x, dy
    assert L.moe_lora_bf16(None, *[F] * 9, f, None) == NULL
    assert lora(L, B.lora_shape(0, 64, 128, 3, 16), 0, x=None, y=None, ws=None) == OK


def test_layer_options_that_do_not_fit():
    from mixture_experts_layer_plan_amd import LayerBuffers
    for kw in (dict(router_proj=True), dict(adapters=(2, 8))):
        with pytest.raises(ValueError):
            LayerBuffers(8, 256, 128, 4, 2, dtype="f32", device="cpu", **kw)
    b = LayerBuffers(8, 256, 128, 4, 2, dtype="bf16", device="cpu", router_proj=True,
                     adapters=(2, 8), scoring=B.scoring("sigmoid"))
    assert b.logits.shape == (8, 4) and b.d_lora_b.shape == (2, 256, 8)


def test_sizes_past_a_launch_or_32_bit_offsets(L):
    sc = B.scoring()
    assert route(L, s_(T=1 << 26, k=1), sc) == UNSUP and route_b(L, s_(T=1 << 26, k=1), sc) == UNSUP
    # the last K step is addressed whole: ranks and experts count to the next 128
    s = B.lora_shape(1, 64, 1 << 24, 2, 8)
    assert lora(L, s, 1 << 40) == UNSUP and lora_b(L, s, 1 << 40) == UNSUP
    assert lora(L, B.lora_shape(1 << 26, 8, 8, 2, 8), 1 << 40) == UNSUP
    assert L.moe_router_logits_bf16(ctypes.byref(s_(T=1, E=8, H=1 << 24)), F, F, F, F, 1 << 40, None) == UNSUP


def test_lora_output_over_its_input(L):
    s = B.lora_shape(70, 64, 64, 3, 16)
    assert lora(L, s, B.moe_lora_workspace_bytes(s, False), x=F, y=F) == UNSUP


def test_the_backwards_workspace_serves_the_forward():
    """A training step keeps one workspace, of the backward's size, for both passes."""
    rng = random.Random(1)

    def log_int(hi):
        return round(hi ** rng.random())
    shapes = [(97, 4992, 272, 3, 64), (110, 6712, 240, 3, 64), (100, 7168, 128, 1, 64), (0, 8, 8, 1, 8)]
    shapes += [(log_int(20000), 8 * log_int(1000), 8 * log_int(1000), log_int(1024), 8 * log_int(16))
               for _ in range(4000)]
    for a in shapes:
        s = B.lora_shape(*a)
        assert B.moe_lora_workspace_bytes(s, True) >= B.moe_lora_workspace_bytes(s, False) >= 0, a
    for T, H, E in [(64, 7168, 256), (20, 7168, 4)] + [(log_int(20000), 128 * log_int(60), log_int(1024))
                                                       for _ in range(4000)]:
        s = B.shape(T, H, 128, E, 1)
        assert B.moe_router_workspace_bytes(s, True) >= B.moe_router_workspace_bytes(s, False), (T, H, E)


def test_routing_that_would_fill_a_launch_exactly(L):
    """Four tokens a workgroup of 256 threads: from 2^26 - 3 tokens on, 2^32 threads."""
    sc = B.scoring()
    for T in ((1 << 26) - 3, (1 << 26) - 1):
        assert route(L, s_(T=T, k=1), sc) == UNSUP and route_b(L, s_(T=T, k=1), sc) == UNSUP


def test_outputs_that_share_bytes_with_their_inputs(L):
    """An output begins inside an input, or an input inside an output, by one row."""
    s = B.lora_shape(70, 64, 128, 3, 16)
    nx, ny = 70 * 64 * 2, 70 * 128 * 2
    f, b = B.moe_lora_workspace_bytes(s, False), B.moe_lora_workspace_bytes(s, True)
    X, Y, FAR = 0x1000000, 0x2000000, 0x3000000
    for x, y in ((X, X + nx - 128), (X + ny - 256, X)):
        assert lora(L, s, f, x=x, y=y, base=FAR) == UNSUP
    for base in (Y + 256, Y - 256):
        assert lora(L, s, f, x=X, y=Y, base=base) == UNSUP
    for kw in (dict(x=X + 128, dy=Y, dxi=FAR), dict(x=Y, dy=X - ny + 128, dxi=FAR),
               dict(x=Y, dy=FAR, dxi=X - 128)):
        assert lora_b(L, s, b, dx=X, **kw) == UNSUP
    r = s_()
    n, ws = 64 * 256 * 2, B.moe_router_workspace_bytes(r, True)
    for x, dxi in ((X + n - 512, FAR), (X - 512, None), (FAR, X + 512)):
        assert L.moe_router_backward_bf16(ctypes.byref(r), x, F, F, dxi, F, X, F, ws, None) == UNSUP
