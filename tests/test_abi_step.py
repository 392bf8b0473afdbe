"""Host-side refusals of the norm, the balance loss and the AdamW step (the fake pointers are
never dereferenced: every call here is refused or has nothing to do)."""
import ctypes

import pytest

B = pytest.importorskip("mixture_experts_layer_plan_amd.binding")

F, BAD = 0x10000, 0x10004
OK, NULL, SHAPE, ALIGN, WS, UNSUP = 0, 1, 2, 3, 4, 5
X, Y, Z, FAR = 0x1000000, 0x2000000, 0x3000000, 0x9000000


@pytest.fixture(scope="module")
def L():
    return B.lib()


# ------------------------------------------------------------------------- norm
def fwd(L, s, f="moe_norm_bf16", x=X, res=None, w=F, b=F, h=None, y=Y, stats=F):
    return getattr(L, f)(ctypes.byref(s), x, res, w, b, h, y, stats, None)


def bwd(L, s, f="moe_norm_backward_bf16", h=X, w=F, stats=F, dy=Y, dh=None, dx=Z, dw=F, db=F, ws=F,
        n=1 << 40):
    return getattr(L, f)(ctypes.byref(s), h, w, stats, dy, dh, dx, dw, db, ws, n, None)


@pytest.mark.parametrize("args", [(-1, 64), (4, 0), (4, 60), (4, 16392), (4, 64, "layer", 0.0),
                                  (4, 64, "layer", -1.0), (4, 64, "rms", float("nan")),
                                  (4, 64, "rms", 2.0)])
def test_norm_shapes(L, args):
    s = B.norm_shape(*args)
    for kind in ("bf16", "f32"):
        assert fwd(L, s, "moe_norm_" + kind) == SHAPE and bwd(L, s, "moe_norm_backward_" + kind) == SHAPE
    assert B.moe_norm_workspace_bytes(s) == 0


def test_norm_pointers(L):
    s = B.norm_shape(4, 64)
    n = B.moe_norm_workspace_bytes(s)
    assert n > 0
    s.kind = 2
    assert fwd(L, s) == SHAPE
    s.kind = 0
    for a in ("x", "y", "stats"):
        assert fwd(L, s, **{a: None}) == NULL and fwd(L, s, **{a: BAD}) == ALIGN
    assert fwd(L, s, res=FAR) == NULL and fwd(L, s, h=FAR) == NULL   # one without the other
    assert fwd(L, s, w=BAD) == ALIGN and fwd(L, s, res=BAD, h=FAR) == ALIGN
    for a in ("h", "stats", "dy", "dx", "ws"):
        assert bwd(L, s, **{a: None}) == NULL
    for a in ("h", "w", "stats", "dy", "dh", "dx", "dw", "db", "ws"):
        assert bwd(L, s, **{a: BAD}) == ALIGN
    assert bwd(L, s, n=n - 1) == WS
    assert L.moe_norm_bf16(None, *[F] * 7, None) == NULL
    assert fwd(L, B.norm_shape(0, 64), x=None, y=None, stats=None) == OK


def test_norm_outputs_over_inputs(L):
    s = B.norm_shape(4, 64)
    for f, size in (("bf16", 512), ("f32", 1024)):
        a, b = "moe_norm_" + f, "moe_norm_backward_" + f
        for off in (16, -16, size - 16, 16 - size):
            assert fwd(L, s, a, y=X + off) == UNSUP
            assert fwd(L, s, a, res=FAR, h=X + off) == UNSUP
            assert fwd(L, s, a, res=FAR, h=FAR + off) == UNSUP
            assert fwd(L, s, a, res=FAR, h=Z, y=FAR + off) == UNSUP
            assert fwd(L, s, a, res=FAR, h=Z, y=Z + off) == UNSUP
            assert bwd(L, s, b, dx=X + off) == UNSUP and bwd(L, s, b, dx=Y + off) == UNSUP
            assert bwd(L, s, b, dh=FAR, dx=FAR + off) == UNSUP
        assert fwd(L, s, a, res=FAR, h=Z, y=Z) == UNSUP and bwd(L, s, b, dx=X) == UNSUP
        row = size // 4
        for off in (0, 16, -16, row - 16, 16 - row):
            assert bwd(L, s, b, dw=FAR, db=FAR + off) == UNSUP
            assert bwd(L, s, b, w=FAR, dw=FAR + off) == UNSUP and bwd(L, s, b, w=FAR, db=FAR + off) == UNSUP
            assert bwd(L, s, b, dx=FAR, dw=FAR + off) == UNSUP and bwd(L, s, b, dx=FAR, db=FAR + off) == UNSUP


# ---------------------------------------------------------------------- balance
def shape(**kw):
    d = dict(T=64, H=128, I=128, E=16, k=2)
    d.update(kw)
    return B.shape(**d)


def loss(L, s, ba, logits=X, idx=Y, start=F, out=F, counts=F, scales=F, ws=F, n=1 << 40):
    return L.moe_balance_loss(ctypes.byref(s), ctypes.byref(ba), logits, idx, start, out, counts, scales,
                              ws, n, None)


def back(L, s, ba, logits=X, idx=Y, start=F, counts=F, scales=F, d_loss=F, d_in=None, dL=Z):
    return L.moe_balance_loss_backward(ctypes.byref(s), ctypes.byref(ba), logits, idx, start, counts,
                                       scales, d_loss, d_in, dL, None)


def test_balance_refusals(L):
    s, ba = shape(), B.balance("sigmoid", 0.01, 3)
    n = B.moe_balance_workspace_bytes(s, ba)
    assert n > 0
    for bad in (shape(k=17), shape(E=1025), shape(T=-1), shape(E=0)):
        assert loss(L, bad, ba) == SHAPE and back(L, bad, ba) == SHAPE
        assert B.moe_balance_workspace_bytes(bad, ba) == 0
    for args in (("softmax", 0.01, 0), ("softmax", 0.01, (1 << 20) + 1), ("softmax", float("inf"), 1),
                 ("softmax", float("nan"), 1)):
        bad = B.balance(*args)
        assert loss(L, s, bad) == SHAPE and back(L, s, bad) == SHAPE
    bad = B.balance()
    bad.score = 2
    assert loss(L, s, bad) == SHAPE
    for a in ("logits", "idx", "start", "out", "counts", "scales", "ws"):
        assert loss(L, s, ba, **{a: None}) == NULL and loss(L, s, ba, **{a: BAD}) == ALIGN
    for a in ("logits", "idx", "start", "counts", "scales", "dL"):
        assert back(L, s, ba, **{a: None}) == NULL and back(L, s, ba, **{a: BAD}) == ALIGN
    assert back(L, s, ba, d_loss=BAD) == ALIGN and back(L, s, ba, d_in=BAD) == ALIGN
    assert loss(L, s, ba, n=n - 1) == WS
    for T in (1 << 26, (1 << 26) - 3):
        assert loss(L, shape(T=T, k=1), ba) == UNSUP and back(L, shape(T=T, k=1), ba) == UNSUP
    size = 64 * 16 * 4
    for off in (16, -16, size - 16, 16 - size):
        assert back(L, s, ba, dL=X + off) == UNSUP and back(L, s, ba, d_in=FAR, dL=FAR + off) == UNSUP
    assert back(L, shape(T=0), ba, logits=None, idx=None, dL=None) == OK
    assert L.moe_balance_loss(None, ctypes.byref(ba), *[F] * 7, n, None) == NULL
    assert L.moe_balance_loss(ctypes.byref(s), None, *[F] * 7, n, None) == NULL
    with pytest.raises(ValueError):
        B.balance("tanh")


# ------------------------------------------------------------------------ AdamW
def ashape(elements=100, n=1, p="bf16", g="bf16", master=False, bits=32):
    return B.adamw_shape(elements, n, p, g, master, bits)


def tensors(s, each, step=0x100000):
    """Tensors far apart, in place, with every pointer that the shape has."""
    arr = (B.moe_adamw_tensor * s.n_tensors)()
    at = X
    for a, n in zip(arr, each):
        a.n = n
        names = ["param", "m", "v"] + (["master"] if s.master else [])
        names += ["m_scale", "v_scale"] if s.state_bits == 8 else []
        a.grad = at
        for i, k in enumerate(names):
            setattr(a, k, at + (i + 1) * step)
            setattr(a, k + "_out", at + (i + 1) * step)
        at += 16 * step
    return arr


def table(L, s, arr, t=F):
    return L.moe_adamw_table(ctypes.byref(s), arr, t, None)


def change(arr, i=0, **kw):
    for k, v in kw.items():
        setattr(arr[i], k, v)
    return arr


@pytest.mark.parametrize("field,value,code", [("elements", -1, SHAPE), ("n_tensors", 0, SHAPE),
                                              ("n_tensors", 65537, SHAPE), ("p_type", 2, SHAPE),
                                              ("g_type", 2, SHAPE), ("master", 2, SHAPE),
                                              ("state_bits", 16, SHAPE), ("elements", 1 << 37, UNSUP)])
def test_adamw_shapes(L, field, value, code):
    s = ashape()
    arr = tensors(s, [100])
    setattr(s, field, value)
    assert table(L, s, arr) == code
    h = B.adamw_hyper(1e-3)
    assert L.moe_adamw_step(ctypes.byref(s), F, ctypes.byref(h), None, None) == code
    assert B.moe_adamw_table_bytes(s) == 0


def test_adamw_master_of_fp32(L):
    s = ashape(p="f32", master=True)
    assert table(L, s, tensors(s, [100])) == SHAPE
    with pytest.raises(ValueError):
        B.adamw_shape(1, 1, "f16")


def test_adamw_tensors(L):
    for master, bits in ((False, 32), (True, 32), (False, 8), (True, 8)):
        s = ashape(300, 2, master=master, bits=bits)
        new = lambda: tensors(s, [100, 200])    # noqa: E731
        names = ["m", "v"] + (["master"] if master else ["param"])
        names += ["m_scale", "v_scale"] if bits == 8 else []
        for k in ["grad", "param_out"] + names + [k + "_out" for k in names]:
            assert table(L, s, change(new(), 1, **{k: None})) == NULL, k
            assert table(L, s, change(new(), 1, **{k: BAD})) == ALIGN, k
        assert table(L, s, change(new(), 1, n=199)) == SHAPE      # elements is the sum
        assert table(L, s, change(new(), 1, n=-1)) == SHAPE
        assert table(L, s, change(new(), 0, weight_decay=float("nan"))) == SHAPE
        assert table(L, s, None) == NULL and table(L, s, new(), None) == NULL
        assert table(L, s, new(), BAD) == ALIGN


def test_adamw_outputs_that_share_bytes(L):
    s = ashape(300, 2, master=True, bits=8)
    new = lambda: tensors(s, [100, 200])    # noqa: E731
    a = new()
    for k in ("param_out", "m_out", "v_out", "master_out", "m_scale_out", "v_scale_out"):
        own = getattr(a[1], k)
        others = [getattr(a[0], o) for o in ("grad", "m", "v", "master", "m_scale", "v_scale", "param_out")]
        others += [a[1].grad] + [getattr(a[1], o) for o in ("m", "v", "master", "m_scale", "v_scale",
                                                            "param_out") if getattr(a[1], o) != own]
        for o in others:
            assert table(L, s, change(new(), 1, **{k: o})) == UNSUP, k
    for k in ("m", "v", "master"):                  # a part of its own input
        assert table(L, s, change(new(), 1, **{k + "_out": getattr(a[1], k) + 16})) == UNSUP, k
    # one tensor twice
    b = new()
    b[1] = b[0]
    s2 = ashape(200, 2, master=True, bits=8)
    assert table(L, s2, b) == UNSUP


def test_adamw_hyper(L):
    out = B.moe_adamw_hyper()
    ok = [1e-3, 0.9, 0.95, 1e-8, 1, 1.0, 7]

    def rc(i, v, o=out):
        a = list(ok)
        a[i] = v
        return L.moe_adamw_hyper_of(*a, ctypes.byref(o))
    assert rc(0, 1e-3) == OK and out.seed == 7
    assert abs(out.one_minus_beta1 - 0.1) < 1e-8 and abs(out.corr1 - 10) < 1e-5 and abs(out.corr2 - 20) < 1e-5
    nan, inf = float("nan"), float("inf")
    for i, v in ((0, nan), (0, inf), (1, 1.0), (1, -0.1), (1, nan), (2, 1.0), (2, -0.1), (3, 0.0), (3, nan),
                 (3, 1e-31), (3, 2.0), (4, 0), (5, inf)):
        assert rc(i, v) == SHAPE, (i, v)
    assert L.moe_adamw_hyper_of(*ok, None) == NULL
    s = ashape()
    h = ctypes.byref(out)
    assert L.moe_adamw_step(ctypes.byref(s), None, h, None, None) == NULL
    assert L.moe_adamw_step(ctypes.byref(s), F, None, None, None) == NULL
    assert L.moe_adamw_step(ctypes.byref(s), F, h, F, None) == NULL          # one of the two
    assert L.moe_adamw_step(ctypes.byref(s), BAD, h, None, None) == ALIGN
    assert L.moe_adamw_step(ctypes.byref(s), F, None, BAD, None) == ALIGN
    assert L.moe_adamw_step(ctypes.byref(ashape(0)), F, h, None, None) == OK  # nothing to do


def test_adamw_values(L):
    def rc(which=0, n=100, c=X, s=Y, o=Z):
        return L.moe_adamw_values(which, n, c, s, o, None)
    assert rc(which=2) == SHAPE and rc(n=-1) == SHAPE
    assert rc(c=None) == NULL and rc(s=None) == NULL and rc(o=None) == NULL
    assert rc(c=BAD) == ALIGN and rc(o=BAD) == ALIGN and rc(s=BAD) == ALIGN
    assert rc(o=X) == UNSUP and rc(o=X - 192) == UNSUP and rc(s=Z + 16) == UNSUP
    assert rc(n=0, c=None, s=None, o=None) == OK


def test_steps_without_a_seed_have_random_bits_of_their_own():
    import numpy as np

    import oracle
    seeds = [B.adamw_hyper(1e-3, step=t).seed for t in range(1, 201)]
    assert len(set(seeds)) == 200
    assert B.adamw_hyper(1e-3, step=5, seed=0).seed == 0 and B.adamw_hyper(1e-3, step=5, seed=9).seed == 9
    # 64 weights of 1 that fall by 2e-4, a twentieth of their step, 200 times: with bits of
    # their own in each step a weight stands still with probability (1 - 0.0512)^200 < 3e-5
    # (below 1 a step is 2^-8, of which 2e-4 is 0.0512)
    p = np.ones(64)
    for seed in seeds:
        p = oracle.round_bf16_at_random(p - 2e-4, oracle.random_bits(seed, 0, 64))
    assert (p < 1).all()
    # the average is off by less than 6 of its deviations: at most 2^-9 a step, 200 steps, 64 weights
    assert abs(p.mean() - (1 - 200 * 2e-4)) < 6 * 2.0 ** -9 * 200 ** 0.5 / 8


def test_scalars_that_fp32_does_not_hold(L):
    out = B.moe_adamw_hyper()
    for lr, scale in ((1e39, 1.0), (-1e300, 1.0), (1e-3, 1e39), (1e-3, -3.5e38)):
        assert L.moe_adamw_hyper_of(lr, 0.9, 0.95, 1e-8, 1, scale, 0, ctypes.byref(out)) == SHAPE, (lr, scale)
    assert L.moe_adamw_hyper_of(3e38, 0.9, 0.95, 1e-8, 1, -3e38, 0, ctypes.byref(out)) == OK


def test_norm_eps_below_the_normal_numbers(L):
    for eps in (1.4e-45, 1e-40, 2.0 ** -127):
        s = B.norm_shape(4, 64, "rms", eps)
        assert s.eps > 0 and fwd(L, s) == SHAPE and bwd(L, s) == SHAPE and B.moe_norm_workspace_bytes(s) == 0
    s = B.norm_shape(0, 64, "rms", 2.0 ** -126)
    assert fwd(L, s, x=None, y=None, stats=None) == OK


def partly(at, size, own):
    """Aligned places of `own` bytes that share some with [at, at + size)"""
    return [p for p in (at, at + 16, at - 16, at + size - 16, at - own + 16)
            if p < at + size and at < p + own and p % 16 == 0]


def test_norm_outputs_over_the_other_inputs(L):
    T, H = 64, 512
    s = B.norm_shape(T, H)
    far = dict(w=0x5000000, b=0x6000000, stats=0x7000000)
    for f, e in (("bf16", 2), ("f32", 4)):
        name, row, n, st = "moe_norm_" + f, H * e, T * H * e, T * 8
        for k in ("w", "b"):
            for p in partly(far[k], row, n):
                assert fwd(L, s, name, **dict(far, y=p)) == UNSUP
                assert fwd(L, s, name, **dict(far, res=FAR, h=p)) == UNSUP
            for p in partly(far[k], row, st):
                assert fwd(L, s, name, **dict(far, stats=p)) == UNSUP
        for at in (X, Y, FAR, Z):
            for p in partly(at, n, st):
                assert fwd(L, s, name, **dict(far, res=FAR, h=Z, stats=p)) == UNSUP
    # no rows, no bytes
    assert fwd(L, B.norm_shape(0, H), y=F + 16, stats=F + 16) == OK


def test_norm_gradients_over_the_other_inputs(L):
    """The same for few rows, whose column sums run beside them, and for many."""
    H = 512
    buf = dict(h=X, w=0x5000000, stats=0x6000000, dy=Y, dh=FAR, dx=Z, dw=0x7000000, db=0x7800000, ws=0xB0000000)
    for T in (16, 256, 2000):
        s = B.norm_shape(T, H)
        for f, e in (("bf16", 2), ("f32", 4)):
            name, row, n, wn = "moe_norm_backward_" + f, H * e, T * H * e, B.moe_norm_workspace_bytes(s)
            size = dict(h=n, w=row, stats=T * 8, dy=n, dh=n, dx=n, dw=row, db=row, ws=wn)
            pairs = [("dx", k) for k in ("h", "w", "stats")]
            pairs += [(d, k) for d in ("dw", "db") for k in ("h", "w", "stats", "dy", "dh", "dx")]
            pairs += [("dw", "db"), ("db", "dw")] + [("ws", k) for k in size if k != "ws"]
            for out, k in pairs:
                for p in partly(buf[k], size[k], size[out]):
                    assert bwd(L, s, name, **dict(buf, **{out: p})) == UNSUP, (T, f, out, k, p - buf[k])
    # without dw and db ws is not looked at (no rows: nothing is launched)
    s = B.norm_shape(0, H)
    assert bwd(L, s, **dict(buf, ws=X, dw=None, db=None)) == OK


def test_balance_buffers_that_share_bytes(L):
    s, ba = shape(T=512, E=64, k=4), B.balance("sigmoid", 0.01, 5)
    n = B.moe_balance_workspace_bytes(s, ba)
    at = dict(logits=X, idx=Y, start=0x4000000, out=0x5000000, counts=0x6000000, scales=0x7000000, ws=0x8000000)
    size = dict(logits=512 * 64 * 4, idx=512 * 4 * 4, start=24, out=4, counts=5 * 64 * 4, scales=20, ws=n)
    for o in ("out", "counts", "scales", "ws"):
        for k in size:
            if k != o:
                for p in partly(at[k], size[k], size[o]):
                    assert loss(L, s, ba, n=n, **dict(at, **{o: p})) == UNSUP, (o, k, p - at[k])


def test_balance_gradient_over_the_other_inputs(L):
    s, ba = shape(T=512, E=64, k=4), B.balance("sigmoid", 0.01, 5)
    at = dict(logits=X, idx=Y, start=0x4000000, counts=0x5000000, scales=0x6000000, d_loss=0x7000000)
    size = dict(idx=512 * 4 * 4, start=24, counts=5 * 64 * 4, scales=20, d_loss=4)
    for k in size:
        for p in partly(at[k], size[k], 512 * 64 * 4):
            assert back(L, s, ba, **dict(at, dL=p)) == UNSUP, (k, p - at[k])
    assert back(L, shape(T=0), ba, **dict(at, dL=0x5000010)) == OK      # no rows, no bytes


def test_adamw_table_over_a_tensor(L):
    """The steps read addresses from it: with a gradient in its place they would go anywhere."""
    for master, bits in ((False, 32), (True, 8)):
        s = ashape(300000, 2, master=master, bits=bits)
        arr = tensors(s, [100000, 200000])
        n = B.moe_adamw_table_bytes(s)
        for i, count in ((0, 100000), (1, 200000)):
            names = ["grad", "m", "v", "param_out", "m_out", "v_out"] + (["master"] if master else ["param"])
            names += ["m_scale", "v_scale_out"] if bits == 8 else []
            for k in names:
                at = getattr(arr[i], k)
                size = (count + 31) // 32 if "scale" in k else count     # or more
                for p in partly(at, size, n):
                    assert table(L, s, arr, p) == UNSUP, (k, p - at)


def test_balance_reads_three_sizes_of_the_shape(L):
    """T, E and k alone: the layer's other limits do not hold for it."""
    ba = B.balance("softmax", 0.01, 3)
    full = B.moe_balance_workspace_bytes(shape(), ba)
    for kw in (dict(H=0), dict(H=100), dict(H=-8, I=-1), dict(flags=1 << 30, I_shared=5, T_minibatch=-2)):
        s = shape(**kw)
        assert B.moe_balance_workspace_bytes(s, ba) == full
        assert loss(L, s, ba, n=full - 1) == WS and back(L, s, ba, dL=F) == UNSUP    # past the shape's check
        assert back(L, shape(T=0, **kw), ba, logits=None, idx=None, dL=None) == OK
    assert loss(L, shape(H=0, k=17), ba) == SHAPE
    s = shape(T=1 << 26, E=64, k=32, H=0)       # T k = 2^31
    assert loss(L, s, ba) == SHAPE
