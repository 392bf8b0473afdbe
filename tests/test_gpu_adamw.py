"""GPU parity of the AdamW step: states and their codes bit for bit, parameters within the
roundings of the formula.

p' = p - lr (u + wd p): u is off by 8 units of itself (two products, a root and a reciprocal
of one unit each, a sum), the two fused products by a unit of each term, the result by half.
bf16 parameters rounded at random go up or down by a rule that ascends in p', so that they lie
between the rule's results at both ends of p's bound."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import digest, np_, say
from step_tol import U, UB, f64

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
KINDS = [(p, g, m, b) for p, g, m in [("f32", "f32", False), ("f32", "bf16", False), ("bf16", "bf16", False),
                                      ("bf16", "f32", False), ("bf16", "bf16", True), ("bf16", "f32", True)]
         for b in (32, 8)]


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_plan_amd import binding
    return binding


def make(sizes, p, g, master, bits, seed=0):
    """Host tensors of a table: gradients and states that span orders of magnitude."""
    rng = np.random.default_rng(seed)
    out = []
    for j, n in enumerate(sizes):
        size = (1e-3 * np.exp2(3 * rng.standard_normal(n))).astype(np.float32)
        t = {"grad": torch.tensor(rng.standard_normal(n).astype(np.float32) * size).to(DT[g])}
        w = torch.tensor((rng.standard_normal(n) * 0.05).astype(np.float32))
        t["param"] = w.to(DT[p])
        if master:
            t["master"] = w
        m = (rng.standard_normal(n) * 0.5).astype(np.float32) * size
        v = (rng.random(n).astype(np.float32) + 0.1) * size * size
        m[::7], v[::7] = 0.0, 0.0                   # untouched so far
        t["grad"][::21] = 0.0
        if bits == 8:
            r = rng.integers(0, 65536, n)
            for k, x in (("m", m), ("v", v)):
                c, s = oracle.encode_state(x, r, k)
                t[k], t[k + "_scale"] = torch.tensor(c), torch.tensor(s)
        else:
            t["m"], t["v"] = torch.tensor(m), torch.tensor(v)
        t["weight_decay"] = 0.1 * (j % 3)
        out.append(t)
    return out


def as_dict(h):
    return {k: getattr(h, k) for k, _ in h._fields_}


def table(B, host, p, g, master, bits, in_place=False):
    """(shape, device tensors, their outputs, table, checks of guard zones)"""
    dev, outs, oks = [], [], []
    for t in host:
        d, o = {}, {}
        for k, v in t.items():
            if k == "weight_decay":
                d[k] = v
                continue
            n = v.numel()
            if k == "grad":
                d[k] = v.cuda()
                continue
            buf = torch.full((n + 128,), 77, dtype=v.dtype, device="cuda")

            def ok(buf=buf, n=n):
                assert bool((buf[:64] == 77).all()) and bool((buf[64 + n:] == 77).all())
            oks.append(ok)
            o[k] = buf[64:64 + n]
            if in_place:
                o[k].copy_(v)
                d[k] = o[k]
            else:
                d[k] = v.cuda()
                d[k + "_out"] = o[k]
        dev.append(d)
        outs.append(o)
    s = B.adamw_shape(sum(t["grad"].numel() for t in host), len(host), p, g, master, bits)
    tab = torch.empty(B.moe_adamw_table_bytes(s), dtype=torch.uint8, device="cuda")
    B.moe_adamw_table(s, dev, tab)
    return s, dev, outs, tab, oks


def verify(host, outs, p, master, bits, h, tensor0=0):
    for j, (t, o) in enumerate(zip(host, outs)):
        n = t["grad"].numel()
        g = t["grad"].float().numpy()
        if bits == 8:
            m = oracle.decode_state(t["m"].numpy(), t["m_scale"].numpy(), "m").astype(np.float32)
            v = oracle.decode_state(t["v"].numpy(), t["v_scale"].numpy(), "v").astype(np.float32)
        else:
            m, v = t["m"].numpy(), t["v"].numpy()
        m2, v2 = oracle.adamw_states(g, m, v, h)
        r = oracle.random_bits(h["seed"], tensor0 + j, n)
        if bits == 8:
            for k, x, rr in (("m", m2, r & 0xFFFF), ("v", v2, r >> 16)):
                c, s = oracle.encode_state(x, rr, k)
                np.testing.assert_array_equal(np_(o[k + "_scale"]), s, err_msg=k)
                np.testing.assert_array_equal(np_(o[k]), c, err_msg=k)
        else:
            np.testing.assert_array_equal(np_(o["m"]).view(np.uint32), m2.view(np.uint32))
            np.testing.assert_array_equal(np_(o["v"]).view(np.uint32), v2.view(np.uint32))
        p0 = f64(t["master"] if master else t["param"])
        p1, lu, lw = oracle.adamw_param(p0, m2, v2, h, t["weight_decay"])
        err = 8 * U * lu + 3 * U * (lu + lw) + U * np.abs(p1) + 1e-42
        got = f64(o["param"])
        if master:
            assert (np.abs(f64(o["master"]) - p1) <= err).all()
            assert torch.equal(o["param"], o["master"].to(torch.bfloat16))
        elif p == "f32":
            assert (np.abs(got - p1) <= err).all()
        else:
            a, b = (oracle.round_bf16_at_random(p1 + e, r) for e in (-err, err))
            assert ((np.minimum(a, b) <= got) & (got <= np.maximum(a, b))).all()
            assert n < 20 or (a == b).mean() > 0.9


SIZES = [[1], [31], [32, 33], [7, 8, 9, 2047, 2048, 2049], [8191, 8192, 8193, 1, 0, 5000], [0, 40, 0]]


@pytest.mark.parametrize("p,g,master,bits", KINDS)
@pytest.mark.parametrize("sizes", SIZES)
def test_parity(B, sizes, p, g, master, bits):
    say(f"adamw {sizes} p={p} g={g} master={master} bits={bits}")
    host = make(sizes, p, g, master, bits, len(sizes))
    for in_place, step in ((False, 1), (True, 1000)):
        h = B.adamw_hyper(3e-3, 0.9, 0.95, 1e-8, step, 0.75, 12345 + step)
        s, dev, outs, tab, oks = table(B, host, p, g, master, bits, in_place)
        B.moe_adamw_step(s, tab, h)
        torch.cuda.synchronize()
        for ok in oks:
            ok()
        verify(host, outs, p, master, bits, as_dict(h))


def test_many_tensors(B):
    """More tensors than one level of the search over tiles and one launch of the table."""
    say("adamw of 300 and 5000 tensors")
    for count in (300, 5000):
        sizes = [(i * 37) % 23 for i in range(count)]
        host = make(sizes, "bf16", "bf16", False, 8, count)
        s, dev, outs, tab, oks = table(B, host, "bf16", "bf16", False, 8)
        h = B.adamw_hyper(1e-2, step=3, seed=9)
        B.moe_adamw_step(s, tab, h)
        torch.cuda.synchronize()
        verify(host, outs, "bf16", False, 8, as_dict(h))


def test_a_run_of_steps_from_zero(B):
    """States that start as zeroed buffers, in place, each step's state the next one's input."""
    say("adamw of six steps from zero")
    for bits in (32, 8):
        host = make([700, 33], "bf16", "bf16", True, bits, 4)
        for t in host:
            for k in ("m", "v", "m_scale", "v_scale"):
                if k in t:
                    t[k] = torch.zeros_like(t[k])
        s, dev, outs, tab, oks = table(B, host, "bf16", "bf16", True, bits, True)
        for step in range(1, 7):
            h = B.adamw_hyper(1e-2, step=step, seed=step)
            before = [{k: v.cpu().clone() if torch.is_tensor(v) else v for k, v in d.items()} for d in dev]
            B.moe_adamw_step(s, tab, h)
            torch.cuda.synchronize()
            verify(before, outs, "bf16", True, bits, as_dict(h))
            for d in dev:
                d["grad"].mul_(-0.5)


@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_that_are_not_finite(B, bits):
    say("adamw with inf and NaN gradients", bits)
    host = make([200], "f32", "f32", False, bits, 1)
    host[0]["grad"][40] = float("nan")
    host[0]["grad"][100] = float("inf")
    s, dev, outs, tab, oks = table(B, host, "f32", "f32", False, bits)
    B.moe_adamw_step(s, tab, B.adamw_hyper(1e-2, seed=3))
    torch.cuda.synchronize()
    o = outs[0]
    clean = [t.clone() for t in (host[0]["grad"],)][0]
    clean[40] = clean[100] = 0.0
    same = dict(host[0], grad=clean)
    s2, _, outs2, tab2, _ = table(B, [same], "f32", "f32", False, bits)
    B.moe_adamw_step(s2, tab2, B.adamw_hyper(1e-2, seed=3))
    torch.cuda.synchronize()
    bad = torch.zeros(200, dtype=torch.bool)
    bad[[40, 100]] = True
    assert torch.isnan(o["param"][[40, 100]]).all()
    assert torch.equal(o["param"].cpu()[~bad], outs2[0]["param"].cpu()[~bad])
    if bits == 8:       # the blocks of 32 around them are lost, and no others
        assert np_(o["m_scale"]).tolist()[1] == 255 and np_(o["v_scale"]).tolist()[3] == 255
        keep = [0, 2, 4, 5, 6]
        assert torch.equal(o["m_scale"][keep], outs2[0]["m_scale"][keep])
        vals = torch.empty((200,), dtype=torch.bfloat16, device="cuda")
        B.moe_adamw_values("m", o["m"].clone(), o["m_scale"].clone(), vals)
        assert torch.isnan(vals[32:64]).all() and torch.isnan(vals[96:128]).all()
        assert torch.isfinite(vals[:32]).all() and torch.isfinite(vals[128:]).all()
    else:
        assert torch.isnan(o["m"][40]) and torch.isinf(o["v"][100])


def test_extreme_magnitudes(B):
    """Subnormal and huge gradients, zero weights, blocks of one value."""
    say("adamw at the ends of the range")
    for bits in (32, 8):
        host = make([640], "f32", "f32", False, bits, 2)
        g = host[0]["grad"]
        g[:32] = 1e-42
        g[32:64] = 1e18
        g[64:96] = 0.0
        g[96:128] *= 1e-25
        g[128] = 1e10
        for k in ("m", "v", "m_scale", "v_scale"):
            if k in host[0]:
                host[0][k][:128 if "scale" not in k else 4] = 0
        h = B.adamw_hyper(1e-2, step=1, grad_scale=1.0, seed=77)
        s, dev, outs, tab, oks = table(B, host, "f32", "f32", False, bits)
        B.moe_adamw_step(s, tab, h)
        torch.cuda.synchronize()
        verify(host, outs, "f32", False, bits, as_dict(h))


@pytest.mark.parametrize("bits", [32, 8])
def test_denominators_below_the_normal_numbers(B, bits):
    """v of tiny gradients is subnormal; its root is not, and with a tiny eps it is the
    denominator."""
    say(f"adamw subnormal v bits={bits}")
    for eps in (1e-30, 1e-12):
        host = make([4096], "f32", "f32", False, bits, 5)
        g = host[0]["grad"]
        g *= torch.logspace(-21, -12, 4096).flip(0)
        for k in ("m", "v", "m_scale", "v_scale"):
            if k in host[0]:
                host[0][k][:] = 0
        h = B.adamw_hyper(1e-2, eps=eps, step=1, seed=78)
        s, dev, outs, tab, oks = table(B, host, "f32", "f32", False, bits)
        B.moe_adamw_step(s, tab, h)
        torch.cuda.synchronize()
        verify(host, outs, "f32", False, bits, as_dict(h))


def test_values_of_codes(B):
    say("adamw values of codes")
    for n in (1, 31, 32, 100, 2048, 5000):
        for which in ("m", "v"):
            rng = np.random.default_rng(n)
            x = (rng.standard_normal(n) * np.exp2(rng.integers(-30, 30, n))).astype(np.float32)
            c, s = oracle.encode_state(np.abs(x) if which == "v" else x, rng.integers(0, 65536, n), which)
            buf = torch.full((n + 128,), 77, dtype=torch.bfloat16, device="cuda")
            out = buf[64:64 + n]
            B.moe_adamw_values(which, torch.tensor(c).cuda(), torch.tensor(s).cuda(), out)
            torch.cuda.synchronize()
            np.testing.assert_array_equal(f64(out), oracle.decode_state(c, s, which))
            assert bool((buf[:64] == 77).all()) and bool((buf[64 + n:] == 77).all())
    every = torch.arange(256, dtype=torch.uint8).cuda()
    scale = torch.full((8,), 127, dtype=torch.uint8, device="cuda")
    out = torch.empty((256,), dtype=torch.bfloat16, device="cuda")
    B.moe_adamw_values("v", every, scale, out)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(f64(out), oracle.step.V_VALUES)


def test_scalars_on_the_device_and_a_graph(B):
    """A captured step replays with the scalars that lie on the device then."""
    say("adamw scalars on the device, graph")
    host = make([3000, 77], "bf16", "bf16", False, 8, 6)
    s, dev, outs, tab, oks = table(B, host, "bf16", "bf16", False, 8)
    names = ("param", "m", "v", "m_scale", "v_scale")
    hd = torch.zeros((40,), dtype=torch.uint8, device="cuda")

    def put(h):
        hd.copy_(torch.frombuffer(bytearray(bytes(h)), dtype=torch.uint8))
    put(B.adamw_hyper(1e-2, step=1, seed=1))
    B.moe_adamw_step(s, tab, hd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_adamw_step(s, tab, hd)
    for step in (1, 2, 50):
        h = B.adamw_hyper(1e-2 / step, step=step, grad_scale=0.5, seed=step)
        put(h)
        graph.replay()
        torch.cuda.synchronize()
        got = digest(*[o[k] for o in outs for k in names])
        B.moe_adamw_step(s, tab, h)
        torch.cuda.synchronize()
        assert digest(*[o[k] for o in outs for k in names]) == got
        verify(host, outs, "bf16", False, 8, as_dict(h))


def test_repeated_and_on_another_stream(B):
    say("adamw repeated, another stream")
    host = make([50000], "bf16", "bf16", True, 8, 3)
    digests = set()
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.current_stream()):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            s, dev, outs, tab, oks = table(B, host, "bf16", "bf16", True, 8)
            B.moe_adamw_step(s, tab, B.adamw_hyper(1e-2, seed=4))
        torch.cuda.synchronize()
        digests.add(digest(*outs[0].values()))
    assert len(digests) == 1


def test_tensors_that_do_not_fit(B):
    say("adamw refusals of the binding")
    host = make([64], "bf16", "bf16", False, 8, 1)
    s = B.adamw_shape(64, 1, "bf16", "bf16", False, 8)
    d = {k: v.cuda() if torch.is_tensor(v) else v for k, v in host[0].items()}
    tab = torch.empty(B.moe_adamw_table_bytes(s), dtype=torch.uint8, device="cuda")
    B.moe_adamw_table(s, [d], tab)
    for k, v in (("grad", d["grad"].float()), ("m", d["m"][:32]), ("v_scale", d["v_scale"][:1]),
                 ("param", d["param"].cpu()), ("m_out", d["m"].float())):
        with pytest.raises(ValueError):
            B.moe_adamw_table(s, [dict(d, **{k: v})], tab)
    with pytest.raises(ValueError):
        B.moe_adamw_table(s, [d, d], tab)
    with pytest.raises(ValueError):
        B.moe_adamw_table(s, [dict(d, master=d["param"].float())], tab)
    with pytest.raises(B.MoeError):
        B.moe_adamw_table(s, [dict(d, m_out=d["v"])], tab)


def test_elements_past_32_bits(B):
    """The last elements of a tensor of more than 2^32 (in 8 bits: 26 GB)."""
    say("adamw of 2^32 + 100 elements")
    n = (1 << 32) + 100
    t = {k: torch.zeros((n,), dtype=torch.bfloat16, device="cuda") for k in ("grad", "param")}
    t.update({k: torch.zeros((n,), dtype=torch.uint8, device="cuda") for k in ("m", "v")})
    t.update({k: torch.zeros(((n + 31) // 32,), dtype=torch.uint8, device="cuda") for k in ("m_scale", "v_scale")})
    tail = make([164], "bf16", "bf16", False, 8, 2)[0]
    first = n - 164                     # a multiple of 32
    for k in ("grad", "param", "m", "v"):
        t[k][first:] = tail[k].cuda()
    for k in ("m_scale", "v_scale"):
        t[k][first // 32:] = tail[k].cuda()
    s = B.adamw_shape(n, 1, "bf16", "bf16", False, 8)
    tab = torch.empty(B.moe_adamw_table_bytes(s), dtype=torch.uint8, device="cuda")
    B.moe_adamw_table(s, [t], tab)
    h = B.adamw_hyper(1e-2, step=2, seed=5)
    B.moe_adamw_step(s, tab, h)
    torch.cuda.synchronize()
    d = as_dict(h)
    m, v = (oracle.decode_state(tail[k].numpy(), tail[k + "_scale"].numpy(), k).astype(np.float32) for k in "mv")
    m2, v2 = oracle.adamw_states(tail["grad"].float().numpy(), m, v, d)
    r = oracle.random_bits(5, 0, 164, first)
    for k, x, rr in (("m", m2, r & 0xFFFF), ("v", v2, r >> 16)):
        c, sc = oracle.encode_state(x, rr, k)
        np.testing.assert_array_equal(np_(t[k][first:]), c)
        np.testing.assert_array_equal(np_(t[k + "_scale"][first // 32:]), sc)
    assert not t["param"][:first:4097].any() and not t["m"][:first:4097].any()


def test_copies_of_masters_at_the_ends_of_bf16(B):
    """Subnormal masters, ties and values past bf16's largest: the conversion is torch's."""
    say("adamw copies of masters")
    w = torch.tensor([1e-40, -1e-40, 2.0 ** -133, 1.5 * 2.0 ** -133, 2.0 ** -126, 3.4e38, -3.4e38, 3.3895e38,
                      1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 0.0, -0.0] * 5)
    n = w.numel()
    z = dict(dtype=torch.float32)
    host = [{"grad": torch.zeros(n, dtype=torch.bfloat16), "param": torch.zeros(n, dtype=torch.bfloat16),
             "master": w, "m": torch.zeros(n, **z), "v": torch.zeros(n, **z), "weight_decay": 0.0}]
    s, dev, outs, tab, oks = table(B, host, "bf16", "bf16", True, 32)
    B.moe_adamw_step(s, tab, B.adamw_hyper(1e-3, seed=1))
    torch.cuda.synchronize()
    assert torch.equal(outs[0]["master"].cpu(), w)
    assert torch.equal(outs[0]["param"].cpu().view(torch.int16), w.bfloat16().view(torch.int16))


def test_nan_weights_stay_nan(B):
    """Also those whose bits are all ones, which a rounding by addition would carry to zero."""
    say("adamw with NaN weights")
    bits = torch.tensor([0x7FFF, -1, 0x7F81, 0x7FC0, 0x7F80, -0x80] * 8, dtype=torch.int16)
    n = bits.numel()
    gbits = torch.tensor([-1, 0x7FFFFFFF, 0x7FC00000] * (n // 3), dtype=torch.int32)
    for gtype in ("bf16", "f32"):
        g = torch.zeros(n, dtype=DT[gtype]) if gtype == "bf16" else gbits.view(torch.float32)
        host = [{"grad": g, "param": bits.view(torch.bfloat16) if gtype == "bf16" else torch.ones(n).bfloat16(),
                 "m": torch.zeros(n), "v": torch.zeros(n), "weight_decay": 0.0}]
        for seed in range(4):
            s, dev, outs, tab, oks = table(B, host, "bf16", gtype, False, 32)
            B.moe_adamw_step(s, tab, B.adamw_hyper(1e-3, seed=seed))
            torch.cuda.synchronize()
            got = outs[0]["param"].cpu()
            # (an infinite weight becomes one too: weight_decay p is 0 times inf)
            assert torch.isnan(got).all()


def test_two_steps_at_once(B):
    """Two tables on two streams given by argument: nothing is shared between calls."""
    say("adamw of two tables at once")
    hosts = [make([300000], "bf16", "bf16", True, 8, k) for k in (1, 2)]
    h = B.adamw_hyper(1e-2, seed=4)
    alone, both = [], []
    for out, streams in ((alone, [None, None]), (both, [torch.cuda.Stream(), torch.cuda.Stream()])):
        tabs = [table(B, host, "bf16", "bf16", True, 8) for host in hosts]
        torch.cuda.synchronize()
        for _ in range(3):
            for (s, _, _, tab, _), st in zip(tabs, streams):
                B.moe_adamw_step(s, tab, h, stream=st)
        torch.cuda.synchronize()
        out += [digest(*t[2][0].values()) for t in tabs]
    assert alone == both
