"""GPU parity of the balance loss, the experts' counts and the gradient against the fp64
oracle; tolerances: step_tol.share_rel, sums of fp32 in their depth."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import digest, np_, say
from step_tol import U, check, share_rel
from test_gpu_norm import guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from mixture_experts_layer_plan_amd import binding
    return binding


def inputs(T, E, k, seed=0, free=0.0):
    rng = np.random.default_rng(seed + 31 * T + E)
    L = (rng.standard_normal((T, E)) * 2 - 0.5 * np.log(1 + rng.permutation(E))).astype(np.float32)
    idx = np.argsort(-L, 1, kind="stable")[:, :k].astype(np.int32)
    idx[rng.random(T) < free] = -1
    return L, idx


def run(B, L, idx, score, coef=0.3, start=None, d_loss=None, d_in=None):
    T, E = L.shape
    n_seq = 1 if start is None else len(start) - 1
    s, ba = B.shape(T, 128, 128, E, idx.shape[1]), B.balance(score, coef, n_seq)
    c = lambda a, t: None if a is None else torch.as_tensor(np.asarray(a), dtype=t).cuda()    # noqa: E731
    Ld, ix, st = c(L, torch.float32), c(idx, torch.int32), c(start, torch.int32)
    dl, di = c(d_loss, torch.float32), c(d_in, torch.float32)
    loss, o1 = guarded((1,), torch.float32)
    counts, o2 = guarded((n_seq, E), torch.int32)
    scales, o3 = guarded((n_seq,), torch.float32)
    dL, o4 = guarded((T, E), torch.float32)
    ws, o5 = guarded((B.moe_balance_workspace_bytes(s, ba),), torch.uint8)
    B.moe_balance_loss(s, ba, Ld, ix, st, loss, counts, scales, ws)
    B.moe_balance_loss_backward(s, ba, Ld, ix, st, counts, scales, dl, di, dL)
    torch.cuda.synchronize()
    for ok in (o1, o2, o3, o4, o5):
        ok()
    return loss, counts, scales, dL


def verify(B, L, idx, score, coef=0.3, start=None, d_loss=None, d_in=None):
    loss, counts, scales, dL = run(B, L, idx, score, coef, start, d_loss, d_in)
    T = len(L)
    rl, rc, rs, where = oracle.balance(L, idx, score, coef, start)
    np.testing.assert_array_equal(np_(counts), rc)
    check(scales, rs, 4 * U * np.abs(rs), "scales")
    tau = share_rel(L)
    # a wavefront's tokens, the chunks by sixteenths, 64 experts, and the rest in 64 bits
    check(loss, np.array([rl]), (tau + (160 + T / 512) * U) * abs(rl) + 1e-38, "loss")
    up = 1.0 if d_loss is None else float(d_loss[0])
    ref = oracle.balance_backward(L, idx, score, coef, start, up, d_in)
    add = 0.0 if d_in is None else np.asarray(d_in, np.float64)
    bound = np.zeros_like(ref)
    for t, i in enumerate(where):
        if i >= 0:
            p = oracle.step.shares(L[t].astype(np.float64), score)
            dot = (p * rc[i]).sum()
            own = abs(up * rs[i]) * p
            bound[t] = own * ((tau + 12 * U) * np.abs(rc[i] - dot) + (tau + 24 * U) * dot) * 1.01
    check(dL, ref, bound + 2 * U * (np.abs(add) + np.abs(ref)) + 1e-38, "d_logits")
    return loss, counts, dL


SIZES = [(1, 1, 1), (1, 4, 1), (3, 8, 2), (16, 8, 2), (17, 60, 6), (64, 64, 6), (33, 65, 5), (200, 128, 8),
         (65, 256, 8), (40, 257, 32), (300, 60, 4), (20, 1000, 9), (11, 1024, 32), (1003, 24, 3),
         (64, 200, 8), (65, 100, 3), (64, 128, 5), (128, 64, 6), (129, 64, 6), (64, 255, 2)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_parity(B, T, E, k, score):
    say(f"balance T={T} E={E} k={k} {score}")
    L, idx = inputs(T, E, k, free=0.1)
    rng = np.random.default_rng(1)
    verify(B, L, idx, score)
    verify(B, L, idx, score, -2.0, None, [2.5], rng.standard_normal((T, E)).astype(np.float32))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("start", [[0, 100], [5, 90], [0, 1, 2, 3, 100], [0, 16, 32, 100], [0, 0, 0, 50, 50, 99],
                                   [0, 15, 17, 33, 64, 64, 65, 80], [100, 100], [0, 0], [99, 100, 100],
                                   list(range(0, 101)), [0] * 70 + [3] * 70 + [77] * 70])
def test_sequences(B, start, score):
    say(f"balance sequences {start[:8]} ({len(start) - 1}) {score}")
    L, idx = inputs(100, 40, 3, free=0.2)
    d_in = np.random.default_rng(2).standard_normal((100, 40)).astype(np.float32)
    _, _, dL = verify(B, L, idx, score, 0.3, start, None, d_in)
    # rows outside every sequence stay as they were, bit for bit
    out = [t for t in range(100) if t < start[0] or t >= start[-1]]
    np.testing.assert_array_equal(np_(dL)[out], d_in[out])


def test_many_sequences(B):
    say("balance of 5000 sequences")
    rng = np.random.default_rng(8)
    L, idx = inputs(6000, 12, 2, free=0.3)
    start = np.sort(rng.integers(0, 6001, 5001))
    verify(B, L, idx, "softmax", 1.0, start)


def test_more_sequences_than_one_grid(B):
    """2^20 sequences of 33 experts, most of them empty: more than a launch of the join takes
    at once."""
    say("balance of 2^20 sequences")
    n = 1 << 20
    L, idx = inputs(300, 33, 2)
    start = np.full(n + 1, 300)
    start[:n - 200] = 0
    start[n - 200:n] = np.arange(200)      # 199 of one token, the last of 101
    loss, counts, scales, dL = run(B, L, idx, "softmax", 1.0, start)
    first = n - 200
    rl, rc, rs, _ = oracle.balance(L, idx, "softmax", 1.0, start[first:])
    np.testing.assert_array_equal(np_(counts[first:]), rc)
    assert not counts[:first].any() and not scales[:first].any()
    check(scales[first:], rs, 4 * U * rs, "scales")
    check(loss, np.array([rl]), (share_rel(L) + 161 * U) * rl, "loss")
    ref = oracle.balance_backward(L, idx, "softmax", 1.0, start[first:])
    assert np.abs(np_(dL) - ref).max() <= (2 * share_rel(L) + 40 * U) * np.abs(rs).max() * rc.max()


@pytest.mark.parametrize("T,E", [(40000, 3), (2100, 1000), (5000, 500)])
def test_chunks_of_several_rounds(B, T, E):
    """More tokens than 1024 chunks of one round hold, with sequences that begin inside."""
    say(f"balance of {T} x {E} in long chunks")
    L, idx = inputs(T, E, 2, free=0.05)
    start = [3, 50, T // 3, T // 3 + 1, T - 5]
    verify(B, L, idx, "sigmoid", 1.0, start)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_no_tokens_or_none_with_an_expert(B, score):
    say("balance without tokens", score)
    for T in (0, 1, 50):
        L, idx = inputs(T, 9, 2)
        idx[:] = -1
        loss, counts, scales, dL = run(B, L, idx, score)
        assert float(loss) == 0 and not counts.any() and not scales.any() and not dL.any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_logits_out_of_play_and_extreme(B, score):
    say("balance with -inf, NaN and the lowest logits", score)
    rng = np.random.default_rng(3)
    L, idx = inputs(60, 24, 4)
    out = rng.random(L.shape) < 0.5
    out[np.arange(60)[:, None], idx] = False      # the chosen ones are in play
    L[out] = -np.inf
    L[rng.random(L.shape) < 0.02] = np.nan
    L[7] = -np.inf                                 # nothing in play, though with experts
    L[8] = np.nan
    verify(B, L, idx, score)
    L, idx = inputs(8, 24, 4)
    L[0] = np.finfo(np.float32).min
    L[1] = 88.0
    L[2] = -300.0
    L[2, 3] = -299.0
    L[3, :] = -200.0
    L[3, 2] = 100.0
    L[4, 5] = np.finfo(np.float32).min
    rows = [1, 2, 3, 4, 5, 6, 7]
    verify(B, L[rows[:3]], idx[rows[:3]], score)
    loss, _, _, dL = run(B, L, idx, score)
    assert torch.isfinite(dL).all() and torch.isfinite(loss).all()
    # equal logits have equal shares, however low
    np.testing.assert_allclose(oracle.step.shares(L[0].astype(np.float64), score), 1 / 24, rtol=1e-12)
    one = np.repeat(L[:1], 4, 0)
    loss, _, _, _ = run(B, one, np.array([[0, 1, 2, 3]] * 4, np.int32), score, 1.0)
    assert abs(float(loss) - 1.0) < 1e-5


def test_bad_experts_are_left_out(B):
    say("balance with ids out of range")
    L, idx = inputs(50, 10, 3)
    idx[4] = [10, -1, 3]
    idx[5] = [2 ** 31 - 1, -2 ** 31, 1000]
    verify(B, L, idx, "softmax")


def test_the_same_expert_twice(B):
    say("balance with a repeated id")
    L, idx = inputs(30, 10, 3)
    idx[:, 1] = idx[:, 0]
    verify(B, L, idx, "sigmoid")


def test_in_place(B):
    say("balance in place")
    L, idx = inputs(70, 20, 4)
    d_in = np.random.default_rng(0).standard_normal(L.shape).astype(np.float32)
    _, counts, scales, ref = run(B, L, idx, "softmax", d_in=d_in)
    s, ba = B.shape(70, 128, 128, 20, 4), B.balance("softmax", 0.3, 1)
    Ld, ix, di = torch.as_tensor(L).cuda(), torch.as_tensor(idx).cuda(), torch.as_tensor(d_in).cuda()
    for target in (di, Ld):
        d0 = torch.as_tensor(d_in).cuda()
        B.moe_balance_loss_backward(s, ba, Ld, ix, None, counts.contiguous(), scales.contiguous(), None,
                                    target if target is di else d0, target)
        assert torch.equal(target, ref)


def test_sequences_that_do_not_ascend_end(B):
    """Unspecified results, but no access out of bounds and no endless loop (the search and
    both walks are bounded whatever the entries hold: see the guards)."""
    say("balance with entries that do not ascend")
    L, idx = inputs(90, 12, 2)
    for start in ([50, 10, 90], [-5, 200, 3], [90, 0, 0], [7, 7, 2 ** 31 - 1], [-2 ** 31, 5, -7]):
        run(B, L, idx, "softmax", start=start)


def test_gradient_against_differences(B):
    """The loss's own change along a direction with the choice held fixed.  A central
    difference is off by its truncation, which the oracle gives, and by the rounding of the
    two losses (their bound in verify)."""
    say("balance by differences")
    for score in ("softmax", "sigmoid"):
        L, idx = inputs(40, 8, 2)
        v = np.random.default_rng(1).standard_normal(L.shape)
        e = 2.0 ** -5
        hi, lo = (L + e * v).astype(np.float32), (L - e * v).astype(np.float32)
        step = hi.astype(np.float64) - lo
        grad = np_(run(B, L, idx, score, 1.0)[3]).astype(np.float64)
        num = float(run(B, hi, idx, score, 1.0)[0]) - float(run(B, lo, idx, score, 1.0)[0])
        rh, rl = (oracle.balance(a, idx, score, 1.0)[0] for a in (hi, lo))
        ref = (oracle.balance_backward(L, idx, score, 1.0) * step).sum()
        noise = 2 * (share_rel(L) + 161 * U) * max(rh, rl)
        bound = abs(rh - rl - ref) + noise + 1e-4 * np.abs(grad * step).sum()
        assert abs(num - (grad * step).sum()) <= bound, (score, num, bound)
        assert bound < 0.2 * abs(ref)                                  # it says something


def test_repeated_calls_and_a_graph(B):
    say("balance repeated and in a graph")
    T, E, k = 700, 60, 4
    start = [0, 100, 333, 690]
    L, idx = inputs(T, E, k, free=0.1)
    want = digest(*run(B, L, idx, "sigmoid", start=start))
    assert digest(*run(B, L, idx, "sigmoid", start=start)) == want
    s, ba = B.shape(T, 128, 128, E, k), B.balance("sigmoid", 0.3, 3)
    d = dict(L=torch.as_tensor(L).cuda(), idx=torch.as_tensor(idx).cuda(),
             start=torch.tensor(start, dtype=torch.int32).cuda())
    o = [torch.empty((1,), device="cuda"), torch.empty((3, E), dtype=torch.int32, device="cuda"),
         torch.empty((3,), device="cuda"), torch.empty((T, E), device="cuda")]
    ws = torch.full((B.moe_balance_workspace_bytes(s, ba),), 255, dtype=torch.uint8, device="cuda")

    def step():
        B.moe_balance_loss(s, ba, d["L"], d["idx"], d["start"], o[0], o[1], o[2], ws)
        B.moe_balance_loss_backward(s, ba, d["L"], d["idx"], d["start"], o[1], o[2], None, None, o[3])
    step()
    torch.cuda.synchronize()
    assert digest(*o) == want
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (5, 6, 7):
        L, idx = inputs(T, E, k, seed=seed, free=0.1)
        d["L"].copy_(torch.as_tensor(L))
        d["idx"].copy_(torch.as_tensor(idx))
        ws.fill_(seed)
        graph.replay()
        torch.cuda.synchronize()
        assert digest(*o) == digest(*run(B, L, idx, "sigmoid", start=start))


def test_a_large_batch(B):
    """Chunks longer than the smallest; sums against 64 bits on the GPU."""
    say("balance of 40000 x 256")
    T, E, k = 40000, 256, 8
    g = torch.Generator(device="cuda").manual_seed(0)
    L = torch.randn((T, E), generator=g, device="cuda")
    idx = torch.topk(L, k, dim=1)[1].to(torch.int32)
    loss, counts, scales, dL = run(B, np_(L), np_(idx), "sigmoid", 0.01)
    assert torch.equal(counts[0].long(), torch.bincount(idx.flatten().long(), minlength=E))
    s = torch.sigmoid(L.double())
    p = s / s.sum(1, keepdim=True)
    c = counts[0].double()
    sc = 0.01 * E / (k * T * T)
    ref = sc * (c * p.sum(0)).sum()
    tau = share_rel(L)
    assert abs(float(loss) - float(ref)) <= (tau + (160 + T / 512) * U) * float(ref)
    dot = (p @ c)[:, None]
    d = sc * p * (c - dot) * (1 - s)
    bound = sc * p * ((tau + 12 * U) * (c - dot).abs() + (tau + 24 * U) * dot)
    assert bool(((dL.double() - d).abs() <= bound + 2 * U * d.abs()).all())


def test_the_largest_batch(B):
    """The last token count that is not refused, of one expert: every share is 1."""
    say("balance of 2^26 - 4 tokens")
    T = (1 << 26) - 4
    s, ba = B.shape(T, 128, 128, 1, 1), B.balance("sigmoid", 0.5, 2)
    L = torch.randn((T, 1), generator=torch.Generator(device="cuda").manual_seed(0), device="cuda")
    idx = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 12345, T - 7], dtype=torch.int32, device="cuda")
    loss, sc = torch.empty(1, device="cuda"), torch.empty(2, device="cuda")
    c = torch.empty((2, 1), dtype=torch.int32, device="cuda")
    ws = torch.empty(B.moe_balance_workspace_bytes(s, ba), dtype=torch.uint8, device="cuda")
    dL = torch.full((T, 1), 9.0, device="cuda")
    B.moe_balance_loss(s, ba, L, idx, start, loss, c, sc, ws)
    B.moe_balance_loss_backward(s, ba, L, idx, start, c, sc, None, None, dL)
    torch.cuda.synchronize()
    assert c[:, 0].tolist() == [12345, T - 7 - 12345]
    # a wavefront adds its 8192 tokens of a chunk one by one, each share within 3 units of 1
    assert abs(float(loss) - 0.5) <= 0.5 * (8192 + 200) * U
    # p (c - p c) with p within 3 units of 1
    assert float(dL.abs().max()) <= float(sc.max()) * T * 8 * U


def test_two_batches_at_once(B):
    """Two workspaces on two streams given by argument."""
    say("balance of two batches at once")
    T, E, k = 3000, 60, 4
    sets = []
    for seed in (1, 2):
        L, idx = inputs(T, E, k, seed=seed)
        want = digest(*run(B, L, idx, "softmax"))
        s, ba = B.shape(T, 128, 128, E, k), B.balance("softmax", 0.3, 1)
        o = [torch.empty((1,), device="cuda"), torch.empty((1, E), dtype=torch.int32, device="cuda"),
             torch.empty((1,), device="cuda"), torch.empty((T, E), device="cuda")]
        ws = torch.empty(B.moe_balance_workspace_bytes(s, ba), dtype=torch.uint8, device="cuda")
        sets.append((s, ba, torch.as_tensor(L).cuda(), torch.as_tensor(idx).cuda(), o, ws, want))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for (s, ba, L, idx, o, ws, _), st in zip(sets, streams):
            B.moe_balance_loss(s, ba, L, idx, None, o[0], o[1], o[2], ws, stream=st)
            B.moe_balance_loss_backward(s, ba, L, idx, None, o[1], o[2], None, None, o[3], stream=st)
    torch.cuda.synchronize()
    for x in sets:
        assert digest(*x[4]) == x[6]


@pytest.mark.parametrize("T,E,n", [(128, 64, 64), (64, 256, 16), (128, 60, 2), (64, 255, 16), (64, 256, 1), (128, 64, 1)])
def test_the_largest_batches_of_one_launch(B, T, E, n):
    """Every row of shares that one workgroup holds, and every count."""
    say(f"balance of {T} x {E} in {n} sequences")
    L, idx = inputs(T, E, 8, free=0.05)
    start = np.linspace(0, T, n + 1).astype(np.int64)
    for score in ("softmax", "sigmoid"):
        verify(B, L, idx, score, 0.5, start)
