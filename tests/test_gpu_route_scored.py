"""GPU parity of scored routing and its gradient against the fp64 oracle.

Tolerances: a weight is scale * z_j / sum z with z = exp(d) q: d is off by 2^-24 of itself
(|d| <= 2 max |l|), exp and the two divisions by a few units, the sum by 6: relative
(2 max |l| + 16) 2^-24.  Gradients are sums of at most E products of such factors."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import digest, np_, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


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


def run(B, L, k, bias, kw, dw=None):
    T, E = L.shape
    s, sc = B.shape(T, 128, 128, E, k), B.scoring(**kw)
    Ld = torch.as_tensor(L, dtype=torch.float32).cuda()
    bd = None if bias is None else torch.as_tensor(bias, dtype=torch.float32).cuda()
    idx, ok1 = guarded((T, k), torch.int32)
    w, ok2 = guarded((T, k), torch.float32)
    B.moe_route_scored(s, sc, Ld, bd, idx, w)
    dL = None
    if dw is not None:
        dL, ok3 = guarded((T, E), torch.float32)
        B.moe_route_scored_backward(s, sc, Ld, idx, torch.as_tensor(dw, dtype=torch.float32).cuda(), dL)
        ok3()
    torch.cuda.synchronize()
    ok1(), ok2()
    return np_(idx), np_(w), None if dL is None else np_(dL)


def check(B, L, k, bias=None, **kw):
    L = np.asarray(L, np.float32)
    rng = np.random.default_rng(9)
    dw = rng.standard_normal((len(L), k)).astype(np.float32)
    idx, w, dL = run(B, L, k, bias, kw, dw)
    b32 = None if bias is None else np.asarray(bias, np.float32)
    ridx, rw = oracle.route_scored(L, k, bias=b32, **kw)
    np.testing.assert_array_equal(idx, ridx)
    big = np.abs(L[np.isfinite(L)]).max(initial=1.0)
    tol = (2 * big + 16) * U
    np.testing.assert_allclose(w, rw, rtol=tol, atol=1e-37)
    grad = dict(score=kw.get("score", "softmax"), renormalise=kw.get("renormalise", True),
                scale=kw.get("scale", 1.0))
    rd = oracle.route_scored_backward(L, ridx, dw, **grad)
    # every term is at most scale max |dw| w, with at most k + 2 roundings on top
    bound = 4 * (tol + (k + 2) * U) * abs(kw.get("scale", 1.0)) * np.abs(dw).max()
    np.testing.assert_allclose(dL, rd, rtol=0, atol=bound)
    return idx, w, dL


SHAPES = [(1, 1, 1), (1, 4, 1), (5, 3, 2), (37, 8, 2), (64, 60, 7), (129, 64, 6), (33, 65, 5),
          (300, 128, 8), (65, 256, 8), (70, 257, 32), (20, 1000, 9), (11, 1024, 32), (4, 16, 16)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_ungrouped(B, T, E, k, score):
    say(f"route_scored T={T} E={E} k={k} {score}")
    rng = np.random.default_rng(T * 31 + E)
    L = rng.standard_normal((T, E)) * 2
    for renorm in (True, False):
        check(B, L, k, None, score=score, renormalise=renorm)
        check(B, L, k, rng.standard_normal(E) * 0.1, score=score, renormalise=renorm, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,keep,top,k", [(256, 8, 4, 2, 8), (256, 8, 4, 1, 8), (64, 64, 5, 2, 3),
                                            (60, 4, 2, 2, 6), (60, 4, 2, 1, 6), (12, 3, 3, 2, 5),
                                            (512, 8, 1, 2, 16), (1024, 16, 3, 2, 32), (66, 3, 2, 2, 7),
                                            (128, 2, 1, 1, 4), (256, 64, 9, 2, 8), (96, 3, 2, 2, 4)])
def test_groups(B, E, G, keep, top, k, score):
    say(f"route_scored groups E={E} G={G} keep={keep} top={top} k={k} {score}")
    rng = np.random.default_rng(E + G)
    L = rng.standard_normal((75, E))
    kw = dict(score=score, n_groups=G, topk_groups=keep, group_top=top)
    check(B, L, k, rng.standard_normal(E) * 0.1, renormalise=True, scale=2.5, **kw)
    check(B, L, k, None, renormalise=False, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_id_and_group(B, score):
    say("route_scored ties", score)
    rng = np.random.default_rng(0)
    L = rng.integers(-1, 2, (200, 32)).astype(np.float32)
    L[L == 0] = np.where(rng.random((L == 0).sum()) < 0.5, -0.0, 0.0)
    check(B, L, 9, None, score=score)
    check(B, L, 9, np.zeros(32), score=score, n_groups=8, topk_groups=4, group_top=2)
    check(B, np.zeros((3, 64)), 8, np.zeros(64), score=score, n_groups=4, topk_groups=2, group_top=2)


def test_scores_that_fp32_cannot_tell_apart(B):
    """Neighbouring fp32 logits whose sigmoids round to the same fp32 value: the larger
    still comes first."""
    say("route_scored near ties")
    base = np.float32(6.0)
    row = [base]
    for _ in range(31):
        row.append(np.nextafter(row[-1], np.float32(9.0), dtype=np.float32))
    L = np.array([row, row[::-1]], np.float32)
    assert len(set((1 / (1 + np.exp(-L[0]))).astype(np.float32))) < 32
    check(B, L, 4, np.zeros(32), score="sigmoid", n_groups=4, topk_groups=2, group_top=2)
    check(B, L, 4, np.full(32, 0.25), score="sigmoid")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_experts_out_of_play(B, score):
    say("route_scored with -inf and NaN logits", score)
    rng = np.random.default_rng(5)
    L = rng.standard_normal((40, 24)).astype(np.float32)
    L[rng.random(L.shape) < 0.6] = -np.inf
    L[rng.random(L.shape) < 0.05] = np.nan
    L[3] = -np.inf
    L[4] = np.nan
    L[5] = -np.inf
    L[5, 7] = 1.0
    lo = np.finfo(np.float32).min
    L[6] = lo                        # the type's lowest value is a number: in play
    L[7] = lo
    L[7, 3] = 0.0
    bias = rng.standard_normal(24) + 5
    for renorm in (True, False):
        idx = run(B, L, 6, None, dict(score=score, renormalise=renorm))[0]
        ridx, rw = oracle.route_scored(L, 6, score, renormalise=renorm)
        np.testing.assert_array_equal(idx, ridx)
        assert (idx[3] == -1).all() and (idx[4] == -1).all() and idx[5].tolist() == [7] + [-1] * 5
        keep = np.ones(40, bool)
        keep[[6, 7]] = False
        check(B, L[keep], 6, None, score=score, renormalise=renorm)
        check(B, L[keep], 6, bias, score=score, renormalise=renorm, n_groups=4, topk_groups=3,
              group_top=2)
    _, w, dL = run(B, L[6:8], 6, None, dict(score=score), np.ones((2, 6), np.float32))
    np.testing.assert_allclose(w, [[1 / 6] * 6, [1.0, 0, 0, 0, 0, 0]], rtol=1e-6)
    assert np.isfinite(dL).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_weights_of_very_negative_logits(B, score):
    say("route_scored weights where the scores underflow", score)
    L = np.array([[-300.0, -301.0, -302.0, -900.0], [-1e4, -1e4, -2e4, -3e4]], np.float32)
    idx, w, dL = run(B, L, 2, None, dict(score=score, renormalise=True), np.ones((2, 2), np.float32))
    assert idx.tolist() == [[0, 1], [0, 1]]
    e = np.exp(-1.0)
    np.testing.assert_allclose(w, [[1 / (1 + e), e / (1 + e)], [0.5, 0.5]], rtol=1e-6)
    assert np.isfinite(dL).all()


def test_backward_ignores_slots_without_an_expert_and_sums_doubled_ids(B):
    say("route_scored_backward odd slots")
    rng = np.random.default_rng(6)
    L = rng.standard_normal((4, 8)).astype(np.float32)
    idx = np.array([[1, -1, 3], [8, 2, -5], [-1, -1, -1], [4, 4, 4]], np.int32)
    dw = rng.standard_normal((4, 3)).astype(np.float32)
    s = B.shape(4, 128, 128, 8, 3)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            sc = B.scoring(score=score, renormalise=renorm)
            dL, ok = guarded((4, 8), torch.float32)
            B.moe_route_scored_backward(s, sc, torch.tensor(L).cuda(), torch.tensor(idx).cuda(),
                                        torch.tensor(dw).cuda(), dL)
            torch.cuda.synchronize()
            ok()
            ref = oracle.route_scored_backward(L, idx, dw, score, renorm)
            np.testing.assert_allclose(np_(dL), ref, rtol=0, atol=64 * U * np.abs(dw).max())


def test_no_tokens_and_repeat(B):
    say("route_scored T=0, determinism")
    run(B, np.zeros((0, 8), np.float32), 2, None, {}, np.zeros((0, 2), np.float32))
    L = np.random.default_rng(1).standard_normal((500, 256)).astype(np.float32)
    kw = dict(score="sigmoid", n_groups=8, topk_groups=4, group_top=2)
    a = run(B, L, 8, np.zeros(256), kw, np.ones((500, 8)))
    b = run(B, L, 8, np.zeros(256), kw, np.ones((500, 8)))
    for x, y in zip(a, b):
        assert x.tobytes() == y.tobytes()


def test_gradient_against_differences(B):
    """Central differences of the kernel's own weights: step 2^-6 leaves a truncation of
    order step^2 and a rounding of 2^-22 / step, both below 2e-3 for these values."""
    say("route_scored gradient against differences")
    rng = np.random.default_rng(8)
    L = (np.arange(12) * 0.5 - 3 + rng.random((6, 12)) * 0.2).astype(np.float32)   # no near ties
    dw = rng.standard_normal((6, 4)).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            kw = dict(score=score, renormalise=renorm, scale=1.5)
            idx, _, dL = run(B, L, 4, None, kw, dw)
            for e in range(12):
                hi, lo = L.copy(), L.copy()
                hi[:, e] += 2.0 ** -6
                lo[:, e] -= 2.0 ** -6
                ih, wh, _ = run(B, hi, 4, None, kw)
                il, wl, _ = run(B, lo, 4, None, kw)
                assert (ih == idx).all() and (il == idx).all()
                num = ((wh.astype(np.float64) - wl) * dw).sum(1) / 2.0 ** -5
                np.testing.assert_allclose(dL[:, e], num, atol=2e-3)


def test_replays_in_a_graph_on_another_stream(B):
    say("route_scored in a captured graph")
    rng = np.random.default_rng(2)
    T, E, k = 77, 64, 6
    s, sc = B.shape(T, 128, 128, E, k), B.scoring(score="sigmoid", n_groups=4, topk_groups=2, group_top=2)
    L = torch.zeros((T, E), device="cuda")
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    w = torch.empty((T, k), device="cuda")
    dL = torch.empty((T, E), device="cuda")
    dw = torch.ones((T, k), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.moe_route_scored(s, sc, L, None, idx, w)
        B.moe_route_scored_backward(s, sc, L, idx, dw, dL)
    for _ in range(3):
        v = torch.tensor(rng.standard_normal((T, E)), dtype=torch.float32).cuda()
        L.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        got = digest(idx, w, dL)
        i2, w2, d2 = (torch.empty_like(t) for t in (idx, w, dL))
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        B.moe_route_scored(s, sc, v, None, i2, w2, st)
        B.moe_route_scored_backward(s, sc, v, i2, dw, d2, st)
        st.synchronize()
        assert digest(i2, w2, d2) == got


@pytest.mark.parametrize("E,G", [(16, 4), (256, 8), (60, 4), (1024, 32)])
def test_biases_of_minus_inf(B, E, G):
    say(f"route_scored bias -inf E={E} G={G}")
    rng = np.random.default_rng(E)
    L = rng.standard_normal((50, E))
    bias = rng.standard_normal(E) * 0.1
    bias[rng.random(E) < 0.6] = -np.inf
    bias[:E // G] = -np.inf                       # a whole group
    bias[E // G:2 * E // G - 1] = -np.inf         # all but one
    for top in (1, 2):
        for keep in (1, 2, G):
            check(B, L, min(8, keep * E // G), bias, score="sigmoid", n_groups=G, topk_groups=keep,
                  group_top=top)


def test_choice_among_scores_near_the_smallest_double(B):
    """Scores from 1e-300 through the subnormals: still in their order (the logits are 2
    apart, so that a subnormal of two units differs from its neighbour)."""
    say("route_scored tiny scores")
    L = -(690.0 + 2.0 * np.arange(24, dtype=np.float32))[None, ::-1].copy()
    idx = run(B, L, 6, None, dict(score="sigmoid", n_groups=4, topk_groups=2, group_top=2))[0]
    assert idx.tolist() == [[23, 22, 21, 20, 19, 18]]
    M = np.concatenate([L, np.zeros((1, 1)), np.full((1, 23), -np.inf)], 1).astype(np.float32)
    idx = run(B, M, 5, None, dict(score="softmax", n_groups=4, topk_groups=4))[0]
    assert idx.tolist() == [[24, 23, 22, 21, 20]]
