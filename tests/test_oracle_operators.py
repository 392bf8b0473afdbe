"""Pins of the oracle's scored routing, router backward and low-rank adapters: brute
force, torch.autograd in fp64 and central differences."""
import itertools

import numpy as np
import pytest
import torch

import oracle


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_choice_and_weights_by_brute_force(score, renorm):
    rng = np.random.default_rng(1)
    E, k, G, keep = 8, 3, 4, 2
    L = rng.standard_normal((40, E))
    bias = rng.standard_normal(E) * 0.3
    idx, w = oracle.route_scored(L, k, score, bias, G, keep, 2, renorm, 1.5)
    for t in range(len(L)):
        s = (torch.softmax if score == "softmax" else lambda v, d: torch.sigmoid(v))(
            torch.tensor(L[t]), 0).numpy()
        c = s + bias
        gs = c.reshape(G, -1).sum(1)      # groups of two: the sum of the best two is the sum
        best_g = max(itertools.combinations(range(G), keep), key=lambda q: sum(gs[list(q)]))
        pool = [e for e in range(E) if e // 2 in best_g]
        best = max(itertools.combinations(pool, k), key=lambda q: sum(c[list(q)]))
        assert sorted(idx[t]) == sorted(best)
        assert list(c[idx[t]]) == sorted(c[idx[t]], reverse=True)
        ref = s[idx[t]] / (s[idx[t]].sum() if renorm else 1.0) * 1.5
        np.testing.assert_allclose(w[t], ref, rtol=1e-13)


def test_plain_softmax_is_the_layers_route():
    rng = np.random.default_rng(2)
    L = rng.integers(-2, 3, (30, 9)).astype(np.float64)
    a, b = oracle.route(L, 4), oracle.route_scored(L, 4)
    assert (a[0] == b[0]).all()
    np.testing.assert_allclose(a[1], b[1], rtol=1e-14)


def test_experts_out_of_play():
    L = np.array([[-np.inf, 1.0, np.nan, 0.5], [-np.inf] * 4, [-400.0, -500.0, -np.inf, -900.0]])
    for score in ("softmax", "sigmoid"):
        idx, w = oracle.route_scored(L, 3, score, renormalise=True)
        assert idx.tolist() == [[1, 3, -1], [-1, -1, -1], [0, 1, 3]]
        np.testing.assert_allclose(w.sum(1), [1.0, 0.0, 1.0], rtol=1e-14)


def test_a_group_with_one_expert_in_play_beats_an_empty_one():
    L = np.array([[-np.inf, -np.inf, 0.1, -np.inf]])
    idx, _ = oracle.route_scored(L, 1, "sigmoid", None, 2, 1, 2)
    assert idx[0, 0] == 2


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_autograd_and_differences(score, renorm):
    rng = np.random.default_rng(3)
    L, dw = rng.standard_normal((7, 12)), rng.standard_normal((7, 4))
    bias = rng.standard_normal(12) * 0.2
    kw = dict(score=score, renormalise=renorm, scale=2.5)
    idx, w = oracle.route_scored(L, 4, bias=bias, n_groups=3, topk_groups=2, group_top=2, **kw)
    got = oracle.route_scored_backward(L, idx, dw, **kw)
    l = torch.tensor(L, requires_grad=True)
    s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    p = torch.gather(s, 1, torch.tensor(idx, dtype=torch.int64))
    if renorm:
        p = p / p.sum(1, keepdim=True)
    (2.5 * p * torch.tensor(dw)).sum().backward()
    np.testing.assert_allclose(got, l.grad.numpy(), rtol=1e-11, atol=1e-14)
    eps = 1e-6
    for t, e in [(0, 0), (1, int(idx[1, 0])), (3, int(idx[3, 2])), (6, 11)]:
        lo, hi = L.copy(), L.copy()
        lo[t, e] -= eps
        hi[t, e] += eps
        f = [oracle.route_scored(v, 4, bias=bias, n_groups=3, topk_groups=2, group_top=2, **kw)
             for v in (lo, hi)]
        assert (f[0][0] == idx).all() and (f[1][0] == idx).all()
        num = ((f[1][1] - f[0][1]) * dw).sum() / (2 * eps)
        np.testing.assert_allclose(got[t, e], num, rtol=1e-6, atol=1e-9)


def test_router_backward_autograd():
    rng = np.random.default_rng(4)
    x, w, dL, dxi = (rng.standard_normal(s) for s in [(6, 5), (3, 5), (6, 3), (6, 5)])
    xt, wt = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    ((xt @ wt.T) * torch.tensor(dL)).sum().backward()
    dw, dx = oracle.router_backward(x, w, dL, dxi)
    np.testing.assert_allclose(dw, wt.grad.numpy(), rtol=1e-12)
    np.testing.assert_allclose(dx, xt.grad.numpy() + dxi, rtol=1e-12)


def test_lora_autograd_and_tokens_without_an_adapter():
    rng = np.random.default_rng(5)
    n, r, hi, ho, T = 3, 2, 5, 4, 9
    idx = np.array([0, 2, -1, 2, 2, 0, 7, 0, -1])
    x, a, b, sc, base, dy = (rng.standard_normal(s) for s in
                             [(T, hi), (n, r, hi), (n, ho, r), (n,), (T, ho), (T, ho)])
    ts = [torch.tensor(v, requires_grad=True) for v in (x, a, b)]
    y = torch.tensor(base).clone()
    ok = torch.tensor((idx >= 0) & (idx < n))
    sel = torch.tensor(np.clip(idx, 0, n - 1))
    add = torch.matmul(ts[2][sel], torch.matmul(ts[1][sel], ts[0][:, :, None]))[:, :, 0]
    y = y + torch.where(ok[:, None], torch.tensor(sc)[sel][:, None] * add, torch.zeros_like(add))
    np.testing.assert_allclose(oracle.lora(idx, x, a, b, sc, base), y.detach().numpy(), rtol=1e-12)
    (y * torch.tensor(dy)).sum().backward()
    dx, da, db = oracle.lora_backward(idx, x, a, b, sc, dy)
    for got, t in zip((dx, da, db), ts):
        np.testing.assert_allclose(got, t.grad.numpy(), rtol=1e-11, atol=1e-14)
    assert not da[1].any() and not db[1].any()


def test_a_bias_of_minus_inf_is_the_last_choice():
    inf = np.inf
    L = np.zeros((1, 8))
    b = np.array([0.0, -inf, -1.0, -1.0, -inf, -inf, -2.0, -inf])
    kw = dict(score="sigmoid", bias=b, n_groups=4, group_top=2)
    # group scores: 0.5 (one expert left), -1 (two), none, -1.5
    assert oracle.route_scored(L, 2, topk_groups=1, **kw)[0].tolist() == [[0, 1]]
    assert oracle.route_scored(L, 4, topk_groups=2, **kw)[0].tolist() == [[0, 2, 3, 1]]
    idx, w = oracle.route_scored(L, 8, topk_groups=4, **kw)
    assert idx.tolist() == [[0, 2, 3, 6, 1, 4, 5, 7]] and np.allclose(w, 1 / 8)
