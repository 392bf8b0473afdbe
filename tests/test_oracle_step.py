"""Pins of the oracle of the norm, the balance loss and the AdamW step: autograd, differences,
hand-made values, and the properties that the 8-bit states are chosen for."""
import numpy as np
import pytest
import torch

import oracle


def t64(a):
    return torch.tensor(np.asarray(a, np.float64), requires_grad=True)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("T,H", [(1, 8), (5, 24), (7, 40)])
def test_norm_gradient_is_autograd(kind, T, H):
    rng = np.random.default_rng(H)
    h, w, b = t64(rng.standard_normal((T, H)) + 1), t64(rng.standard_normal(H)), t64(rng.standard_normal(H))
    dy, dh = rng.standard_normal((T, H)), rng.standard_normal((T, H))
    x = h - h.mean(1, keepdim=True) if kind == "layer" else h
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-3) * w + b
    (y * torch.tensor(dy)).sum().backward()
    ry, _, _ = oracle.norm(h.detach().numpy(), w.detach().numpy(), b.detach().numpy(), kind, 1e-3)
    np.testing.assert_allclose(ry, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    dx, dw, db = oracle.norm_backward(h.detach().numpy(), w.detach().numpy(), dy, dh, kind, 1e-3)
    np.testing.assert_allclose(dx, h.grad.numpy() + dh, rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(dw, w.grad.numpy(), rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(db, b.grad.numpy(), rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_gradient_by_differences(kind):
    rng = np.random.default_rng(1)
    h, w, dy = rng.standard_normal((2, 16)), rng.standard_normal(16), rng.standard_normal((2, 16))
    dx, dw, _ = oracle.norm_backward(h, w, dy, None, kind, 1e-2)
    e = 1e-6
    for i in range(16):
        hp, hm = h.copy(), h.copy()
        hp[0, i] += e
        hm[0, i] -= e
        d = ((oracle.norm(hp, w, None, kind, 1e-2)[0] - oracle.norm(hm, w, None, kind, 1e-2)[0]) * dy).sum()
        assert abs(d / (2 * e) - dx[0, i]) < 1e-7


def test_norm_by_hand():
    y, _, rstd = oracle.norm(np.array([[1.0, 3.0]]), kind="layer", eps=3.0)
    np.testing.assert_allclose(y, [[-0.5, 0.5]])
    y, _, _ = oracle.norm(np.array([[3.0, 1.0]]), kind="rms", eps=4.0)
    np.testing.assert_allclose(y, [[1.0, 1 / 3]])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_is_autograd(score):
    rng = np.random.default_rng(3)
    T, E, k = 11, 6, 2
    L = rng.standard_normal((T, E)) * 2
    idx = np.argsort(-L, 1)[:, :k].copy()
    idx[3] = -1
    idx[4, 1] = -1
    start = [1, 4, 4, 9]                      # a token before, two behind, an empty sequence
    l = t64(L)
    s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    p = s / s.sum(1, keepdim=True)
    loss = 0.0
    for a, b in ((1, 4), (4, 9)):
        use = [t for t in range(a, b) if (idx[t] >= 0).any()]
        c = torch.tensor([sum((idx[t] == e).sum() for t in use) for e in range(E)], dtype=torch.float64)
        loss = loss + 0.3 / 2 * E / (k * len(use) ** 2) * (c * p[use].sum(0)).sum()
    (2.5 * loss).backward()
    got, counts, scales, _ = oracle.balance(L, idx, score, 0.3, start)
    assert abs(got - float(loss.detach())) < 1e-12 and counts.sum() == 2 * 2 + 5 * 2 - 1 and scales[1] == 0
    d = oracle.balance_backward(L, idx, score, 0.3, start, 2.5, np.ones((T, E)))
    np.testing.assert_allclose(d - 1, l.grad.numpy(), rtol=1e-9, atol=1e-14)


def test_balance_of_an_even_load_is_its_coefficient():
    L = np.zeros((8, 4))
    idx = np.array([[t % 4, (t + 1) % 4] for t in range(8)])
    loss, counts, _, _ = oracle.balance(L, idx, "softmax", 0.7)
    assert abs(loss - 0.7) < 1e-15 and (counts == 4).all()
    assert not np.abs(oracle.balance_backward(L, idx, "softmax", 0.7)).any()


def test_states_against_torch_adamw():
    rng = np.random.default_rng(0)
    p0, lr, wd = rng.standard_normal(50), 1e-2, 0.1
    ref = torch.nn.Parameter(torch.tensor(p0))
    opt = torch.optim.AdamW([ref], lr=lr, betas=(0.9, 0.95), eps=1e-8, weight_decay=wd)
    p, m, v = p0.copy(), np.zeros(50), np.zeros(50)
    for step in range(1, 6):
        g = rng.standard_normal(50).astype(np.float32)
        h = dict(lr=lr, beta1=0.9, one_minus_beta1=0.1, beta2=0.95, one_minus_beta2=0.05, eps=1e-8,
                 corr1=1 / (1 - 0.9 ** step), corr2=1 / (1 - 0.95 ** step), grad_scale=1.0)
        m, v = oracle.adamw_states(g, m, v, h)
        p, _, _ = oracle.adamw_param(p, m, v, h, wd)
        ref.grad = torch.tensor(g.astype(np.float64))
        opt.step()
        np.testing.assert_allclose(p, ref.detach().numpy(), rtol=0, atol=step * lr * 1e-6)


@pytest.mark.parametrize("which", ["m", "v"])
def test_codes_round_trip_and_stay_between_neighbours(which):
    rng = np.random.default_rng(5)
    n = 200                                    # a block that ends early
    x = (rng.standard_normal(n) * np.exp2(rng.integers(-20, 20, n))).astype(np.float32)
    x[5] = 0.0
    x = np.abs(x) if which == "v" else x
    for r in (0, 1, 32768, 65535):
        codes, scales = oracle.encode_state(x, np.full(n, r), which)
        y = oracle.decode_state(codes, scales, which)
        assert y[5] == 0
        again = oracle.encode_state(y.astype(np.float32), np.full(n, 65535), which)
        assert (again[0] == codes).all() and (again[1] == scales).all()   # on the grid: stays
        s = np.repeat(np.exp2(scales - 127.0), 32)[:n]
        top = (448 if which == "m" else 1.875) * s
        assert (np.abs(y) <= top).all()
        # a value below the top binade is off by less than a step of an eighth of its binade
        step = np.maximum(np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 1e-300))) - 3),
                          s * (2.0 ** -9 if which == "m" else 1.125 * 2.0 ** -31))
        assert (np.abs(y - x) <= step).all()
    if which == "v":
        assert (codes[x > 0] > 0).all()


@pytest.mark.parametrize("which", ["m", "v"])
def test_rounding_at_random_is_right_on_average(which):
    n = 32
    x = np.linspace(0.011, 1.0, n).astype(np.float32)
    draws = 3000
    mean = np.zeros(n)
    for i in range(draws):
        r = oracle.random_bits(i, 0, n)
        c = oracle.encode_state(x, (r & 0xFFFF) if which == "m" else r >> 16, which)
        mean += oracle.decode_state(*c, which) / draws
    # a draw deviates by at most half a step (an eighth of the value) in the root mean square
    assert (np.abs(mean - x) <= 5 * x / 16 / np.sqrt(draws)).all()


def test_nearest_rounding_would_freeze_v():
    """Why v is rounded at random: a state that decays by 0.1 % a step."""
    v = np.full(32, 1.0, np.float32)
    half = np.full(32, 32767)
    c, s = oracle.encode_state(v, half, "v")
    near = rnd = oracle.decode_state(c, s, "v")
    for step in range(1000):
        near = oracle.decode_state(*oracle.encode_state((near * 0.999).astype(np.float32), half, "v"), "v")
        r = oracle.random_bits(step, 0, 32)
        rnd = oracle.decode_state(*oracle.encode_state((rnd * 0.999).astype(np.float32), r >> 16, "v"), "v")
    assert (near == 1.0).all()
    assert abs(rnd.mean() - 0.999 ** 1000) < 0.05


def test_states_that_are_not_finite_or_vanish():
    x = np.zeros(64, np.float32)
    x[3] = np.inf
    c, s = oracle.encode_state(x, np.zeros(64, int), "m")
    assert s[0] == 255 and s[1] == 1 and np.isnan(oracle.decode_state(c, s, "m")[:32]).all()
    tiny = np.full(32, 1e-44, np.float32)
    c, s = oracle.encode_state(tiny, np.zeros(32, int), "v")
    assert (c == 1).all() or (oracle.decode_state(c, s, "v") > 0).all()


def test_bf16_at_random():
    p = np.array([1.0 + 2.0 ** -9, -1.0 - 2.0 ** -9, 1.0])
    lo = oracle.round_bf16_at_random(p, np.zeros(3, np.int64))
    hi = oracle.round_bf16_at_random(p, np.full(3, 0xFFFF))
    assert lo.tolist() == [1.0, -1.0, 1.0] and hi.tolist() == [1.0 + 2.0 ** -7, -1.0 - 2.0 ** -7, 1.0]
