"""Derived error bounds of the router projection's and the adapters' kernels.

U32 = 2^-24 and UB = 2^-8 are the rounding units of fp32 and bf16 (half an eps).
* An fp32 sum of K products of bf16 values (exact in fp32) in 32-deep matrix steps: at most
  32 roundings inside a step, one per step of K / 32 and at most 64 joining the parts:
  |error| <= (K / 32 + 96) U32 sum |products|.
* An fp32 operand split into two bf16 halves is off by at most UB^2 of itself.
* A result rounded to bf16 is off by at most UB of itself, plus what came before.
"""
import numpy as np

U32, UB = 2.0 ** -24, 2.0 ** -8


def depth(K):
    return (K / 32 + 96) * U32


def abs64(t):
    return np.abs(t.detach().to("cpu").double().numpy())


def dot_bound(a, b):
    """a [m, K], b [n, K] -> bound of the error of a b^T in fp32"""
    return depth(a.shape[1]) * (abs64(a) @ abs64(b).T)


def check(got, ref, bound, name=""):
    """Every element within its bound; an element without an error bound must be equal."""
    g = got.detach().to("cpu").double().numpy()
    assert g.shape == ref.shape, name
    bad = ~(np.abs(g - ref) <= bound)
    assert not bad.any(), (name, int(bad.sum()), float(np.abs(g - ref)[bad].max()))


def bf16_of(ref, err):
    """Bound of round_bf16(v) with |v - ref| <= err."""
    return err + UB * (np.abs(ref) + err) + 1e-40


def lora_bounds(idx, x, a, b, scale, base):
    """(|u|, bound of u, bound of y before its rounding), u = scale A x per token"""
    X, A, Bm, S = abs64(x), abs64(a), abs64(b), abs64(scale)
    n = A.shape[0]
    T, r = X.shape[0], A.shape[1]
    uabs, yerr = np.zeros((T, r)), np.zeros((T, Bm.shape[1]))
    uerr = np.zeros((T, r))
    for i in range(n):
        at = np.nonzero(idx == i)[0]
        if not len(at):
            continue
        m = S[i] * (X[at] @ A[i].T)             # >= |u|
        e = (depth(X.shape[1]) + U32) * m       # the sum, then the scale
        uabs[at], uerr[at] = m, e
        full = (m + e) @ Bm[i].T
        add = 0 if base is None else abs64(base)[at]
        yerr[at] = e @ Bm[i].T + (UB * UB + depth(2 * r)) * full + U32 * (full + add)
    return uabs, uerr, yerr


def outer_bound(idx, n, p, perr, q):
    """Bound of sum_t p_t (x) q_t per adapter: p fp32 known to perr and split, q exact."""
    Q = abs64(q)
    out = np.zeros((n, p.shape[1], Q.shape[1]))
    for i in range(n):
        at = np.nonzero(idx == i)[0]
        if len(at):
            full = (p[at] + perr[at]).T @ Q[at]
            out[i] = perr[at].T @ Q[at] + (UB * UB + depth(2 * len(at))) * full
    return out
