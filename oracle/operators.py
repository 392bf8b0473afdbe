"""fp64 oracle of scored routing, the router projection's backward and the low-rank
adapters.  TEST INFRASTRUCTURE ONLY (see the package docstring)."""
from __future__ import annotations

import numpy as np

from .moe import _f64, _i64


def log_scores(row, score):
    """log s of one token's logits; -inf for experts out of play (logit -inf or NaN)."""
    row = np.where(np.isnan(row), -np.inf, row)
    if score == "sigmoid":
        return -np.logaddexp(0.0, -row)
    top = row.max()
    if top == -np.inf:
        return row
    return row - (top + np.log(np.exp(row - top).sum()))


def route_scored(logits, k, score="softmax", bias=None, n_groups=1, topk_groups=1, group_top=1,
                 renormalise=True, scale=1.0):
    """(topk_idx int32 [T, k], topk_w float64 [T, k]); -1 and 0 in slots left over."""
    L = _f64(logits)
    T, E = L.shape
    b = np.zeros(E) if bias is None else _f64(bias)
    per = E // n_groups
    idx = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        ls = log_scores(L[t], score)
        play = [e for e in range(E) if ls[e] > -np.inf]
        # without bias and groups the order of the scores is that of the logits
        c = {e: (L[t, e] if bias is None and n_groups == 1 else np.exp(ls[e]) + b[e]) for e in play}
        gs = []
        for g in range(n_groups):
            # a bias of -inf leaves its expert out of the group's score
            mem = sorted((c[e] for e in play if e // per == g and c[e] > -np.inf),
                         reverse=True)[:group_top]
            gs.append((-sum(mem) if mem else np.inf, g))
        kept = {g for _, g in sorted(gs)[:topk_groups]}
        sel = sorted((e for e in play if e // per in kept), key=lambda e: (-c[e], e))[:k]
        if not sel:
            continue
        s = ls[sel]
        if renormalise:
            s = s - s.max()
            p = np.exp(s) / np.exp(s).sum()
        else:
            p = np.exp(s)
        idx[t, :len(sel)] = sel
        w[t, :len(sel)] = scale * p
    return idx, w


def route_scored_backward(logits, topk_idx, d_topk_w, score="softmax", renormalise=True, scale=1.0):
    """d_logits of sum(w * d_topk_w) with the choice held fixed."""
    L, idx, dw = _f64(logits), _i64(topk_idx), _f64(d_topk_w)
    T, E = L.shape
    out = np.zeros((T, E))
    for t in range(T):
        ls = log_scores(L[t], score)
        ok = (idx[t] >= 0) & (idx[t] < E)
        sel, g = idx[t][ok], scale * dw[t][ok]
        if not len(sel):
            continue
        # ds_e log s_e is the local derivative: sigmoid 1 - s on the diagonal, softmax
        # delta - s
        lp = ls[sel]
        if renormalise:
            p = np.exp(lp - lp.max())
            p /= p.sum()
            dlog = p * (g - (p * g).sum())     # d / d log s of the chosen
        else:
            dlog = np.exp(lp) * g
        if score == "sigmoid":
            one_minus = np.exp(-np.logaddexp(0.0, L[t][sel]))
            for e, v in zip(sel, dlog * one_minus):
                out[t, e] += v
        else:
            for e, v in zip(sel, dlog):
                out[t, e] += v
            out[t] -= np.exp(ls) * dlog.sum()
    return out


def router_backward(x, w, d_logits, dx_in=None):
    x, w, dL = _f64(x), _f64(w), _f64(d_logits)
    dx = dL @ w
    return dL.T @ x, dx if dx_in is None else dx + _f64(dx_in)


def lora(idx, x, a, b, scale, base=None):
    """y = base + scale_a B_a (A_a x), token by token; ids outside [0, n) have no adapter."""
    x, a, b, scale, idx = _f64(x), _f64(a), _f64(b), _f64(scale), _i64(idx)
    y = np.zeros((x.shape[0], b.shape[1])) if base is None else _f64(base).copy()
    for t, i in enumerate(idx):
        if 0 <= i < a.shape[0]:
            y[t] += scale[i] * (b[i] @ (a[i] @ x[t]))
    return y


def lora_backward(idx, x, a, b, scale, dy, dx_in=None):
    """(dx, d_a, d_b)"""
    x, a, b, scale, dy, idx = _f64(x), _f64(a), _f64(b), _f64(scale), _f64(dy), _i64(idx)
    dx = np.zeros_like(x) if dx_in is None else _f64(dx_in).copy()
    da, db = np.zeros_like(a), np.zeros_like(b)
    for t, i in enumerate(idx):
        if 0 <= i < a.shape[0]:
            v = scale[i] * (b[i].T @ dy[t])
            dx[t] += a[i].T @ v
            da[i] += np.outer(v, x[t])
            db[i] += np.outer(dy[t], scale[i] * (a[i] @ x[t]))
    return dx, da, db
