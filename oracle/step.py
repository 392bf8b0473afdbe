"""fp64 oracle of the norm in front of the layer, the balance loss and the AdamW step.
TEST INFRASTRUCTURE ONLY (see the package docstring).

The AdamW states are the exception to fp64: their update is defined as fp32 operations, each
rounded, so that their 8-bit codes are whole numbers to compare exactly."""
from __future__ import annotations

import numpy as np

from .moe import _f64, _i64

F32 = np.float32


# ------------------------------------------------------------------------- norm
def norm(h, w=None, b=None, kind="layer", eps=1e-5):
    """(y, xh, rstd) of the rows of h"""
    h = _f64(h)
    H = h.shape[1]
    d = h - (h.sum(1, keepdims=True) / H if kind == "layer" else 0.0)
    rstd = 1.0 / np.sqrt((d * d).sum(1, keepdims=True) / H + eps)
    xh = d * rstd
    y = xh if w is None else xh * _f64(w)
    return (y if b is None else y + _f64(b)), xh, rstd


def norm_backward(h, w, dy, dh_in=None, kind="layer", eps=1e-5):
    """(dx, dw, db), from the Jacobian of one row at a time"""
    _, xh, rstd = norm(h, kind=kind, eps=eps)
    dy = _f64(dy)
    g = dy if w is None else dy * _f64(w)
    T, H = dy.shape
    dx = np.zeros((T, H))
    centre = np.full((H,), 1.0 / H) if kind == "layer" else np.zeros(H)
    for t in range(T):
        # d xh = rstd (I - 1 centre^T - xh xh^T / H) d h
        dx[t] = rstd[t] * (g[t] - centre * g[t].sum() - xh[t] * (xh[t] @ g[t]) / H)
    if dh_in is not None:
        dx = dx + _f64(dh_in)
    return dx, (dy * xh).sum(0), dy.sum(0)


# ---------------------------------------------------------------------- balance
def shares(row, score):
    """p of one token; 0 for experts out of play"""
    row = np.where(np.isnan(row), -np.inf, row)
    ls = -np.logaddexp(0.0, -row) if score == "sigmoid" else row
    top = ls.max()
    if top == -np.inf:
        return np.zeros_like(row)
    z = np.exp(ls - top)
    return z / z.sum()


def balance(logits, topk_idx, score="softmax", coef=1.0, seq_start=None):
    """(loss, counts int64 [n_seq, E], scales [n_seq], sequence of each token or -1)"""
    L, idx = _f64(logits), _i64(topk_idx)
    T, E = L.shape
    k = idx.shape[1]
    start = [0, T] if seq_start is None else [int(v) for v in seq_start]
    n_seq = len(start) - 1
    where = np.full(T, -1)
    counts = np.zeros((n_seq, E), np.int64)
    psum = np.zeros((n_seq, E))
    N = np.zeros(n_seq)
    for i in range(n_seq):
        for t in range(start[i], start[i + 1]):
            own = [e for e in idx[t] if 0 <= e < E]
            if not own:
                continue
            where[t] = i
            N[i] += 1
            for e in own:
                counts[i, e] += 1
            psum[i] += shares(L[t], score)
    n = (N > 0).sum()
    scales = np.array([coef * E / (k * v * v * n) if v else 0.0 for v in N])
    return float((scales * (counts * psum).sum(1)).sum()), counts, scales, where


def balance_backward(logits, topk_idx, score="softmax", coef=1.0, seq_start=None, d_loss=1.0,
                     d_in=None):
    L = _f64(logits)
    _, counts, scales, where = balance(logits, topk_idx, score, coef, seq_start)
    out = np.zeros_like(L) if d_in is None else _f64(d_in).copy()
    for t, i in enumerate(where):
        if i < 0:
            continue
        p, c = shares(L[t], score), counts[i]
        g = d_loss * scales[i] * p * (c - (p * c).sum())
        if score == "sigmoid":
            row = np.where(p > 0, L[t], 0.0)
            g = g * np.exp(-np.logaddexp(0.0, row))
        out[t] += g
    return out


# ------------------------------------------------------------------------ AdamW
def random_bits(seed, tensor, n, first=0):
    """32 random bits for the elements first .. first + n of a table's tensor"""
    def mix(x):
        x = x & 0xFFFFFFFF
        x = x ^ (x >> 16)
        x = (x * 0x5BE0CD19) & 0xFFFFFFFF
        x = x ^ (x >> 15)
        x = (x * 0xBB67AE85) & 0xFFFFFFFF
        return x ^ (x >> 16)
    out = np.empty(n, np.int64)
    for j in range(n):
        i = first + j
        key = (mix(mix(tensor + 1) + seed) + (i >> 32) * 0x3C6EF373) & 0xFFFFFFFF
        out[j] = mix((i & 0xFFFFFFFF) ^ key)
    return out


def adamw_states(g, m, v, h):
    """m', v' in fp32, each product and sum rounded"""
    g, m, v = (np.asarray(a, F32) for a in (g, m, v))
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        g = g * F32(h["grad_scale"])
        return (m * F32(h["beta1"]) + g * F32(h["one_minus_beta1"]),
                v * F32(h["beta2"]) + (g * F32(h["one_minus_beta2"])) * g)


def adamw_param(p, m, v, h, weight_decay):
    """p' in 64 bits from the new states, and |lr u| and |lr weight_decay p|"""
    p, m, v = _f64(p), _f64(m), _f64(v)
    u = m * h["corr1"] / (np.sqrt(v * h["corr2"]) + h["eps"])
    wd = float(F32(weight_decay)) * p
    return p - h["lr"] * (u + wd), abs(h["lr"]) * np.abs(u), abs(h["lr"]) * np.abs(wd)


def _neighbours(c):
    """value of m's code magnitudes and of v's codes, from the bits"""
    E, f = c >> 3, c & 7
    m = np.where(E == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * np.exp2(E - 7.0))
    v = np.where(c == 0, 0.0, (1 + f / 8) * np.exp2(E - 31.0))
    return m, v


M_VALUES = _neighbours(np.arange(127))[0]      # 0 .. 448
V_VALUES = _neighbours(np.arange(256))[1]      # 0, 1.125 * 2^-31 .. 1.875


def encode_state(x, r16, which):
    """(codes, scale bytes) of one tensor's fp32 state: for each block the smallest power of
    two that brings it into the codes' range (2^-126 at least), and for each value the upper
    neighbour where its distance from the lower one, in steps, plus a random number in (0, 1)
    reaches 1."""
    x = np.asarray(x, F32)
    n = x.size
    table = M_VALUES if which == "m" else V_VALUES
    codes, scales = np.zeros(n, np.uint8), np.zeros((n + 31) // 32, np.uint8)
    for b in range(len(scales)):
        blk = x[32 * b:32 * b + 32].astype(np.float64)
        top = np.abs(blk).max()
        if not top < 2.0 ** 126:
            scales[b] = 255
            continue
        X = -126
        while top > table[-1] * 2.0 ** X:
            X += 1
        scales[b] = X + 127
        for j, val in enumerate(blk):
            # the scaling is exact but for results that fp32 holds as subnormals
            y = float(F32(abs(F32(val)) * F32(2.0 ** -X)))
            rnd = (int(r16[32 * b + j]) * 16 + 8) / 2 ** 20
            if which == "m":
                if y < 2.0 ** -6:      # steps of 2^-9
                    c = int(np.floor(y / 2.0 ** -9 + rnd))
                else:
                    c = int(np.searchsorted(table, y, side="right")) - 1
                    step = 2.0 ** (np.floor(np.log2(y)) - 3)
                    c += int((y - table[c]) / step + rnd >= 1)
                c |= int(np.signbit(x[32 * b + j])) << 7
            elif val <= 0:
                c = 0
            else:
                c = int(np.searchsorted(table, y, side="right")) - 1
                if c < 1:
                    c = 1              # v > 0 does not become 0
                else:
                    step = 2.0 ** (np.floor(np.log2(y)) - 3)
                    c += int((y - table[c]) / step + rnd >= 1)
            codes[32 * b + j] = c
    return codes, scales


def decode_state(codes, scales, which):
    codes = np.asarray(codes).astype(np.int64)
    s = np.exp2(np.asarray(scales).astype(np.float64) - 127.0)
    s = np.where(np.asarray(scales) == 255, np.nan, s)
    s = np.repeat(s, 32)[:codes.size]
    if which == "v":
        return V_VALUES[codes] * s
    return np.where(codes > 127, -1.0, 1.0) * M_VALUES[codes & 127] * s


def round_bf16_at_random(p, r):
    """p (64 bits) on bf16's grid: the neighbour that 16 random bits say"""
    u = np.asarray(p, F32).view(np.uint32).astype(np.int64)
    u = (u + ((r ^ (r >> 16)) & 0xFFFF)) & 0xFFFF0000
    return u.astype(np.uint32).view(F32).astype(np.float64)
