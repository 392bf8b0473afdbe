"""Derived error bounds of the norm's, the balance loss's and the AdamW step's kernels.

U = 2^-24 and UB = 2^-8 are half a step of fp32 and bf16 relative to the value.
Norm: a sum over a row of H <= 16384 values is at most 32 additions in a thread, 6 in its
wavefront and 16 over the wavefronts: D = 56 roundings.
  mean         off by dmu <= D U mean|h|
  variance     of the differences to that mean: + dmu^2 (their first order sums to 0), and
               (D + 3) U of itself; rstd half of that relative, and 4 U for its root and quotient
  xh           off by rstd dmu + |xh| ((D + 8) U + (rstd dmu)^2)
"""
import numpy as np

U, UB = 2.0 ** -24, 2.0 ** -8
D = 56


def f64(t):
    return t.detach().to("cpu").double().numpy() if hasattr(t, "detach") else np.asarray(t, np.float64)


def rounded(ref, err, bf16):
    """bound of v rounded to the type, |v - ref| <= err"""
    u = UB if bf16 else U
    return err + u * (np.abs(ref) + err) + 1e-38


def check(got, ref, bound, name=""):
    g = f64(got)
    assert g.shape == ref.shape, name
    bad = ~(np.abs(g - ref) <= bound)
    assert not bad.any(), (name, int(bad.sum()), float(np.abs(g - ref)[bad].max()),
                           float(np.broadcast_to(bound, ref.shape)[bad].min()))


def xh_err(h, xh, rstd, kind):
    dmu = D * U * np.abs(h).mean(1, keepdims=True) if kind == "layer" else 0.0
    rel = (D + 8) * U + (rstd * dmu) ** 2
    return rstd * dmu + np.abs(xh) * rel, rel


def norm_bounds(h, w, b, xh, rstd, kind):
    """of y before its rounding"""
    e, _ = xh_err(h, xh, rstd, kind)
    w = 1.0 if w is None else np.abs(f64(w))
    b = 0.0 if b is None else np.abs(f64(b))
    return w * e + 3 * U * (w * np.abs(xh) + b)


def norm_back_bounds(h, w, dy, dh, xh, rstd, kind):
    """of (dx, dw, db) before their roundings"""
    e, rel = xh_err(h, xh, rstd, kind)
    dy = f64(dy)
    g = np.abs(dy if w is None else dy * f64(w))
    T = len(dy)
    m = lambda a: a.mean(1, keepdims=True)    # noqa: E731
    ax = np.abs(xh)
    gx = np.abs(m((dy if w is None else dy * f64(w)) * xh))
    e_mg = (D + 2) * U * m(g) if kind == "layer" else 0.0
    e_mgx = m(g * e) + (D + 3) * U * m(g * ax)
    terms = g + m(g) + ax * (gx + e_mgx)
    dx = rstd * (U * g + e_mg + e * (gx + e_mgx) + ax * e_mgx + (rel + 6 * U) * terms)
    if dh is not None:
        dx = dx + 2 * U * np.abs(f64(dh))
    # rows of a workgroup one after the other and workgroups by sixteenths, or every 8th row or
    # more in a thread: at most 128 + T / 8
    depth = (128 + T / 8) * U
    return dx, (np.abs(dy) * e).sum(0) + depth * (np.abs(dy) * ax).sum(0), depth * np.abs(dy).sum(0)


def share_rel(logits):
    """Relative error of a token's shares: an exponential of l - top has the rounding of the
    difference (at most 2 max|l|) and 2 units, the sigmoid's factor 5, the sum over at most
    1024 experts 24, the reciprocal and the product 3."""
    l = f64(logits)
    big = np.abs(l[np.isfinite(l)]).max(initial=0.0)
    return (2 * big + 34) * U
