"""Plain 64-bit forms of the gated recurrence and the residual RMS-Norm, with
the largest error a float32 implementation of the same formulas can make.

U is float32's half step.  The relative errors of one gate, from the error
bounds of the operations it is made of (2^x instruction 4 U, reciprocal 2 U,
each float32 operation U, the logarithm 6.5 U), are
  e = exp(-|x|):              3 U |x| + 4 U
  sigmoid(x), sigmoid(-x):    (6 |x| + 12) U
  softplus(x):                (3 |x| + 13) U
  alpha = exp(-l), l = A sp:  (l (3 |x| + 17) + 4) U
with |x| of x = za + bias standing for |za| + |bias| (each is multiplied by
log2(e) and rounded before the sum), and for a = (1 - beta) alpha the same
whether the factors or their exponents are put together (an exponent's error
is three roundings of it at most),
and they enter a sum of products through its majorant, the same recurrence on
absolute values (H for the states, G for their gradients): every term of h[t]
is a product with one more factor a per step, whatever the order in which the
products are formed.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}


def double(t):
    return None if t is None else t.detach().cpu().double()


def bounds_of(offsets, n_seq, rows):
    if offsets is None:
        return [rows // n_seq * s for s in range(n_seq + 1)]
    return [int(o) for o in offsets.cpu()]


def recurrence(za, zb, v, A, bias, off, h0=None, dy=None, dhT=None):
    """Values and error bounds in float64 on the CPU: dict of (value, bound).
    Rows outside the sequences hold NaN."""
    za, zb, v, A, bias, h0, dy, dhT = map(double, (za, zb, v, A, bias, h0, dy, dhT))
    rows, D = za.shape
    n = len(off) - 1
    A = torch.ones(D, dtype=torch.float64) if A is None else A
    bias = torch.zeros(D, dtype=torch.float64) if bias is None else bias
    x = za + bias
    sp = torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))
    lam = A * sp
    alpha, beta, keep, sig = torch.exp(-lam), torch.sigmoid(zb), torch.sigmoid(-zb), torch.sigmoid(x)
    far = lambda t: torch.nan_to_num(t.abs(), posinf=200.0).clamp(max=200.0)   # exp(-200) is 0 in float32
    size = far(za.abs() + bias.abs())
    e_s = (6 * far(zb) + 12) * U
    e_sp = (3 * size + 13) * U
    e_alpha = (lam.clamp(max=200.0) * (3 * size + 17) + 4) * U
    e_a, e_b, e_sig = e_s + e_alpha + U, e_s + U, (6 * size + 12) * U
    a, b = keep * alpha, beta * v
    nan = lambda *s: torch.full(s, float("nan"), dtype=torch.float64)
    y, Ey, before, H, Eb = nan(rows, D), nan(rows, D), nan(rows, D), nan(rows, D), nan(rows, D)
    hT, EhT = nan(n, D), nan(n, D)
    for s in range(n):
        h = torch.zeros(D, dtype=torch.float64) if h0 is None else h0[s].clone()
        M, E = h.abs(), torch.zeros(D, dtype=torch.float64)
        for t in range(off[s], off[s + 1]):
            before[t], H[t], Eb[t] = h, M, E
            E = a[t] * E + (e_a[t] + 4 * U) * a[t] * M + (e_b[t] + 4 * U) * b[t].abs() + 1e-37
            h = a[t] * h + b[t]
            M = a[t] * M + b[t].abs()
            y[t], Ey[t] = h, E
        hT[s], EhT[s] = h, E
    out = {"y": (y, Ey), "hT": (hT, EhT)}
    if dy is None:
        return out
    g, G, Eg = nan(rows, D), nan(rows, D), nan(rows, D)
    dh0, Edh0 = nan(n, D), nan(n, D)
    for s in range(n):
        r = torch.zeros(D, dtype=torch.float64) if dhT is None else dhT[s].clone()
        M, E = r.abs(), torch.zeros(D, dtype=torch.float64)
        for t in range(off[s + 1] - 1, off[s] - 1, -1):
            g[t], G[t], Eg[t] = dy[t] + r, dy[t].abs() + M, E + 4 * U * (dy[t].abs() + M) + 1e-37
            r, M, E = a[t] * g[t], a[t] * G[t], a[t] * Eg[t] + (e_a[t] + 4 * U) * a[t] * G[t]
        dh0[s], Edh0[s] = r, E
    W = v.abs() + alpha * H
    dlog, Edlog = g * a * before, a * (Eg * H + G * Eb + (e_a + 4 * U) * G * H)
    out["dv"] = beta * g, beta * (Eg + (e_b + 2 * U) * G)
    out["dzb"] = (g * (v - alpha * before) * beta * keep,
                  beta * keep * (Eg * W + G * (alpha * Eb + (e_alpha + 4 * U) * W) + (2 * e_s + 4 * U) * G * W))
    out["dza"] = -A * sig * dlog, A * sig * (Edlog + (e_sig + 4 * U) * G * a * H)
    inside = torch.zeros(rows, dtype=torch.bool)
    for s in range(n):
        inside[off[s]:off[s + 1]] = True
    # Column sums over n rows in any order: at most n + 64 roundings of each term.
    k = (int(inside.sum()) + 64) * U
    col = lambda val, err: (val[inside].sum(0), (err + k * (val.abs() + err))[inside].sum(0) + 1e-37)
    out["dA"] = col(-sp * dlog, sp * (Edlog + (e_sp + 4 * U) * G * a * H))
    out["dbias"] = col(*out["dza"])
    out["dh0"] = dh0, Edh0
    return out


def within(got, value, bound, what="", where=None):
    """got is value, computed within `bound` and rounded to got's type."""
    g = got.detach().cpu().double().reshape(value.shape)
    lim = bound + HALF[got.dtype] * (value.abs() + bound) + 1e-37
    if where is not None:
        g, value, lim = g[where], value[where], lim[where]
    bad = ~((g - value).abs() <= lim)
    assert not bad.any(), (what, int(bad.sum()), bad.numel(),
                           float((g - value).abs()[bad].max()), float(lim[bad].min()),
                           torch.nonzero(bad)[:4].tolist())


def norm_sum(x, residual):
    """s by its definition: the float32 sum rounded to the type."""
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


# Sum of squares: every lane adds at most 64 terms in order and at most 16
# partial sums follow; its relative error is halved by the square root, whose
# result and the products with it take a few roundings more.
E_NORM = (0.5 * (64 + 16) + 8) * U


def rmsnorm(s, gamma, eps):
    """n in float64, its error bound, and s / sqrt(mean + eps)."""
    s = double(s)
    hat = s / torch.sqrt(s.square().mean(1, keepdim=True) + eps)
    y = hat if gamma is None else hat * double(gamma)
    return y, E_NORM * y.abs(), hat


def rmsnorm_backward(s, dout, gamma, ds, eps):
    s, dout = double(s), double(dout)
    inv = 1.0 / torch.sqrt(s.square().mean(1, keepdim=True) + eps)
    hat = s * inv
    w = dout if gamma is None else dout * double(gamma)
    m, M = (w * hat).mean(1, keepdim=True), (w * hat).abs().mean(1, keepdim=True)
    dx = inv * (w - hat * m)
    E = inv * (3 * E_NORM) * (w.abs() + hat.abs() * M)
    if ds is not None:
        dx = dx + double(ds)
        E = E + 2 * U * (double(ds).abs() + dx.abs())
    col = dout * hat
    k = (s.shape[0] + 64) * U + E_NORM
    return {"dx": (dx, E), "dgamma": (col.sum(0), k * col.abs().sum(0) + 1e-37)}
