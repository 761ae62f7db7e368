"""Plain 64-bit forms of the layer norm, the short convolution and the selective
scan, with the largest error a float32 implementation of the same formulas can
make.

As in tests/_layers.py U is float32's half step and the relative errors of the
gates follow from the operations they are made of:
  sigmoid(x):                     (6 |x| + 12) U
  softplus(x):                    (3 |x| + 13) U, |x| standing for |dt| + |bias|
  delta = softplus ln 2 / ln 2:   2 U more
  a = exp(-A delta):              (l (3 |x| + 17) + 4) U with l = A delta; where a
                                  chunk's decay is one exponential of the summed
                                  delta, whose sum of up to `len` terms a lane adds
                                  at most half of in order, l len / 2 U more
Errors go through a sum of products by its majorant, the same recurrence on
absolute values (M for the states, G for their gradients).
"""
from __future__ import annotations

import torch

from tests._layers import U, double, within  # noqa: F401  (within: for the tests)

TINY = 1e-37
# The 2^x and reciprocal instructions and what is made of them flush results below
# 2^-126 to zero: exp(-90) = 8e-40 is 0.  So delta, a and the sigmoids are off by
# 2^-126 besides, and products with them by that times the other factor (du = 1e3
# at delta = exp(-88) = 6e-39: 6e-36, more than TINY).
FLUSH = 2.0 ** -126


def far(t):
    return torch.nan_to_num(t.abs(), posinf=200.0).clamp(max=200.0)   # exp(-200) is 0 in float32


# ---------------------------------------------------------------- layer norm

# Sums along a row: every lane adds at most 64 terms in order, at most 16 + 5
# partial sums follow.
SUMS = (64 + 21) * U


def _centred(s, eps):
    s = double(s)
    mean = s.mean(1, keepdim=True)
    c = s - mean
    e_mean = (SUMS + 2 * U) * s.abs().mean(1, keepdim=True)
    e_c = e_mean + U * c.abs()
    var = c.square().mean(1, keepdim=True) + eps
    e_var = 2 * (e_c * c.abs()).mean(1, keepdim=True) + e_c.square().mean(1, keepdim=True) + (SUMS + 4 * U) * var
    part = e_var / var
    assert (part < 0.5).all(), "the float32 variance says nothing"
    inv = 1.0 / torch.sqrt(var)
    e_inv = part / (1 - part) + 5 * U                       # relative; half would do for a small part
    hat = c * inv
    return c, hat, inv, e_c, e_inv, inv * e_c + hat.abs() * (e_inv + 2 * U)


def layernorm(s, gamma, beta, eps):
    """n in float64 and its error bound."""
    _, hat, _, _, _, e_hat = _centred(s, eps)
    g = torch.ones(hat.shape[1], dtype=torch.float64) if gamma is None else double(gamma)
    b = torch.zeros(hat.shape[1], dtype=torch.float64) if beta is None else double(beta)
    y = hat * g + b
    return y, g.abs() * e_hat + 2 * U * ((hat * g).abs() + b.abs()) + TINY


def layernorm_backward(s, dout, gamma, ds, eps):
    c, hat, inv, e_c, e_inv, e_hat = _centred(s, eps)
    dout = double(dout)
    w = dout if gamma is None else dout * double(gamma)
    mean = lambda t: t.mean(1, keepdim=True)
    mw, m = mean(w), mean(w * hat)
    e_mw = (SUMS + 2 * U) * mean(w.abs())
    e_m = mean(w.abs() * e_hat) + (SUMS + 4 * U) * mean((w * hat).abs())
    inner = w - mw - hat * m
    size = w.abs() + mw.abs() + (hat * m).abs()
    e_inner = e_mw + hat.abs() * e_m + e_hat * m.abs() + 4 * U * size
    dx = inv * inner
    E = inv * e_inner + (e_inv + 2 * U) * inv * size
    if ds is not None:
        dx = dx + double(ds)
        E = E + 2 * U * (double(ds).abs() + dx.abs())
    k = (dout.shape[0] + 64) * U
    return {"dx": (dx, E + TINY),
            "dgamma": ((dout * hat).sum(0), (dout.abs() * e_hat).sum(0) + k * (dout * hat).abs().sum(0) + TINY),
            "dbeta": (dout.sum(0), k * dout.abs().sum(0) + TINY)}


# ---------------------------------------------------------------- activation

def silu(x, e_x):
    """silu(x) and its bound, for x with the error e_x."""
    s = torch.sigmoid(x)
    y = x * s
    return y, 1.1 * e_x + torch.nan_to_num(y).abs() * (6 * far(x) + 15) * U + far(x) * FLUSH + TINY


def dsilu(x, e_x):
    """sig (1 + x (1 - sig)) and its bound; its own slope is at most 0.5."""
    s = torch.sigmoid(x)
    size = 1 + x.abs() * (1 - s)
    e_s = (6 * far(x) + 12) * U
    E = 0.5 * e_x + s * (size * (e_s + 5 * U) + x.abs() * (s * e_s + 2 * U)) + size * FLUSH + TINY
    return s * (1 + x * (1 - s)), E


# --------------------------------------------------------------- convolution

def conv(x, w, bias, off, act, x0=None, dy=None, dxT=None):
    """(value, bound) of every output; rows outside the sequences hold NaN."""
    x, w, bias, x0, dy, dxT = map(double, (x, w, bias, x0, dy, dxT))
    rows, D = x.shape
    K, n = w.shape[1], len(off) - 1
    bias = torch.zeros(D, dtype=torch.float64) if bias is None else bias
    nan = lambda *s: torch.full(s, float("nan"), dtype=torch.float64)
    zeros = lambda *s: torch.zeros(*s, dtype=torch.float64)
    y, Ey, dx, Edx = (nan(rows, D) for _ in range(4))
    xT, dx0, Edx0 = nan(n, K - 1, D), zeros(n, K - 1, D), zeros(n, K - 1, D)
    dw, Mw, Ew, db, Mb, Eb = zeros(D, K), zeros(D, K), zeros(D, K), zeros(D), zeros(D), zeros(D)
    for s in range(n):
        a, b = off[s], off[s + 1]
        T = b - a
        seq = torch.cat([zeros(K - 1, D) if x0 is None else x0[s], x[a:b]])
        pre = bias + sum(w[:, j] * seq[j:j + T] for j in range(K))
        e_pre = (K + 1) * U * (bias.abs() + sum((w[:, j] * seq[j:j + T]).abs() for j in range(K)))
        y[a:b], Ey[a:b] = silu(pre, e_pre) if act else (pre, e_pre)
        xT[s] = seq[T:]
        if dy is None:
            continue
        f, ef = dsilu(pre, e_pre) if act else (torch.ones_like(pre), torch.zeros_like(pre))
        d = dy[a:b] * f
        ed = dy[a:b].abs() * (ef + 2 * U * f.abs())
        g, M, E = zeros(T + K - 1, D), zeros(T + K - 1, D), zeros(T + K - 1, D)
        for j in range(K):
            g[j:j + T] += w[:, j] * d
            M[j:j + T] += (w[:, j] * d).abs()
            E[j:j + T] += w[:, j].abs() * ed
            dw[:, j] += (d * seq[j:j + T]).sum(0)
            Mw[:, j] += (d * seq[j:j + T]).abs().sum(0)
            Ew[:, j] += (ed * seq[j:j + T].abs()).sum(0)
        db += d.sum(0)
        Mb += d.abs().sum(0)
        Eb += ed.sum(0)
        if dxT is not None:
            g[T:] += dxT[s]
            M[T:] += dxT[s].abs()
        E = E + (K + 2) * U * M + TINY
        dx0[s], Edx0[s], dx[a:b], Edx[a:b] = g[:K - 1], E[:K - 1], g[K - 1:], E[K - 1:]
    out = {"y": (y, Ey + TINY), "xT": (xT, torch.zeros_like(xT))}
    if dy is not None:
        k = (off[-1] - off[0] + 64) * U
        out.update(dx=(dx, Edx), dx0=(dx0, Edx0), dw=(dw, Ew + k * Mw + TINY), dbias=(db, Eb + k * Mb + TINY))
    return out


# ---------------------------------------------------------------------- scan

def scan(x, dt, A, B, C, off, skip=None, bias=None, z=None, h0=None, dy=None, dhT=None):
    """(value, bound) of every output; rows outside the sequences hold NaN.
    B, C [rows, groups, N]."""
    x, dt, A, B, C, skip, bias, z, h0, dy, dhT = map(double, (x, dt, A, B, C, skip, bias, z, h0, dy, dhT))
    rows, D = x.shape
    G, N = B.shape[1:]
    n, per = len(off) - 1, D // G
    zero = torch.zeros(D, dtype=torch.float64)
    skip, bias = zero if skip is None else skip, zero if bias is None else bias
    wide = lambda t: t.repeat_interleave(per, 1)                       # [rows, D, N]
    raw = dt + bias
    size = far(dt.abs() + bias.abs())
    delta = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    e_d = (3 * size + 15) * U
    length = torch.zeros(rows, 1, 1, dtype=torch.float64)
    inside = torch.zeros(rows, dtype=torch.bool)
    for s in range(n):
        length[off[s]:off[s + 1]] = off[s + 1] - off[s]
        inside[off[s]:off[s + 1]] = True
    lam = A * delta[:, :, None]
    a = torch.exp(-lam)
    e_a = (lam.clamp(max=200.0) * (3 * size[:, :, None] + 17 + length / 2) + 4) * U
    u, e_u = delta * x, e_d + 2 * U
    Bw, Cw = wide(B), wide(C)
    b = u[:, :, None] * Bw
    e_b = (e_u + 2 * U)[:, :, None]
    nan = lambda *s: torch.full(s, float("nan"), dtype=torch.float64)
    before, M, E = nan(rows, D, N), nan(rows, D, N), nan(rows, D, N)   # in front of each row
    after, Ma, Ea = nan(rows, D, N), nan(rows, D, N), nan(rows, D, N)
    hT, EhT = nan(n, D, N), nan(n, D, N)
    grow, take = (e_a + 4 * U) * a + FLUSH, (e_b + 3 * U) * b.abs() + FLUSH * (x[:, :, None] * Bw).abs() + TINY
    for s in range(n):
        h = torch.zeros(D, N, dtype=torch.float64) if h0 is None else h0[s].clone()
        m, e = h.abs(), torch.zeros(D, N, dtype=torch.float64)
        for t in range(off[s], off[s + 1]):
            before[t], M[t], E[t] = h, m, e
            e = a[t] * e + grow[t] * m + take[t]
            h = a[t] * h + b[t]
            m = a[t] * m + b[t].abs()
            after[t], Ma[t], Ea[t] = h, m, e
        hT[s], EhT[s] = h, e
    inner = (Cw * after).sum(2) + skip * x
    M_in = (Cw.abs() * Ma).sum(2) + (skip * x).abs()
    e_in = (Cw.abs() * Ea).sum(2) + (N + 4) * U * M_in
    if z is None:
        y, Ey = inner, e_in
    else:
        gate, e_gate = silu(z, torch.zeros_like(z))
        y, Ey = inner * gate, gate.abs() * e_in + M_in * (e_gate + 2 * U * gate.abs())
    out = {"y": (y, Ey + TINY), "hT": (hT, EhT)}
    if dy is None:
        return out
    d = dy if z is None else dy * gate
    e_dd = torch.zeros_like(d) if z is None else dy.abs() * (e_gate + 2 * U * gate.abs())
    g, Gm, Eg, r, Rm, Er = (nan(rows, D, N) for _ in range(6))
    dh0, Edh0 = nan(n, D, N), nan(n, D, N)
    push = d[:, :, None] * Cw
    e_push = e_dd[:, :, None] * Cw.abs() + 2 * U * push.abs() + TINY
    for s in range(n):
        v = torch.zeros(D, N, dtype=torch.float64) if dhT is None else dhT[s].clone()
        m, e = v.abs(), torch.zeros(D, N, dtype=torch.float64)
        for t in range(off[s + 1] - 1, off[s] - 1, -1):
            g[t], Gm[t] = push[t] + v, push[t].abs() + m
            Eg[t] = e + e_push[t] + 2 * U * Gm[t]
            v, m, e = a[t] * g[t], a[t] * Gm[t], a[t] * Eg[t] + grow[t] * Gm[t]
            r[t], Rm[t], Er[t] = v, m, e
        dh0[s], Edh0[s] = v, e
    p, Pm = r * before, Rm * M
    Ep = Er * M + Rm * E + 2 * U * Pm
    du, dum, Edu = (g * Bw).sum(2), (Gm * Bw.abs()).sum(2), (Eg * Bw.abs()).sum(2)
    Edu = Edu + (N + 4) * U * dum
    dl, dlm, Edl = (p * A).sum(2), (Pm * A).sum(2), (Ep * A).sum(2)
    Edl = Edl + (N + 4) * U * dlm
    sig, e_sig = torch.sigmoid(raw), (6 * size + 12) * U
    # The product's error besides: |d| is known to e_dd.
    dx = du * delta + d * skip
    Edx = Edu * delta + dum * (delta * (e_d + 3 * U) + FLUSH) + skip.abs() * (e_dd + 3 * U * d.abs())
    ddt = (du * x - dl) * sig
    Mddt = (dum * x.abs() + dlm) * sig
    Eddt = sig * (Edu * x.abs() + Edl) + Mddt * (e_sig + 5 * U) + (dum * x.abs() + dlm) * FLUSH
    groups = lambda t: t.view(rows, G, per, N).sum(2)
    k = (per + 64) * U
    au = u.abs()[:, :, None]
    dB, EdB = groups(g * u[:, :, None]), groups(Eg * au + Gm * au * (e_u[:, :, None] + 2 * U + k) + Gm * FLUSH * x.abs()[:, :, None])
    ad, ed3 = d.abs()[:, :, None], e_dd[:, :, None]
    dC, EdC = groups(d[:, :, None] * after), groups(ad * Ea + Ma * (ed3 + ad * (2 * U + k)))
    q = (int(inside.sum()) + 64) * U
    col = lambda val, size_, err: (val[inside].sum(0), (err + q * size_)[inside].sum(0) + TINY)
    d3 = delta[:, :, None]
    out["dA"] = col(-d3 * p, d3 * Pm, d3 * Ep + d3 * Pm * (e_d[:, :, None] + 4 * U) + FLUSH * Pm)
    out["dskip"] = col(d * x, (d * x).abs(), x.abs() * (e_dd + 2 * U * d.abs()))
    out["dbias"] = col(ddt, Mddt, Eddt)
    out.update(dx=(dx, Edx + TINY), ddt=(ddt, Eddt + TINY), dB=(dB, EdB + TINY), dC=(dC, EdC + TINY), dh0=(dh0, Edh0))
    if z is not None:
        f, ef = dsilu(z, torch.zeros_like(z))
        out["dz"] = dy * inner * f, dy.abs() * (f.abs() * e_in + M_in * (ef + 3 * U * f.abs())) + TINY
    return out
