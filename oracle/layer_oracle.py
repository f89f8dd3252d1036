"""fp64 references of the layer operators around the scan (tests only).

Each function also returns the same sums taken over absolute values, which the
tests' error bounds are multiples of. Plain loops over tokens, from the
definitions; numpy float64 throughout.
"""

from __future__ import annotations

import numpy as np

__all__ = ["silu", "softplus", "selective_scan", "conv1d", "group_norm", "delta_rule", "delta_magnitudes", "head_norm"]


def silu(z):
    with np.errstate(over="ignore"):
        return z / (1.0 + np.exp(-z))


def softplus(v):
    return np.logaddexp(v, 0.0)


def selective_scan(x, dt, A, B, C, D=None, z=None, h0=None):
    """x, dt, z [L, E]; A [E, N]; B, C [L, G, N]; h0 [E, N]. dt as it enters
    the recurrence. Returns y, y_abs [L, E], h, h_abs [E, N]."""
    L, E = x.shape
    G, N = B.shape[1:]
    h = np.zeros((E, N)) if h0 is None else h0.astype(np.float64).copy()
    ha = np.abs(h)
    y, ya = np.zeros((L, E)), np.zeros((L, E))
    per = E // G
    for t in range(L):
        Bt, Ct = np.repeat(B[t], per, 0), np.repeat(C[t], per, 0)
        decay = np.exp(dt[t][:, None] * A)
        u = (dt[t] * x[t])[:, None] * Bt
        h = decay * h + u
        ha = decay * ha + np.abs(u)
        y[t] = (h * Ct).sum(1)
        ya[t] = (ha * np.abs(Ct)).sum(1)
    if D is not None:
        y += D * x
        ya += np.abs(D * x)
    if z is not None:
        y, ya = y * silu(z), ya * np.abs(silu(z))
    return y, ya, h, ha


def conv1d(x, w, bias=None, act=True, state=None):
    """x [L, CH]; w [CH, K]; state [CH, K-1]. Returns out, the sums of
    absolute values before the activation [L, CH], and the last K-1 inputs."""
    L, CH = x.shape
    K = w.shape[1]
    line = np.concatenate([np.zeros((K - 1, CH)) if state is None else state.T.astype(np.float64), x])
    z = np.zeros((L, CH)) if bias is None else np.tile(bias, (L, 1))
    za = np.abs(z)
    for k in range(K):
        z = z + line[k:k + L] * w[:, k]
        za = za + np.abs(line[k:k + L] * w[:, k])
    return (silu(z) if act else z), za, line[L:].T


def group_norm(x, ngroups, eps, w=None, bias=None, z=None, center=True, gate_first=False, act=False):
    """x, z [R, C]. Returns out [R, C]."""
    R, C = x.shape
    gate = None if z is None else silu(z)
    v = (x * gate if gate is not None and gate_first else x).reshape(R, ngroups, -1)
    if center:
        v = v - v.mean(2, keepdims=True)
    o = (v / np.sqrt((v * v).mean(2, keepdims=True) + eps)).reshape(R, C)
    if w is not None:
        o = o * w
    if bias is not None:
        o = o + bias
    if gate is not None and not gate_first:
        o = o * gate
    return silu(o) if act else o


def delta_rule(x, a, beta, k, q, scale=1.0, S0=None):
    """One head. x [L, P]; decays a and beta [L]; k, q [L, N]; S0 [P, N].
    Returns y [L, P], S [P, N]."""
    L, P = x.shape
    S = np.zeros((P, k.shape[1])) if S0 is None else S0.astype(np.float64).copy()
    y = np.zeros((L, P))
    for t in range(L):
        S = a[t] * S
        S = S + np.outer(beta[t] * (x[t] - S @ k[t]), k[t])
        y[t] = scale * (S @ q[t])
    return y, S


def delta_magnitudes(x, a, beta, k, q, scale=1.0, S0=None, block=64, cut=False):
    """What rounding errors of ``delta_rule`` are multiples of, for keys and
    betas whose transitions do not grow (beta |k|^2 <= 2): an error of a row of
    the state, in the 2-norm, is then passed on with the decay and no more.

    Token by token: E_t = a E_{t-1} + a |s| (1 + beta |k|^2) + beta |x| |k|.
    In blocks, whose solution is U = T R with R = beta (x - e^g S0 k) and
    T = (1 + A)^-1: |U| <= K = |T| |1 + A| |T| beta (|x| + e^g |S0| |k|), and
    E <- e^g E + e^g |S0| + sum_j e^(g - g_j) |k_j| K_j.
    With ``cut`` for states that are joined from what a segment makes of the state
    that enters it, S0 M, and of none, B: |S0 M| <= |S0| and |B| <= |S| + |S0|, so
    both have 3 max|S| in |S0|'s place.
    Returns (token [P], block [P], y's token and block form [L, P], y's block
    terms themselves [L, P]): the latter what roundings of the operands of y's
    products alone are multiples of."""
    L, P = x.shape
    S = np.zeros((P, k.shape[1])) if S0 is None else S0.astype(np.float64).copy()
    kn, qn = np.linalg.norm(k, axis=1), np.linalg.norm(q, axis=1)
    assert np.all(beta * kn * kn <= 2.0 + 1e-6), "the transitions grow"
    et, eb = np.zeros(P), np.zeros(P)
    yt, yb, yo = np.zeros((L, P)), np.zeros((L, P)), np.zeros((L, P))
    norm = lambda m: np.linalg.norm(m, axis=1)  # noqa: E731
    top = norm(S)
    if cut:
        for t in range(L):
            S = a[t] * S
            S = S + np.outer(beta[t] * (x[t] - S @ k[t]), k[t])
            top = np.maximum(top, norm(S))
        S = np.zeros((P, k.shape[1])) if S0 is None else S0.astype(np.float64).copy()
    for t0 in range(0, L, block):
        t1 = min(L, t0 + block)
        n, kk, qq, xx, bb = t1 - t0, k[t0:t1], q[t0:t1], x[t0:t1], beta[t0:t1]
        with np.errstate(divide="ignore"):
            g = np.cumsum(np.log(a[t0:t1]))
        i, j = np.indices((n, n))
        dec = np.where(i >= j, np.exp(np.where(i >= j, g[:, None] - g[None, :], 0.0)), 0.0)
        IA = np.eye(n) + np.where(i > j, bb[:, None] * dec * (kk @ kk.T), 0.0)
        T = np.abs(np.linalg.inv(IA))
        s0 = 3 * top if cut else norm(S)
        K = T @ np.abs(IA) @ T @ (bb[:, None] * (np.abs(xx) + np.exp(g)[:, None] * s0 * kn[t0:t1, None]))
        att = dec * np.abs(qq @ kk.T)
        for r in range(n):
            t = t0 + r
            et = a[t] * et + a[t] * norm(S) * (1 + beta[t] * kn[t] ** 2) + beta[t] * np.abs(x[t]) * kn[t]
            S = a[t] * S
            S = S + np.outer(beta[t] * (x[t] - S @ k[t]), k[t])
            yt[t] = abs(scale) * (qn[t] * et + norm(S) * qn[t])
            own = (dec[r][:, None] * kn[t0:t1, None] * K).sum(0)
            yb[t] = abs(scale) * qn[t] * (np.exp(g[r]) * (eb + s0) + own)
            yo[t] = abs(scale) * (np.exp(g[r]) * s0 * qn[t] + att[r] @ K)
        eb = np.exp(g[-1]) * (eb + s0) + (np.exp(g[-1] - g)[:, None] * kn[t0:t1, None] * K).sum(0)
    return et, eb, yt, yb, yo


def head_norm(x, eps, w=None, l2=False, angle=None, pairs=False):
    """x [.., heads, D]; angle [.., R / 2] of each token. Returns the result and
    what its rounding errors are multiples of."""
    sq = (x * x).sum(-1, keepdims=True)
    v = x / np.sqrt((sq if l2 else sq / x.shape[-1]) + eps)
    if w is not None:
        v = v * w
    mag = np.abs(v)
    if angle is not None:
        half = angle.shape[-1]
        a = np.arange(half) * 2 if pairs else np.arange(half)
        b = a + 1 if pairs else a + half
        c, s = np.cos(angle)[..., None, :], np.sin(angle)[..., None, :]
        out, m = v.copy(), mag.copy()
        out[..., a] = v[..., a] * c - v[..., b] * s
        out[..., b] = v[..., b] * c + v[..., a] * s
        m[..., a] = m[..., b] = mag[..., a] + mag[..., b]
        v, mag = out, m
    return v, mag
