"""The gated delta rule in blocks as the matrix cores take it, in numpy: fp32
operands as sums of bf16 terms, products in fp32. And what its roundings come to
in the 2-norm, for bounds that a worst case element by element is too wide for.

Of one block, with S0 the state that enters it (delta_blocks.h has the names):
    R = X - e^g K S0^T;  U = T R;  Y = scale (e^g Q S0^T + M U);  S = e^g_end S0 + U'^T K

Bounds. u = 2^-24. An operand of n terms is off by at most 2^-8n, with whatever
sign; the terms of a sum are off independently of one another, so a product's sum
is off by the root of its terms' squares, times 2^-8n for each operand that is
rounded (taken at its greatest, where the root mean square is less than 3/5 of it).
fp32 sums: a product of three terms each has 6 pairs, so an entry adds up to
6 (N + 64 + 64) values and the substitution 192, 1728 with N = 128; each addition is off
by at most u of its partial sum, with a root mean square of u / sqrt(12) of
it: sqrt(1728 / 12) u = 12 u = 2^-20.4 and 2^-20 as the bound. With two terms of
bf16 io the same sums are far below 2^-16.
"""

from __future__ import annotations

import numpy as np
import torch

F32 = np.float32
OPERANDS = ("K", "S", "T", "R", "Q", "S of y", "M", "U of y", "U'", "K of the state")


def bf16(v):
    return torch.from_numpy(np.ascontiguousarray(v, dtype=F32)).to(torch.bfloat16).float().numpy()


def terms(v, n):
    out, v = [], np.asarray(v, F32)
    for _ in range(n):
        out.append(bf16(v))
        v = v - out[-1]
    return out


def mul(a, b, na, nb, acc=None):
    """acc + a b, of the pairs of terms that are as large as the longer one's last."""
    ta, tb = terms(a, na), terms(b, nb)
    r = np.zeros((a.shape[0], b.shape[1]), F32) if acc is None else np.asarray(acc, F32)
    for i in range(na):
        for j in range(nb):
            if i + j < max(na, nb):
                r = r + ta[i] @ tb[j]
    return r


def delta_in_terms(x, a, beta, k, q, scale, S0, terms_of, block=64):
    """One head as layer_oracle.delta_rule, fp32 throughout; terms_of names the
    terms of each operand (three where it names none)."""
    n = [terms_of.get(o, 3) for o in OPERANDS]
    x, a, beta, k, q = (np.asarray(v, F32) for v in (x, a, beta, k, q))
    S = np.zeros((x.shape[1], k.shape[1]), F32) if S0 is None else np.asarray(S0, F32)
    y = np.zeros(x.shape, F32)
    scale = F32(scale)
    for t0 in range(0, len(x), block):
        part = slice(t0, min(len(x), t0 + block))
        X, b, K, Q = x[part], beta[part], k[part], q[part]
        g = np.cumsum(np.log2(a[part].astype(np.float64)))
        i, j = np.indices((len(X), len(X)))
        dec = np.where(i >= j, np.exp2(np.where(i >= j, g[:, None] - g[None], 0.0)), 0.0).astype(F32)
        A = np.where(i > j, b[:, None] * dec * (K @ K.T), 0).astype(np.float64)
        T = np.linalg.inv(np.eye(len(X)) + A).astype(F32) * b[None]
        M = scale * dec * (Q @ K.T)
        eg, ed = np.exp2(g).astype(F32)[:, None], np.exp2(g[-1] - g).astype(F32)[:, None]
        R = X - eg * mul(K, S.T, n[0], n[1])
        U = mul(T, R, n[2], n[3])
        y[part] = mul(M, U, n[6], n[7], acc=scale * eg * mul(Q, S.T, n[4], n[5]))
        S = mul((ed * U).T, K, n[8], n[9], acc=eg[-1, 0] * S)
    return y, S


def rms_bounds(x, a, beta, k, q, scale, S0, fp32, block=64):
    """(y, state): the 2-norms of what the roundings of one head come to, stored
    roundings of y aside. For transitions that do not grow: the error of a state is
    passed on with the decay at the most."""
    one, two = (2.0 ** -20, 2.0 ** -20) if fp32 else (2.0 ** -8, 2.0 ** -16)
    S = np.zeros((x.shape[1], k.shape[1])) if S0 is None else S0.astype(np.float64)
    sq, es, ey = lambda m: m * m, 0.0, 0.0  # noqa: E731
    for t0 in range(0, len(x), block):
        part = slice(t0, min(len(x), t0 + block))
        X, b, K, Q = x[part], beta[part], k[part], q[part]
        g = np.cumsum(np.log(a[part]))
        i, j = np.indices((len(X), len(X)))
        dec = np.where(i >= j, np.exp(np.where(i >= j, g[:, None] - g[None], 0.0)), 0.0)
        T = np.linalg.inv(np.eye(len(X)) + np.where(i > j, b[:, None] * dec * (K @ K.T), 0)) * b[None]
        M = scale * dec * (Q @ K.T)
        eg, ed = np.exp(g)[:, None], np.exp(g[-1] - g)[:, None]
        R = X - eg * (K @ S.T)
        U = T @ R
        # off in R: its own rounding, and of S and K in what is taken off
        eR = two ** 2 * (sq(R) + 2 * sq(eg) * (sq(K) @ sq(S).T))
        # off in U: T's rounding, and R's through T
        eU = two ** 2 * (sq(T) @ sq(R)) + sq(T) @ eR
        own = eU + 2 * two ** 2 * sq(U)
        ey += np.sum(scale ** 2 * sq(eg) * (2 * one ** 2 * (sq(Q) @ sq(S).T) + np.sum(sq(Q), 1, keepdims=True) * es / x.shape[1]))
        ey += np.sum(2 * one ** 2 * (sq(M) @ sq(U)) + sq(M) @ eU)
        es = eg[-1, 0] ** 2 * (es + two ** 2 * np.sum(sq(S))) + np.sum(sq(ed * np.linalg.norm(K, axis=1, keepdims=True)) * own)
        S = eg[-1, 0] * S + (ed * U).T @ K
    return np.sqrt(ey), np.sqrt(es)
