"""fp64 references of the layer operators around the scan (tests only).

Each function also returns the same sums taken over absolute values, which the
tests' error bounds are multiples of. Plain loops over tokens, from the
definitions; numpy float64 throughout.
"""

from __future__ import annotations

import numpy as np

__all__ = ["silu", "softplus", "selective_scan", "conv1d", "group_norm"]


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
