"""Inputs, references and error bounds shared by the tests of the layer
operators around the scan.

Bounds. u = 2^-24 is half a step of fp32, and every fp32 operation of a kernel
is off by at most u relative to its result (the hardware's exp2, log2,
reciprocal and reciprocal root by at most 1 ulp = 2 u). A result stored in
bf16 is off by 2^-8 of itself more.

- softplus: log(1 + e^v): argument product u |v| log2(e) -> 2 u |v|, exp2 2 u,
  1 + e rounded and corrected to first order, log, reciprocal and three
  products: below (16 + 2 |v|) u relative for the |v| <= 8 drawn here: 32 u.
- scan: a term of y_t entered k steps ago passed k decays exp2(d A2) (2 u for
  exp2, its argument off by 34 u relative: A2, d and one product; a factor e^-r
  is then off by 34 u r, and r e^-r < 0.37) and k fused adds: at most
  (3 k + 34 * 64) u for decays down to e^-64, below which a term is lost
  beside any other. Summed over N states and with d x B and D: (N + 40) u.
  Together (3 L + N + 2300) u of the sum of absolute values.
- silu: argument product and exp2 2 u |z| + 2 u, sum, reciprocal, product: for
  |z| <= 10 at most 26 u relative.
- conv: K products and adds: (K + 1) u of the sum of absolute values; through
  the SiLU (slope below 1.1) and its own error.
"""

from __future__ import annotations

import numpy as np
import torch

from oracle import layer_oracle as ref
from ssd_testutil import np64

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
IO = {"fp32": torch.float32, "bf16": torch.bfloat16}


def within(got, want, bound, what):
    got, want = np64(got) if isinstance(got, torch.Tensor) else got, np.asarray(want)
    assert got.shape == want.shape, f"{what}: shape {got.shape}, expected {want.shape}"
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    over = np.abs(got - want) - bound
    if over.size and np.max(over) > 0:
        i = np.unravel_index(np.argmax(over), over.shape)
        raise AssertionError(f"{what}: off by {np.abs(got - want)[i]:.3e} at {i}, allowed "
                             f"{np.broadcast_to(bound, want.shape)[i]:.3e}")


class Selective:
    """Seeded inputs of a selective scan: [b, L, ..], cut from wider buffers
    where ``views``; ``lens`` packs sequences (b = 1)."""

    def __init__(self, b, L, E, N, G=1, io="fp32", dt="fp32", gate=True, skip=True, init=True, pre=True, views=False,
                 lens=None, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.io, self.lens, self.b, self.L, self.E, self.N, self.G = IO[io], lens, b, L, E, N, G
        T = self.io

        def draw(*shape, scale=1.0):
            return torch.randn(shape, generator=g) * scale

        def rows(width, dtype, scale=1.0):
            if not views:
                return draw(b, L, width, scale=scale).to(dtype)
            wide = draw(b + 1, L + 2, width + 5, scale=scale).to(dtype)
            return wide[:b, 1:L + 1, 3:width + 3]

        self.x, self.z = rows(E, T), (rows(E, T) if gate else None)
        self.B, self.C = (rows(G * N, T, N ** -0.5).unflatten(-1, (G, N)) for _ in range(2))
        self.A = -torch.exp(torch.rand((E, N), generator=g) * 2.8)
        self.D = draw(E) if skip else None
        n = len(lens) if lens is not None else b
        self.init = draw(n, E, N, scale=0.5) if init else None
        if pre:
            self.dt = rows(E, IO[dt], 0.5)
            self.bias = draw(E, scale=0.5) - 2.0
            self.pre = dict(bias=self.bias, softplus=True, limit=(1e-3, 0.5))
        else:
            self.dt, self.bias, self.pre = (rows(E, IO[dt], 0.5).abs() * 0.2), None, None
        self.cu = None
        if lens is not None:
            self.cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)

    def to(self, dev):
        """Device copies that keep the strides of views."""
        def move(t):
            if t is None:
                return None
            if t.is_contiguous():
                return t.to(dev)
            base = t._base if t._base is not None else t
            return base.to(dev).as_strided(t.shape, t.stride(), t.storage_offset())

        pre = None if self.pre is None else dict(self.pre, bias=self.pre["bias"].to(dev))
        return dict(x=move(self.x), dt=move(self.dt), A=self.A.to(dev), B=move(self.B), C=move(self.C),
                    D=move(self.D), z=move(self.z), dt_pre=pre), move(self.init), move(self.cu)

    def reference(self):
        """(y, bound of y, states, bound of states), rows or sequences in turn."""
        x, B, C, A = np64(self.x), np64(self.B), np64(self.C), np64(self.A)
        dt = np64(self.dt)
        if self.pre is not None:
            dt = np.clip(ref.softplus(dt + np64(self.bias)), 1e-3, 0.5)
        z, D = (None if t is None else np64(t) for t in (self.z, self.D))
        if self.lens is None:
            spans = [(i, 0, self.L) for i in range(self.b)]
        else:
            spans = [(0, int(a), int(b)) for a, b in zip(self.cu[:-1], self.cu[1:])]
        y, ya = np.zeros(x.shape), np.zeros(x.shape)
        hs, has = [], []
        for s, (i, a, b) in enumerate(spans):
            h0 = None if self.init is None else np64(self.init[s])
            r = ref.selective_scan(x[i, a:b], dt[i, a:b], A, B[i, a:b], C[i, a:b], D,
                                   None if z is None else z[i, a:b], h0)
            y[i, a:b], ya[i, a:b] = r[0], r[1]
            hs.append(r[2]), has.append(r[3])
        f = (3 * self.L + self.N + 2300 + 26) * U
        return y, ya * f + np.abs(y) * HALF[self.io], np.stack(hs), np.stack(has) * f


def conv_reference(x, w, bias, act, states, spans, io):
    """x [b, L, CH] float64, spans [(row, first, last)] with a state each.
    Returns out, its bound, the last states."""
    out, bound = np.zeros(x.shape), np.zeros(x.shape)
    last = []
    for s, (i, a, b) in enumerate(spans):
        o, za, st = ref.conv1d(x[i, a:b], w, bias, act, None if states is None else states[s])
        out[i, a:b] = o
        bound[i, a:b] = 1.1 * (w.shape[1] + 1) * U * za + (26 * U + HALF[io]) * np.abs(o)
        last.append(st)
    return out, bound, np.stack(last)


def norm_bound(x, ngroups, eps, w, bias, z, center, gate_first, act, io, out):
    """v carries the gate's 27 u; the mean adds at most 64 adds' and the
    product's u of mean|v|; the squares' mean (66 u and the doubled errors of
    v - mu) halves in the root (2 u, and a Newton step): 40 u of o and the
    mean's error, through weight and slope of what follows; then the stored
    rounding."""
    R, C = x.shape
    gate = None if z is None else ref.silu(z)
    v = (x * gate if gate is not None and gate_first else x).reshape(R, ngroups, -1)
    mean_abs = np.abs(v).mean(2, keepdims=True)
    c = v - v.mean(2, keepdims=True) if center else v
    sd = np.sqrt((c * c).mean(2, keepdims=True) + eps)
    dmu = 66 * U * mean_abs if center else np.zeros_like(mean_abs)
    # error of v - mu relative to the group's deviation, and of the deviation itself
    dv = 28 * U * np.abs(v) + dmu
    dsd = np.sqrt((dv * dv).mean(2, keepdims=True)) + 40 * U * sd
    rel = (dv + U * np.abs(c)) / sd + np.abs(c) / sd * (dsd / sd + 4 * U)
    wn = 1.0 if w is None else np.abs(w)
    err = rel.reshape(R, C) * wn
    core = (c / sd).reshape(R, C) * (1.0 if w is None else w)
    err = err + 3 * U * (np.abs(core) + (0.0 if bias is None else np.abs(bias)))
    if gate is not None and not gate_first:
        err = err * np.abs(gate)
    if act:
        err = 1.1 * err
    return err + (28 * U + HALF[io]) * np.abs(out)
