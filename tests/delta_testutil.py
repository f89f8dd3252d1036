"""Inputs, references and error bounds shared by the tests of the gated delta
rule and of the norm of heads.

Bounds. u = 2^-24. A two-term operand (a bf16 and the bf16 of what it leaves) is
off by at most 2^-8 * 2^-8 = 2^-16; with fp32 io there are three terms, 2^-24, and the
bounds for two below are wider than they need be.

- decay exp2(d A log2 e): its argument r is off by (32 + 3) u r (layer_testutil's
  softplus, A's and d's products), exp2 by 2 u, and e^-r r < 0.37; summed over
  up to 64 tokens of a block in 64 bits: (36 * 64 + 2) u for decays down to
  e^-64, below which a term is lost beside any other.
- beta: a sigmoid of |v| <= 10: 26 u.
- a token's products: S k over N columns (N + 1) u, the decay and beta above,
  difference, product, update: (N + 2400) u of delta_magnitudes' token form.
- in blocks, what reaches a state is made of products of two-term operands: the
  state and the keys in R (2^-16 each with fp32 io), R and T in U, U and the keys
  in the update: at most 6 * 2^-16, the products of two second terms left out
  (2^-16 at each of the three: 3 * 2^-16), sums of up to N and 2 * 64 terms and
  the substitution's 3 * 64 operations: 9 * 2^-16 + (2 N + 512) u of the block form.
- y: its own products are, with bf16 io, of operands rounded once: state,
  decayed scores and solutions 2^-8 each, two in a product: 2 * 2^-8 + 2^-16 of the
  block's terms; with fp32 io of two-term operands, 3 * 2^-16. Then the stored
  rounding.
- all of a state, in its 2-norm over random inputs: nine roundings of 2^-16 do
  not add up with one sign, but they may: 9 * 2^-16 of the norm (1.4e-4). One
  operand rounded to bf16 alone gives some 2^-8 / sqrt(12) = 1.1e-3.
- norm of a head: squares and sum (D + 2) u, halved by the root (2 u and a Newton
  step 3 u), products with the root and the weight: (D / 2 + 8) u. The angle:
  reduced in 64 bits, to 2^-25 of half a turn in fp32, so 2 u pi, sine and cosine
  4 u more, two products and a sum 3 u: (D / 2 + 22) u of |v_a| + |v_b|.
"""

from __future__ import annotations

import numpy as np
import torch

from layer_testutil import HALF, IO, U, within  # noqa: F401
from oracle import layer_oracle as ref
from ssd_testutil import np64


class Delta:
    """Seeded inputs of the rule: [b, L, ..], cut from wider buffers where
    ``views``; ``lens`` packs sequences (b = 1)."""

    def __init__(self, b, L, H, P, N, G=1, io="fp32", dt="fp32", init=True, pre=True, sigmoid=True, views=False, lens=None,
                 scale=0.3, seed=0, decay=2.8):
        g = torch.Generator().manual_seed(seed)
        T = self.io = IO[io]
        self.lens, self.b, self.L, self.H, self.P, self.N, self.G = lens, b, L, H, P, N, G
        self.scale, self.sigmoid = scale, sigmoid

        def draw(*shape, scale=1.0):
            return torch.randn(shape, generator=g) * scale

        def rows(heads, width, dtype, value):
            v = value if width is None else value.flatten(2)
            if views:
                wide = torch.full((b + 1, L + 2, v.shape[2] + 5), float("nan"))
                wide = wide.to(dtype)
                wide[:b, 1:L + 1, 3:v.shape[2] + 3] = v.to(dtype)
                v = wide[:b, 1:L + 1, 3:v.shape[2] + 3]
            else:
                v = v.to(dtype)
            return v if width is None else v.unflatten(-1, (heads, width))

        unit = lambda v: v / v.norm(dim=-1, keepdim=True).clamp(min=1e-6)  # noqa: E731
        self.x = rows(H, P, T, draw(b, L, H, P))
        # a little below length one, so that rounding to the io type keeps beta |k|^2 <= 2
        self.B, self.C = (rows(G, N, T, 0.98 * unit(draw(b, L, G, N))) for _ in range(2))
        self.beta = rows(H, None, IO[dt], draw(b, L, H) if sigmoid else torch.rand((b, L, H), generator=g) * 2.0)
        self.A = -torch.exp(torch.rand((H,), generator=g) * decay)
        n = len(lens) if lens is not None else b
        self.init = draw(n, H, P, N, scale=0.5) if init else None
        if pre:
            self.dt = rows(H, None, IO[dt], draw(b, L, H, scale=0.5))
            self.bias = draw(H, scale=0.5) - 3.0
            self.pre = dict(bias=self.bias, softplus=True, limit=(1e-3, 0.3))
        else:
            self.dt, self.bias, self.pre = rows(H, None, IO[dt], draw(b, L, H).abs() * 0.1), None, None
        self.cu = None if lens is None else torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)

    def to(self, dev):
        """Device copies that keep the strides of views."""
        def move(t):
            if t is None or t.is_contiguous():
                return None if t is None else t.to(dev)
            base = t._base if t._base is not None else t
            return base.to(dev).as_strided(t.shape, t.stride(), t.storage_offset())

        pre = None if self.pre is None else dict(self.pre, bias=self.pre["bias"].to(dev))
        return dict(x=move(self.x), dt=move(self.dt), A=self.A.to(dev), B=move(self.B), C=move(self.C),
                    beta=move(self.beta), dt_pre=pre, scale=self.scale, beta_sigmoid=self.sigmoid), move(self.init), move(self.cu)

    def reference(self, cut=False):
        """(y, bound of y, states, bound of states), rows or sequences in turn."""
        x, B, C, A = np64(self.x), np64(self.B), np64(self.C), np64(self.A)
        dt, beta = np64(self.dt), np64(self.beta)
        if self.sigmoid:
            beta = 1.0 / (1.0 + np.exp(-beta))
        if self.pre is not None:
            dt = np.clip(ref.softplus(dt + np64(self.bias)), np.float32(1e-3), np.float32(0.3))
        a = np.exp(dt * A)
        if self.lens is None:
            spans = [(i, 0, self.L) for i in range(self.b)]
        else:
            spans = [(0, int(f), int(e)) for f, e in zip(self.cu[:-1], self.cu[1:])]
        scale = float(np.float32(self.scale))
        y, yb = np.zeros(x.shape), np.zeros(x.shape)
        S = np.zeros((len(spans), self.H, self.P, self.N))
        Sb = np.zeros((len(spans), self.H, self.P, 1))
        fp32 = self.io == torch.float32
        ct, cb = (self.N + 2400) * U, 9 * 2.0 ** -16 + (2 * self.N + 512) * U
        cy = 3 * 2.0 ** -16 if fp32 else 2 * 2.0 ** -8 + 2.0 ** -16
        for s, (i, f, e) in enumerate(spans):
            for h in range(self.H):
                g = h // (self.H // self.G)
                args = (x[i, f:e, h], a[i, f:e, h], beta[i, f:e, h], B[i, f:e, g], C[i, f:e, g], scale,
                        None if self.init is None else np64(self.init[s, h]))
                y[i, f:e, h], S[s, h] = ref.delta_rule(*args)
                et, eb, yt, ybl, yo = ref.delta_magnitudes(*args, cut=cut)
                Sb[s, h, :, 0] = ct * et + cb * eb
                yb[i, f:e, h] = ct * yt + cb * ybl + cy * yo + HALF[self.io] * np.abs(y[i, f:e, h])
        return y, yb, S, Sb


def near(got, want, what, part=9 * 2.0 ** -16):
    """The whole state, in its 2-norm."""
    got = np64(got)
    off = np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-30)
    assert off <= part, f"{what}: off by {off:.2e} of its norm, allowed {part:.2e}"
