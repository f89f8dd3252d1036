"""GPU tests of the gated delta rule's accuracy in the 2-norm (bounds:
delta_terms.py, shown to tell on the CPU in test_delta_terms.py): fp32 io's three
terms, and keys that a block's triangular system finds hardest."""

import numpy as np
import pytest
import torch

import mamba_ssd_scan_fwd_amd as ssd
from delta_terms import rms_bounds
from delta_testutil import HALF, Delta
from oracle import layer_oracle as ref
from ssd_testutil import np64, note
from test_delta_terms import FP32_OFF
from test_gpu_delta import is_cut

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def in_blocks(s):
    d = ssd.DeltaDesc(batch=s.b, seqlen=s.L, nheads=s.H, headdim=s.P, dstate=s.N, ngroups=s.G,
                      io_dtype=int(s.io == torch.bfloat16), scale=1.0)
    return ssd.delta_rule_workspace_bytes(d, len(s.lens) if s.lens else 0) > 0


def run(s):
    kw, h0, cu = s.to(DEV)
    if cu is None:
        return ssd.delta_rule(init_state=h0, **kw)
    return ssd.delta_rule_varlen(cu_seqlens=cu, init_states=h0, **kw)


def exact(s, bounds=False):
    """For pre = sigmoid = False: (y, S), and with `bounds` the 2-norms of what
    they may be off by."""
    x, B, C, dt, beta, A = (np64(t) for t in (s.x, s.B, s.C, s.dt, s.beta, s.A))
    spans = [(i, 0, s.L) for i in range(s.b)] if s.lens is None else [(0, int(f), int(e)) for f, e in zip(s.cu[:-1], s.cu[1:])]
    scale = float(np.float32(s.scale))
    y, S, ey, es = np.zeros(x.shape), np.zeros((len(spans), s.H, s.P, s.N)), 0.0, 0.0
    for n, (i, f, e) in enumerate(spans):
        for h in range(s.H):
            g = h // (s.H // s.G)
            args = (x[i, f:e, h], np.exp(dt[i, f:e, h] * A[h]), beta[i, f:e, h], B[i, f:e, g], C[i, f:e, g], scale, np64(s.init[n, h]))
            y[i, f:e, h], S[n, h] = ref.delta_rule(*args)
            if bounds:
                r = rms_bounds(*args, fp32=s.io == torch.float32)
                ey, es = ey + r[0] ** 2, es + r[1] ** 2
    return (y, S, np.sqrt(ey), np.sqrt(es)) if bounds else (y, S)


def off(got, want):
    return float(np.linalg.norm(np64(got) - want) / np.linalg.norm(want))


@pytest.mark.parametrize("L,P,N,views,lens", [
    (300, 48, 32, False, None), (300, 48, 64, False, None), (300, 48, 128, False, None), (300, 33, 77, True, None),
    (300, 33, 27, True, None), (300, 24, 61, False, [100, 0, 130, 70]), (300, 24, 128, False, [64, 65, 171]),
    # cut into segments
    (1100, 24, 32, False, None), (1100, 24, 64, False, None), (1100, 24, 128, False, None), (1300, 17, 50, True, None),
    (2200, 16, 64, False, [1500, 0, 700]),
])
def test_fp32_keeps_three_terms(L, P, N, views, lens):
    """Without a decay and with betas as they are given, so that nothing but the
    products is rounded. In segments the entering states have three products more
    behind them (the first walk's and the join's), each with errors of its own: the
    root of the two forms' squares, 1.5 of the bound, and 2 as the limit there."""
    s = Delta(1, L, 2 if L < 1000 else 1, P, N, 1, "fp32", "fp32", pre=False, sigmoid=False, views=views, lens=lens, seed=L + N)
    s.A.zero_()
    cut = is_cut(s, len(lens) if lens else 0)
    assert in_blocks(s) and cut == (L > 1000)
    note(f"[gpu] delta rule, three terms: L={L} P={P} N={N} lens={lens}")
    got, want = run(s), exact(s)
    note(f"   y {off(got[0], want[0]):.2e}, states {off(got[1], want[1]):.2e}")
    for name, g, w in zip(("y", "states"), got, want):
        assert off(g, w) < FP32_OFF * (2 if cut else 1), name


@pytest.mark.parametrize("io,P,N,views", [("bf16", 64, 64, False), ("bf16", 80, 128, False), ("bf16", 33, 100, True),
                                          ("bf16", 32, 200, False), ("fp32", 48, 64, False)])
@pytest.mark.parametrize("keys,low,high", [(1, 0.9, 1.1), (1, 1.9, 2.0), (3, 1.9, 2.0)])
@pytest.mark.parametrize("decay,length", [(0.0, 0.98), (1.0, 0.5), (0.3, 1.4)])
def test_keys_that_repeat_within_a_block(io, P, N, views, keys, low, high, decay, length):
    """Betas up to what a key's length allows; keys of length one and not. The
    values that a key answers replace one another, so y is a small difference of
    many of a block's solutions."""
    s = Delta(1, 200, 2, P, N, 1, io, io, pre=False, sigmoid=False, views=views, seed=keys + N)
    g = torch.Generator().manual_seed(keys)
    s.A.fill_(-decay)
    few = torch.randn((keys, 1, N), generator=g)
    few = few / few.norm(dim=-1, keepdim=True) * length
    s.B.copy_(few[torch.randint(0, keys, (200,), generator=g)][None])
    if keys == 1:
        s.C.copy_(s.B)
    s.beta.copy_((low + (high - low) * torch.rand((1, 200, 2), generator=g)) * (0.98 / length) ** 2)
    assert in_blocks(s)
    note(f"[gpu] delta rule: {keys} keys, betas {low} to {high}, decay {decay}, length {length} {io} P={P} N={N}")
    y, h = run(s)
    yr, hr, ey, es = exact(s, bounds=True)
    note(f"   y {off(y, yr):.2e}, states {off(h, hr):.2e}")
    assert np.linalg.norm(np64(y) - yr) < ey + HALF[s.io] * np.linalg.norm(yr)
    assert np.linalg.norm(np64(h) - hr) < es
