"""GPU tests of the layer operators at the edges of what their documentation
allows, beside those of test_gpu_layer.py: offsets, unusual values, and the
kernels that only large calls reach. Bounds as derived in layer_testutil."""

import numpy as np
import pytest
import torch

import mamba_ssd_scan_fwd_amd as ssd
from layer_testutil import Selective, conv_reference, within
from ssd_testutil import note, np64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
GUARD = 4096


@pytest.mark.parametrize("cu", [[70, 80, 100], [64, 100, 100], [99, 100], [65, 64, 63, 100], [100, 100, 100]])
def test_offsets_that_begin_behind_a_piece_stay_inside(cu):
    """No offset before the end of the first 64 tokens, a piece of the first
    walk: whatever the values, nothing around the outputs is written."""
    E, N, L, S = 48, 16, 100, len(cu) - 1
    s = Selective(1, L, E, N, init=False, seed=47)
    kw, _, _ = s.to(DEV)
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    note(f"[gpu] offsets behind the first piece {cu}")
    ybuf = torch.full((2 * GUARD + L * E,), 9.0, device=DEV)
    fbuf = torch.full((2 * GUARD + S * E * N,), 9.0, device=DEV)
    y, f = ybuf[GUARD:-GUARD].view(1, L, E), fbuf[GUARD:-GUARD].view(S, E, N)
    ssd.selective_scan_varlen(cu_seqlens=c, y=y, final_states=f, **kw)
    cbuf = torch.full((2 * GUARD + S * E * 3,), 9.0, device=DEV)
    ssd.conv1d_varlen(kw["x"], torch.ones((E, 4), device=DEV), cu_seqlens=c, y=y,
                      conv_states_out=cbuf[GUARD:-GUARD].view(S, E, 3))
    torch.cuda.synchronize()
    for buf in (ybuf, fbuf, cbuf):
        assert (buf[:GUARD] == 9.0).all() and (buf[-GUARD:] == 9.0).all()


@pytest.mark.parametrize("cu,L,io", [([20, 60, 80], 100, "fp32"), ([70, 90, 90, 200], 230, "bf16"),
                                     ([1, 2, 300], 300, "fp32"), ([150, 150, 151], 260, "bf16")])
def test_offsets_that_begin_behind_the_first_token(cu, L, io):
    """A slice of a longer array of offsets: its sequences are computed, the
    tokens before and behind them left alone."""
    E, N, K, S = 48, 16, 4, len(cu) - 1
    s = Selective(1, L, E, N, io=io, dt=io, lens=[1] * S, seed=L)
    s.cu = torch.tensor(cu, dtype=torch.int32)
    kw, h0, c = s.to(DEV)
    note(f"[gpu] offsets {cu} of {L} tokens, {io}")
    for k in ("x", "dt", "z", "B", "C"):  # not read
        kw[k][:, :cu[0]] = float("nan")
        kw[k][:, cu[-1]:] = float("nan")
    y = torch.full((1, L, E), 7.0, dtype=s.io, device=DEV)
    f = torch.full((S, E, N), 7.0, device=DEV)
    ssd.selective_scan_varlen(cu_seqlens=c, init_states=h0, y=y, final_states=f, **kw)
    yr, yb, hr, hb = s.reference()
    within(y[:, cu[0]:cu[-1]], yr[:, cu[0]:cu[-1]], yb[:, cu[0]:cu[-1]], "y")
    within(f, hr, hb, "final_states")
    assert (y[:, :cu[0]] == 7.0).all() and (y[:, cu[-1]:] == 7.0).all()
    g = torch.Generator().manual_seed(48)
    w, c0 = torch.randn((E, K), generator=g), torch.randn((S, E, K - 1), generator=g)
    y.fill_(7.0)
    last = torch.full((S, E, K - 1), 7.0, device=DEV)
    ssd.conv1d_varlen(kw["x"], w.to(DEV), cu_seqlens=c, conv_states_in=c0.to(DEV), conv_states_out=last, y=y)
    want, bound, end = conv_reference(np64(s.x), np64(w), None, True, np64(c0), [(0, a, b) for a, b in zip(cu, cu[1:])], s.io)
    within(y[:, cu[0]:cu[-1]], want[:, cu[0]:cu[-1]], bound[:, cu[0]:cu[-1]], "conv")
    assert np.array_equal(np64(last), end)
    assert (y[:, :cu[0]] == 7.0).all() and (y[:, cu[-1]:] == 7.0).all()
