"""GPU tests of the layer operators at the edges of what their documentation
allows, beside those of test_gpu_layer.py: offsets, unusual values, and the
kernels that only large calls reach. Bounds as derived in layer_testutil."""

import pytest
import torch

import mamba_ssd_scan_fwd_amd as ssd
from layer_testutil import Selective
from ssd_testutil import note

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
