"""GPU test of the norm of heads: angles of any size, against 60 digits."""

from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import mamba_ssd_scan_fwd_amd as ssd
from delta_testutil import U
from ssd_testutil import note

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
getcontext().prec = 60
TURN = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")


def test_angles_of_any_size():
    """Off by at most 2^-26 of a turn, the reduced angle's rounding to fp32, and 3 * 2^-53
    of the turns, those of 1 / (2 pi) and of two products in 64 bits; sine and cosine 4 u
    more, the norm 16 u."""
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 1999999999, 123456789, 4095, 1], dtype=torch.int32)
    freq = torch.tensor([1.0, 0.7310585975646973, 2.5, 10000.0, 16777215.0, 1e-4])
    x = torch.zeros((len(pos), 1, 12))
    x[..., :6] = 1.0
    note("[gpu] head norm: angles of up to 2^55")
    out = ssd.head_norm(x.to(DEV), positions=pos.to(DEV), inv_freq=freq.to(DEV), eps=0.0).double().cpu().numpy()[:, 0] / np.sqrt(2.0)
    for i, p in enumerate(pos.tolist()):
        for j, f in enumerate(freq.tolist()):
            turns = Decimal(p) * Decimal(f) / TURN
            part = float(turns - turns.to_integral_value()) * 2 * np.pi
            bound = 2 * np.pi * (2.0 ** -26 + 3 * 2.0 ** -53 * abs(float(turns))) + (4 + 16) * U
            off = max(abs(out[i, j] - np.cos(part)), abs(out[i, j + 6] - np.sin(part)))
            assert off <= bound, (p, f, off, bound)
