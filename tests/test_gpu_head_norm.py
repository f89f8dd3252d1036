"""GPU tests of the norm of heads with rotation, against the fp64 definition
(oracle/layer_oracle.py) within bounds derived in delta_testutil."""

import numpy as np
import pytest
import torch

import mamba_ssd_scan_fwd_amd as ssd
from delta_testutil import HALF, IO, U, within
from oracle import layer_oracle as ref
from ssd_testutil import note, np64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

CASES = [
    # leading, Hq, Hk, D, R, io, l2, pairs, weights, views
    ((1, 1), 1, 0, 1, 0, "fp32", False, False, False, False),
    ((3,), 2, 1, 2, 2, "fp32", True, True, True, False),
    ((5,), 3, 2, 7, 4, "bf16", False, False, True, True),
    ((2, 9), 4, 4, 16, 16, "bf16", False, False, True, True),
    ((2, 33), 16, 16, 128, 0, "bf16", True, False, False, True),
    ((1, 70), 32, 8, 128, 128, "bf16", False, False, True, True),
    ((1, 1), 32, 8, 128, 128, "bf16", False, True, True, False),
    ((3, 11), 24, 24, 80, 32, "fp32", False, True, True, True),
    ((3, 11), 5, 3, 96, 90, "bf16", True, False, True, True),
    ((7,), 3, 1, 129, 64, "fp32", False, False, True, True),
    ((7,), 3, 1, 130, 130, "bf16", False, True, False, True),
    ((4, 5), 2, 2, 256, 128, "fp32", False, False, True, False),
    ((4, 5), 2, 1, 511, 510, "bf16", True, True, True, False),
    ((6,), 2, 0, 512, 512, "fp32", False, False, True, True),
    ((5,), 1, 1, 300, 298, "fp32", False, True, True, True),
    ((2, 3000), 3, 2, 64, 64, "bf16", False, False, True, False),
]


def rows(shape, io, views, g):
    """[.., heads, D], cut from a wider buffer where views."""
    width = shape[-2] * shape[-1]
    if not views:
        return torch.randn(shape, generator=g).to(io)
    wide = torch.randn((*shape[:-2], width + 5), generator=g).to(io)
    return wide[..., 3:width + 3].unflatten(-1, shape[-2:])


def device(t):
    if t.is_contiguous():
        return t.to(DEV)
    base = t._base if t._base is not None else t
    return base.to(DEV).as_strided(t.shape, t.stride(), t.storage_offset())


def check(got, x, w, eps, l2, angle, pairs, what):
    want, mag = ref.head_norm(np64(x), eps, None if w is None else np64(w), l2, angle, pairs)
    within(got, want, (x.shape[-1] / 2 + 22) * U * mag + HALF[x.dtype] * np.abs(want), what)


@pytest.mark.parametrize("lead,Hq,Hk,D,R,io,l2,pairs,weights,views", CASES)
def test_head_norm_matches_the_definition(lead, Hq, Hk, D, R, io, l2, pairs, weights, views):
    g = torch.Generator().manual_seed(D + R)
    q = rows((*lead, Hq, D), IO[io], views, g)
    k = rows((*lead, Hk, D), IO[io], views, g) if Hk else None
    wq, wk = (1.0 + 0.3 * torch.randn((D,), generator=g) for _ in range(2)) if weights else (None, None)
    pos = freq = angle = None
    if R:
        pos = torch.randint(-5, 1 << 22, lead, generator=g, dtype=torch.int32)
        freq = torch.exp(-torch.arange(R // 2) * (9.0 / max(R // 2, 1)))
        angle = np64(pos)[..., None] * np64(freq)
    eps = 1e-5
    note(f"[gpu] head norm {lead} Hq={Hq} Hk={Hk} D={D} R={R} {io} l2={l2} pairs={pairs}")
    move = lambda t: None if t is None else device(t)  # noqa: E731
    out = ssd.head_norm(move(q), move(k), move(wq), move(wk) if Hk else None, positions=move(pos), inv_freq=move(freq),
                        eps=eps, l2=l2, pairs=pairs)
    out = out if Hk else (out,)
    check(out[0], q, wq, eps, l2, angle, pairs, "q")
    if Hk:
        check(out[1], k, wk, eps, l2, angle, pairs, "k")


@pytest.mark.parametrize("size", [1e-21, 1e-19, 1e18])
@pytest.mark.parametrize("l2", [False, True])
def test_heads_of_extreme_size_and_of_zeros(size, l2):
    g = torch.Generator().manual_seed(1)
    x = torch.randn((4, 3, 64), generator=g) * size
    x[1] = 0.0
    note(f"[gpu] head norm of size {size} l2={l2}")
    out = ssd.head_norm(x.to(DEV), eps=1e-30 if size < 1e-20 else 0.0 if size > 1 else 1e-38, l2=l2)
    keep = [0, 2, 3]
    eps = float(np.float32(1e-30 if size < 1e-20 else 0.0 if size > 1 else 1e-38))
    want, mag = ref.head_norm(np64(x[keep]), eps, l2=l2)
    # squares below 2^-149 are lost: 64 of them beside eps and the sum
    lost = 64 * 2.0 ** -149 / (eps + (np64(x[keep]) ** 2).mean(-1, keepdims=True))
    within(out[keep], want, (32 + 22) * U * mag + lost * mag, "out")
    if size < 1:
        assert (out[1] == 0).all()


def test_nan_and_infinity_stay_in_their_head():
    g = torch.Generator().manual_seed(2)
    q, k = torch.randn((9, 6, 128), generator=g).to(DEV), torch.randn((9, 2, 128), generator=g).to(DEV)
    pos, freq = torch.arange(9, dtype=torch.int32, device=DEV), torch.rand(32, generator=g).to(DEV)
    note("[gpu] head norm: NaN and infinities beside others")
    want = ssd.head_norm(q, k, positions=pos, inv_freq=freq)
    q[3, 2, 5], k[7, 1, 100] = float("nan"), float("inf")
    got = ssd.head_norm(q, k, positions=pos, inv_freq=freq)
    assert torch.isnan(got[0][3, 2]).all()
    assert torch.isnan(got[1][7, 1, 100]) and (got[1][7, 1, 64:100] == 0).all()
    got[0][3, 2], got[1][7, 1] = want[0][3, 2], want[1][7, 1]
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_positions_at_the_ends_of_their_type():
    x = torch.randn((4, 2, 8), generator=torch.Generator().manual_seed(3))
    pos = torch.tensor([0, -1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    # whole turns and halves of them: the angle's digits are all in the position
    freq = torch.tensor([1.0, 0.5, 2.0 ** -20, 0.1])
    note("[gpu] head norm: positions of 2^31")
    out = ssd.head_norm(x.to(DEV), positions=pos.to(DEV), inv_freq=freq.to(DEV))
    angle = np64(pos)[:, None] * np64(freq)
    want, mag = ref.head_norm(np64(x), float(np.float32(1e-5)), angle=angle)
    # 2^31 radians are 3.4e8 turns, of which a product and a constant in 64 bits lose 3 * 2^-53 each way
    lost = 2 * np.pi * 3.5e8 * 4 * 2.0 ** -53
    within(out, want, ((4 + 22) * U + lost) * mag + U * np.abs(want), "out")
