"""GPU tests of the layer operators around the scan, against the fp64
definitions (oracle/layer_oracle.py) within bounds derived in layer_testutil."""

import numpy as np
import pytest
import torch

import mamba_ssd_scan_fwd_amd as ssd
from layer_testutil import HALF, IO, Selective, U, conv_reference, norm_bound, within
from oracle import layer_oracle as ref
from ssd_testutil import note, np64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


# ---- selective scan, prompts ---------------------------------------------------

SCAN = [
    # b, L, E, N, G, io, dt, gate, skip, init, pre, views
    (1, 1, 1, 1, 1, "fp32", "fp32", False, False, False, False, False),
    (2, 3, 5, 16, 1, "fp32", "fp32", True, True, True, True, False),
    (1, 31, 64, 16, 1, "bf16", "bf16", True, True, False, True, False),
    (3, 32, 65, 16, 1, "bf16", "fp32", True, False, True, True, True),
    (2, 33, 130, 5, 2, "fp32", "fp32", False, True, True, True, True),
    (1, 64, 48, 17, 3, "bf16", "bf16", True, True, True, False, True),
    (1, 65, 64, 32, 1, "fp32", "fp32", True, True, True, True, False),
    (2, 130, 40, 33, 1, "bf16", "bf16", True, True, True, True, False),
    (1, 257, 128, 16, 1, "fp32", "fp32", True, True, True, True, True),
    (1, 300, 96, 64, 2, "bf16", "bf16", True, True, True, True, True),
    (1, 70, 20, 100, 1, "fp32", "fp32", True, True, True, True, False),
    (1, 67, 12, 256, 2, "bf16", "fp32", True, True, True, True, False),
    (2, 129, 7, 200, 1, "fp32", "fp32", True, True, False, True, True),
    (1, 100, 203, 16, 1, "bf16", "bf16", True, True, True, True, True),
    (1, 70, 198, 14, 2, "bf16", "fp32", True, True, True, True, True),
    (1, 45, 131, 52, 1, "fp32", "fp32", True, True, True, True, True),
]


@pytest.mark.parametrize("b,L,E,N,G,io,dt,gate,skip,init,pre,views", SCAN)
def test_selective_scan_matches_the_recurrence(b, L, E, N, G, io, dt, gate, skip, init, pre, views):
    s = Selective(b, L, E, N, G, io, dt, gate, skip, init, pre, views, seed=L + E)
    kw, h0, _ = s.to(DEV)
    note(f"[gpu] selective scan b={b} L={L} E={E} N={N} G={G} {io}/{dt}")
    y, hT = ssd.selective_scan(init_state=h0, **kw)
    yr, yb, hr, hb = s.reference()
    within(y, yr, yb, "y")
    within(hT, hr, hb, "final_state")


@pytest.mark.parametrize("io,N,init", [("fp32", 16, True), ("bf16", 16, False), ("bf16", 24, True), ("fp32", 128, True)])
def test_selective_scan_packed(io, N, init):
    lens = [5, 0, 1, 64, 33, 0, 0, 150, 2, 1, 1, 31, 0]
    s = Selective(1, sum(lens), 70, N, 1, io, io, True, True, init, True, True, lens=lens, seed=N)
    kw, h0, cu = s.to(DEV)
    note(f"[gpu] selective scan packed {io} N={N} init={init}")
    y, hT = ssd.selective_scan_varlen(cu_seqlens=cu, init_states=h0, **kw)
    yr, yb, hr, hb = s.reference()
    within(y, yr, yb, "y")
    within(hT, hr, hb, "final_states")


def test_selective_scan_packed_leaves_what_lies_behind():
    lens = [40, 60]
    s = Selective(1, 130, 33, 16, lens=lens, seed=3)
    kw, h0, cu = s.to(DEV)
    y = torch.full((1, 130, 33), 7.0, device=DEV)
    note("[gpu] selective scan: tokens behind the last sequence")
    # what lies behind is not read either
    for k in ("x", "dt", "z", "B", "C"):
        kw[k][:, 100:] = float("nan")
    _, hT = ssd.selective_scan_varlen(cu_seqlens=cu, init_states=h0, y=y, **kw)
    yr, yb, hr, hb = s.reference()
    within(y[:, :100], yr[:, :100], yb[:, :100], "y")
    assert torch.equal(y[:, 100:], torch.full_like(y[:, 100:], 7.0))
    within(hT, hr, hb, "final_states")


def test_selective_scan_sequences_do_not_meet():
    lens = [50, 0, 70, 1, 80]
    s = Selective(1, sum(lens), 64, 16, lens=lens, seed=4)
    kw, h0, cu = s.to(DEV)
    note("[gpu] selective scan: a sequence of NaN and infinities beside others")
    want, hw = ssd.selective_scan_varlen(cu_seqlens=cu, init_states=h0, **kw)
    kw["x"][:, 50:120] = float("nan")
    kw["B"][:, 50:120] = float("inf")
    h0[2] = float("inf")
    got, hg = ssd.selective_scan_varlen(cu_seqlens=cu, init_states=h0, **kw)
    others = torch.tensor([t for t in range(sum(lens)) if not 50 <= t < 120], device=DEV)
    assert torch.equal(got[:, others], want[:, others])
    assert torch.equal(hg[[0, 1, 3, 4]], hw[[0, 1, 3, 4]])
    assert torch.isnan(got[:, 50:120]).all()


@pytest.mark.parametrize("lens", [None, [90, 0, 140, 30]])
def test_selective_scan_state_in_place_and_same_bits(lens):
    L = 260
    s = Selective(1, L, 64, 16, lens=lens, seed=5)
    kw, h0, cu = s.to(DEV)
    note("[gpu] selective scan: final state over the initial state")

    def run(init, final):
        if lens is None:
            return ssd.selective_scan(init_state=init, final_state=final, **kw)
        return ssd.selective_scan_varlen(cu_seqlens=cu, init_states=init, final_states=final, **kw)

    y, hT = run(h0, None)
    again = run(h0, None)
    assert torch.equal(y, again[0]) and torch.equal(hT, again[1])
    state = h0.clone()
    yi, hi = run(state, state)
    assert hi.data_ptr() == state.data_ptr()
    assert torch.equal(y, yi) and torch.equal(hT, hi)


@pytest.mark.parametrize("E,N,G,io,lens", [
    (99, 16, 1, "bf16", None), (130, 13, 2, "fp32", None), (127, 30, 1, "bf16", [200, 0, 3, 157]), (81, 70, 1, "fp32", None),
    (300, 1, 3, "bf16", [1, 1, 358]), (97, 129, 1, "bf16", None)])
def test_selective_scan_state_in_place_at_odd_channels(E, N, G, io, lens):
    # the channels behind the last whole 64 share a workgroup with some before
    # them, which must be written once, from the state as it was
    s = Selective(1 if lens else 3, 360, E, N, G, io, io, True, True, True, True, True, lens=lens, seed=E)
    kw, h0, cu = s.to(DEV)
    note(f"[gpu] selective scan in place E={E} N={N} G={G} {io} lens={lens}")
    if lens is None:
        y, hT = ssd.selective_scan(init_state=h0, final_state=h0, **kw)
    else:
        y, hT = ssd.selective_scan_varlen(cu_seqlens=cu, init_states=h0, final_states=h0, **kw)
    yr, yb, hr, hb = s.reference()
    within(y, yr, yb, "y")
    within(hT, hr, hb, "final_state")


def test_selective_scan_time_major_and_own_workspace():
    s = Selective(3, 100, 64, 16, seed=6)
    kw, h0, _ = s.to(DEV)
    y, hT = ssd.selective_scan(init_state=h0, **kw)
    note("[gpu] selective scan: time-major inputs")
    tm = {k: kw[k].transpose(0, 1).contiguous().transpose(0, 1) for k in ("x", "dt", "z", "B", "C")}
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV)
    y2, h2 = ssd.selective_scan(init_state=h0, workspace=ws, **dict(kw, **tm))
    assert torch.equal(y, y2) and torch.equal(hT, h2)


def test_selective_scan_carries_over_calls():
    s = Selective(2, 150, 64, 16, seed=7)
    kw, h0, _ = s.to(DEV)
    note("[gpu] selective scan: two calls in turn")
    cut = 71
    part = lambda a, b: {k: (v[:, a:b] if k in ("x", "dt", "z", "B", "C") else v) for k, v in kw.items()}  # noqa: E731
    y1, h = ssd.selective_scan(init_state=h0, **part(0, cut))
    y2, h = ssd.selective_scan(init_state=h, **part(cut, 150))
    yr, yb, hr, hb = s.reference()
    within(torch.cat([y1, y2], 1), yr, yb, "y")
    within(h, hr, hb, "final_state")


# ---- selective scan, single tokens ----------------------------------------------

STEP = [(1, 1, 1, 1, "fp32", "fp32"), (3, 70, 16, 1, "bf16", "bf16"), (5, 64, 5, 2, "fp32", "fp32"),
        (2, 130, 24, 1, "bf16", "fp32"), (4, 33, 64, 3, "fp32", "fp32"), (2, 12, 256, 1, "bf16", "bf16"),
        (67, 2048, 16, 1, "bf16", "bf16")]


@pytest.mark.parametrize("b,E,N,G,io,dt", STEP)
def test_selective_step_matches_the_recurrence(b, E, N, G, io, dt):
    s = Selective(b, 1, E, N, G, io, dt, views=True, seed=b + E)
    kw, h0, _ = s.to(DEV)
    note(f"[gpu] selective step b={b} E={E} N={N} G={G} {io}/{dt}")
    one = {k: (v[:, 0] if k in ("x", "dt", "z", "B", "C") else v) for k, v in kw.items()}
    state = h0.clone()
    y = ssd.selective_step(state=state, **one)
    yr, yb, hr, hb = s.reference()
    within(y, yr[:, 0], yb[:, 0], "y")
    within(state, hr, hb, "state")


@pytest.mark.parametrize("b,slots", [(9, [3, -1, 11, 3, 0, 12, 3, 99, 5]), (300, None)])
def test_selective_step_slots(b, slots):
    E, N, pool = 96, 16, 12 if slots else 400
    if slots is None:
        g = torch.Generator().manual_seed(1)
        slots = torch.randperm(pool, generator=g)[:b].tolist()
        slots[7], slots[290], slots[299], slots[150] = slots[6], slots[3], slots[290], -5
    s = Selective(b, 1, E, N, io="bf16", dt="bf16", init=False, seed=8)
    kw, _, _ = s.to(DEV)
    one = {k: (v[:, 0].contiguous() if k in ("x", "dt", "z", "B", "C") else v) for k, v in kw.items()}
    before = torch.randn((pool, E, N), generator=torch.Generator().manual_seed(2))
    state, y = before.to(DEV), torch.full((b, E), 3.0, dtype=torch.bfloat16, device=DEV)
    note(f"[gpu] selective step: slots of {b} rows, some padding, some repeated")
    ssd.selective_step(state=state, y=y, state_slots=torch.tensor(slots, dtype=torch.int32, device=DEV), **one)
    first = {}
    for r, k in enumerate(slots):
        if 0 <= k < pool:
            first.setdefault(k, r)
    rows = sorted(first.values())
    dead = [r for r in range(b) if r not in set(rows)]
    s.init = torch.zeros((b, E, N))
    for k, r in first.items():
        s.init[r] = before[k]
    yr, yb, hr, hb = s.reference()
    within(y[rows], yr[rows, 0], yb[rows, 0], "y")
    assert torch.equal(y[dead], torch.full_like(y[dead], 3.0))
    within(state[[slots[r] for r in rows]], hr[rows], hb[rows], "state")
    rest = [k for k in range(pool) if k not in first]
    assert torch.equal(state[rest].cpu(), before[rest])


def test_selective_steps_continue_a_prompt():
    s = Selective(2, 40, 64, 16, io="bf16", dt="bf16", seed=9)
    kw, h0, _ = s.to(DEV)
    note("[gpu] selective scan then steps")
    part = {k: (v[:, :30] if k in ("x", "dt", "z", "B", "C") else v) for k, v in kw.items()}
    y0, state = ssd.selective_scan(init_state=h0, **part)
    ys = [y0]
    for t in range(30, 40):
        one = {k: (v[:, t] if k in ("x", "dt", "z", "B", "C") else v) for k, v in kw.items()}
        ys.append(ssd.selective_step(state=state, **one)[:, None])
    yr, yb, hr, hb = s.reference()
    within(torch.cat(ys, 1), yr, yb, "y")
    within(state, hr, hb, "state")


# ---- short convolution -------------------------------------------------------------

def conv_inputs(b, L, CH, K, io, seed, views):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((b + 1, L + 2, CH + 5), generator=g).to(IO[io])
    x = x[:b, 1:L + 1, 3:CH + 3] if views else x[:b, :L, :CH].contiguous()
    w, bias = torch.randn((CH, K), generator=g) * K ** -0.5, torch.randn(CH, generator=g) * 0.3
    return x, w, bias, g


def on_device(t):
    base = t._base if t._base is not None else t
    return base.to(DEV).as_strided(t.shape, t.stride(), t.storage_offset())


@pytest.mark.parametrize("b,L,CH,K,io,act,bias,state,views", [
    (1, 1, 1, 4, "fp32", True, True, True, False),
    (2, 2, 64, 4, "bf16", True, True, True, False),
    (1, 9, 520, 3, "bf16", True, False, False, False),
    (3, 65, 37, 4, "fp32", False, True, True, True),
    (2, 130, 640, 2, "bf16", True, True, True, True),
    (1, 300, 24, 1, "fp32", True, True, False, False),
    (2, 77, 516, 4, "fp32", True, True, True, False),
    (1, 1000, 2048, 4, "bf16", True, True, True, False),
    (2, 40, 1001, 4, "bf16", True, True, True, True),
    (1, 90, 11, 3, "bf16", True, True, True, False),
    (1, 33, 517, 2, "fp32", True, True, True, True),
    (2, 21, 7, 4, "bf16", True, True, True, True),
])
def test_conv1d_matches_the_definition(b, L, CH, K, io, act, bias, state, views):
    x, w, bv, g = conv_inputs(b, L, CH, K, io, L + CH, views)
    s0 = torch.randn((b, CH, K - 1), generator=g) if state else None
    out = torch.empty((b, CH, K - 1), device=DEV)
    note(f"[gpu] conv1d b={b} L={L} CH={CH} K={K} {io}")
    y = ssd.conv1d(on_device(x), w.to(DEV), bv.to(DEV) if bias else None, silu=act,
                   conv_state_in=None if s0 is None else s0.to(DEV), conv_state_out=out)
    want, bound, last = conv_reference(np64(x), np64(w), np64(bv) if bias else None, act,
                                       None if s0 is None else np64(s0), [(i, 0, L) for i in range(b)], IO[io])
    within(y, want, bound, "y")
    assert np.array_equal(np64(out), last)


@pytest.mark.parametrize("io,K,split,state", [("bf16", 4, True, True), ("fp32", 4, False, True), ("bf16", 3, False, False),
                                              ("fp32", 2, True, True)])
def test_conv1d_packed(io, K, split, state):
    lens = [3, 0, 1, 64, 2, 0, 0, 200, 1, 1, 9, 0]
    T, tail = sum(lens), 7
    H, P, G, N = 3, 16, 2, 16
    CH = H * P + 2 * G * N
    x, w, bv, g = conv_inputs(1, T + tail, CH, K, io, K, not split)
    s0 = torch.randn((len(lens), CH, K - 1), generator=g) if state else None
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
    out = torch.empty((len(lens), CH, K - 1), device=DEV)
    note(f"[gpu] conv1d packed {io} K={K} split={split}")
    kw = dict(cu_seqlens=cu, conv_states_in=None if s0 is None else s0.to(DEV), conv_states_out=out)
    if split:
        xs = ssd.conv1d_split_varlen(on_device(x), w.to(DEV), bv.to(DEV), nheads=H, headdim=P, ngroups=G, dstate=N, **kw)
        assert [tuple(o.shape) for o in xs] == [(1, T + tail, H, P), (1, T + tail, G, N), (1, T + tail, G, N)]
        y = torch.cat([o.flatten(2) for o in xs], 2)
    else:
        y = torch.full((1, T + tail, CH), 5.0, dtype=IO[io], device=DEV)
        ssd.conv1d_varlen(on_device(x), w.to(DEV), bv.to(DEV), y=y, **kw)
        assert torch.equal(y[:, T:], torch.full_like(y[:, T:], 5.0))
    ends = np.cumsum(lens)
    spans = [(0, int(e) - n, int(e)) for n, e in zip(lens, ends)]
    want, bound, last = conv_reference(np64(x), np64(w), np64(bv), True, None if s0 is None else np64(s0), spans, IO[io])
    within(y[:, :T], want[:, :T], bound[:, :T], "y")
    assert np.array_equal(np64(out), last)


def test_conv1d_gives_what_conv1d_split_gives():
    H, P, G, N, L = 4, 32, 1, 64, 100
    x, w, bv, _ = conv_inputs(2, L, H * P + 2 * G * N, 4, "bf16", 1, False)
    a = (x.to(DEV), w.to(DEV), bv.to(DEV))
    kw = dict(nheads=H, headdim=P, ngroups=G, dstate=N)
    note("[gpu] conv1d beside conv1d_split")
    want = torch.cat([o.flatten(2) for o in ssd.conv1d_split(*a, **kw)], 2)
    y = ssd.conv1d(*a)
    # two evaluations of the same sums and SiLU in fp32, each stored in bf16
    z, za, _ = ref.conv1d(np64(x[0]), np64(w), np64(bv), True)
    within(y[:1], np64(want[:1]), 2 * (1.1 * 5 * U * za + (26 * U + 2.0 ** -8) * np.abs(z))[None], "y")


@pytest.mark.parametrize("b,CH,K,io,act,views", [(1, 1, 4, "fp32", True, False), (3, 64, 4, "bf16", True, False),
                                                 (5, 37, 3, "fp32", False, True), (300, 1028, 4, "bf16", True, False),
                                                 (2, 516, 2, "fp32", True, False), (4, 40, 1, "bf16", True, True),
                                                 (70, 1027, 4, "bf16", True, True), (3, 6, 3, "fp32", True, True)])
def test_conv1d_step_matches_the_definition(b, CH, K, io, act, views):
    x, w, bv, g = conv_inputs(b, 1, CH, K, io, b + CH, views)
    pool = b + 3
    before = torch.randn((pool, CH, K - 1), generator=g)
    slots = torch.randperm(pool, generator=g)[:b]
    state = before.to(DEV)
    note(f"[gpu] conv1d step b={b} CH={CH} K={K} {io}")
    y = ssd.conv1d_step(on_device(x)[:, 0], w.to(DEV), bv.to(DEV), state, silu=act, state_slots=slots.int().to(DEV))
    want, bound, last = conv_reference(np64(x), np64(w), np64(bv), act, np64(before[slots]),
                                       [(i, 0, 1) for i in range(b)], IO[io])
    within(y, want[:, 0], bound[:, 0], "y")
    expect = np64(before)
    expect[slots.numpy()] = last
    assert np.array_equal(np64(state), expect)


def test_conv1d_step_padding_and_repeated_slots():
    b, CH, K, pool = 7, 64, 4, 5
    slots = [2, -1, 2, 5, 0, 0, 4]
    x, w, bv, g = conv_inputs(b, 1, CH, K, "fp32", 11, False)
    before = torch.randn((pool, CH, K - 1), generator=g)
    state, y = before.to(DEV), torch.full((b, CH), 3.0, device=DEV)
    note("[gpu] conv1d step: padding and repeated slots")
    ssd.conv1d_step(x[:, 0].to(DEV), w.to(DEV), bv.to(DEV), state, y=y,
                    state_slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
    rows = [0, 4, 6]
    want, bound, last = conv_reference(np64(x[rows]), np64(w), np64(bv), True, np64(before[[2, 0, 4]]),
                                       [(i, 0, 1) for i in range(3)], torch.float32)
    within(y[rows], want[:, 0], bound[:, 0], "y")
    assert torch.equal(y[[1, 2, 3, 5]], torch.full((4, CH), 3.0, device=DEV))
    expect = np64(before)
    expect[[2, 0, 4]] = last
    assert np.array_equal(np64(state), expect)


# ---- group norm --------------------------------------------------------------------

@pytest.mark.parametrize("shape,G,io,center,gate,first,act,weights,views", [
    ((1, 1), 1, "fp32", False, False, False, False, True, False),
    ((3, 8), 1, "fp32", True, True, True, False, True, False),
    ((2, 5, 130), 2, "bf16", True, True, False, False, True, True),
    ((7, 512), 8, "bf16", False, True, True, False, True, False),
    ((4, 3, 640), 5, "fp32", True, False, False, True, True, False),
    ((300, 2048), 1, "bf16", False, True, True, False, True, False),
    ((2, 9, 4096), 1, "bf16", True, True, False, False, True, True),
    ((5, 4104), 1, "fp32", True, True, True, False, False, False),
    ((3, 8200), 1, "bf16", False, True, False, False, True, False),
    ((2, 16384), 1, "fp32", True, True, True, False, True, False),
    ((2, 16383), 1, "bf16", True, False, False, False, True, False),
    ((70, 24), 3, "bf16", True, False, False, True, False, False),
    ((1001, 8192), 128, "fp32", True, True, False, False, True, False),
    ((64, 96), 96, "fp32", False, True, True, False, True, False),
    ((9, 3009), 3, "bf16", True, True, True, False, True, True),
    ((5, 2, 1001), 1, "fp32", True, True, False, False, True, True),
    ((6, 4999), 1, "bf16", False, True, True, False, True, True),
    ((40, 9 * 11), 9, "bf16", True, True, False, False, True, True),
    ((40, 12 * 3), 12, "fp32", True, False, False, True, True, True),
    ((2, 12345), 1, "bf16", True, True, False, False, True, False),
])
def test_group_norm_matches_the_definition(shape, G, io, center, gate, first, act, weights, views):
    g = torch.Generator().manual_seed(sum(shape))
    C = shape[-1]

    def draw(shift):
        if not views:
            return (torch.randn(shape, generator=g) + shift).to(IO[io])
        wide = (torch.randn((*shape[:-1], 2 * C + 16), generator=g) + shift).to(IO[io])
        return wide[..., 8:C + 8]

    x, z = draw(0.5), draw(0.0) if gate else None
    w, bias = (1 + 0.3 * torch.randn(C, generator=g), 0.3 * torch.randn(C, generator=g)) if weights else (None, None)
    note(f"[gpu] group norm {shape} G={G} {io} center={center} gate={gate}/{first}")
    dev = lambda t: None if t is None else on_device(t)  # noqa: E731
    o = ssd.group_norm(dev(x), dev(w), dev(bias), dev(z), ngroups=G, center=center, gate_first=first, silu=act)
    assert o.shape == x.shape and o.dtype == x.dtype
    flat = lambda t: None if t is None else np64(t).reshape(-1, C)  # noqa: E731
    vec = lambda t: None if t is None else np64(t)  # noqa: E731
    want = ref.group_norm(flat(x), G, 1e-5, vec(w), vec(bias), flat(z), center, first, act)
    bound = norm_bound(flat(x), G, 1e-5, vec(w), vec(bias), flat(z), center, first, act, IO[io], want)
    within(o.reshape(-1, C), want, bound, "out")


# ---- the operators together ---------------------------------------------------------

def test_selective_layer_prompt_then_tokens():
    """conv1d -> selective_scan -> group_norm on a projection's views, then
    token by token from slots; the same tokens in one go as the reference."""
    b, L, new, E, N, K = 2, 50, 6, 128, 16, 4
    g = torch.Generator().manual_seed(21)
    T = L + new
    xz = (torch.randn((b, T, 2 * E), generator=g)).to(torch.bfloat16).to(DEV)
    bc = (torch.randn((b, T, 2 * N), generator=g) * N ** -0.5).to(torch.bfloat16).to(DEV)
    dt = (torch.randn((b, T, E), generator=g) * 0.5).to(torch.bfloat16).to(DEV)
    w, bias = torch.randn((E, K), generator=g).to(DEV) * 0.5, torch.randn(E, generator=g).to(DEV) * 0.1
    A, D = -torch.exp(torch.rand((E, N), generator=g) * 2.8).to(DEV), torch.randn(E, generator=g).to(DEV)
    nw = (1 + 0.2 * torch.randn(E, generator=g)).to(DEV)
    pre = dict(bias=torch.full((E,), -2.0, device=DEV), softplus=True)
    note("[gpu] selective layer: prompt, then tokens")

    def prompt(n):
        x, z = xz[:, :n, :E], xz[:, :n, E:]
        B, C = bc[:, :n, :N].unsqueeze(2), bc[:, :n, N:].unsqueeze(2)
        conv = torch.empty((b, E, K - 1), device=DEV)
        u = ssd.conv1d(x, w, bias, conv_state_out=conv)
        y, h = ssd.selective_scan(u, dt[:, :n], A, B, C, D, z, dt_pre=pre)
        return ssd.group_norm(y, nw, ngroups=4, center=False), conv, h

    whole, conv_end, h_end = prompt(T)
    out, conv, h = prompt(L)
    pool_c, pool_h = torch.zeros((5, E, K - 1), device=DEV), torch.zeros((5, E, N), device=DEV)
    slots = torch.tensor([4, 1], dtype=torch.int32, device=DEV)
    pool_c[slots.long()], pool_h[slots.long()] = conv, h
    outs = [out]
    for t in range(L, T):
        u = ssd.conv1d_step(xz[:, t, :E], w, bias, pool_c, state_slots=slots)
        y = ssd.selective_step(u, dt[:, t], A, bc[:, t, :N].unsqueeze(1), bc[:, t, N:].unsqueeze(1), D, xz[:, t, E:],
                               pool_h, state_slots=slots, dt_pre=pre)
        outs.append(ssd.group_norm(y, nw, ngroups=4, center=False)[:, None])
    got = torch.cat(outs, 1)
    assert torch.equal(pool_c[slots.long()], conv_end)
    # both sides store u, y and the norm in bf16 from fp32 values that differ
    # in their last bits: a step of bf16 in u (2^-7 of it) and in y may differ
    # here and there; the norm leaves them relative to the group's size
    diff = (got.double() - whole.double()).norm() / whole.double().norm()
    assert diff < 2.0 ** -7, diff
    assert (pool_h[slots.long()] - h_end).norm() / h_end.norm() < 2.0 ** -7


def test_ssd_layer_prompt_then_tokens():
    """conv1d_split_varlen -> forward_varlen -> group_norm over packed
    requests, then conv1d_split_step -> decode_step -> group_norm."""
    H, P, G, N, K = 8, 32, 1, 64, 4
    CH, E = H * P + 2 * G * N, H * P
    lens, new = [20, 33, 7], 4
    S = len(lens)
    g = torch.Generator().manual_seed(22)
    rows = [torch.randn((n + new, CH), generator=g).to(torch.bfloat16).to(DEV) for n in lens]
    zs = [torch.randn((n + new, E), generator=g).to(torch.bfloat16).to(DEV) for n in lens]
    dts = [torch.rand((n + new, H), generator=g).to(DEV) * 0.1 for n in lens]
    w, bias = torch.randn((CH, K), generator=g).to(DEV) * 0.5, torch.randn(CH, generator=g).to(DEV) * 0.1
    A, D, nw = -torch.rand(H, generator=g).to(DEV) * 4, torch.randn(H, generator=g).to(DEV), torch.ones(E, device=DEV)
    heads = dict(nheads=H, headdim=P, ngroups=G, dstate=N)
    note("[gpu] SSD layer: packed prompts, then tokens")

    def prompt(extra):
        ln = [n + extra for n in lens]
        cu = torch.tensor([0] + list(np.cumsum(ln)), dtype=torch.int32, device=DEV)
        cat = lambda parts: torch.cat([p[:n] for p, n in zip(parts, ln)])[None]  # noqa: E731
        conv = torch.empty((S, CH, K - 1), device=DEV)
        x, B, C = ssd.conv1d_split_varlen(cat(rows), w, bias, cu_seqlens=cu, conv_states_out=conv, **heads)
        y, h = ssd.forward_varlen(x, cat(dts), A, B, C, D, cu_seqlens=cu)
        o = ssd.group_norm(y.flatten(2), nw, None, cat(zs), ngroups=2, center=False, gate_first=True)
        return o[0].split(ln), conv, h

    whole, conv_end, h_end = prompt(new)
    part, conv, h = prompt(0)
    got = [[p] for p in part]
    for t in range(new):
        at = [n + t for n in lens]
        pick = lambda parts: torch.stack([p[i] for p, i in zip(parts, at)])  # noqa: E731
        x, B, C = ssd.conv1d_split_step(pick(rows), w, bias, conv, **heads)
        y = ssd.decode_step(x, pick(dts), A, B, C, D, h)
        o = ssd.group_norm(y.flatten(1), nw, None, pick(zs), ngroups=2, center=False, gate_first=True)
        for s in range(S):
            got[s].append(o[s:s + 1])
    assert torch.equal(conv, conv_end)
    for s in range(S):
        a, b = torch.cat(got[s]).double(), whole[s].double()
        # the prompt path rounds its products' operands and chunk states to
        # bf16 (2^-8 each, several of them), the token path only its outputs
        assert (a - b).norm() / b.norm() < 2e-2
    assert (h - h_end).norm() / h_end.norm() < 2e-2


# ---- streams and graphs --------------------------------------------------------------

def _layer_calls(seed):
    """One call of every operator on fixed buffers; returns (run, outputs)."""
    E, N, K, lens = 64, 16, 4, [70, 0, 90, 1]
    s = Selective(1, sum(lens), E, N, io="bf16", dt="bf16", lens=lens, seed=seed)
    kw, h0, cu = s.to(DEV)
    one = {k: (v[:, 0] if k in ("x", "dt", "z", "B", "C") else v) for k, v in kw.items()}
    g = torch.Generator().manual_seed(seed)
    w, bias = torch.randn((E, K), generator=g).to(DEV), torch.randn(E, generator=g).to(DEV)
    state, conv = torch.randn((3, E, N), generator=g).to(DEV), torch.randn((3, E, K - 1), generator=g).to(DEV)
    slot = torch.tensor([2], dtype=torch.int32, device=DEV)

    def run():
        last = torch.empty((len(lens), E, K - 1), device=DEV)
        u = ssd.conv1d_varlen(kw["x"], w, bias, cu_seqlens=cu, conv_states_out=last)
        y, h = ssd.selective_scan_varlen(cu_seqlens=cu, init_states=h0, **dict(kw, x=u))
        o = ssd.group_norm(y, ngroups=4)
        st, cs = state.clone(), conv.clone()
        t = ssd.conv1d_step(one["x"], w, bias, cs, state_slots=slot)
        yt = ssd.selective_step(state=st, state_slots=slot, **dict(one, x=t))
        return [u, last, y, h, o, t, cs, yt, st]

    return run


def test_layer_operators_on_another_stream():
    run = _layer_calls(31)
    want = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    note("[gpu] layer operators on a side stream")
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_stream_argument_orders_workspace_and_outputs():
    s = Selective(1, 400, 64, 16, seed=33)
    kw, h0, _ = s.to(DEV)
    want = ssd.selective_scan(init_state=h0, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    note("[gpu] selective scan: stream argument")
    got = ssd.selective_scan(init_state=h0, stream=side, **kw)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_layer_operators_replay_from_a_captured_graph():
    run = _layer_calls(32)
    want = run()
    torch.cuda.synchronize()
    note("[gpu] layer operators captured and replayed")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(4):
        for o in out:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out))
        eager = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, eager))


def test_every_operator_takes_a_stream():
    s = Selective(1, 40, 64, 16, io="bf16", dt="bf16", seed=34)
    kw, h0, _ = s.to(DEV)
    one = {k: (v[:, 0] if k in ("x", "dt", "z", "B", "C") else v) for k, v in kw.items()}
    g = torch.Generator().manual_seed(35)
    w, conv = torch.randn((64, 4), generator=g).to(DEV), torch.randn((1, 64, 3), generator=g).to(DEV)
    cu = torch.tensor([0, 7, 40], dtype=torch.int32, device=DEV)

    def run(**on):
        st, cs = h0.clone(), conv.clone()
        torch.cuda.synchronize()
        out = [ssd.selective_scan_varlen(cu_seqlens=cu, **kw, **on)[0], ssd.selective_step(state=st, **one, **on),
               ssd.conv1d(kw["x"], w, **on), ssd.conv1d_varlen(kw["x"], w, cu_seqlens=cu, **on),
               ssd.conv1d_step(one["x"], w, None, cs, **on), ssd.group_norm(kw["x"], **on)]
        torch.cuda.synchronize()
        return [*out, st, cs]

    note("[gpu] every layer operator with a stream argument")
    side = torch.cuda.Stream()
    for a, b in zip(run(), run(stream=side)):
        assert torch.equal(a, b)


# ---- far offsets, alignment, odd shapes --------------------------------------------------


def test_rows_far_apart():
    """Token strides that take the last rows past 2^32 bytes and 2^31 elements."""
    L, E, N, far = 1100, 64, 16, (1 << 21) + 24
    s = Selective(1, L, E, N, io="bf16", dt="bf16", seed=41)
    kw, h0, _ = s.to(DEV)
    note("[gpu] rows more than 2^32 bytes apart")
    base = torch.empty(L * far, dtype=torch.bfloat16, device=DEV)
    wide = base.view(1, L, far)
    moved = dict(kw)
    at = 0
    for k in ("x", "dt", "z"):
        wide[:, :, at:at + E] = kw[k]
        moved[k] = wide[:, :, at:at + E]
        at += E + 8
    for k in ("B", "C"):
        wide[:, :, at:at + N] = kw[k][:, :, 0]
        moved[k] = wide[:, :, at:at + N].unsqueeze(2)
        at += N + 8
    want = ssd.selective_scan(init_state=h0, **kw)
    got = ssd.selective_scan(init_state=h0, **moved)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    w = torch.randn((E, 4), generator=torch.Generator().manual_seed(1)).to(DEV)
    assert torch.equal(ssd.conv1d(kw["x"], w), ssd.conv1d(moved["x"], w))
    assert torch.equal(ssd.group_norm(kw["x"], None, None, kw["z"], ngroups=2),
                       ssd.group_norm(moved["x"], None, None, moved["z"], ngroups=2))


def test_slots_behind_two_to_the_31_elements():
    E, N, K = 8192, 16, 4
    pool = (1 << 31) // (E * N) + 3
    s = Selective(2, 1, E, N, io="bf16", dt="bf16", seed=42)
    kw, h0, _ = s.to(DEV)
    one = {k: (v[:, 0] if k in ("x", "dt", "z", "B", "C") else v) for k, v in kw.items()}
    note("[gpu] state pool of more than 2^31 elements")
    state = torch.zeros((pool, E, N), device=DEV)
    slots = torch.tensor([pool - 1, 1], dtype=torch.int32, device=DEV)
    state[slots.long()] = h0
    y = ssd.selective_step(state=state, state_slots=slots, **one)
    yr, yb, hr, hb = s.reference()
    within(y, yr[:, 0], yb[:, 0], "y")
    within(state[slots.long()], hr, hb, "state")
    assert not state[pool - 2].any() and not state[0].any()
    del state
    pool = (1 << 31) // (E * (K - 1)) + 3
    conv = torch.zeros((pool, E, K - 1), device=DEV)
    slots = torch.tensor([1, pool - 1], dtype=torch.int32, device=DEV)
    x, w, bv, g = conv_inputs(2, 1, E, K, "bf16", 43, False)
    before = torch.randn((2, E, K - 1), generator=g)
    conv[slots.long()] = before.to(DEV)
    y = ssd.conv1d_step(x[:, 0].to(DEV), w.to(DEV), bv.to(DEV), conv, state_slots=slots)
    want, bound, last = conv_reference(np64(x), np64(w), np64(bv), True, np64(before), [(i, 0, 1) for i in range(2)],
                                       torch.bfloat16)
    within(y, want[:, 0], bound[:, 0], "y")
    assert np.array_equal(np64(conv[slots.long()]), last)
    assert not conv[pool - 2].any()


@pytest.mark.parametrize("io", ["fp32", "bf16"])
def test_unaligned_views_give_the_same_bits(io):
    """The element-wise accesses compute what the wide ones do."""
    b, L, E, N = 2, 70, 128, 16
    s = Selective(b, L, E, N, io=io, dt=io, seed=44)
    kw, h0, _ = s.to(DEV)
    note(f"[gpu] unaligned views {io}")

    def shifted(t, by):
        wide = torch.zeros((*t.shape[:2], t[0, 0].numel() + 9), dtype=t.dtype, device=DEV)
        flat = t.flatten(2)
        wide[..., by:by + flat.shape[2]] = flat
        return wide[..., by:by + flat.shape[2]].view(t.shape) if t.dim() == 3 else \
            wide[..., by:by + flat.shape[2]].unflatten(2, t.shape[2:])

    off = {k: (shifted(v, 3) if k in ("x", "dt", "z", "B", "C") else v) for k, v in kw.items()}
    want, got = ssd.selective_scan(init_state=h0, **kw), ssd.selective_scan(init_state=h0, **off)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    first = lambda d: {k: (v[:, 0] if k in ("x", "dt", "z", "B", "C") else v) for k, v in d.items()}  # noqa: E731
    s1, s2 = h0.clone(), h0.clone()
    assert torch.equal(ssd.selective_step(state=s1, **first(kw)), ssd.selective_step(state=s2, **first(off)))
    assert torch.equal(s1, s2)
    w = torch.randn((E, 4), generator=torch.Generator().manual_seed(2)).to(DEV)
    c1, c2 = (torch.zeros((b, E, 3), device=DEV) for _ in range(2))
    assert torch.equal(ssd.conv1d(kw["x"], w, conv_state_out=c1), ssd.conv1d(off["x"], w, conv_state_out=c2))
    assert torch.equal(c1, c2)
    assert torch.equal(ssd.conv1d_step(kw["x"][:, 1], w, None, c1), ssd.conv1d_step(off["x"][:, 1], w, None, c2))
    assert torch.equal(c1, c2)
    assert torch.equal(ssd.group_norm(kw["x"], None, None, kw["z"]), ssd.group_norm(off["x"], None, None, off["z"]))


@pytest.mark.parametrize("lens", [[1] * 200, [1, 2, 3, 0] * 40, [0, 0, 777, 0], [300, 1, 1, 1, 300], [2] * 64 + [500]])
def test_many_short_and_a_few_long_sequences(lens):
    T = sum(lens)
    s = Selective(1, T, 66, 16, lens=lens, io="bf16", dt="bf16", seed=T)
    kw, h0, cu = s.to(DEV)
    note(f"[gpu] packed: {len(lens)} sequences, {T} tokens")
    state = h0.clone()
    y, _ = ssd.selective_scan_varlen(cu_seqlens=cu, init_states=state, final_states=state, **kw)
    yr, yb, hr, hb = s.reference()
    within(y, yr, yb, "y")
    within(state, hr, hb, "final_states")
    w = torch.randn((66, 4), generator=torch.Generator().manual_seed(3))
    c0 = torch.randn((len(lens), 66, 3), generator=torch.Generator().manual_seed(4))
    out = torch.empty((len(lens), 66, 3), device=DEV)
    yc = ssd.conv1d_varlen(kw["x"], w.to(DEV), cu_seqlens=cu, conv_states_in=c0.to(DEV), conv_states_out=out)
    ends = np.cumsum(lens)
    want, bound, last = conv_reference(np64(s.x), np64(w), None, True, np64(c0),
                                       [(0, int(e) - n, int(e)) for n, e in zip(lens, ends)], torch.bfloat16)
    within(yc, want, bound, "conv")
    assert np.array_equal(np64(out), last)


@pytest.mark.parametrize("cu", [[0, 50, 30, 100], [0, 1 << 30, 100], [-5, 40, 100], [20, 60, 80], [0, 0, 0], [100, 0, 100]])
def test_bad_offsets_stay_inside(cu):
    """Arrays of offsets that are no such thing: any values, but no access
    outside (y, states and what surrounds them)."""
    E, N, L, S = 48, 16, 100, len(cu) - 1
    s = Selective(1, L, E, N, init=False, seed=45)
    kw, _, _ = s.to(DEV)
    c = torch.tensor(cu, dtype=torch.int32, device=DEV)
    note(f"[gpu] bad offsets {cu}")
    guard = 4096
    ybuf = torch.full((2 * guard + L * E,), 9.0, device=DEV)
    fbuf = torch.full((2 * guard + S * E * N,), 9.0, device=DEV)
    y = ybuf[guard:guard + L * E].view(1, L, E)
    f = fbuf[guard:guard + S * E * N].view(S, E, N)
    ssd.selective_scan_varlen(cu_seqlens=c, y=y, final_states=f, **kw)
    w = torch.ones((E, 4), device=DEV)
    cbuf = torch.full((2 * guard + S * E * 3,), 9.0, device=DEV)
    ssd.conv1d_varlen(kw["x"], w, cu_seqlens=c, y=y, conv_states_out=cbuf[guard:guard + S * E * 3].view(S, E, 3))
    torch.cuda.synchronize()
    for buf in (ybuf, fbuf, cbuf):
        assert (buf[:guard] == 9.0).all() and (buf[-guard:] == 9.0).all()


def test_group_norm_of_rows_without_spread():
    """A constant row (variance 0) and one of infinities: what the formula gives."""
    x = torch.zeros((4, 256), device=DEV)
    x[1], x[2], x[3, 7] = 3.0, float("inf"), float("nan")
    note("[gpu] group norm of constant and non-finite rows")
    b = torch.full((256,), 0.5, device=DEV)
    o = ssd.group_norm(x, None, b)
    assert torch.equal(o[:2], torch.full((2, 256), 0.5, device=DEV))
    assert torch.isnan(o[2:]).all()
    o = ssd.group_norm(x, center=False)
    assert torch.equal(o[0], torch.zeros(256, device=DEV))
    want = 3.0 / np.sqrt(9.0 + 1e-5)
    assert (np64(o[1]) - want).max() <= 6 * U * want
    assert torch.isnan(o[2:]).all()


def test_selective_scan_of_zero_steps_and_long_decays():
    """dt = 0 carries the state over unchanged; a decay of exp(-large) forgets it."""
    b, L, E, N = 1, 90, 64, 16
    s = Selective(b, L, E, N, skip=False, gate=False, pre=False, seed=46)
    kw, h0, _ = s.to(DEV)
    note("[gpu] selective scan: zero steps, infinite decays")
    kw["dt"].zero_()
    y, h = ssd.selective_scan(init_state=h0, **kw)
    assert torch.equal(h, h0)
    kw["dt"].fill_(1.0e4)
    y, h = ssd.selective_scan(init_state=h0, **kw)
    # every decay is exp(-1e4 |A|) = 0: only the last token is left
    want = 1.0e4 * np64(kw["x"][0, -1])[:, None] * np64(kw["B"][0, -1])
    within(h[0], want, 3 * U * np.abs(want), "final_state")
