"""GPU tests of the layer operators at the edges of what their documentation
allows, beside those of test_gpu_layer.py: offsets, unusual values, and the
kernels that only large calls reach. Bounds as derived in layer_testutil."""

import ctypes

import numpy as np
import pytest
import torch

import mamba_ssd_scan_fwd_amd as ssd
from layer_testutil import IO, Selective, U, conv_reference, norm_bound, within
from oracle import layer_oracle as ref
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


# ---- kernels that only large calls reach -------------------------------------------
# (sizes just past the rules at the launches: several rows a workgroup, memory-side
# cache passed by, long tiles)


def first_rows(slots, pool):
    """Rows that have their slot, and the others."""
    first = {}
    for r, k in enumerate(slots):
        if 0 <= k < pool:
            first.setdefault(k, r)
    rows = sorted(first.values())
    return rows, [r for r in range(len(slots)) if r not in set(rows)]


def some_slots(b, pool, seed):
    """A permutation with padding, and with slots named again in the same four
    rows, the same two, the next ones and far behind."""
    slots = torch.randperm(pool, generator=torch.Generator().manual_seed(seed))[:b].tolist()
    slots[1], slots[6], slots[10], slots[11], slots[13], slots[b - 1] = slots[0], slots[4], slots[9], slots[9], slots[11], slots[2]
    slots[17], slots[20], slots[21] = -1, pool, -1
    return slots


@pytest.mark.parametrize("b,E,N,io,shift", [(67, 8192, 16, "bf16", 0), (131, 8192, 16, "bf16", 0), (70, 4096, 64, "fp32", 1),
                                            (36, 8192, 20, "bf16", 3), (401, 2050, 24, "bf16", 1)])
def test_selective_step_of_many_rows(b, E, N, io, shift):
    """Four rows a workgroup (from 8192 workgroups of one row on), the last
    four incomplete; from 64 MiB of states on past the cache; the pool at any
    element."""
    pool = b + 9
    slots = some_slots(b, pool, b)
    s = Selective(b, 1, E, N, io=io, dt=io, init=False, views=True, seed=b)
    kw, _, _ = s.to(DEV)
    one = {k: (v[:, 0] if k in ("x", "dt", "z", "B", "C") else v) for k, v in kw.items()}
    before = torch.randn((pool, E, N), generator=torch.Generator().manual_seed(b + 1))
    state = torch.empty(pool * E * N + shift, device=DEV)[shift:].view(pool, E, N).copy_(before)
    y = torch.full((b, E), 3.0, dtype=s.io, device=DEV)
    note(f"[gpu] selective step of {b} rows, E={E} N={N} {io}")
    ssd.selective_step(state=state, y=y, state_slots=torch.tensor(slots, dtype=torch.int32, device=DEV), **one)
    rows, dead = first_rows(slots, pool)
    assert len(dead) >= 8
    s.init = torch.zeros((b, E, N))
    s.init[rows] = before[[slots[r] for r in rows]]
    yr, yb, hr, hb = s.reference()
    within(y[rows], yr[rows, 0], yb[rows, 0], "y")
    assert (y[dead] == 3.0).all()
    within(state[[slots[r] for r in rows]], hr[rows], hb[rows], "state")
    rest = sorted(set(range(pool)) - {slots[r] for r in rows})
    assert torch.equal(state[rest].cpu(), before[rest])


@pytest.mark.parametrize("b,CH,K,io,shift", [(257, 8192, 4, "bf16", 0), (411, 4100, 3, "fp32", 1), (2049, 512, 2, "bf16", 3)])
def test_conv1d_step_of_many_rows(b, CH, K, io, shift):
    """Two rows a workgroup, the last pair incomplete."""
    pool = b + 9
    slots = some_slots(b, pool, b)
    g = torch.Generator().manual_seed(b + 2)
    x = torch.randn((b, CH + 5), generator=g).to(IO[io])[:, 3:CH + 3]
    w, bias = torch.randn((CH, K), generator=g) * K ** -0.5, torch.randn(CH, generator=g) * 0.3
    before = torch.randn((pool, CH, K - 1), generator=g)
    state = torch.empty(pool * CH * (K - 1) + shift, device=DEV)[shift:].view(pool, CH, K - 1).copy_(before)
    y = torch.full((b, CH), 3.0, dtype=IO[io], device=DEV)
    note(f"[gpu] conv1d step of {b} rows, CH={CH} K={K} {io}")
    ssd.conv1d_step(x._base.to(DEV)[:, 3:CH + 3], w.to(DEV), bias.to(DEV), state, y=y,
                    state_slots=torch.tensor(slots, dtype=torch.int32, device=DEV))
    rows, dead = first_rows(slots, pool)
    at = [slots[r] for r in rows]
    want, bound, last = conv_reference(np64(x[rows])[:, None], np64(w), np64(bias), True, np64(before[at]),
                                       [(i, 0, 1) for i in range(len(rows))], IO[io])
    within(y[rows], want[:, 0], bound[:, 0], "y")
    assert (y[dead] == 3.0).all()
    expect = np64(before)
    expect[at] = last
    assert np.array_equal(np64(state), expect)


@pytest.mark.parametrize("b,L,CH,K,io", [(2, 4500, 4099, 4, "bf16"), (2, 8200, 4099, 4, "bf16"), (1, 9001, 2049, 3, "fp32"),
                                         (3, 2900, 8192, 2, "bf16"), (1, 33000, 1030, 4, "bf16")])
def test_conv1d_of_large_inputs(b, L, CH, K, io):
    """Outputs of 64 to 256 MiB: inputs past the cache, tiles of 32 and 64
    tokens. Windows against the definition, everything against short calls."""
    g = torch.Generator(device=DEV).manual_seed(L)
    x = torch.randn((b, L, CH + 5), generator=g, device=DEV).to(IO[io])[:, :, 3:CH + 3]
    w, bias = torch.randn((CH, K), generator=g, device=DEV) * K ** -0.5, torch.randn(CH, generator=g, device=DEV) * 0.3
    s0 = torch.randn((b, CH, K - 1), generator=g, device=DEV)
    size = b * L * CH * x.element_size()
    assert 64 << 20 <= size < 256 << 20
    note(f"[gpu] conv1d b={b} L={L} CH={CH} K={K} {io}")
    last = torch.empty_like(s0)
    y = ssd.conv1d(x, w, bias, conv_state_in=s0, conv_state_out=last)
    line = torch.cat([s0.transpose(1, 2), x.float()], 1)  # token t at t + K - 1
    assert torch.equal(last, line[:, L:].transpose(1, 2))
    for a in list(range(0, L, 999)) + [L - 130]:
        z = min(a + 999, L)
        part = ssd.conv1d(x[:, a:z], w, bias, conv_state_in=line[:, a:a + K - 1].transpose(1, 2).contiguous())
        assert torch.equal(y[:, a:z], part), a
    for a, z in ((0, 70), (L // 2, L // 2 + 70), (L - 70, L)):
        want, bound, _ = conv_reference(np64(x[:, a:z]), np64(w), np64(bias), True,
                                        np64(line[:, a:a + K - 1].transpose(1, 2)), [(i, 0, z - a) for i in range(b)], IO[io])
        within(y[:, a:z], want, bound, f"y from {a}")


@pytest.mark.parametrize("T", [33000, 66000, 132000])
def test_conv1d_packed_in_long_tiles(T):
    """Tiles of 16, 32 and 64 tokens with sequences that end inside them."""
    CH, K, S = 64, 4, 700
    g = torch.Generator().manual_seed(T)
    cu = torch.cat([torch.zeros(1, dtype=torch.long), torch.randint(0, T - 50, (S - 1,), generator=g).sort()[0],
                    torch.tensor([T - 9])])
    cu[101], cu[103], cu[301:305] = cu[100], cu[102] + 1, cu[300]
    cu = cu.sort()[0]
    x, w = torch.randn((1, T, CH), generator=g).to(torch.bfloat16), torch.randn((CH, K), generator=g)
    s0 = torch.randn((S, CH, K - 1), generator=g)
    y = torch.full((1, T, CH), 7.0, dtype=torch.bfloat16, device=DEV)
    last = torch.empty((S, CH, K - 1), device=DEV)
    note(f"[gpu] conv1d packed, {T} tokens")
    ssd.conv1d_varlen(x.to(DEV), w.to(DEV), cu_seqlens=cu.int().to(DEV), conv_states_in=s0.to(DEV), conv_states_out=last, y=y)
    spans = [(0, a, b) for a, b in zip(cu.tolist(), cu.tolist()[1:])]
    want, bound, end = conv_reference(np64(x), np64(w), None, True, np64(s0), spans, torch.bfloat16)
    within(y[:, :T - 9], want[:, :T - 9], bound[:, :T - 9], "y")
    assert (y[:, T - 9:] == 7.0).all()
    assert np.array_equal(np64(last), end)


@pytest.mark.parametrize("R,C,G,io,gate,first,center", [
    (6000, 4101, 3, "bf16", True, True, False), (4000, 5001, 1, "fp32", False, False, True), (3000, 9001, 1, "bf16", True, False, True),
    (2900, 4097, 1, "fp32", True, True, True), (21000, 2050, 205, "bf16", True, False, False)])
def test_group_norm_of_large_inputs(R, C, G, io, gate, first, center):
    """More than 128 MiB: inputs past the cache, groups that end inside a
    pack. Some rows against the definition, all against short calls."""
    g = torch.Generator(device=DEV).manual_seed(R)
    x = torch.randn((R, C + 3), generator=g, device=DEV).to(IO[io])[:, 1:C + 1]
    z = torch.randn((R, C + 3), generator=g, device=DEV).to(IO[io])[:, 2:C + 2] if gate else None
    w, bias = 1 + 0.3 * torch.randn(C, generator=g, device=DEV), 0.3 * torch.randn(C, generator=g, device=DEV)
    assert R * C * x.element_size() * (3 if gate else 2) > 128 << 20
    kw = dict(ngroups=G, center=center, gate_first=first)
    note(f"[gpu] group norm {R} x {C} G={G} {io}")
    o = ssd.group_norm(x, w, bias, z, **kw)
    for a in range(0, R, 511):
        part = ssd.group_norm(x[a:a + 511], w, bias, None if z is None else z[a:a + 511], **kw)
        assert torch.equal(o[a:a + 511], part), a
    rows = [0, 1, 2, R // 2, R - 3, R - 2, R - 1]
    pick = lambda t: None if t is None else np64(t[rows])  # noqa: E731
    want = ref.group_norm(pick(x), G, 1e-5, np64(w), np64(bias), pick(z), center, first, False)
    bound = norm_bound(pick(x), G, 1e-5, np64(w), np64(bias), pick(z), center, first, False, IO[io], want)
    within(o[rows], want, bound, "out")


# ---- streams ------------------------------------------------------------------------


def test_group_norm_of_a_constant_row():
    x = torch.full((3, 256), 3.0, device=DEV)
    x[1], x[2] = -3.0, 0.0
    note("[gpu] group norm of constant rows")
    o = np64(ssd.group_norm(x, center=False))
    want = 3.0 / np.sqrt(9.0 + 1e-5)
    assert np.abs(o[0] - want).max() <= 6 * U * want and np.abs(o[1] + want).max() <= 6 * U * want
    assert np.all(o[2] == 0.0)


def same_block(t):
    """Whether the allocator gives a freed block of t's size out again at once."""
    a = torch.empty_like(t)
    at = a.data_ptr()
    del a
    return torch.empty_like(t).data_ptr() == at


def test_memory_of_a_call_on_another_stream_is_kept_until_it_ran():
    """The call waits behind a sleep on its stream; its inputs are dropped, and
    blocks of their sizes overwritten on the caller's stream, before it runs.
    Then its output is read behind a sleep on the caller's stream and dropped,
    and blocks of its size overwritten on the other."""
    s = Selective(1, 2000, 64, 16, seed=34)
    kw, h0, _ = s.to(DEV)
    want, hT = ssd.selective_scan(init_state=h0, **kw)
    names = ("x", "dt", "z", "B", "C")
    note("[gpu] selective scan: memory in use on two streams")
    here, side = torch.cuda.current_stream(), torch.cuda.Stream()
    held = torch.empty_like(kw["x"])
    assert same_block(held)
    mine = dict(kw, **{k: kw[k].clone() for k in names})
    start = h0.clone()
    side.wait_stream(here)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    y, h = ssd.selective_scan(init_state=start, stream=side, **mine)
    del mine, start
    junk = [torch.full_like(kw[k], float("nan")) for k in names for _ in range(2)] + [torch.full_like(h0, float("nan"))]
    here.wait_stream(side)
    torch.cuda._sleep(20_000_000)
    kept, keph = y.clone(), h.clone()
    del y, h
    with torch.cuda.stream(side):
        junk += [torch.full_like(want, float("nan")) for _ in range(3)] + [torch.full_like(hT, float("nan")) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(kept, want) and torch.equal(keph, hT)


# ---- unusual values --------------------------------------------------------------------


@pytest.mark.parametrize("io,L", [("fp32", 50), ("bf16", 300)])
def test_a_step_size_of_nan_is_not_clamped_away(io, L):
    """dt is clamped to its limits, infinities too; a NaN stays NaN and takes
    its channel from its token on, and no other."""
    s = Selective(1, L, 70, 16, io=io, dt=io, gate=False, seed=49)
    kw, h0, _ = s.to(DEV)
    want, hw = ssd.selective_scan(init_state=h0, **kw)
    note(f"[gpu] selective scan and step: NaN step sizes, {io}")
    t, e = L - 11, 33
    dt = kw["dt"].clone()
    dt[0, t, e] = float("nan")
    y, h = ssd.selective_scan(init_state=h0, **dict(kw, dt=dt))
    assert torch.isnan(y[0, t:, e]).all() and torch.isnan(h[0, e]).all()
    others = torch.arange(70, device=DEV) != e
    assert torch.equal(y[:, :, others], want[:, :, others]) and torch.equal(h[:, others], hw[:, others])
    assert torch.equal(y[0, :t, e], want[0, :t, e])
    state = h0.clone()
    one = {k: (v[:, t] if k in ("x", "dt", "B", "C") else v) for k, v in dict(kw, dt=dt, z=None).items()}
    y1 = ssd.selective_step(state=state, **one)
    assert torch.isnan(y1[0, e]) and torch.isnan(state[0, e]).all()
    assert torch.isfinite(y1[:, others]).all() and torch.isfinite(state[:, others]).all()
    # beyond the limits on both sides: the same as dt at them
    pre = dict(limit=(1e-3, 0.5))
    near = {k: (v[:, t] if k in ("x", "B", "C") else v) for k, v in dict(kw, z=None, dt_pre=pre).items() if k != "dt"}
    for far, at in ((float("-inf"), 1e-3), (float("inf"), 0.5)):
        a, b = h0.clone(), h0.clone()
        ya = ssd.selective_step(state=a, dt=torch.full((1, 70), far, device=DEV), **near)
        yb = ssd.selective_step(state=b, dt=torch.full((1, 70), at, device=DEV), **near)
        assert torch.equal(ya, yb) and torch.equal(a, b)


def test_decays_of_the_lowest_value():
    """A of the type's lowest value: a step of zero keeps the state (0 times it
    is no infinity), any other forgets it."""
    E, N, lowest = 40, 16, torch.finfo(torch.float32).min
    s = Selective(2, 7, E, N, gate=False, skip=False, pre=False, seed=50)
    kw, h0, _ = s.to(DEV)
    kw["A"][:, 3:9] = lowest
    kw["dt"].zero_()
    note("[gpu] selective scan and step: decays of the lowest value")
    _, h = ssd.selective_scan(init_state=h0, **kw)
    assert torch.equal(h, h0)
    one = {k: (v[:, 0] if k in ("x", "dt", "B", "C") else v) for k, v in dict(kw, z=None).items()}
    state = h0.clone()
    ssd.selective_step(state=state, **one)
    assert torch.equal(state, h0)
    one["dt"] = torch.full((2, E), 0.25, device=DEV)
    ssd.selective_step(state=state, **one)
    u = (0.25 * one["x"])[:, :, None] * one["B"][:, :1]
    assert torch.equal(state[:, :, 3:9], u[:, :, 3:9])


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("size", [3e-21, 1e-20, 1e-19, 1e18])
def test_group_norm_of_rows_of_extreme_size(size, center):
    """eps = 0 and squares below the smallest normal number: the statistics
    are then as exact as subnormal sums of squares are. Of C squares and adds
    each is off by 2^-150, as is their mean; the root halves that; 8 U for the
    rest, and for the centre (a mean off by 66 U of mean|x|, the square of
    which does not count here) 70 U of a deviation."""
    C = 256
    x = (torch.randn((5, C), generator=torch.Generator().manual_seed(51)) * size).float()
    note(f"[gpu] group norm of rows of size {size}")
    o = np64(ssd.group_norm(x.to(DEV), eps=0.0, center=center))
    want = ref.group_norm(np64(x), 1, 0.0, center=center)
    v = np64(x) - (np64(x).mean(1, keepdims=True) if center else 0.0)
    var = (v * v).mean(1, keepdims=True)
    rel = 0.5 * (2 * C * 2.0 ** -150 / (C * var) + 2.0 ** -150 / var) + 8 * U
    within(o, want, np.abs(want) * rel * 1.01 + (70 * U if center else 0.0), "out")


# ---- calls at once, graphs, the C ABI ------------------------------------------------------


def scans(seed, lens=None):
    """A scan that is cut into segments (so it has a workspace), and its result."""
    s = Selective(1, 900, 96, 16, io="bf16", dt="bf16", lens=lens, seed=seed)
    kw, h0, cu = s.to(DEV)

    def run():
        u = ssd.conv1d(kw["x"], w) if cu is None else ssd.conv1d_varlen(kw["x"], w, cu_seqlens=cu)
        a = dict(kw, x=u)
        y, h = (ssd.selective_scan(init_state=h0, **a) if cu is None else
                ssd.selective_scan_varlen(cu_seqlens=cu, init_states=h0, **a))
        return [y, h, ssd.group_norm(y, ngroups=3)]

    w = torch.randn((96, 4), generator=torch.Generator().manual_seed(seed)).to(DEV)
    return run


def test_two_streams_at_once():
    runs = [scans(61), scans(62, [300, 0, 7, 593])]
    wants = [r() for r in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    note("[gpu] two streams at once")
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for r, st, g in zip(runs, streams, got):
            with torch.cuda.stream(st):
                g.append(r())
    torch.cuda.synchronize()
    for want, outs in zip(wants, got):
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_two_graphs_replayed_at_once():
    """Each graph has its own workspace: replays on two streams, with eager
    calls between, all give the same bits."""
    runs = [scans(63), scans(64, [1] * 40 + [860])]
    wants = [r() for r in runs]
    note("[gpu] two graphs at once")
    torch.cuda.synchronize()
    graphs, outs = [], []
    for r in runs:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            r()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(r())
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(4):
        for out in outs:
            for o in out:
                o.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        eager = [r() for r in runs]
        torch.cuda.synchronize()
        for want, out, e in zip(wants, outs, eager):
            assert all(torch.equal(a, b) for a, b in zip(want, out))
            assert all(torch.equal(a, b) for a, b in zip(want, e))


@pytest.mark.parametrize("own", [False, True])
def test_workspace_of_the_c_abi(own):
    """A null workspace is allocated and freed in stream order; one of exactly
    the size asked for is enough, and nothing behind it is written."""
    s = Selective(1, 1500, 64, 16, seed=65)
    kw, h0, _ = s.to(DEV)
    want, hw = ssd.selective_scan(init_state=h0, **kw)
    d = ssd.SelectiveDesc(batch=1, seqlen=1500, channels=64, dstate=16, ngroups=1, io_dtype=0, dt_dtype=0,
                          dt_bias=kw["dt_pre"]["bias"].data_ptr(), dt_softplus=1, dt_clamp=1, dt_min=1e-3, dt_max=0.5)
    n = ssd.selective_scan_workspace_bytes(d)
    assert n > 0
    ws = torch.full((n + GUARD,), 255, dtype=torch.uint8, device=DEV)
    y, h = torch.empty_like(want), torch.empty_like(hw)
    note(f"[gpu] selective scan through the C ABI, own workspace {own}")
    torch.cuda.synchronize()
    p = [kw[k].data_ptr() for k in ("x", "dt", "A", "B", "C", "D", "z")] + [t.data_ptr() for t in (h0, y, h)]
    for _ in range(3):
        st = ssd.load_library().ssd_selective_scan(ctypes.byref(d), *p, ws.data_ptr() if own else None, n if own else 0, None)
        assert st == 0
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(h, hw)
    assert (ws[n:] == 255).all()


def test_outputs_of_more_than_two_to_the_31_elements():
    """The second of two rows lies behind 2^31 elements in part: its last
    tokens against the definition (scan) and against a call on their own."""
    b, L, E, N, tail = 2, 540_001, 2048, 16, 150
    g = torch.Generator(device=DEV).manual_seed(66)
    draw = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    x, z, dt, B, C = draw(b, L, E), draw(b, L, E), draw(b, L, E), draw(b, L, 1, N), draw(b, L, 1, N)
    A = -torch.exp(torch.rand((E, N), generator=g, device=DEV) * 2.8)
    assert x.numel() > 1 << 31
    note("[gpu] outputs of more than 2^31 elements")
    # steps of 0.05 and more, so that 1280 tokens back nothing is left (e^-64)
    pre = dict(softplus=True, limit=(0.05, 0.5))
    y, h = ssd.selective_scan(x, dt, A, B, C, None, z, dt_pre=pre)
    _, before = ssd.selective_scan(x[:, :-tail], dt[:, :-tail], A, B[:, :-tail], C[:, :-tail], dt_pre=pre)
    d = np.clip(ref.softplus(np64(dt[:, -tail:])), 0.05, 0.5)
    f = (3 * 1280 + N + 2300 + 26) * U
    for i in range(b):
        # (before is itself off by f of its terms' absolute values, bounded by
        # those that 1280 steps of 0.5 of |x B| below 6 x 6 can leave)
        yr, ya, hr, ha = ref.selective_scan(np64(x[i, -tail:]), d[i], np64(A), np64(B[i, -tail:]), np64(C[i, -tail:]), None,
                                            np64(z[i, -tail:]), np64(before[i]))
        left = np.exp(-np.cumsum(d[i], 0)) * 1280 * 0.5 * 36.0  # of any state, |A| being 1 at least
        gate = np.abs(ref.silu(np64(z[i, -tail:]))) * np.abs(np64(C[i, -tail:, 0])).sum(1)[:, None]
        within(y[i, -tail:], yr, f * (ya + left * gate) + np.abs(yr) * 2.0 ** -8, "y")
        within(h[i], hr, f * (ha + left[-1][:, None]), "final_state")
    w = torch.randn((E, 4), generator=g, device=DEV)
    line = x[:, -tail - 3:]
    assert torch.equal(ssd.conv1d(x, w)[:, -tail:], ssd.conv1d(line, w)[:, 3:])
    assert torch.equal(ssd.group_norm(x, None, None, z, ngroups=4)[:, -tail:],
                       ssd.group_norm(x[:, -tail:], None, None, z[:, -tail:], ngroups=4))


def test_a_stream_given_inside_a_capture():
    """A captured call on a second stream that forks from the capturing one
    and joins it again."""
    s = Selective(1, 500, 64, 16, io="bf16", dt="bf16", seed=67)
    kw, h0, _ = s.to(DEV)
    want, hw = ssd.selective_scan(init_state=h0, **kw)
    note("[gpu] selective scan: stream argument inside a capture")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        y, h = ssd.selective_scan(init_state=h0, stream=side, **kw)
        here.wait_stream(side)
        o = ssd.group_norm(y)
    norm = ssd.group_norm(want)
    for _ in range(3):
        for t in (y, h, o):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(h, hw) and torch.equal(o, norm)
