"""GPU tests of the gated delta rule, against the fp64 recurrence
(oracle/layer_oracle.py) within bounds derived in delta_testutil."""

import numpy as np
import pytest
import torch

import mamba_ssd_scan_fwd_amd as ssd
from delta_testutil import Delta, near, within
from ssd_testutil import note

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOKENS = ("x", "dt", "B", "C", "beta")

RULE = [
    # b, L, H, P, N, G, io, dt, init, pre, sigmoid, views
    (1, 1, 1, 1, 1, 1, "fp32", "fp32", False, False, False, False),
    (2, 3, 2, 5, 7, 1, "fp32", "fp32", True, True, True, False),
    (1, 15, 2, 16, 16, 2, "bf16", "bf16", True, True, True, False),
    (3, 16, 2, 64, 32, 1, "bf16", "fp32", False, True, True, True),
    (1, 17, 4, 20, 64, 2, "fp32", "fp32", True, True, True, True),
    (2, 37, 2, 128, 128, 1, "bf16", "bf16", False, True, True, False),
    (1, 63, 2, 64, 128, 1, "fp32", "fp32", True, True, True, False),
    (2, 64, 2, 64, 64, 2, "bf16", "bf16", True, True, True, True),
    (1, 65, 3, 33, 100, 3, "bf16", "fp32", True, True, False, True),
    (2, 128, 2, 128, 128, 1, "bf16", "bf16", True, False, True, False),
    (1, 130, 2, 64, 64, 1, "fp32", "fp32", True, True, False, True),
    (1, 200, 2, 96, 96, 2, "bf16", "bf16", True, True, True, False),
    (1, 129, 2, 256, 256, 1, "bf16", "bf16", True, True, True, True),
    (1, 70, 1, 256, 255, 1, "fp32", "fp32", True, True, True, False),
    (2, 300, 2, 48, 24, 1, "bf16", "fp32", False, True, True, True),
    (1, 300, 1, 131, 77, 1, "fp32", "fp32", True, True, True, True),
    (1, 520, 2, 64, 128, 1, "bf16", "bf16", True, True, True, False),
    # blocks that end early, of many heads
    (8, 13, 32, 128, 128, 4, "bf16", "bf16", True, True, True, False),
    (2, 20, 200, 128, 100, 1, "bf16", "fp32", True, True, True, True),
    (1, 50, 300, 64, 64, 300, "fp32", "fp32", False, True, True, False),
]


@pytest.mark.parametrize("b,L,H,P,N,G,io,dt,init,pre,sigmoid,views", RULE)
def test_rule_matches_the_recurrence(b, L, H, P, N, G, io, dt, init, pre, sigmoid, views):
    s = Delta(b, L, H, P, N, G, io, dt, init, pre, sigmoid, views, seed=L + P)
    kw, h0, _ = s.to(DEV)
    note(f"[gpu] delta rule b={b} L={L} H={H} P={P} N={N} G={G} {io}/{dt}")
    y, hT = ssd.delta_rule(init_state=h0, **kw)
    yr, yb, hr, hb = s.reference()
    within(y, yr, yb, "y")
    within(hT, hr, hb, "final_state")
    near(hT, hr, "final_state")


PACKED = [[5, 0, 1, 64, 33, 0, 0, 150, 2, 1, 1, 31, 0], [200], [64, 64, 128], [1] * 40,
          [64, 0, 1, 300, 33, 0, 0, 150, 63, 65, 0]]


@pytest.mark.parametrize("lens", PACKED)
@pytest.mark.parametrize("io,P,N,init", [("fp32", 20, 16, True), ("bf16", 64, 128, False), ("bf16", 40, 50, True),
                                         ("fp32", 64, 64, False)])
def test_rule_packed(io, P, N, init, lens):
    s = Delta(1, sum(lens), 2, P, N, 1, io, io, init, True, True, True, lens=lens, seed=N)
    kw, h0, cu = s.to(DEV)
    note(f"[gpu] delta rule packed {io} P={P} N={N} init={init} lens={lens}")
    y, hT = ssd.delta_rule_varlen(cu_seqlens=cu, init_states=h0, **kw)
    yr, yb, hr, hb = s.reference()
    within(y, yr, yb, "y")
    within(hT, hr, hb, "final_states")


@pytest.mark.parametrize("io", ["fp32", "bf16"])
def test_packed_leaves_what_lies_outside(io):
    lens = [40, 60]
    s = Delta(1, 130, 2, 33, 64, 1, io, io, lens=lens, seed=3)
    kw, h0, cu = s.to(DEV)
    cu = cu + 10
    for k in TOKENS:
        kw[k] = torch.roll(kw[k], 10, 1)
        kw[k][:, :10] = kw[k][:, 110:] = float("nan")
    y = torch.full((1, 130, 2, 33), 7.0, device=DEV, dtype=s.io)
    note(f"[gpu] delta rule: tokens before and behind the sequences {io}")
    _, hT = ssd.delta_rule_varlen(cu_seqlens=cu, init_states=h0, y=y, **kw)
    yr, yb, hr, hb = s.reference()
    within(y[:, 10:110], yr[:, :100], yb[:, :100], "y")
    assert (y[:, :10] == 7.0).all() and (y[:, 110:] == 7.0).all()
    within(hT, hr, hb, "final_states")


@pytest.mark.parametrize("io", ["fp32", "bf16"])
def test_sequences_and_rows_do_not_meet(io):
    lens = [50, 0, 130, 1, 80]
    s = Delta(1, sum(lens), 2, 64, 64, 2, io, io, lens=lens, seed=4)
    kw, h0, cu = s.to(DEV)
    note(f"[gpu] delta rule: NaN and infinities beside others {io}")
    want, hw = ssd.delta_rule_varlen(cu_seqlens=cu, init_states=h0, **kw)
    others = torch.tensor([t for t in range(sum(lens)) if not 50 <= t < 180], device=DEV)
    # row 7 of head 1's values alone
    one = dict(kw, x=kw["x"].clone())
    one["x"][:, 60, 1, 7] = float("nan")
    got, hg = ssd.delta_rule_varlen(cu_seqlens=cu, init_states=h0, **one)
    rows = [p for p in range(64) if p != 7]
    assert torch.equal(got[:, :, 0], want[:, :, 0]) and torch.equal(got[:, :, 1, rows], want[:, :, 1, rows])
    assert torch.equal(got[:, others], want[:, others])
    assert torch.isnan(got[:, 60:180, 1, 7]).all() and torch.isnan(hg[2, 1, 7]).all()
    # keys, states and steps of a whole sequence
    kw["B"][:, 70, 0] = float("inf")
    kw["dt"][:, 75] = float("nan")
    kw["beta"][:, 77] = float("nan")
    h0[2] = float("inf")
    got, hg = ssd.delta_rule_varlen(cu_seqlens=cu, init_states=h0, **kw)
    assert torch.equal(got[:, others], want[:, others])
    assert torch.equal(hg[[0, 1, 3, 4]], hw[[0, 1, 3, 4]])
    assert torch.isnan(got[:, 77:180]).all()


@pytest.mark.parametrize("lens", [None, [90, 0, 140, 30]])
@pytest.mark.parametrize("io,P,N", [("bf16", 64, 128), ("fp32", 50, 30), ("fp32", 64, 64)])
def test_state_in_place_and_same_bits(io, P, N, lens):
    s = Delta(1, 260, 2, P, N, 1, io, io, lens=lens, seed=5)
    kw, h0, cu = s.to(DEV)
    note(f"[gpu] delta rule: final state over the initial state {io} P={P} N={N} lens={lens}")

    def run(init, final):
        if lens is None:
            return ssd.delta_rule(init_state=init, final_state=final, **kw)
        return ssd.delta_rule_varlen(cu_seqlens=cu, init_states=init, final_states=final, **kw)

    y, hT = run(h0, None)
    again = run(h0, None)
    assert torch.equal(y, again[0]) and torch.equal(hT, again[1])
    state = h0.clone()
    yi, hi = run(state, state)
    assert hi.data_ptr() == state.data_ptr()
    assert torch.equal(y, yi) and torch.equal(hT, hi)


def test_time_major_own_workspace_and_outputs():
    s = Delta(3, 100, 2, 64, 64, io="bf16", dt="bf16", seed=6)
    kw, h0, _ = s.to(DEV)
    y, hT = ssd.delta_rule(init_state=h0, **kw)
    note("[gpu] delta rule: time-major inputs, a workspace of noise")
    tm = {k: kw[k].transpose(0, 1).contiguous().transpose(0, 1) for k in TOKENS}
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(y)
    y2, none = ssd.delta_rule(init_state=h0, workspace=ws, y=out, return_final_state=False, **dict(kw, **tm))
    assert none is None and y2.data_ptr() == out.data_ptr() and torch.equal(y, y2)


@pytest.mark.parametrize("io", ["fp32", "bf16"])
def test_rule_carries_over_calls(io):
    s = Delta(2, 250, 2, 64, 64, io=io, dt=io, seed=7)
    kw, h0, _ = s.to(DEV)
    note(f"[gpu] delta rule: two calls in turn {io}")
    cut = 71
    part = lambda a, b: {k: (v[:, a:b] if k in TOKENS else v) for k, v in kw.items()}  # noqa: E731
    y1, h = ssd.delta_rule(init_state=h0, **part(0, cut))
    y2, h = ssd.delta_rule(init_state=h, **part(cut, 250))
    yr, yb, hr, hb = s.reference()
    within(torch.cat([y1, y2], 1), yr, 2 * yb, "y")
    within(h, hr, 2 * hb, "final_state")


# ---- long sequences of few heads: the time axis in segments -------------------------


def is_cut(s, S=0):
    """Whether the call's workspace holds more than the blocks' records."""
    d = ssd.DeltaDesc(batch=s.b, seqlen=s.L, nheads=s.H, headdim=s.P, dstate=s.N, ngroups=s.G, io_dtype=int(s.io == torch.bfloat16),
                      scale=1.0)
    slots = s.L // 64 + S if S else s.b * -(-s.L // 64)
    return ssd.delta_rule_workspace_bytes(d, S) > slots * s.H * (18944 if s.io == torch.bfloat16 else 37376)


@pytest.mark.parametrize("L,H,P,N,io,views", [(1100, 2, 64, 64, "bf16", False), (1025, 1, 128, 128, "bf16", False),
                                              (1300, 1, 40, 77, "bf16", True), (1100, 1, 20, 64, "fp32", False),
                                              (1088, 1, 33, 100, "fp32", True), (1100, 1, 16, 256, "bf16", False),
                                              (2200, 1, 16, 32, "bf16", False)])
def test_long_rule_in_segments(L, H, P, N, io, views):
    s = Delta(1, L, H, P, N, 1, io, "fp32", views=views, seed=L)
    assert is_cut(s)
    kw, h0, _ = s.to(DEV)
    note(f"[gpu] delta rule in segments L={L} H={H} P={P} N={N} {io}")
    y, hT = ssd.delta_rule(init_state=h0, **kw)
    yr, yb, hr, hb = s.reference(cut=True)
    within(y, yr, yb, "y")
    within(hT, hr, hb, "final_state")
    near(hT, hr, "final_state")
    again = ssd.delta_rule(init_state=h0, final_state=h0, **kw)
    assert torch.equal(y, again[0]) and torch.equal(hT, h0)


@pytest.mark.parametrize("lens", [[1500, 0, 700], [3, 2000], [0, 0, 1600, 0], [640, 640, 641]])
@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_long_packed_rule_in_segments(lens, io):
    s = Delta(1, sum(lens), 1, 24, 64, 1, io, "fp32", lens=lens, seed=len(lens))
    assert is_cut(s, len(lens))
    kw, h0, cu = s.to(DEV)
    note(f"[gpu] delta rule packed in segments {lens} {io}")
    y, hT = ssd.delta_rule_varlen(cu_seqlens=cu, init_states=h0, **kw)
    yr, yb, hr, hb = s.reference(cut=True)
    within(y, yr, yb, "y")
    within(hT, hr, hb, "final_states")
    again = ssd.delta_rule_varlen(cu_seqlens=cu, init_states=h0, final_states=h0, **kw)
    assert torch.equal(y, again[0]) and torch.equal(hT, h0)


@pytest.mark.parametrize("cu", [[0, 50, 30, 1000], [0, 1 << 30, 100], [-5, 400, 1000], [20, 600, 800], [0, 0, 0], [1000, 0, 1000],
                                [990, 64, 1000, 3]])
@pytest.mark.parametrize("H,P,io", [(1, 16, "bf16"), (64, 16, "bf16"), (1, 16, "fp32"), (64, 16, "fp32"), (2, 5, "bf16")])
def test_bad_offsets_stay_inside(cu, H, P, io):
    """Whatever the offsets hold, nothing outside the arrays is touched."""
    T, N = 1000, 32
    s = Delta(1, T, H, P, N, 1, io, "fp32", init=False, seed=12)
    kw, _, _ = s.to(DEV)
    S = len(cu) - 1
    y = torch.full((1, T + 64, H, P), 7.0, device=DEV, dtype=s.io)
    h = torch.full((S + 2, H, P, N), 5.0, device=DEV)
    note(f"[gpu] delta rule: offsets {cu} H={H}")
    ssd.delta_rule_varlen(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV), y=y[:, :T], final_states=h[1:S + 1], **kw)
    assert (y[:, T:] == 7.0).all() and (h[0] == 5.0).all() and (h[S + 1] == 5.0).all()


# ---- decays and betas at their borders ---------------------------------------------


@pytest.mark.parametrize("io", ["fp32", "bf16"])
def test_without_decay_and_with_whole_ones(io):
    """A = 0 keeps the state; beta = 1 and keys of length one replace what a key
    answers (the same key twice: the second value is what is left of it)."""
    L, P, N = 150, 64, 64
    s = Delta(1, L, 1, P, N, 1, io, io, init=False, pre=False, sigmoid=False, seed=8, scale=1.0)
    kw, _, _ = s.to(DEV)
    kw["A"] = torch.zeros(1, device=DEV)
    kw["beta"] = torch.ones_like(kw["beta"])
    kw["B"] = torch.zeros_like(kw["B"])
    t = torch.arange(L, device=DEV)
    kw["B"][0, t, 0, t % N] = 1.0
    kw["C"] = kw["B"].clone()
    note(f"[gpu] delta rule: keys of one channel {io}")
    y, hT = ssd.delta_rule(**kw)
    # products with 0 and 1 of values of x as they came; later ones of what is left
    # in the state and of the difference to it: each one operand's rounding, 2^-8 of
    # up to 2 max|x| and 1 max|x| in y, 2^-16 in the state (2^-24 with fp32 io)
    top = float(kw["x"].float().abs().max())
    if io == "bf16":  # (of fp32, the terms are products and sums of their own)
        assert torch.equal(y[:, :N], kw["x"][:, :N])
    assert (y.float() - kw["x"].float()).abs().max() <= (3 * 2.0 ** -16 if io == "fp32" else 4 * 2.0 ** -8) * top
    last = torch.stack([kw["x"][0, max(i for i in range(L) if i % N == n), 0] for n in range(N)], 1)
    assert (hT[0, 0] - last.float()).abs().max() <= 9 * 2.0 ** -16 * top


@pytest.mark.parametrize("io", ["fp32", "bf16"])
def test_decays_that_end_everything(io):
    """A decay of the lowest value, or a step of infinity, empties the state; the
    tokens behind it decay among themselves as if it had not been there."""
    L, cut = 150, 70
    s = Delta(1, L, 2, 64, 64, 1, io, "fp32", pre=False, seed=9)
    s.dt[0, cut] = 1e30
    kw, h0, _ = s.to(DEV)
    note(f"[gpu] delta rule: a step of 1e30 {io}")
    y, hT = ssd.delta_rule(init_state=h0, **kw)
    # the reference: a decay of exactly 0 there
    sr = Delta(1, L, 2, 64, 64, 1, io, "fp32", pre=False, seed=9)
    a = Delta(1, L - cut, 2, 64, 64, 1, io, "fp32", pre=False, seed=9)
    for k in TOKENS:
        setattr(a, k, getattr(sr, k)[:, cut:])
    a.A, a.init = sr.A, None
    yr, yb, hr, hb = a.reference()
    within(y[:, cut:], yr, yb, "y")
    within(hT, hr, hb, "final_state")
    kw["dt"][0, cut] = float("inf")
    y2, h2 = ssd.delta_rule(init_state=h0, **kw)
    assert torch.equal(y, y2) and torch.equal(hT, h2)


def test_steps_of_zero_keep_the_state():
    s = Delta(1, 100, 2, 64, 64, 1, "bf16", "fp32", pre=False, sigmoid=False, seed=10)
    kw, h0, _ = s.to(DEV)
    kw["dt"].zero_()
    kw["beta"].zero_()
    kw["A"].fill_(torch.finfo(torch.float32).min)
    note("[gpu] delta rule: steps and betas of zero")
    y, hT = ssd.delta_rule(init_state=h0, **kw)
    assert torch.equal(hT, h0)
    assert torch.isfinite(y).all()


# ---- single tokens --------------------------------------------------------------------

STEP = [(1, 1, 1, 1, 1, "fp32", "fp32"), (3, 2, 20, 16, 1, "bf16", "bf16"), (5, 4, 64, 5, 2, "fp32", "fp32"),
        (2, 6, 33, 100, 3, "bf16", "fp32"), (4, 2, 128, 128, 1, "bf16", "bf16"), (2, 2, 256, 256, 2, "fp32", "fp32"),
        (2, 1, 255, 253, 1, "bf16", "bf16"), (70, 32, 128, 128, 16, "bf16", "bf16"), (67, 32, 128, 60, 32, "fp32", "fp32"),
        # two and four rows of the state to a team, the last of them short
        (33, 32, 50, 64, 8, "fp32", "fp32"), (130, 32, 70, 61, 4, "bf16", "bf16"), (300, 32, 36, 64, 1, "bf16", "fp32")]


@pytest.mark.parametrize("b,H,P,N,G,io,dt", STEP)
def test_step_matches_the_recurrence(b, H, P, N, G, io, dt):
    s = Delta(b, 1, H, P, N, G, io, dt, views=True, seed=b + P)
    kw, h0, _ = s.to(DEV)
    note(f"[gpu] delta step b={b} H={H} P={P} N={N} G={G} {io}/{dt}")
    one = {k: (v[:, 0] if k in TOKENS else v) for k, v in kw.items()}
    state = h0.clone()
    y = ssd.delta_step(state=state, **one)
    yr, yb, hr, hb = s.reference()
    within(y, yr[:, 0], yb[:, 0], "y")
    within(state, hr, hb, "state")


@pytest.mark.parametrize("b,H,P,N,slots", [(9, 2, 20, 24, [3, -1, 11, 3, 0, 12, 3, 99, 5]), (300, 32, 16, 64, None)])
def test_step_slots(b, H, P, N, slots):
    pool = 12 if slots else 400
    if slots is None:
        g = torch.Generator().manual_seed(1)
        slots = torch.randperm(pool, generator=g)[:b].tolist()
        slots[7], slots[290], slots[299], slots[150] = slots[6], slots[3], slots[290], -5
    s = Delta(b, 1, H, P, N, io="bf16", dt="bf16", init=False, seed=8)
    kw, _, _ = s.to(DEV)
    one = {k: (v[:, 0].contiguous() if k in TOKENS else v) for k, v in kw.items()}
    before = torch.randn((pool, H, P, N), generator=torch.Generator().manual_seed(2))
    state, y = before.to(DEV), torch.full((b, H, P), 3.0, dtype=torch.bfloat16, device=DEV)
    note(f"[gpu] delta step: slots of {b} rows, some padding, some repeated")
    ssd.delta_step(state=state, y=y, state_slots=torch.tensor(slots, dtype=torch.int32, device=DEV), **one)
    first = {}
    for r, k in enumerate(slots):
        if 0 <= k < pool:
            first.setdefault(k, r)
    rows = sorted(first.values())
    dead = [r for r in range(b) if r not in set(rows)]
    s.init = torch.zeros((b, H, P, N))
    for k, r in first.items():
        s.init[r] = before[k]
    yr, yb, hr, hb = s.reference()
    within(y[rows], yr[rows, 0], yb[rows, 0], "y")
    assert (y[dead] == 3.0).all()
    within(state[[slots[r] for r in rows]], hr[rows], hb[rows], "state")
    kept = [k for k in range(pool) if k not in first]
    assert torch.equal(state[kept].cpu(), before[kept])


def test_steps_continue_a_prompt():
    L, more = 70, 6
    s = Delta(2, L + more, 2, 64, 64, io="bf16", dt="bf16", seed=11)
    kw, h0, _ = s.to(DEV)
    note("[gpu] delta rule over a prompt, then steps")
    part = {k: (v[:, :L] if k in TOKENS else v) for k, v in kw.items()}
    ys = [ssd.delta_rule(init_state=h0, final_state=h0, **part)[0]]
    for t in range(L, L + more):
        one = {k: (v[:, t] if k in TOKENS else v) for k, v in kw.items()}
        ys.append(ssd.delta_step(state=h0, **one)[:, None])
    yr, yb, hr, hb = s.reference()
    within(torch.cat(ys, 1), yr, 2 * yb, "y")
    within(h0, hr, 2 * hb, "state")
