"""GPU tests of the gated delta rule and the norm of heads as a layer uses them:
together, on streams, from graphs, through the C ABI, at far offsets."""

import ctypes

import numpy as np
import pytest
import torch

import mamba_ssd_scan_fwd_amd as ssd
from delta_testutil import Delta, within
from ssd_testutil import note

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOKENS = ("x", "dt", "B", "C", "beta")


def off(a, b):
    a, b = a.double(), b.double()
    return float((a - b).norm() / b.norm())


# ---- the operators together ---------------------------------------------------------


class Layer:
    """conv1d_split -> head_norm -> delta_rule -> group_norm with a gate."""

    def __init__(self, seed, H=8, P=64, G=4, N=64, K=4):
        g = torch.Generator().manual_seed(seed)
        self.H, self.P, self.G, self.N, self.K = H, P, G, N, K
        self.E, self.CH = H * P, H * P + 2 * G * N
        self.heads = dict(nheads=H, headdim=P, ngroups=G, dstate=N)
        self.w, self.b = torch.randn((self.CH, K), generator=g).to(DEV) * 0.5, torch.randn(self.CH, generator=g).to(DEV) * 0.1
        self.A, self.nw = -torch.exp(torch.rand(H, generator=g) * 2).to(DEV), (1 + 0.2 * torch.randn(P, generator=g)).to(DEV)
        self.rule = dict(scale=N ** -0.5, beta_sigmoid=True, dt_pre=dict(bias=torch.full((H,), -3.0, device=DEV), softplus=True))
        # the last three of a row: a head's step, beta and gate
        self.width = self.CH + 2 * H + self.E
        self.freq = torch.exp(-torch.arange(N // 2) * (9.0 / (N // 2))).to(DEV)
        self.g = g

    def draw(self, *lead):
        return torch.randn((*lead, self.width), generator=self.g).to(torch.bfloat16).to(DEV)

    def parts(self, row):
        return row[..., :self.CH].contiguous(), row[..., self.CH:self.CH + self.H], row[..., self.CH + self.H:self.CH + 2 * self.H], \
            row[..., self.CH + 2 * self.H:]

    def qk(self, C, B, pos):
        return ssd.head_norm(C, B, positions=pos, inv_freq=self.freq, l2=True)

    def out(self, y, z):
        return ssd.group_norm(y.flatten(-2), None, None, z, ngroups=self.H, center=False, gate_first=False)

    def prompt(self, row, pos):
        xbc, dt, beta, z = self.parts(row)
        conv = torch.empty((row.shape[0], self.CH, self.K - 1), device=DEV)
        x, B, C = ssd.conv1d_split(xbc, self.w, self.b, conv_state_out=conv, **self.heads)
        q, k = self.qk(C, B, pos)
        y, h = ssd.delta_rule(x, dt, self.A, k, q, beta, **self.rule)
        return self.out(y, z), conv, h

    def packed(self, row, pos, cu):
        xbc, dt, beta, z = self.parts(row)
        conv = torch.empty((len(cu) - 1, self.CH, self.K - 1), device=DEV)
        x, B, C = ssd.conv1d_split_varlen(xbc, self.w, self.b, cu_seqlens=cu, conv_states_out=conv, **self.heads)
        q, k = self.qk(C, B, pos)
        y, h = ssd.delta_rule_varlen(x, dt, self.A, k, q, beta, cu_seqlens=cu, **self.rule)
        return self.out(y, z), conv, h

    def token(self, row, pos, conv, h, slots):
        xbc, dt, beta, z = self.parts(row)
        x, B, C = ssd.conv1d_split_step(xbc, self.w, self.b, conv, state_slots=slots, **self.heads)
        q, k = self.qk(C, B, pos)
        y = ssd.delta_step(x, dt, self.A, k, q, beta, h, state_slots=slots, **self.rule)
        return self.out(y, z)


def positions(*lead):
    return torch.arange(lead[-1], dtype=torch.int32, device=DEV).expand(lead).contiguous()


# Both sides store the convolution, the keys and queries, y and the output in bf16 from
# fp32 values that differ in their last bits: now and then a step of bf16, 2^-7 of the
# value, in each. The prompts round the states, scores and solutions of y's products to bf16, a half
# step of 2^-8 each. A state sees the first kind alone.
Y_OFF, H_OFF = 4 * 2.0 ** -8, 2.0 ** -7


@pytest.mark.parametrize("L", [9, 100])
def test_layer_prompt_then_tokens(L):
    b, new = 3, 5
    m, T = Layer(21), L + new
    row, pos = m.draw(b, T), positions(b, T)
    note(f"[gpu] delta layer: prompts of {L}, then tokens")
    whole, conv_end, h_end = m.prompt(row, pos)
    first, conv, h = m.prompt(row[:, :L], pos[:, :L].contiguous())
    pool_c, pool_h = torch.zeros((6, *conv.shape[1:]), device=DEV), torch.zeros((6, *h.shape[1:]), device=DEV)
    slots = torch.tensor([4, 1, 5], dtype=torch.int32, device=DEV)
    pool_c[slots.long()], pool_h[slots.long()] = conv, h
    outs = [first] + [m.token(row[:, t], pos[:, t].contiguous(), pool_c, pool_h, slots)[:, None] for t in range(L, T)]
    assert torch.equal(pool_c[slots.long()], conv_end)
    assert off(torch.cat(outs, 1)[:, L:], whole[:, L:]) < Y_OFF and off(torch.cat(outs, 1), whole) < Y_OFF
    assert off(pool_h[slots.long()], h_end) < H_OFF
    assert not pool_h[[0, 2, 3]].any() and not pool_c[[0, 2, 3]].any()


def test_layer_packed_prompts_then_tokens():
    lens, new = [20, 133, 1, 70], 3
    m = Layer(22)
    rows = [m.draw(n + new) for n in lens]
    note("[gpu] delta layer: packed prompts, then tokens")

    def packed(extra):
        ln = [n + extra for n in lens]
        cu = torch.tensor([0] + list(np.cumsum(ln)), dtype=torch.int32, device=DEV)
        o, conv, h = m.packed(torch.cat([r[:n] for r, n in zip(rows, ln)])[None], torch.cat([positions(n) for n in ln])[None], cu)
        return o[0].split(ln), conv, h

    whole, conv_end, h_end = packed(new)
    part, conv, h = packed(0)
    got = [[p] for p in part]
    for t in range(new):
        row = torch.stack([r[n + t] for r, n in zip(rows, lens)])
        pos = torch.tensor([n + t for n in lens], dtype=torch.int32, device=DEV)
        o = m.token(row, pos, conv, h, None)
        for s in range(len(lens)):
            got[s].append(o[s:s + 1])
    assert torch.equal(conv, conv_end)
    for s in range(len(lens)):
        assert off(torch.cat(got[s]), whole[s]) < Y_OFF
    assert off(h, h_end) < H_OFF


# ---- streams and graphs --------------------------------------------------------------


def calls(seed):
    """Every kernel once on fixed buffers: (name, inputs, call)."""
    out = []

    def rule(name, *a, **kw):
        s = Delta(*a, seed=seed, **kw)
        k, h0, cu = s.to(DEV)
        if cu is None:
            out.append((name, lambda **on: list(ssd.delta_rule(init_state=h0, **k, **on))))
        else:
            # rows of no sequence are left as they are
            out.append((name, lambda **on: list(ssd.delta_rule_varlen(cu_seqlens=cu, init_states=h0, **k, **on))))
        return k, h0

    k, h0 = rule("walk", 2, 9, 2, 20, 24, 1, "bf16", "bf16")
    rule("blocks", 2, 200, 4, 64, 64, 2, "bf16", "bf16")
    rule("blocks fp32", 2, 150, 4, 64, 64, 2, "fp32", "fp32")
    rule("packed", 1, 373, 4, 128, 128, 1, "bf16", "bf16", lens=[100, 0, 200, 73])
    rule("segments", 1, 1100, 1, 64, 64, 1, "bf16", "bf16")
    one = {n: (v[:, 4] if n in TOKENS else v) for n, v in k.items()}

    def step(**on):
        st = h0.clone()
        torch.cuda.current_stream().synchronize() if on else None
        y = ssd.delta_step(state=st, **one, **on)
        return [y, st]

    g = torch.Generator().manual_seed(seed)
    q, kk = torch.randn((2, 70, 6, 128), generator=g).to(DEV), torch.randn((2, 70, 2, 128), generator=g).to(DEV)
    pos, freq = positions(2, 70), torch.rand(64, generator=g).to(DEV)
    out.append(("step", step))
    out.append(("head norm", lambda **on: list(ssd.head_norm(q, kk, positions=pos, inv_freq=freq, **on))))
    return out


def run_all(cs, **on):
    return [t for _, f in cs for t in f(**on)]


def same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_stream_argument_and_current_stream():
    cs = calls(31)
    want = run_all(cs)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    note("[gpu] delta rule, step, head norm on a side stream")
    with torch.cuda.stream(side):
        got = run_all(cs)
    side.synchronize()
    assert same(want, got)
    side.wait_stream(torch.cuda.current_stream())
    for name, f in cs:
        if name == "step":
            continue
        a, b = f(), f(stream=side)
        side.synchronize()
        assert same(a, b), name
    step = dict(cs)["step"]
    a, b = step(), step(stream=side)
    torch.cuda.synchronize()
    assert same(a, b)


def test_two_streams_at_once():
    runs = [calls(32), calls(33)]
    wants = [run_all(r) for r in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    note("[gpu] delta rule: two streams at once")
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for r, st, g in zip(runs, streams, got):
            with torch.cuda.stream(st):
                g.append(run_all(r))
    torch.cuda.synchronize()
    for want, outs in zip(wants, got):
        assert all(same(want, o) for o in outs)


def test_two_graphs_replayed_at_once():
    """Each graph has its own workspaces: replays on two streams, with eager
    calls between, all give the same bits."""
    runs = [calls(34), calls(35)]
    wants = [run_all(r) for r in runs]
    note("[gpu] delta rule: two graphs at once")
    torch.cuda.synchronize()
    graphs, outs = [], []
    for r in runs:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            run_all(r)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(run_all(r))
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(4):
        for out in outs:
            for o in out:
                o.zero_()
        torch.cuda.synchronize()
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        eager = [run_all(r) for r in runs]
        torch.cuda.synchronize()
        for want, out, e in zip(wants, outs, eager):
            assert same(want, out) and same(want, e)


def test_a_stream_given_inside_a_capture():
    s = Delta(1, 500, 4, 64, 64, 2, "bf16", "bf16", seed=67)
    kw, h0, _ = s.to(DEV)
    want = list(ssd.delta_rule(init_state=h0, **kw))
    norm = ssd.head_norm(want[0], l2=True)
    note("[gpu] delta rule: stream argument inside a capture")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        y, h = ssd.delta_rule(init_state=h0, stream=side, **kw)
        here.wait_stream(side)
        o = ssd.head_norm(y, l2=True)
    for _ in range(3):
        for t in (y, h, o):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same([*want, norm], [y, h, o])


def test_memory_of_a_call_on_another_stream_is_kept_until_it_ran():
    """The call waits behind a sleep on its stream; its inputs are dropped, and
    blocks of their sizes overwritten on the caller's stream, before it runs."""
    s = Delta(1, 2000, 4, 64, 64, 2, "bf16", "bf16", seed=36)
    kw, h0, _ = s.to(DEV)
    want = list(ssd.delta_rule(init_state=h0, **kw))
    note("[gpu] delta rule: memory in use on two streams")
    here, side = torch.cuda.current_stream(), torch.cuda.Stream()
    mine = dict(kw, **{k: kw[k].clone() for k in TOKENS})
    start = h0.clone()
    side.wait_stream(here)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = list(ssd.delta_rule(init_state=start, stream=side, **mine))
    del mine, start
    junk = [torch.full_like(kw[k], float("nan")) for k in TOKENS for _ in range(2)] + [torch.full_like(h0, float("nan"))]
    here.wait_stream(side)
    assert same(want, got) and junk


# ---- the C ABI -----------------------------------------------------------------------


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("L,lens", [(300, None), (1500, None), (400, [100, 0, 300])])
def test_workspace_of_the_c_abi(own, L, lens):
    """A null workspace is allocated and freed in stream order; one of exactly
    the size asked for is enough, and nothing behind it is written."""
    s = Delta(1, L, 2, 64, 128, 1, "bf16", "bf16", lens=lens, seed=65)
    kw, h0, cu = s.to(DEV)
    S = 0 if lens is None else len(lens)
    want, hw = ssd.delta_rule_varlen(cu_seqlens=cu, init_states=h0, **kw) if S else ssd.delta_rule(init_state=h0, **kw)
    pre = kw["dt_pre"]
    d = ssd.DeltaDesc(batch=1, seqlen=L, nheads=2, headdim=64, dstate=128, ngroups=1, io_dtype=1, dt_dtype=1, beta_sigmoid=1,
                      scale=kw["scale"], dt_bias=pre["bias"].data_ptr(), dt_softplus=1, dt_clamp=1, dt_min=1e-3, dt_max=0.3)
    n = ssd.delta_rule_workspace_bytes(d, S)
    assert n > 0
    ws = torch.full((n + 4096,), 255, dtype=torch.uint8, device=DEV)
    y, h = torch.empty_like(want), torch.empty_like(hw)
    note(f"[gpu] delta rule through the C ABI L={L} {lens}, own workspace {own}")
    torch.cuda.synchronize()
    p = [kw[k].data_ptr() for k in ("x", "dt", "A", "B", "C", "beta")] + [t.data_ptr() for t in (h0, y, h)]
    at = [ws.data_ptr() if own else None, n if own else 0, None]
    for _ in range(3):
        if S:
            st = ssd.load_library().ssd_delta_rule_varlen(ctypes.byref(d), cu.data_ptr(), S, *p, *at)
        else:
            st = ssd.load_library().ssd_delta_rule(ctypes.byref(d), *p, *at)
        assert st == 0
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(h, hw)
    assert (ws[n:] == 255).all()


# ---- alignment --------------------------------------------------------------------------


def shifted(t, by=1):
    """t's values, dense, ``by`` elements behind an aligned address."""
    flat = torch.empty(t.numel() + by, dtype=t.dtype, device=DEV)
    flat[by:] = t.flatten()
    return flat[by:].view(t.shape)


@pytest.mark.parametrize("io,L,H,P,N,lens", [("bf16", 150, 2, 64, 64, None), ("bf16", 150, 2, 128, 128, [70, 0, 80]),
                                             ("bf16", 1100, 1, 64, 64, None), ("fp32", 150, 2, 64, 64, None),
                                             ("bf16", 150, 2, 33, 200, None), ("bf16", 9, 2, 20, 24, None), ("fp32", 9, 2, 20, 24, [4, 5])])
def test_arrays_at_odd_addresses(io, L, H, P, N, lens):
    """Outputs, states and parameters need the alignment of their elements alone."""
    s = Delta(1, L, H, P, N, 1, io, io, lens=lens, seed=52)
    kw, h0, cu = s.to(DEV)
    rule = (lambda h, **a: ssd.delta_rule(init_state=h, **a)) if lens is None else \
        (lambda h, final_state=None, **a: ssd.delta_rule_varlen(cu_seqlens=cu, init_states=h, final_states=final_state, **a))
    want = rule(h0, **kw)
    note(f"[gpu] delta rule, step, head norm: odd addresses {io} L={L} P={P} N={N}")
    out = shifted(torch.zeros_like(want[0])), shifted(torch.zeros_like(want[1]))
    odd = dict(kw, A=shifted(kw["A"]), dt_pre=dict(kw["dt_pre"], bias=shifted(kw["dt_pre"]["bias"])))
    got = rule(shifted(h0), y=out[0], final_state=out[1], **odd)
    assert got[0].data_ptr() == out[0].data_ptr() and same(want, got)
    one = {k: (v[:, 0] if k in TOKENS else v) for k, v in kw.items()}
    st, so = h0[:1].clone(), shifted(h0[:1])
    y, yo = ssd.delta_step(state=st, **one), shifted(torch.zeros_like(want[0][:, 0]))
    ssd.delta_step(state=so, y=yo, **one)
    assert torch.equal(y, yo) and torch.equal(st, so)
    q, w, pos, freq = kw["x"], torch.rand(P, device=DEV), positions(1, L), torch.rand(P // 2, device=DEV)
    for pairs in (False, True):
        n = ssd.head_norm(q, q, w, w, positions=pos, inv_freq=freq, pairs=pairs)
        m = shifted(torch.zeros_like(q)), shifted(torch.zeros_like(q))
        ssd.head_norm(shifted(q), q, shifted(w), w, positions=shifted(pos), inv_freq=shifted(freq), pairs=pairs, q_out=m[0], k_out=m[1])
        assert same(n, m)


# ---- far offsets, many heads -----------------------------------------------------------


@pytest.mark.parametrize("io,L", [("bf16", 1100), ("fp32", 1100), ("bf16", 1090)])
def test_rows_far_apart(io, L):
    """Token strides that take the last rows past 2^32 bytes and 2^31 elements."""
    H, P, N = 2, 64, 32
    shift = 3 if L % 4 else 8  # unaligned rows too
    far = (1 << 21) + 24
    s = Delta(1, L, H, P, N, 1, io, io, seed=41)
    kw, h0, _ = s.to(DEV)
    note(f"[gpu] delta rule: rows more than 2^32 bytes apart {io} L={L}")
    base = torch.empty(L * far, dtype=s.io, device=DEV)
    wide, moved, at = base.view(1, L, far), dict(kw), shift
    for k in TOKENS:
        v = kw[k].flatten(2)
        wide[:, :, at:at + v.shape[2]] = v
        part = wide[:, :, at:at + v.shape[2]]
        moved[k] = part if kw[k].dim() == 3 else part.unflatten(2, kw[k].shape[2:])
        at += v.shape[2] + 8
    y, h = ssd.delta_rule(init_state=h0, **moved)
    yr, yb, hr, hb = s.reference(cut=True)
    within(y, yr, yb, "y")
    within(h, hr, hb, "final_state")
    cu = torch.tensor([0, L], dtype=torch.int32, device=DEV)
    yp, hp = ssd.delta_rule_varlen(cu_seqlens=cu, init_states=h0, **moved)
    within(yp, yr, yb, "y packed")
    within(hp, hr, hb, "final_states packed")
    freq, pos = torch.rand(8, device=DEV), positions(1, L)
    for a, b in zip(ssd.head_norm(kw["x"], kw["x"], positions=pos, inv_freq=freq),
                    ssd.head_norm(moved["x"], moved["x"], positions=pos, inv_freq=freq)):
        assert torch.equal(a, b)


def test_short_rows_far_apart():
    """The same token after token, and of single tokens of many rows."""
    b, H, P, N, far = 1100, 1, 16, 5, (1 << 21) + 24
    s = Delta(b, 2, H, P, N, 1, "bf16", "bf16", seed=42)
    kw, h0, _ = s.to(DEV)
    note("[gpu] delta rule and step: rows of the batch more than 2^32 bytes apart")
    wide, moved, at = torch.empty(b * far, dtype=s.io, device=DEV).view(b, far), dict(kw), 3
    for k in TOKENS:
        v = kw[k].reshape(b, -1)
        wide[:, at:at + v.shape[1]] = v
        moved[k] = wide[:, at:at + v.shape[1]].unflatten(1, kw[k].shape[1:])
        at += v.shape[1] + 8
    y, h = ssd.delta_rule(init_state=h0, **moved)
    yr, yb, hr, hb = s.reference()
    within(y, yr, yb, "y")
    within(h, hr, hb, "final_state")
    state = h0.clone()
    for t in range(2):
        one = {k: (v[:, t] if k in TOKENS else v) for k, v in moved.items()}
        within(ssd.delta_step(state=state, **one), yr[:, t], yb[:, t], "y of a step")
    within(state, hr, hb, "state of steps")


def test_slots_behind_two_to_the_31_elements():
    H, P, N = 32, 128, 128
    pool = (1 << 31) // (H * P * N) + 3
    s = Delta(2, 1, H, P, N, 1, "bf16", "bf16", seed=43)
    kw, h0, _ = s.to(DEV)
    one = {k: (v[:, 0] if k in TOKENS else v) for k, v in kw.items()}
    note("[gpu] delta step: a pool of more than 2^31 elements")
    state = torch.zeros((pool, H, P, N), device=DEV)
    slots = torch.tensor([pool - 1, 1], dtype=torch.int32, device=DEV)
    state[slots.long()] = h0
    y = ssd.delta_step(state=state, state_slots=slots, **one)
    yr, yb, hr, hb = s.reference()
    within(y, yr[:, 0], yb[:, 0], "y")
    within(state[slots.long()], hr, hb, "state")
    assert not state[pool - 2].any() and not state[0].any()


def test_outputs_of_more_than_two_to_the_31_elements():
    """The second of two rows lies behind 2^31 elements in part: against calls of
    that row alone, which may cut it in other segments (nine roundings of 2^-16 of a
    state's terms, and y's operands of 2^-8, on either side), batched and packed."""
    b, L, H, P, N = 2, 540_001, 16, 128, 32
    g = torch.Generator(device=DEV).manual_seed(66)
    draw = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    x, dt, beta = draw(b, L, H, P), draw(b, L, H), draw(b, L, H)
    note("[gpu] delta rule and head norm: outputs of more than 2^31 elements")
    C, B = ssd.head_norm(draw(b, L, 1, N), draw(b, L, 1, N), l2=True)
    A = -torch.exp(torch.rand((H,), generator=g, device=DEV))
    assert x.numel() > 1 << 31
    kw = dict(beta_sigmoid=True, dt_pre=dict(bias=torch.full((H,), -3.0, device=DEV), softplus=True))
    y, h = ssd.delta_rule(x, dt, A, B, C, beta, **kw)
    alone, ha = ssd.delta_rule(x[1:], dt[1:], A, B[1:], C[1:], beta[1:], **kw)
    assert off(h[1:], ha) < 18 * 2.0 ** -16
    for t in range(0, L, 60_000):
        assert off(y[1:, t:t + 60_000], alone[:, t:t + 60_000]) < 4 * 2.0 ** -8
    del alone
    flat = lambda t: t.flatten(0, 1)[None]  # noqa: E731
    cu = torch.tensor([0, L, 2 * L], dtype=torch.int32, device=DEV)
    yp, hp = ssd.delta_rule_varlen(flat(x), flat(dt), A, flat(B), flat(C), flat(beta), cu_seqlens=cu, **kw)
    assert off(hp, h) < 18 * 2.0 ** -16
    for t in range(0, L, 60_000):
        assert off(yp.view_as(y)[:, t:t + 60_000], y[:, t:t + 60_000]) < 4 * 2.0 ** -8
    del yp, y
    freq, pos = torch.rand(64, device=DEV), positions(b, L)
    q = ssd.head_norm(x, positions=pos, inv_freq=freq)
    for t in (0, L - 200):
        part = slice(t, t + 200)
        assert torch.equal(q[:, part], ssd.head_norm(x[:, part], positions=pos[:, part].contiguous(), inv_freq=freq))


@pytest.mark.parametrize("P,N,L", [(1, 3, 3), (16, 8, 70)])
def test_as_many_heads_as_are_allowed(P, N, L):
    H, some = 65535, [0, 1, 40000, 65534]
    g = torch.Generator(device=DEV).manual_seed(67)
    draw = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    x, dt, beta, A = draw(1, L, H, P), draw(1, L, H), draw(1, L, H), -torch.rand((H,), generator=g, device=DEV)
    C, B = ssd.head_norm(draw(1, L, 1, N), draw(1, L, 1, N), l2=True)
    note(f"[gpu] delta rule: {H} heads of {P} x {N}")
    kw = dict(beta_sigmoid=True, dt_pre=dict(softplus=True))
    y, h = ssd.delta_rule(x, dt, A, B, C, beta, **kw)
    few = lambda t: t[:, :, some].contiguous()  # noqa: E731
    ya, ha = ssd.delta_rule(few(x), few(dt), A[some], B, C, few(beta), **kw)
    # fp32 both: three-term operands in blocks, 2^-22 each at the most
    assert off(few(y), ya) < 2.0 ** -18 and off(h[:, some], ha) < 2.0 ** -18
    s1, s2 = h.clone(), h[:, some].contiguous()
    y1 = ssd.delta_step(x[:, 0], dt[:, 0], A, B[:, 0], C[:, 0], beta[:, 0], s1, **kw)
    y2 = ssd.delta_step(few(x)[:, 0], few(dt)[:, 0], A[some], B[:, 0], C[:, 0], few(beta)[:, 0], s2, **kw)
    assert torch.equal(y1[:, some], y2) and torch.equal(s1[:, some], s2)


def test_head_norm_of_large_inputs():
    """Inputs beyond the memory-side cache, which are read past it."""
    L, Hq, Hk, D = 40_000, 32, 8, 128
    g = torch.Generator(device=DEV).manual_seed(68)
    qk = torch.randn((L, (Hq + Hk) * D + 8), generator=g, device=DEV, dtype=torch.bfloat16)
    q, k = qk[:, :Hq * D].unflatten(1, (Hq, D)), qk[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    w, freq, pos = torch.rand((2, D), generator=g, device=DEV), torch.rand((D // 2,), generator=g, device=DEV), positions(L)
    note("[gpu] head norm of 400 MB")
    got = ssd.head_norm(q, k, w[0], w[1], positions=pos, inv_freq=freq)
    parts = [ssd.head_norm(q[t:t + 5000], k[t:t + 5000], w[0], w[1], positions=pos[t:t + 5000], inv_freq=freq)
             for t in range(0, L, 5000)]
    assert torch.equal(got[0], torch.cat([p[0] for p in parts])) and torch.equal(got[1], torch.cat([p[1] for p in parts]))


# ---- unusual values --------------------------------------------------------------------


@pytest.mark.parametrize("io,L,H,P,N", [("bf16", 9, 2, 20, 24), ("fp32", 9, 2, 20, 24), ("bf16", 200, 2, 64, 64),
                                        ("fp32", 200, 2, 64, 64), ("bf16", 200, 2, 33, 200)])
def test_steps_of_nan_and_betas_without_end(io, L, H, P, N):
    """dt is clamped to its limits, infinities too; a NaN stays NaN and takes its
    head from its token on, and no other. A beta of infinity is a whole one."""
    s = Delta(1, L, H, P, N, 1, io, io, seed=49)
    kw, h0, _ = s.to(DEV)
    want, hw = ssd.delta_rule(init_state=h0, **kw)
    note(f"[gpu] delta rule and step: NaN steps, betas of infinity {io} L={L}")
    t = L - 5
    dt = kw["dt"].clone()
    dt[0, t, 1] = float("nan")
    y, h = ssd.delta_rule(init_state=h0, **dict(kw, dt=dt))
    assert torch.isnan(y[0, t:, 1]).all() and torch.isnan(h[0, 1]).all()
    assert torch.equal(y[:, :, 0], want[:, :, 0]) and torch.equal(h[:, 0], hw[:, 0])
    assert torch.equal(y[0, :max(0, t - 64), 1], want[0, :max(0, t - 64), 1])
    one = {k: (v[:, t] if k in TOKENS else v) for k, v in dict(kw, dt=dt).items()}
    state = h0.clone()
    y1 = ssd.delta_step(state=state, **one)
    assert torch.isnan(y1[0, 1]).all() and torch.isnan(state[0, 1]).all()
    assert torch.isfinite(y1[0, 0]).all() and torch.isfinite(state[0, 0]).all()
    ends = []
    for big in (float("inf"), 1e30):
        dt, beta = kw["dt"].clone(), kw["beta"].clone()
        dt[0, t, 0], dt[0, t - 1, 0], beta[0, t, 1], beta[0, t - 2, 1] = big, -big, big, -big
        a = dict(kw, dt=dt, beta=beta)
        one = {k: (v[:, t] if k in TOKENS else v) for k, v in a.items()}
        state = h0.clone()
        ends.append([*ssd.delta_rule(init_state=h0, **a), ssd.delta_step(state=state, **one), state])
        assert all(torch.isfinite(e).all() for e in ends[-1])
    assert same(*ends)


def test_dead_weights_of_the_state_do_not_grow():
    """Keys of length one and betas of 2: each token turns the state over in its
    key's direction, and the state keeps its length (A = 0, x = 0)."""
    L, P, N = 256, 64, 64
    g = torch.Generator().manual_seed(50)
    B = torch.randn((1, L, 1, N), generator=g)
    B = (B / B.norm(dim=-1, keepdim=True)).to(DEV)
    h0 = torch.randn((1, 1, P, N), generator=g).to(DEV)
    zero = torch.zeros((1, L, 1), device=DEV)
    note("[gpu] delta rule: reflections")
    y, h = ssd.delta_rule(torch.zeros((1, L, 1, P), device=DEV), zero, torch.zeros(1, device=DEV), B, B, zero + 2.0, h0)
    # each of 256 reflections rounds sums of 64 terms in fp32, in blocks of 64 of three-term operands
    assert abs(float(h.double().norm() / h0.double().norm()) - 1) < 256 * 64 * 2.0 ** -24
    assert torch.isfinite(y).all()
