"""GPU tests of the gated delta rule over packs of uneven sequences, whose short ones
go token after token and whose long ones in blocks."""

import random

import pytest
import torch

import mamba_ssd_scan_fwd_amd as ssd
from delta_testutil import Delta, near, within
from ssd_testutil import note

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOKENS = ("x", "dt", "B", "C", "beta")


def apart(s, S):
    """Whether the call's sequences go each in its own form: its workspace holds
    records of fewer blocks than all sequences would have."""
    d = ssd.DeltaDesc(batch=1, seqlen=s.L, nheads=s.H, headdim=s.P, dstate=s.N, ngroups=s.G, io_dtype=int(s.io == torch.bfloat16),
                      scale=1.0)
    return 0 < ssd.delta_rule_workspace_bytes(d, S) < (s.L // 64 + S) * s.H * (18944 if s.io == torch.bfloat16 else 37376)


SHAPES = [("fp32", 2, 64, 64, False), ("fp32", 3, 33, 90, True), ("bf16", 4, 64, 64, False), ("bf16", 3, 96, 64, False), ("bf16", 4, 32, 128, False),
          ("bf16", 5, 20, 61, True), ("bf16", 2, 24, 200, False)]
PACKS = [[1] * 200 + [900] + [1] * 200, [900] + [2] * 300, [0, 0] + [3] * 300 + [500], [4] * 300,
         [1] * 150 + [190, 0, 191, 400] + [2] * 200 + [64, 65, 128, 0, 250] + [1] * 200]


@pytest.mark.parametrize("lens", PACKS)
@pytest.mark.parametrize("io,H,P,N,views", SHAPES)
def test_short_and_long_sequences_of_a_pack(io, H, P, N, views, lens):
    s = Delta(1, sum(lens), H, P, N, 1, io, io, views=views, lens=lens, seed=N + len(lens))
    kw, h0, cu = s.to(DEV)
    note(f"[gpu] delta rule, uneven pack: {io} H={H} P={P} N={N}, {len(lens)} sequences of {sum(lens)} tokens, apart {apart(s, len(lens))}")
    y, h = ssd.delta_rule_varlen(cu_seqlens=cu, init_states=h0, **kw)
    yr, yb, hr, hb = s.reference()
    within(y, yr, yb, "y")
    within(h, hr, hb, "final_states")
    near(h, hr, "final_states")
    # each sequence's states in place, and the same bits
    again, _ = ssd.delta_rule_varlen(cu_seqlens=cu, init_states=h0, final_states=h0, **kw)
    assert torch.equal(y, again) and torch.equal(h, h0)


def test_these_packs_take_either_form():
    some = [apart(Delta(1, sum(p), H, P, N, io=io, init=False, lens=p), len(p)) for io, H, P, N, _ in SHAPES for p in PACKS]
    assert sum(some) >= len(some) // 2
    # without a call for it no sequence is told apart
    assert not apart(Delta(1, 2000, 8, 64, 64, lens=[1000, 1000]), 2)


@pytest.mark.parametrize("io", ["fp32", "bf16"])
def test_what_lies_outside_an_uneven_pack_is_left(io):
    lens = [1] * 200 + [600] + [2] * 200
    T = sum(lens)
    s = Delta(1, T + 30, 4, 48, 64, 1, io, io, lens=lens, seed=3)
    kw, h0, cu = s.to(DEV)
    cu = cu + 10
    for k in TOKENS:
        kw[k] = torch.roll(kw[k], 10, 1)
        kw[k][:, :10] = kw[k][:, T + 10:] = float("nan")
    assert apart(s, len(lens))
    y = torch.full((1, T + 30, 4, 48), 7.0, device=DEV, dtype=s.io)
    note(f"[gpu] delta rule, uneven pack: tokens before and behind the sequences {io}")
    _, h = ssd.delta_rule_varlen(cu_seqlens=cu, init_states=h0, y=y, **kw)
    yr, yb, hr, hb = s.reference()
    within(y[:, 10:T + 10], yr[:, :T], yb[:, :T], "y")
    assert (y[:, :10] == 7.0).all() and (y[:, T + 10:] == 7.0).all()
    within(h, hr, hb, "final_states")


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("io,P", [("fp32", 16), ("bf16", 16), ("bf16", 9)])
def test_offsets_of_any_kind_stay_inside(io, P, seed):
    T, S, N = 1000, 400, 32
    r = random.Random(seed)
    cu = [r.choice([0, T, T, r.randrange(-50, T + 50), 1 << 30]) for _ in range(S + 1)] if seed else [0, T] * (S // 2) + [0]
    s = Delta(1, T, 2, P, N, 1, io, "fp32", init=False, seed=12)
    kw, _, _ = s.to(DEV)
    assert apart(s, S)
    y = torch.full((1, T + 64, 2, P), 7.0, device=DEV, dtype=s.io)
    h = torch.full((S + 2, 2, P, N), 5.0, device=DEV)
    d = ssd.DeltaDesc(batch=1, seqlen=T, nheads=2, headdim=P, dstate=N, ngroups=1, io_dtype=int(io == "bf16"), scale=1.0)
    need = ssd.delta_rule_workspace_bytes(d, S)
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device=DEV)
    note(f"[gpu] delta rule, uneven pack: offsets that do not rise, seed {seed} {io}")
    ssd.delta_rule_varlen(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV), y=y[:, :T], final_states=h[1:S + 1], workspace=ws, **kw)
    assert (y[:, T:] == 7.0).all() and (h[0] == 5.0).all() and (h[S + 1] == 5.0).all() and (ws[need:] == 255).all()


def test_many_sequences_are_gone_through():
    """More offsets than one turn of the search, long sequences in its first, last and a middle one."""
    lens = [1] * 9000
    for i in (0, 4095, 4096, 8191, 8999):
        lens[i] = 500 + i % 7
    s = Delta(1, sum(lens), 1, 16, 16, 1, "bf16", "bf16", init=False, lens=lens, seed=5)
    assert apart(s, len(lens))
    kw, _, cu = s.to(DEV)
    note("[gpu] delta rule, uneven pack: 9000 sequences")
    y, h = ssd.delta_rule_varlen(cu_seqlens=cu, **kw)
    yr, yb, hr, hb = s.reference()
    within(y, yr, yb, "y")
    within(h, hr, hb, "final_states")


def test_uneven_packs_in_a_graph_follow_the_offsets():
    """The lengths are read as the graph runs: other offsets, other sequences in blocks."""
    lens = [1] * 200 + [700] + [1] * 200
    s = Delta(1, sum(lens), 4, 64, 64, 1, "bf16", "bf16", lens=lens, seed=6)
    kw, h0, cu = s.to(DEV)
    assert apart(s, len(lens))
    other = torch.flip(cu[-1] - cu, [0]).contiguous()
    other[1:100] += 300
    run = lambda c: ssd.delta_rule_varlen(cu_seqlens=c, init_states=h0, **kw)  # noqa: E731
    wants = [run(cu), run(other)]
    now = cu.clone()
    note("[gpu] delta rule, uneven pack: a graph")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run(now)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = run(now)
    for turn in (0, 1, 0, 1):
        now.copy_([cu, other][turn])
        y.zero_(), h.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, wants[turn][0]) and torch.equal(h, wants[turn][1])
        eager = run([cu, other][turn])
        assert torch.equal(y, eager[0]) and torch.equal(h, eager[1])
