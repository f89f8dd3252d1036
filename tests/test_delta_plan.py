"""The plan of a call of the gated delta rule, on the CPU: which form a call takes,
seen by the workspace it asks for, and calls that no form can launch."""

import pytest

from test_delta_host import OK, SHAPE, BASE, NAMES, bytes_of, call, rule

FAR = {n: BASE + (i << 40) for i, n in enumerate(NAMES)}
SMALL = dict(nheads=32, ngroups=1, headdim=32, dstate=64)


@pytest.mark.parametrize("io", [0, 1])
def test_blocks_with_too_many_workgroups_go_token_after_token(io):
    """64 tokens go in blocks, unless the walk over blocks would have 2^32 threads:
    2^23 workgroups of 512, where the walk token after token has as many of 256."""
    kw = dict(SMALL, seqlen=64, io_dtype=io, dt_dtype=io)
    st, need = bytes_of(batch=1 << 10, **kw)
    assert st == OK and need > 0
    assert bytes_of(batch=1 << 18, **kw) == (OK, 0)


@pytest.mark.parametrize("L", [4, 16, 64])
@pytest.mark.parametrize("S", [None, 1 << 19])
def test_calls_that_no_form_can_launch_are_refused_by_the_query_too(L, S):
    kw = dict(SMALL, batch=1 if S else 1 << 19, seqlen=(L << 19) if S else L)
    assert bytes_of(S=S or 0, **kw)[0] == SHAPE
    assert call(rule(**kw), S=S, **FAR) == SHAPE


@pytest.mark.parametrize("P,N", [(8, 8), (16, 16), (32, 32), (64, 16)])
@pytest.mark.parametrize("batch,L", [(16, 16), (4096, 8), (16384, 8)])
def test_records_are_paid_for(P, N, batch, L):
    """A block's record of 18.5 KB for a few tokens of a small state: token after token
    takes half the time, and none of the workspace."""
    kw = dict(batch=batch, seqlen=L, nheads=32, ngroups=1, headdim=P, dstate=N)
    assert bytes_of(**kw) == (OK, 0)
    assert bytes_of(**dict(kw, seqlen=128, batch=16))[1] > 0


@pytest.mark.parametrize("io,H,P,N,S,T", [(0, 8, 64, 64, 256, 4096 + 255), (0, 2, 32, 32, 1001, 8192 + 1000), (0, 4, 64, 64, 256, 2048 + 255),
                                          (1, 4, 64, 64, 256, 512 + 255), (1, 16, 60, 61, 256, 512 + 255)])
def test_a_pack_that_may_hold_a_long_sequence_has_blocks_for_it(io, H, P, N, S, T):
    """The host knows the mean length alone. By it alone these go token after token,
    where a sequence of nearly all tokens takes 4 to 18 times what it does in blocks."""
    kw = dict(nheads=H, headdim=P, dstate=N, ngroups=H, io_dtype=io, dt_dtype=io)
    st, need = bytes_of(S=S, batch=1, seqlen=T, **kw)
    assert st == OK and need >= (T // 64) * H * (18944 if io else 37376)
    # with fewer tokens than a long sequence has, token after token and no workspace
    assert bytes_of(S=30, batch=1, seqlen=30, **kw) == (OK, 0)
