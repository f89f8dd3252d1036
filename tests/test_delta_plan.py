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
