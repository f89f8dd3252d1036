"""Refusals of the layer operators, on the CPU: the C ABI with fake device
addresses (no call reaches a kernel) and the binding's own checks."""

import ctypes
import os

import pytest
import torch

import mamba_ssd_scan_fwd_amd as ssd
from mamba_ssd_scan_fwd_amd.binding import Conv1dDesc, GroupNormDesc, SelectiveDesc

OK, NULLP, SHAPE, UNSUP, ALIGN, WS, ALIAS = range(7)
BASE = 0x7F0000000000  # fake device addresses: never dereferenced


def lib():
    if not os.path.exists(ssd.lib_path()):
        pytest.skip("libssd.so not built (python -m mamba_ssd_scan_fwd_amd.build)")
    return ssd.load_library()


class Stride(tuple):
    """(token, batch) of a descriptor's stride."""

    def __new__(cls, token, batch):
        return super().__new__(cls, (token, batch))


def fill(d, kw):
    for k, v in kw.items():
        if isinstance(v, Stride):
            setattr(d, k.replace("stride", "token"), v[0])
            setattr(d, k.replace("stride", "batch"), v[1])
        else:
            setattr(d, k, v)
    return d


def sel(**kw):
    return fill(SelectiveDesc(batch=2, seqlen=100, channels=64, dstate=16, ngroups=2, io_dtype=1, dt_dtype=1), kw)


def conv(**kw):
    widths = kw.pop("out_channels", (64, 0, 0))
    d = fill(Conv1dDesc(batch=2, seqlen=100, channels=64, conv_width=4, silu=1, io_dtype=1), kw)
    d.out0, d.out1, d.out2 = widths
    return d


def norm(**kw):
    return fill(GroupNormDesc(batch=2, rows=100, channels=64, ngroups=2, io_dtype=1, eps=1e-5), kw)


def pointers(*names):
    return {n: BASE + (i << 32) for i, n in enumerate(names)}


def scan(d, ws_bytes=1 << 30, S=None, **over):
    p = pointers("x", "dt", "A", "B", "C", "D", "z", "h0", "y", "hT", "ws", "cu")
    p.update(over)
    mid = [p[k] for k in ("x", "dt", "A", "B", "C", "D", "z", "h0", "y", "hT", "ws")]
    if S is None:
        return lib().ssd_selective_scan(ctypes.byref(d), *mid, ws_bytes, None)
    return lib().ssd_selective_scan_varlen(ctypes.byref(d), p["cu"], S, *mid, ws_bytes, None)


def step(d, n=8, **over):
    p = pointers("x", "dt", "A", "B", "C", "D", "z", "state", "slots", "y")
    p.update(over)
    return lib().ssd_selective_step(ctypes.byref(d), *[p[k] for k in ("x", "dt", "A", "B", "C", "D", "z", "state", "slots")],
                                    n, p["y"], None)


def conv_call(d, cu=None, S=0, **over):
    p = pointers("x", "w", "b", "in", "out_st", "o0")
    p.update(o1=None, o2=None)
    p.update(over)
    return lib().ssd_conv1d(ctypes.byref(d), cu, S, *[p[k] for k in ("x", "w", "b", "in", "out_st", "o0", "o1", "o2")], None)


def conv_step(d, n=8, **over):
    p = pointers("x", "w", "b", "state", "slots", "o0")
    p.update(o1=None, o2=None)
    p.update(over)
    return lib().ssd_conv1d_step(ctypes.byref(d), *[p[k] for k in ("x", "w", "b", "state", "slots")], n,
                                 *[p[k] for k in ("o0", "o1", "o2")], None)


def norm_call(d, **over):
    p = pointers("x", "w", "b", "z", "out")
    p.update(over)
    return lib().ssd_group_norm(ctypes.byref(d), *[p[k] for k in ("x", "w", "b", "z", "out")], None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), SHAPE), (dict(seqlen=0), SHAPE), (dict(channels=0), SHAPE), (dict(dstate=0), SHAPE),
    (dict(ngroups=0), SHAPE), (dict(ngroups=3), SHAPE), (dict(batch=70000), SHAPE), (dict(seqlen=1 << 31), SHAPE),
    (dict(channels=(1 << 20) + 2), SHAPE), (dict(dstate=257), UNSUP), (dict(io_dtype=2), UNSUP), (dict(dt_dtype=5), UNSUP),
    (dict(io_dtype=0, dt_dtype=1), UNSUP), (dict(dt_clamp=1, dt_min=2.0, dt_max=1.0), SHAPE),
    (dict(dt_clamp=1, dt_min=float("nan"), dt_max=1.0), SHAPE), (dict(dt_bias=BASE + 2), ALIGN),
    (dict(x_stride=Stride(63, 0)), SHAPE), (dict(x_stride=Stride(64, 63)), SHAPE), (dict(B_stride=Stride(31, 0)), SHAPE),
    (dict(z_stride=Stride(1 << 22, 0)), SHAPE), (dict(dt_stride=Stride(64, -5)), SHAPE),
    (dict(C_stride=Stride(-32, 0)), SHAPE), (dict(x_stride=Stride(64, 1 << 41)), SHAPE),
])
def test_selective_scan_refuses_descriptors(kw, code):
    assert scan(sel(**kw)) == code
    assert scan(sel(**dict(kw, batch=kw.get("batch", 1))), S=3) == code
    n = ctypes.c_size_t(0)
    assert lib().ssd_selective_scan_workspace_bytes(ctypes.byref(sel(**kw)), 0, ctypes.byref(n)) == code
    if kw not in (dict(seqlen=1 << 31),):
        assert step(sel(**dict(kw, seqlen=kw.get("seqlen", 1)))) == code


@pytest.mark.parametrize("name", ["x", "dt", "A", "B", "C", "y"])
def test_selective_scan_refuses_null_and_misaligned(name):
    assert scan(sel(), **{name: None}) == NULLP
    assert scan(sel(), **{name: BASE + (99 << 32) + 1}) == ALIGN
    assert step(sel(seqlen=1), **{name: None}) == NULLP
    assert step(sel(seqlen=1), **{name: BASE + (99 << 32) + 1}) == ALIGN


def test_selective_scan_refuses_other_calls():
    L = lib()
    d = sel()
    n = ctypes.c_size_t(0)
    assert L.ssd_selective_scan_workspace_bytes(None, 0, ctypes.byref(n)) == NULLP
    assert L.ssd_selective_scan_workspace_bytes(ctypes.byref(d), 0, None) == NULLP
    assert L.ssd_selective_scan_workspace_bytes(ctypes.byref(d), -1, ctypes.byref(n)) == SHAPE
    assert L.ssd_selective_scan_workspace_bytes(ctypes.byref(d), 3, ctypes.byref(n)) == SHAPE  # packed: batch 1
    assert scan(d, S=3) == SHAPE
    one = sel(batch=1)
    assert scan(one, S=0) == SHAPE and scan(one, S=1 << 31) == SHAPE
    assert scan(one, S=3, cu=None) == NULLP
    assert scan(one, S=3, cu=BASE + 2) == ALIGN
    for bad in ("D", "h0", "hT"):
        assert scan(d, **{bad: BASE + (99 << 32) + 2}) == ALIGN
    assert scan(d, ws=BASE + (99 << 32) + 128) == ALIGN
    long = sel(seqlen=4096)
    assert L.ssd_selective_scan_workspace_bytes(ctypes.byref(long), 0, ctypes.byref(n)) == OK and n.value > 0
    assert scan(long, ws_bytes=n.value - 1) == WS


@pytest.mark.parametrize("out,over", [("y", "x"), ("y", "z"), ("y", "A"), ("y", "h0"), ("y", "hT"), ("hT", "dt"),
                                      ("hT", "B"), ("ws", "x"), ("ws", "hT"), ("ws", "y"), ("ws", "h0")])
def test_selective_scan_refuses_overlap(out, over):
    p = pointers("x", "dt", "A", "B", "C", "D", "z", "h0", "y", "hT", "ws", "cu")
    d = sel(seqlen=4096)
    assert scan(d, **{out: p[over]}) == ALIAS
    # one element into the other array
    assert scan(d, **{out: p[over] + 256}) == ALIAS


def test_selective_scan_refuses_partly_overlapping_states():
    p = pointers("x", "dt", "A", "B", "C", "D", "z", "h0")
    assert scan(sel(), hT=p["h0"] + 16) == ALIAS


def test_overlap_follows_the_extent_of_views():
    # 2 rows of 100 tokens, 300 elements apart: y behind the dense size of x
    # lies inside the view's extent all the same
    x = pointers("x")["x"]
    assert scan(sel(x_stride=Stride(300, 0)), y=x + 2 * 100 * 64 * 2) == ALIAS


def test_selective_step_refuses():
    d = sel(seqlen=1)
    assert step(sel(seqlen=2)) == SHAPE
    assert step(d, n=0) == SHAPE and step(d, n=1 << 31) == SHAPE
    assert step(d, n=1, slots=None) == SHAPE  # without a slot map every row needs its slot
    assert step(d, state=None) == NULLP
    assert step(d, state=BASE + 2) == ALIGN and step(d, slots=BASE + 2) == ALIGN
    p = pointers("x", "dt", "A", "B", "C", "D", "z", "state", "slots", "y")
    for out in ("state", "y"):
        for other in ("x", "A", "z", "slots", "C"):
            assert step(d, **{out: p[other]}) == ALIAS, (out, other)
    assert step(d, y=p["state"]) == ALIAS


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), SHAPE), (dict(seqlen=0), SHAPE), (dict(channels=0, out_channels=(0, 0, 0)), SHAPE),
    (dict(out_channels=(63, 0, 0)), SHAPE), (dict(out_channels=(0, 64, 0)), SHAPE), (dict(out_channels=(65, -1, 0)), SHAPE),
    (dict(conv_width=0), UNSUP), (dict(conv_width=5), UNSUP), (dict(io_dtype=3), UNSUP),
    (dict(x_stride=Stride(10, 0)), SHAPE), (dict(batch=70000), SHAPE),
])
def test_conv1d_refuses_descriptors(kw, code):
    assert conv_call(conv(**kw)) == code
    assert conv_step(conv(**dict(kw, seqlen=kw.get("seqlen", 1)))) == code


def test_conv1d_refuses_other_calls():
    L = lib()
    d, p = conv(), pointers("x", "w", "b", "in", "out_st", "o0")
    assert L.ssd_conv1d(None, None, 0, *[None] * 9) == NULLP
    for name in ("x", "w", "o0"):
        assert conv_call(d, **{name: None}) == NULLP
        assert conv_call(d, **{name: BASE + (99 << 32) + 1}) == ALIGN
    assert conv_call(conv(out_channels=(32, 16, 16)), o1=BASE + (20 << 32)) == NULLP
    assert conv_call(d, S=2) == SHAPE                          # sequences without offsets
    assert conv_call(d, cu=BASE + (30 << 32), S=2) == SHAPE    # packed: batch 1
    one = conv(batch=1)
    assert conv_call(one, cu=BASE + (30 << 32), S=0) == SHAPE
    assert conv_call(one, cu=BASE + (30 << 32) + 2, S=2) == ALIGN
    for out in ("o0", "out_st"):
        for other in ("x", "w", "b", "in"):
            assert conv_call(d, **{out: p[other]}) == ALIAS, (out, other)
    assert conv_call(d, o0=p["out_st"]) == ALIAS
    assert conv_call(d, out_st=p["in"]) == ALIAS               # not in place
    assert conv_call(conv(out_channels=(32, 16, 16)), o1=p["o0"], o2=BASE + (40 << 32)) == ALIAS


def test_conv1d_step_refuses():
    d = conv(seqlen=1)
    p = pointers("x", "w", "b", "state", "slots", "o0")
    assert conv_step(conv(seqlen=2)) == SHAPE
    assert conv_step(d, n=0) == SHAPE and conv_step(d, n=1, slots=None) == SHAPE
    for name in ("x", "w", "state", "o0"):
        assert conv_step(d, **{name: None}) == NULLP
    for out in ("state", "o0"):
        for other in ("x", "w", "b", "slots"):
            assert conv_step(d, **{out: p[other]}) == ALIAS, (out, other)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), SHAPE), (dict(rows=0), SHAPE), (dict(channels=0), SHAPE), (dict(ngroups=0), SHAPE),
    (dict(ngroups=3), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(io_dtype=9), UNSUP),
    (dict(channels=16385, ngroups=1), UNSUP), (dict(silu=1), UNSUP), (dict(x_stride=Stride(1, 0)), SHAPE),
    (dict(z_stride=Stride(64, 3)), SHAPE),
])
def test_group_norm_refuses_descriptors(kw, code):
    assert norm_call(norm(**kw)) == code


def test_group_norm_refuses_other_calls():
    p = pointers("x", "w", "b", "z", "out")
    assert lib().ssd_group_norm(None, *[None] * 6) == NULLP
    assert norm_call(norm(), x=None) == NULLP and norm_call(norm(), out=None) == NULLP
    assert norm_call(norm(), z=BASE + (9 << 32) + 1) == ALIGN and norm_call(norm(), w=BASE + (9 << 32) + 2) == ALIGN
    for other in ("x", "w", "b", "z"):
        assert norm_call(norm(), out=p[other]) == ALIAS


def test_workspace_follows_the_cut_of_the_time_axis():
    n = ctypes.c_size_t(0)

    def need(**kw):
        S = kw.pop("S", 0)
        assert lib().ssd_selective_scan_workspace_bytes(ctypes.byref(sel(**kw)), S, ctypes.byref(n)) == OK
        return n.value

    # enough rows and channels fill the card: no segments, no workspace
    assert need(batch=64, channels=8192, seqlen=4096) == 0
    assert need(batch=1, channels=64, seqlen=32) == 0
    assert need(batch=1, channels=64, seqlen=8192) > 0
    # a workspace grows with the channels and states, and not with the tokens
    # once the segments are as many as are of use
    assert need(batch=1, channels=64, seqlen=1 << 20) <= 2 * need(batch=1, channels=64, seqlen=1 << 19)
    assert need(batch=1, S=5, seqlen=8192) > 0


def test_binding_refuses_host_tensors_and_wrong_ranks():
    lib()
    x = torch.zeros(2, 8, 16)
    with pytest.raises(ValueError, match="device tensor"):
        ssd.selective_scan(x, x, torch.zeros(16, 4), x, x)
    with pytest.raises(ValueError, match="device tensor"):
        ssd.conv1d(x, torch.zeros(16, 4))
    with pytest.raises(ValueError, match="device tensor"):
        ssd.conv1d_step(x[:, 0], torch.zeros(16, 4), None, torch.zeros(2, 16, 3))
    with pytest.raises(ValueError, match="device tensor"):
        ssd.selective_step(x[:, 0], x[:, 0], torch.zeros(16, 4), x[:, :1], x[:, :1], None, None, torch.zeros(2, 16, 4))
    with pytest.raises(ValueError, match="device tensor"):
        ssd.group_norm(x)
    with pytest.raises(ValueError, match="dimensions"):
        ssd.group_norm(torch.zeros(2, 2, 2, 2))


def test_strides_of_views():
    from mamba_ssd_scan_fwd_amd.binding import _marshal

    lib()

    def of(t, lead=2):
        return _marshal().strides(t, lead)

    wide = torch.zeros(3, 10, 20)
    assert of(wide) == (0, 0)  # dense
    assert of(wide[:, :, 5:12]) == (20, 200)
    assert of(wide[:, 2:6]) == (20, 200)
    assert of(wide[:, ::2]) == (40, 200)
    assert of(wide.transpose(0, 1)) == (200, 20)
    assert of(wide[:1]) == (0, 0)
    assert of(wide[:, :1]) == (20, 200)
    assert of(wide[:1, :, :4]) == (20, 184)
    assert of(wide[:, 3], 1) == (20, 200)
    assert of(wide[:, :, 4:12].unflatten(2, (2, 4))) == (20, 200)
    for bad in (wide[:, :, ::2], wide.transpose(1, 2), wide[:, :, 4:12].unflatten(2, (2, 4))[..., :3],
                wide[:, :1].expand(3, 10, 20), wide[:1].expand(3, 10, 20)):
        with pytest.raises(ValueError):
            of(bad)
    with pytest.raises(ValueError):
        of(wide[:1, 0].expand(3, 20), 1)


def test_structs_are_as_long_as_the_headers():
    # 5 sizes, 2 types, pointer, 2 flags, 2 limits, 5 pairs of strides; 6
    # sizes, 3 ints (padded), 1 pair; 4 sizes, 4 ints, eps (padded), 2 pairs
    assert ctypes.sizeof(SelectiveDesc) == 40 + 8 + 8 + 8 + 8 + 80
    assert ctypes.sizeof(Conv1dDesc) == 48 + 16 + 16
    assert ctypes.sizeof(GroupNormDesc) == 32 + 16 + 8 + 32


@pytest.mark.parametrize("token,batch", [(1 << 62, 0), ((1 << 63) - 1, 0), (1 << 57, 0), (-(1 << 63), 0), (1 << 62, 1 << 62),
                                         (0, (1 << 63) - 1), (0, -(1 << 63)), (64, 1 << 62)])
def test_strides_of_any_size_are_refused_without_overflow(token, batch):
    # (products of what is refused must not overflow either: the sanitized
    # build of build.py ends the test there)
    s = Stride(token, batch)
    assert scan(sel(x_stride=s)) == SHAPE and scan(sel(B_stride=s)) == SHAPE
    assert step(sel(seqlen=1, z_stride=s)) == SHAPE
    assert conv_call(conv(x_stride=s)) == SHAPE and conv_step(conv(seqlen=1, x_stride=s)) == SHAPE
    assert norm_call(norm(z_stride=s)) == SHAPE


def test_outputs_of_any_size_are_refused_without_overflow():
    # rows that lie over one another make a small input of any number of rows;
    # the dense output of as many does not fit (64 x 2^16 x 2^31 and more)
    s, n = Stride(1 << 20, 1 << 20), (1 << 31) - 1
    assert scan(sel(batch=65535, seqlen=n, channels=1 << 20, ngroups=1, x_stride=s, dt_stride=s, z_stride=s,
                    B_stride=Stride(16, 16), C_stride=Stride(16, 16))) == SHAPE
    assert conv_call(conv(batch=65535, seqlen=n, channels=1 << 20, out_channels=(1 << 20, 0, 0), x_stride=s)) == SHAPE
    few = Stride(4, 4)
    assert norm_call(norm(batch=n, rows=n, channels=4, ngroups=1, x_stride=few, z_stride=few)) == SHAPE
    assert norm_call(norm(batch=1 << 20, rows=1 << 20, channels=4, ngroups=1, x_stride=few, z_stride=few)) == SHAPE


def test_workspace_size_from_public_names():
    lib()
    desc = ssd.SelectiveDesc(batch=1, seqlen=8192, channels=64, dstate=16, ngroups=1, io_dtype=0, dt_dtype=0)
    assert ssd.selective_scan_workspace_bytes(desc) > 0
    assert ssd.selective_scan_workspace_bytes(desc, 5) > 0
    desc.seqlen = 32
    assert ssd.selective_scan_workspace_bytes(desc) == 0
    with pytest.raises(ssd.SSDError):
        ssd.selective_scan_workspace_bytes(desc, -1)
