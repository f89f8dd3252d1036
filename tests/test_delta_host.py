"""Refusals of the gated delta rule and of the norm of heads, on the CPU: the C
ABI with fake device addresses (no call reaches a kernel), the binding's own
checks, and the compiled marshalling without memory."""

import ctypes

import pytest
import torch

import mamba_ssd_scan_fwd_amd as ssd
from mamba_ssd_scan_fwd_amd.binding import DeltaDesc, HeadNormDesc
from test_layer_host import ALIAS, ALIGN, BASE, NULLP, OK, SHAPE, UNSUP, WS, Stride, fill, lib, pointers
from test_layer_marshal import run

FAR = BASE + (99 << 32)
INPUTS = ("x", "dt", "A", "B", "C", "beta")
NAMES = (*INPUTS, "h0", "y", "hT", "ws", "cu", "state", "slots")


def rule(**kw):
    return fill(DeltaDesc(batch=2, seqlen=100, nheads=4, headdim=64, dstate=64, ngroups=2, io_dtype=1, dt_dtype=1, scale=1.0), kw)


def heads(**kw):
    return fill(HeadNormDesc(batch=2, rows=100, q_heads=4, k_heads=2, headdim=64, rot=32, io_dtype=1, eps=1e-5), kw)


def call(d, ws_bytes=1 << 40, S=None, **over):
    p = dict(pointers(*NAMES), **over)
    mid = [p[k] for k in (*INPUTS, "h0", "y", "hT", "ws")]
    if S is None:
        return lib().ssd_delta_rule(ctypes.byref(d), *mid, ws_bytes, None)
    return lib().ssd_delta_rule_varlen(ctypes.byref(d), p["cu"], S, *mid, ws_bytes, None)


def step(d, n=8, **over):
    p = dict(pointers(*NAMES), **over)
    return lib().ssd_delta_step(ctypes.byref(d), *[p[k] for k in (*INPUTS, "state", "slots")], n, p["y"], None)


def norm(d, **over):
    names = ("q", "k", "qw", "kw", "pos", "freq", "qo", "ko")
    p = dict(pointers(*names), **over)
    return lib().ssd_head_norm(ctypes.byref(d), *[p[k] for k in names], None)


def bytes_of(S=0, **kw):
    n = ctypes.c_size_t(0)
    st = lib().ssd_delta_rule_workspace_bytes(ctypes.byref(rule(**kw)), S, ctypes.byref(n))
    return st, n.value


BAD = [
    (dict(batch=0), SHAPE), (dict(seqlen=0), SHAPE), (dict(nheads=0), SHAPE), (dict(headdim=0), SHAPE), (dict(dstate=0), SHAPE),
    (dict(ngroups=0), SHAPE), (dict(ngroups=3), SHAPE), (dict(nheads=65536), SHAPE), (dict(seqlen=1 << 31), SHAPE),
    (dict(batch=1 << 31), SHAPE), (dict(headdim=257), UNSUP), (dict(dstate=257), UNSUP), (dict(io_dtype=2), UNSUP),
    (dict(dt_dtype=5), UNSUP), (dict(io_dtype=0, dt_dtype=1), UNSUP), (dict(nheads=65534, ngroups=1, headdim=17), SHAPE),
    (dict(dt_clamp=1, dt_min=2.0, dt_max=1.0), SHAPE), (dict(dt_clamp=1, dt_min=float("nan"), dt_max=1.0), SHAPE),
    (dict(dt_bias=BASE + 2), ALIGN), (dict(x_stride=Stride(255, 0)), SHAPE), (dict(x_stride=Stride(256, 255)), SHAPE),
    (dict(B_stride=Stride(127, 0)), SHAPE), (dict(beta_stride=Stride(3, 0)), SHAPE), (dict(dt_stride=Stride(4, -5)), SHAPE),
    (dict(C_stride=Stride(-128, 0)), SHAPE), (dict(x_stride=Stride(256, 1 << 41)), SHAPE),
]


@pytest.mark.parametrize("kw,code", BAD)
def test_rule_refuses_descriptors(kw, code):
    assert call(rule(**kw)) == code
    assert call(rule(**dict(kw, batch=kw.get("batch", 1))), S=3) == code
    assert bytes_of(**kw)[0] == code
    if kw != dict(seqlen=1 << 31):
        assert step(rule(**dict(kw, seqlen=kw.get("seqlen", 1)))) == code


@pytest.mark.parametrize("name", [*INPUTS, "y"])
def test_rule_refuses_null_and_misaligned(name):
    for f, d in ((call, rule()), (step, rule(seqlen=1))):
        assert f(d, **{name: None}) == NULLP
        assert f(d, **{name: FAR + 1}) == ALIGN


def test_rule_refuses_other_calls():
    L, d, n = lib(), rule(), ctypes.c_size_t(0)
    assert L.ssd_delta_rule_workspace_bytes(None, 0, ctypes.byref(n)) == NULLP
    assert L.ssd_delta_rule_workspace_bytes(ctypes.byref(d), 0, None) == NULLP
    assert bytes_of(S=-1)[0] == SHAPE and bytes_of(S=3)[0] == SHAPE  # packed: batch 1
    assert call(d, S=3) == SHAPE
    one = rule(batch=1)
    assert call(one, S=0) == SHAPE and call(one, S=1 << 31) == SHAPE
    assert call(one, S=3, cu=None) == NULLP and call(one, S=3, cu=BASE + 2) == ALIGN
    for bad in ("h0", "hT"):
        assert call(d, **{bad: FAR + 2}) == ALIGN
    assert call(d, ws=FAR + 128) == ALIGN
    st, need = bytes_of(seqlen=4096)
    assert st == OK and need > 0
    assert call(rule(seqlen=4096), ws_bytes=need - 1) == WS
    assert ssd.load_library().ssd_delta_rule(None, *[BASE] * 10, 0, None) == NULLP
    assert ssd.load_library().ssd_delta_rule_varlen(None, BASE, 1, *[BASE] * 10, 0, None) == NULLP
    assert ssd.load_library().ssd_delta_step(None, *[BASE] * 8, 1, BASE, None) == NULLP


@pytest.mark.parametrize("out,over", [("y", "x"), ("y", "beta"), ("y", "A"), ("y", "h0"), ("y", "hT"), ("hT", "dt"), ("hT", "B"),
                                      ("ws", "x"), ("ws", "hT"), ("ws", "y"), ("ws", "h0"), ("y", "C"), ("ws", "beta")])
def test_rule_refuses_overlap(out, over):
    p = pointers(*NAMES)
    d = rule(seqlen=4096)
    assert call(d, **{out: p[over]}) == ALIAS
    if over != "A":  # of 16 bytes
        assert call(d, **{out: p[over] + 256}) == ALIAS
    one = rule(seqlen=4096, batch=1)
    assert call(one, S=3, **{out: p[over]}) == ALIAS
    assert call(one, S=3, y=p["cu"]) == ALIAS and call(one, S=3, hT=p["cu"] + 4) == ALIAS


def test_rule_refuses_partly_overlapping_states():
    assert call(rule(), hT=pointers(*NAMES)["h0"] + 16) == ALIAS


def test_step_refuses():
    d = rule(seqlen=1)
    assert step(rule(seqlen=2)) == SHAPE
    assert step(d, n=0) == SHAPE and step(d, n=1 << 31) == SHAPE
    assert step(d, n=1, slots=None) == SHAPE  # without a slot map every row needs its slot
    assert step(d, state=None) == NULLP
    assert step(d, state=BASE + 2) == ALIGN and step(d, slots=BASE + 2) == ALIGN
    p = pointers(*NAMES)
    for out in ("state", "y"):
        for other in ("x", "A", "beta", "slots", "C"):
            assert step(d, **{out: p[other]}) == ALIAS, (out, other)
    assert step(d, y=p["state"]) == ALIAS


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), SHAPE), (dict(rows=0), SHAPE), (dict(q_heads=0), SHAPE), (dict(k_heads=-1), SHAPE), (dict(headdim=0), SHAPE),
    (dict(batch=1 << 31), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(rot=-2), SHAPE), (dict(rot=66), SHAPE), (dict(rot=31), SHAPE),
    (dict(eps=-1e-5), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(io_dtype=2), UNSUP), (dict(headdim=513), UNSUP),
    (dict(q_heads=(1 << 14) + 1), SHAPE), (dict(k_heads=(1 << 14) + 1), SHAPE), (dict(q_stride=Stride(255, 0)), SHAPE),
    (dict(k_stride=Stride(127, 0)), SHAPE), (dict(q_stride=Stride(-256, 0)), SHAPE), (dict(k_stride=Stride(128, 1 << 62)), SHAPE),
])
def test_head_norm_refuses_descriptors(kw, code):
    assert norm(heads(**kw)) == code


def test_head_norm_refuses_other_calls():
    d, p = heads(), pointers("q", "k", "qw", "kw", "pos", "freq", "qo", "ko")
    assert lib().ssd_head_norm(None, *p.values(), None) == NULLP
    for name in ("q", "k", "pos", "freq", "qo", "ko"):
        assert norm(d, **{name: None}) == NULLP, name
    for name in p:
        assert norm(d, **{name: FAR + 1}) == ALIGN, name
    for out in ("qo", "ko"):
        for other in p:
            if other != out:
                assert norm(d, **{out: p[other]}) == ALIAS, (out, other)
    # a view's extent: 200 tokens, 900 elements apart
    assert norm(heads(q_stride=Stride(900, 90000)), ko=p["q"] + 2 * 150 * 900) == ALIAS
    # without keys or a rotation their arguments do not matter, whatever they are
    assert norm(heads(k_heads=0, rot=0), q=None, k=BASE + 1, ko=BASE + 1, kw=BASE + 1, pos=BASE + 1, freq=BASE + 1) == NULLP
    assert norm(heads(k_heads=0, rot=0), qo=p["q"], k=BASE + 1, ko=BASE + 1, kw=BASE + 1, pos=BASE + 1, freq=BASE + 1) == ALIAS


@pytest.mark.parametrize("token,batch", [(1 << 62, 0), ((1 << 63) - 1, 0), (1 << 57, 0), (-(1 << 63), 0), (1 << 62, 1 << 62),
                                         (0, (1 << 63) - 1), (0, -(1 << 63)), (256, 1 << 62)])
def test_strides_of_any_size_are_refused_without_overflow(token, batch):
    s = Stride(token, batch)
    assert call(rule(x_stride=s)) == SHAPE and call(rule(beta_stride=s)) == SHAPE and call(rule(C_stride=s)) == SHAPE
    assert step(rule(seqlen=1, B_stride=s)) == SHAPE
    assert norm(heads(q_stride=s)) == SHAPE and norm(heads(k_stride=s)) == SHAPE


def test_sizes_of_any_kind_are_refused_without_overflow():
    """Sizes that are each in range and whose product is not."""
    n = (1 << 31) - 1
    one = Stride(1, 1)
    small = dict(nheads=1, ngroups=1, headdim=1, dstate=1, x_stride=one, dt_stride=one, beta_stride=one, B_stride=one, C_stride=one)
    assert call(rule(batch=n, seqlen=n, **small)) == SHAPE
    assert call(rule(batch=1, seqlen=n, nheads=65535, ngroups=1, headdim=16, dstate=256, io_dtype=1)) == SHAPE
    assert bytes_of(S=n, batch=1, seqlen=n, nheads=65535, ngroups=1, headdim=16, dstate=256)[0] == SHAPE
    assert step(rule(seqlen=1, batch=1, nheads=65535, ngroups=1, headdim=16, dstate=256), n=n) == SHAPE
    assert norm(heads(batch=n, rows=n, q_heads=1, k_heads=0, headdim=1, rot=0, q_stride=one)) == SHAPE


def test_launches_of_too_many_threads_are_refused():
    """2^26 rows and heads of 256 threads each and more: refused before a launch."""
    many = dict(batch=1 << 20, seqlen=1, nheads=64, ngroups=1, headdim=5, dstate=5)
    far = {n: BASE + (i << 40) for i, n in enumerate(NAMES)}
    assert call(rule(**many), **far) == SHAPE
    assert call(rule(**dict(many, batch=1, seqlen=10)), S=1 << 20, **far) == SHAPE
    assert step(rule(**many), n=1 << 20, **far) == SHAPE


def test_workspace_follows_the_way_that_is_taken():
    # token after token needs none, blocks a record for each block and head, and
    # whether a type, an alignment or a stride is one or another does not matter
    assert bytes_of(batch=1, seqlen=4) == (OK, 0)
    assert bytes_of(headdim=5, seqlen=4096) == (OK, 0)
    st, need = bytes_of(batch=2, seqlen=640, nheads=64, ngroups=1)
    assert st == OK and need == 2 * 10 * 64 * 18944
    st, fp32 = bytes_of(batch=2, seqlen=640, nheads=64, ngroups=1, io_dtype=0, dt_dtype=0)
    assert st == OK and fp32 == 2 * 10 * 64 * 37376
    st, packed = bytes_of(S=7, batch=1, seqlen=1280, nheads=64, ngroups=1)
    assert st == OK and packed >= (20 + 7) * 64 * 18944
    # grows with the tokens and no faster
    assert bytes_of(batch=1, nheads=2, seqlen=1 << 20)[1] <= 2 * bytes_of(batch=1, nheads=2, seqlen=1 << 19)[1]
    lib()
    d = rule(seqlen=4096)
    assert ssd.delta_rule_workspace_bytes(d) == bytes_of(seqlen=4096)[1]
    with pytest.raises(ssd.SSDError):
        ssd.delta_rule_workspace_bytes(d, -1)


def test_structs_are_as_long_as_the_headers():
    # 6 sizes, 2 types, pointer, 2 flags, 2 limits, flag, scale, 5 pairs of
    # strides; 6 sizes, 3 ints, eps, 2 pairs
    assert ctypes.sizeof(DeltaDesc) == 48 + 8 + 8 + 8 + 8 + 8 + 80
    assert ctypes.sizeof(HeadNormDesc) == 48 + 16 + 32


def test_binding_refuses_host_tensors_and_wrong_ranks():
    lib()
    x, v, s = torch.zeros(2, 8, 4, 16), torch.zeros(2, 8, 4), torch.zeros(2, 4, 16, 16)
    for f in (lambda: ssd.delta_rule(x, v, v, x, x, v),
              lambda: ssd.delta_rule_varlen(x[:1], v[:1], v, x[:1], x[:1], v[:1], cu_seqlens=torch.zeros(2, dtype=torch.int32)),
              lambda: ssd.delta_step(x[:, 0], v[:, 0], v, x[:, 0], x[:, 0], v[:, 0], s), lambda: ssd.head_norm(x)):
        with pytest.raises(ValueError, match="device tensor"):
            f()
    with pytest.raises(ValueError, match="dimensions"):
        ssd.head_norm(torch.zeros(2, 2))
    with pytest.raises(ValueError, match="cu_seqlens"):
        ssd.delta_rule_varlen(x, v, v, x, x, v, cu_seqlens=None)


def test_marshalling_refuses_wrong_arguments():
    """With device tensors that have no memory: what is refused before any is looked for."""
    out = run("""
def rule(**kw):
    a = dict(x=dev(2, 3, 4, 8), dt=dev(2, 3, 4), A=dev(4), B=dev(2, 3, 2, 8), C=dev(2, 3, 2, 8), beta=dev(2, 3, 4), cu=None,
             init=None, y=None, final=None, ws=None)
    a.update(kw)
    return m.delta_prompts(a["x"], a["dt"], a["A"], a["B"], a["C"], a["beta"], a["cu"], a["init"], a["y"], a["final"], True,
                           a["ws"], 1.0, False, *pre(), 0)

def token(**kw):
    a = dict(x=dev(2, 4, 8), dt=dev(2, 4), A=dev(4), B=dev(2, 2, 8), C=dev(2, 2, 8), beta=dev(2, 4), state=dev(5, 4, 8, 8),
             slots=None, y=None)
    a.update(kw)
    return m.delta_token(*a.values(), 1.0, False, *pre(), 0)

def norm(q, k=None, qw=None, kw=None, pos=None, freq=None, qo=None, ko=None):
    return m.head_norm(q, k, qw, kw, pos, freq, 1e-5, False, False, qo, ko, 0)

i32, bf = torch.int32, torch.bfloat16
cases = [lambda: rule(A=None), lambda: rule(A=dev(5)), lambda: rule(A=dev(4, dtype=bf)), lambda: rule(x=dev(2, 3, 4)),
         lambda: rule(x=None), lambda: rule(x=dev(2, 3, 4, 8, dtype=torch.float16)), lambda: rule(B=dev(2, 3, 2, 8, dtype=bf)),
         lambda: rule(C=dev(2, 3, 2, 9)), lambda: rule(C=dev(2, 3, 1, 8)), lambda: rule(beta=dev(2, 3, 4, dtype=bf)),
         lambda: rule(beta=dev(2, 3, 1)), lambda: rule(dt=dev(2, 3)), lambda: rule(init=dev(3, 4, 8, 8)),
         lambda: rule(init=dev(2, 4, 8, 8, dtype=bf)), lambda: rule(final=dev(2, 4, 8, 8).transpose(2, 3)),
         lambda: rule(y=dev(2, 3, 4, 9)), lambda: rule(y=dev(2, 3, 4, 8, dtype=bf)),
         lambda: rule(cu=dev(3, dtype=i32)), lambda: rule(cu=dev(3)), lambda: rule(x=dev(2, 3, 4, 16)[..., ::2]),
         lambda: rule(B=dev(2, 1, 2, 8).expand(2, 3, 2, 8)),
         lambda: token(state=dev(5, 4, 8)), lambda: token(state=dev(5, 4, 8, 9)), lambda: token(state=dev(5, 4, 8, 8, dtype=bf)),
         lambda: token(state=dev(5, 4, 8, 16)[..., :8]), lambda: token(slots=dev(3, dtype=i32)), lambda: token(slots=dev(2)),
         lambda: token(x=dev(2, 3, 4, 8)), lambda: token(state=None),
         lambda: norm(dev(2, 4)), lambda: norm(dev(2, 4, 8), dev(2, 3, 4, 8)), lambda: norm(dev(2, 4, 8), dev(2, 4, 9)),
         lambda: norm(dev(2, 4, 8), dev(2, 4, 8, dtype=bf)), lambda: norm(dev(2, 4, 8), dev(2, 0, 8)),
         lambda: norm(dev(2, 4, 8), None, None, dev(8)), lambda: norm(dev(2, 4, 8), None, None, None, None, None, None, dev(2, 4, 8)),
         lambda: norm(dev(2, 4, 8), None, dev(9)), lambda: norm(dev(2, 4, 8), pos=dev(2, dtype=i32)),
         lambda: norm(dev(2, 4, 8), freq=dev(2)), lambda: norm(dev(2, 4, 8), pos=dev(2), freq=dev(2)),
         lambda: norm(dev(2, 4, 8), pos=dev(3, dtype=i32), freq=dev(2)), lambda: norm(dev(2, 4, 8), pos=dev(2, dtype=i32), freq=dev(2, 2)),
         lambda: norm(dev(2, 4, 8), qo=dev(2, 4, 8, dtype=bf)), lambda: norm(dev(2, 4, 8, dtype=torch.float16)),
         lambda: norm(dev(2, 4, 16)[..., ::2])]
with FakeTensorMode():
    for i, f in enumerate(cases):
        try:
            f()
            print("taken", i)
        except (ValueError, TypeError) as e:
            print("refused", i, *str(e).splitlines()[:1])
        except BaseException as e:
            print("other", i, type(e).__name__, *str(e).splitlines()[:1])
print("alive", len(cases))
""")
    lines = out.splitlines()
    assert lines[-1] == "alive %d" % (len(lines) - 1)
    assert not [ln for ln in lines[:-1] if not ln.startswith("refused")]


def test_tensors_without_memory_and_streams_that_are_none():
    """Inside vmap a tensor has no address, and a stream is a number: the calls
    raise and the process, with the interpreter's lock in order, goes on."""
    out = run("""
calls = dict(
    delta_prompts=lambda x, s=0: m.delta_prompts(x, dev(2, 3, 4), dev(4), dev(2, 3, 1, 8), dev(2, 3, 1, 8), dev(2, 3, 4), None, None,
                                                 None, None, True, None, 1.0, False, *pre(), s),
    delta_packed=lambda x, s=0: m.delta_prompts(x, dev(1, 3, 4), dev(4), dev(1, 3, 1, 8), dev(1, 3, 1, 8), dev(1, 3, 4),
                                                dev(3, dtype=torch.int32), None, None, None, True, None, 1.0, False, *pre(), s),
    delta_token=lambda x, s=0: m.delta_token(x, dev(2, 4), dev(4), dev(2, 1, 8), dev(2, 1, 8), dev(2, 4), dev(2, 4, 8, 8), None,
                                             None, 1.0, False, *pre(), s),
    head_norm=lambda x, s=0: m.head_norm(x, x, None, None, None, None, 1e-5, True, False, None, None, s),
)
shapes = dict(delta_prompts=(2, 3, 4, 8), delta_packed=(1, 3, 4, 8), delta_token=(2, 4, 8), head_norm=(2, 4, 8))
with FakeTensorMode():
    for name, f in calls.items():
        try:
            torch.vmap(lambda x: (f(x), x)[1])(dev(5, *shapes[name]))
        except RuntimeError as e:
            print("raised", name)
        try:
            f(dev(*shapes[name]), "0")
        except TypeError as e:
            print("raised", name)
print("alive", sum(range(10)))
""")
    names = ["delta_prompts", "delta_packed", "delta_token", "head_norm"]
    assert out.splitlines() == ["raised " + n for n in names for _ in range(2)] + ["alive 45"]
