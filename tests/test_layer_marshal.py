"""The compiled marshalling of the layer operators, on the CPU: what it does
with arguments that have no memory or are no handles. Each test runs its calls
in a process of its own, since what it guards against ends the process."""

import os
import subprocess
import sys

import pytest

import mamba_ssd_scan_fwd_amd as ssd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Device tensors without a device: shapes and types, no memory.
HEAD = """
import sys, warnings
sys.path.insert(0, {root!r})
warnings.simplefilter("ignore")
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from mamba_ssd_scan_fwd_amd.binding import _marshal
m = _marshal()

def dev(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="cuda")

def pre():
    return None, False, None

E, N, G, K = 8, 4, 1, 4
calls = dict(
    selective_prompts=lambda x, s=0: m.selective_prompts(x, x, dev(E, N), dev(2, 3, G, N), dev(2, 3, G, N), None, None, None,
                                                         None, None, None, True, None, *pre(), s),
    selective_packed=lambda x, s=0: m.selective_prompts(x, x, dev(E, N), dev(1, 3, G, N), dev(1, 3, G, N), None, None,
                                                        dev(3, dtype=torch.int32), None, None, None, True, None, *pre(), s),
    selective_step=lambda x, s=0: m.selective_step(x, x, dev(E, N), dev(2, G, N), dev(2, G, N), None, None, dev(2, E, N), None,
                                                   None, *pre(), s),
    conv_prompts=lambda x, s=0: m.conv_prompts(x, dev(E, K), None, None, True, None, None, None, None, s),
    conv_token=lambda x, s=0: m.conv_token(x, dev(E, K), None, None, True, dev(2, E, K - 1), None, None, s),
    group_norm=lambda x, s=0: m.group_norm(x, None, None, None, 1, 1e-5, True, False, False, None, s),
)
shapes = dict(selective_prompts=(2, 3, E), selective_packed=(1, 3, E), selective_step=(2, E), conv_prompts=(2, 3, E),
              conv_token=(2, E), group_norm=(2, E))
"""


def run(body):
    if not os.path.exists(ssd.lib_path()):
        pytest.skip("libssd.so not built (python -m mamba_ssd_scan_fwd_amd.build)")
    r = subprocess.run([sys.executable, "-c", HEAD.format(root=ROOT) + body], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stdout[-500:], r.stderr[-1500:])
    return r.stdout


def test_tensors_without_memory_raise():
    """Inside vmap a tensor has no address: the call raises and the process,
    with the interpreter's lock in order, goes on."""
    out = run("""
with FakeTensorMode():
    for name, f in calls.items():
        try:
            torch.vmap(lambda x: (f(x), x)[1])(dev(5, *shapes[name]))
        except RuntimeError as e:
            print("raised", name, type(e).__name__)
print("alive", sum(range(10)))
""")
    lines = out.splitlines()
    assert [ln.split()[1] for ln in lines if ln.startswith("raised")] == [
        "selective_prompts", "selective_packed", "selective_step", "conv_prompts", "conv_token", "group_norm"]
    assert lines[-1] == "alive 45"


def test_a_stream_that_is_no_handle_raises():
    out = run("""
with FakeTensorMode():
    for name, f in calls.items():
        try:
            f(dev(*shapes[name]), "0")
        except TypeError as e:
            print("raised", name)
print("alive", sum(range(10)))
""")
    lines = out.splitlines()
    assert len([ln for ln in lines if ln.startswith("raised")]) == 6 and lines[-1] == "alive 45"


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """(It would be launched on with the wrong device current.)"""
    import torch

    from mamba_ssd_scan_fwd_amd import binding

    class Marshal:
        def __getattr__(self, name):
            return lambda *a: pytest.fail("called")

    class Part:
        def __init__(self, index):
            self.device = torch.device("cuda", index)

    monkeypatch.setattr(binding, "_marshal", Marshal)
    monkeypatch.setattr(binding, "_On", lambda *a: pytest.fail("switched"))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for x, stream in ((0, 1), (1, 0)):
        with pytest.raises(ValueError, match="stream is on cuda:%d, expected cuda:%d" % (stream, x)):
            binding.group_norm(Part(x), stream=Part(stream))
        with pytest.raises(ValueError, match="stream"):
            binding.selective_scan(Part(x), None, None, None, None, stream=Part(stream))
