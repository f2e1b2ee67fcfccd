"""How the Python calls reach the library (CPU): the device and stream of a launch, without and with torch's shortcuts
for them."""
import importlib.util
import os

import pytest
import torch

from moe_grouped_expert_amd import _binding as b

SHORT = ("_cuda_getDevice", "_cuda_getCurrentRawStream")


def fresh(monkeypatch):
    """A second copy of the binding, as this torch makes it."""
    spec = importlib.util.spec_from_file_location("moe_grouped_expert_amd._binding_copy", os.path.abspath(b.__file__))
    mod = importlib.util.module_from_spec(spec)
    monkeypatch.setitem(__import__("sys").modules, spec.name, mod)
    spec.loader.exec_module(mod)
    return mod


class Stream:
    def __init__(self, n):
        self.cuda_stream = 1000 + n


class Lib:
    def __init__(self):
        self.seen = []

    def some_call(self, args, stream):
        self.seen.append(stream)
        return 0


@pytest.mark.parametrize("shortcuts", [True, False])
def test_stream_and_device_of_a_call(monkeypatch, shortcuts):
    """A call on the current device takes its current stream; one on another device makes that current first."""
    entered = []

    class Device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            entered.append(self.d.index)

        def __exit__(self, *a):
            pass

    for n in SHORT:
        monkeypatch.delattr(torch._C, n, raising=False)
    if shortcuts:
        monkeypatch.setattr(torch._C, SHORT[0], lambda: 1, raising=False)
        monkeypatch.setattr(torch._C, SHORT[1], lambda i: 1000 + i, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream(getattr(d, "index", d)))
    monkeypatch.setattr(torch.cuda, "device", Device)
    mod = fresh(monkeypatch)
    mod._LIB = Lib()
    a = mod.CombineArgs()
    mod._call("some_call", a, torch.device("cuda", 1))
    assert mod._LIB.seen == [1001] and entered == []
    mod._call("some_call", a, torch.device("cuda", 3))
    assert mod._LIB.seen == [1001, 1003] and entered == [3]
