"""The current stream of the binding's calls, also where torch lacks the private
names that it takes it from."""
import importlib.util
import sys
from types import SimpleNamespace

import pytest
import torch

from fp4_precision_b200 import qfp4 as Q

PRIVATE = ("_cuda_getCurrentRawStream", "_cuda_getDevice")


def binding_without(monkeypatch, names):
    """The binding as imported where torch._C lacks `names`."""
    spec = importlib.util.spec_from_file_location("fp4_precision_b200.qfp4_plain", Q.__file__)
    m = importlib.util.module_from_spec(spec)
    with monkeypatch.context() as without:  # (torch itself uses them)
        without.setitem(sys.modules, spec.name, m)
        for n in names:
            without.delattr(torch._C, n, raising=False)
        spec.loader.exec_module(m)
    return m


def test_without_the_private_names(monkeypatch):
    monkeypatch.setattr(torch.cuda, "init", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda i: SimpleNamespace(cuda_stream=1000 + i))
    m = binding_without(monkeypatch, PRIVATE)
    assert m._stream(None).value == 1003
    seen = []
    m._go(lambda *a: seen.append(a) or m.OK, "call", 3, "arguments")
    assert seen == [("arguments", 1003)]


@pytest.mark.gpu
def test_is_torch_s_current_stream(monkeypatch):
    plain = binding_without(monkeypatch, PRIVATE)
    for s in (torch.cuda.default_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            assert (Q._stream(None).value or 0) == (plain._stream(None).value or 0) == s.cuda_stream
