"""The device that a call of the binding launches on (no GPU: torch's calls
are replaced)."""
import ast
import inspect

import torch

import pytest

from speculative_decoding_verification_temperature_gb300 import api


@pytest.fixture
def devices(monkeypatch):
    """Two devices, the first is current; what was entered, in order."""
    seen = []

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            seen.append(("enter", self.device))

        def __exit__(self, *exc):
            seen.append(("exit", self.device))
            return False

    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(api, "_devices", None)
    return seen


def launch(seen, rc=0):
    def fn(*args):
        seen.append(("call", args))
        return rc
    return fn


def test_the_current_device_is_not_entered_again(devices):
    assert api._call(torch.device("cuda", 0), launch(devices, 3), 1, 2) == 3
    assert devices == [("call", (1, 2))]


def test_another_device_is_entered_for_the_call(devices):
    dev = torch.device("cuda", 1)
    assert api._call(dev, launch(devices), 7) == 0
    assert devices == [("enter", dev), ("call", (7,)), ("exit", dev)]


def test_one_device_is_never_asked_for(devices, monkeypatch):
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_device", None)
    api._call(torch.device("cuda", 0), launch(devices))
    assert devices == [("call", ())]


def test_every_launch_goes_to_its_tensors_device():
    """Each call that takes a stream is made through _call."""
    tree = ast.parse(inspect.getsource(api))
    made = direct = 0
    for node in ast.walk(tree):
        if not isinstance(node, ast.Call):
            continue
        if not any(isinstance(a, ast.Call) and isinstance(a.func, ast.Name)
                   and a.func.id in ("_stream", "_raw_stream")
                   for a in node.args):
            continue
        if ast.unparse(node.func) == "_call":
            made += 1
        else:
            direct += 1
    assert made >= 20 and direct == 0
