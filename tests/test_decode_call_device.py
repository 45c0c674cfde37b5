"""A prepared call is launched on its tensors' device, whichever is current (CPU: the device calls
of torch and the library are stand-ins, nothing is launched)."""

import ctypes

import pytest
import torch

from bucketized_guidance_step_gb300 import decode, gs


class Machine:
    """Two devices of which one is current, and a library that notes what it is asked to launch."""

    def __init__(self, current):
        self.current, self.launched, self.status = current, [], gs.GS_OK

    def gs_pages_free(self, *args):
        self.launched.append((self.current, args))
        return self.status


@pytest.fixture
def machine(monkeypatch):
    m = Machine(0)

    class Guard:
        def __init__(self, device):
            self.to = device if isinstance(device, int) else torch.device(device).index

        def __enter__(self):
            self.back, m.current = m.current, self.to

        def __exit__(self, *_):
            m.current = self.back

    monkeypatch.setattr(decode, "load", lambda: m)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: m.current)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: m.current)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0 if i == 1 else 1000 + i)
    return m


@pytest.mark.parametrize("current", [0, 1, 2])
def test_the_tensors_device_is_current_during_the_launch(machine, current):
    machine.current = current
    call = decode.Call("gs_pages_free", (7, 8), torch.device("cuda:1"), ())
    call()
    call()
    assert machine.launched == [(1, (7, 8, 0))] * 2 and machine.current == current


def test_the_device_before_is_current_again_after_an_error(machine):
    machine.status = gs.GS_ERR_INVALID_ARG
    with pytest.raises(decode.GSError):
        decode.Call("gs_pages_free", (), torch.device("cuda:1"), ())()
    assert machine.launched == [(1, (0,))] and machine.current == 0


def test_the_workspace_is_asked_for_on_the_tensors_device(machine, monkeypatch):
    asked = []

    def need(args, n):
        asked.append(machine.current)
        ctypes.cast(n, ctypes.POINTER(ctypes.c_int64)).contents.value = 40
        return gs.GS_OK

    machine.gs_guided_logits_workspace = need
    for name in ("zeros", "empty"):
        make = getattr(torch, name)
        monkeypatch.setattr(torch, name, lambda *a, make=make, device=None, **kw: make(*a, **kw))
    a = decode.GuidedLogitsArgs()
    work = decode._zeroed("gs_guided_logits_workspace", a, torch.device("cuda:1"))
    assert asked == [1] and a.workspace == work.data_ptr() and a.workspace_bytes == 40
