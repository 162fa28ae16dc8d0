"""The calls around the codec launch with their tensors' device current.

A default stream's handle is 0 on every device, so a launch with another device
current would run there, on memory of a device it does not own. One GPU is
enough to see the order of things: the context that makes the device current is
replaced by one that records whether it is entered when the library is called.
"""
import pytest
import torch

import bit_tensor_activation_amd as B
from bit_tensor_activation_amd import api
from helpers import say

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


class Device:
    """Stands for torch.cuda.device: notes what is made current and left."""
    made, entered = [], False

    def __init__(self, idx):
        Device.made.append(idx)

    def __enter__(self):
        Device.entered = True

    def __exit__(self, *_):
        Device.entered = False


class Library:
    """libbtq, noting for each launching call whether a device was entered."""

    def __init__(self, lib):
        self.lib, self.seen = lib, []

    def __getattr__(self, name):
        fn = getattr(self.lib, name)
        if name.endswith("_bytes"):
            return fn

        def call(*args):
            self.seen.append(Device.entered)
            return fn(*args)
        return call


@pytest.fixture
def lib(monkeypatch):
    watched = Library(api._lib.load())
    monkeypatch.setattr(api._lib, "load", lambda: watched)
    Device.made.clear()
    return watched


def calls():
    x = torch.randn((2, 3, 64), device=DEV)
    w, sw = torch.ones((2, 8, 64), dtype=torch.int8, device=DEV), torch.ones((2, 8), device=DEV)
    q, s = torch.ones((2, 3, 64), dtype=torch.int8, device=DEV), torch.ones((2, 3), device=DEV)
    r = torch.randn((3, 64), device=DEV)
    y, n, ns = torch.empty((2, 3, 8), device=DEV), torch.empty_like(q[0]), torch.empty_like(s[0])
    ws = torch.empty(B.btq_int8_linear_workspace_bytes(2, 3, 64), dtype=torch.uint8, device=DEV)
    # (outputs given: allocations have a context of their own)
    return {"quantize_rows": lambda **kw: B.btq_quantize_rows(x, q, s, **kw),
            "int8_matmul": lambda **kw: B.btq_int8_matmul(q, s, w, sw, y=y, **kw),
            "int8_linear": lambda **kw: B.btq_int8_linear(x, w, sw, y=y, workspace=ws, **kw),
            "block_norm": lambda **kw: B.btq_block_norm(r, r, post="rms", residual_out=r, n=n,
                                                        n_scale=ns, **kw)}


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("name", ["quantize_rows", "int8_matmul", "int8_linear", "block_norm"])
def test_tensors_of_a_device_that_is_not_current(name, given, lib, monkeypatch):
    say(f"case: {name} with another device current, stream given: {given}")
    call = calls()[name]
    kw = dict(stream=torch.cuda.current_stream(DEV)) if given else {}
    with monkeypatch.context() as m:
        m.setattr(torch._C, "_cuda_getDevice", lambda: 5)
        m.setattr(torch.cuda, "device", Device)
        call(**kw)
    torch.cuda.synchronize()
    assert lib.seen == [True] and not Device.entered and Device.made == [0]
    call(**kw)   # and without a context where the device is current
    torch.cuda.synchronize()
    assert lib.seen == [True, False]
