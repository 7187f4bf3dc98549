"""Checks of the routed-expert binding itself."""
import os
import subprocess
import sys

import pytest
import torch

from helpers import DEV, require_gpu
from mx9_dual_axis_amd import routed

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Memory:
    """Stands for a tensor: notes the streams that it is said to be used on."""

    def __init__(self):
        self.streams = []

    def record_stream(self, stream):
        self.streams.append(stream)


def test_a_routing_used_on_another_stream_holds_all_its_memory():
    """Nothing of a routing, its workspace included, may go back to the
    allocator while another stream still works on it."""
    r = object.__new__(routed.MXRouting)
    names = ("idx", "weight", "slot", "src", "counts", "offs", "live", "prob", "loss", "_workspace")
    for n in names:
        object.__setattr__(r, n, Memory())
    object.__setattr__(r, "_ptrs", ())
    stream = object()
    r.record_stream(stream)
    assert [getattr(r, n).streams for n in names] == [[stream]] * len(names)


@pytest.mark.gpu
def test_memory_recorded_on_a_stream_is_not_handed_out():
    """While a stream that a dropped routing was recorded on is at work, new
    tensors get other memory."""
    require_gpu()
    T = 1 << 20                                           # idx, weight and slot: blocks of 8 MiB each
    plan = routed.mx_routing(T, 4, 2, align=1, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a, z = torch.randn(8192, 8192, device=DEV), torch.randn(T, 4, device=DEV)
        (a @ a).sum()
        side.synchronize()
        b = [a @ a for _ in range(8)]                     # some 10 ms each
        routed.mx_route(z, out=plan)
        done = torch.cuda.Event()
        done.record(side)
    plan.record_stream(side)
    held = {t.data_ptr() for t in (plan.idx, plan.weight, plan.slot)}
    del plan
    new = [torch.empty((T, 2), dtype=torch.int32, device=DEV) for _ in range(3)]
    at_work = not done.query()
    torch.cuda.synchronize()
    del b
    if not at_work:
        pytest.skip("the other stream was done too early to tell")
    assert held.isdisjoint(t.data_ptr() for t in new)


def test_the_package_needs_no_private_name_of_torch():
    """The calls' quick ways to the current device and stream are private to
    torch: without them (a torch built without a GPU, a later one) the package
    imports and its public ones are used."""
    code = """
import torch
for n in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, n):
        delattr(torch._C, n)
from mx9_dual_axis_amd import routed
torch.cuda.current_device = lambda: 3
class Stream:
    cuda_stream = 77
torch.cuda.current_stream = lambda i: Stream if i == 3 else None
assert routed._device() == 3 and routed._stream(3) == 77
seen = []
routed._run(3, lambda *a: seen.append(a), 5)
assert seen == [(5, 77)]
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)
