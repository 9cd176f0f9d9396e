"""A workspace is allocated and its first bytes are cleared on the device that it is asked for, whichever is current:
on CPU, with the library, the allocation and the devices replaced."""

import pytest
import torch

from gated_deltanet_linear_tree_gb300 import build

MAKE = {"workspace": (2, 8, 4, 128), "prefill_workspace": (10, 2, 4, 128), "attend_workspace": (10, 2, 8, 4, 128)}


@pytest.fixture
def world(monkeypatch):
    """(canopy, log): device 0 is current; the log holds (event, device) in order."""
    build.build()
    from gated_deltanet_linear_tree_gb300 import canopy
    canopy.load()
    log, current = [], [0]

    def index_of(device):
        device = torch.device(device if not isinstance(device, int) else f"cuda:{device}")
        return current[-1] if device.index is None else device.index

    class Device:
        def __init__(self, device):
            self.index = index_of(device)

        def __enter__(self):
            current.append(self.index)

        def __exit__(self, *e):
            current.pop()

    class Lib:
        canopy_workspace_bytes = canopy_prefill_workspace_bytes = canopy_attend_workspace_bytes = \
            staticmethod(lambda *a: 8192)

        @staticmethod
        def canopy_workspace_init(p, n, stream):
            log.append(("clear", current[-1], stream))
            return 0

    real = torch.empty

    def empty(*a, device=None, **kw):
        log.append(("allocate", index_of(device)))
        return real(*a, **kw)

    monkeypatch.setattr(canopy, "load", lambda: Lib)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(canopy, "_stream", lambda: ("stream of", current[-1]))
    return canopy, log


@pytest.mark.parametrize("name", MAKE)
@pytest.mark.parametrize("device,index", [("cuda", 0), ("cuda:0", 0), ("cuda:1", 1), (torch.device("cuda", 2), 2),
                                          (1, 1)])
def test_cleared_on_its_own_device(world, name, device, index):
    canopy, log = world
    ws = getattr(canopy, name)(*MAKE[name], device=device)
    assert ws.dtype == torch.uint8 and ws.numel() == 8192
    assert log == [("allocate", index), ("clear", index, ("stream of", index))]


@pytest.mark.parametrize("name", MAKE)
def test_on_the_current_device_by_default(world, name):
    canopy, log = world
    with torch.cuda.device(3):
        getattr(canopy, name)(*MAKE[name])
    assert log == [("allocate", 3), ("clear", 3, ("stream of", 3))]


def test_error_word_read_on_the_workspaces_device(world, monkeypatch):
    """...behind the calls of that device's stream, which set its bits."""
    canopy, log = world
    ws = torch.zeros(8, dtype=torch.uint8).as_subclass(type("OnGpu", (torch.Tensor,), {"get_device": lambda t: 1,
                                                                                        "device": torch.device("cuda", 1)}))
    lib = type("Lib", (), {"canopy_read_device_error": staticmethod(lambda p, e, stream: log.append(stream) or 0)})
    monkeypatch.setattr(canopy, "load", lambda: lib)
    assert canopy.read_device_error(ws) == 0
    assert log == [("stream of", 1)]
