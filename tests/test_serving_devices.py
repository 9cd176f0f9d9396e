"""Which tensors of a step, prefill or accept have to be on one device: the
Python side's checks, on CPU tensors that say they are on one GPU or another.
No call reaches the library: its entry points are replaced."""

import pytest
import torch

from gated_deltanet_linear_tree_gb300 import build


class OnGpu(torch.Tensor):
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.index


def on(index, *shape, dtype=torch.float32):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)
    t.index = index
    return t


@pytest.fixture(scope="module")
def canopy():
    build.build()
    from gated_deltanet_linear_tree_gb300 import canopy
    canopy.load()
    return canopy


@pytest.fixture
def no_calls(canopy, monkeypatch):
    lib = type("Lib", (), {"canopy_prefill_workspace_bytes": staticmethod(lambda *a: 8)})  # no entry point to call
    monkeypatch.setattr(canopy, "load", lambda: lib)


STEP = dict(q=(2, 2, 32), k=(2, 2, 32), v=(2, 4, 32), g=(2, 4), beta=(2, 4), S=(2, 4, 32, 32), out=(2, 4, 32),
            S_out=(2, 4, 32, 32), err=(1,))
PREFILL = dict(q=(9, 2, 32), k=(9, 2, 32), v=(9, 4, 32), g=(9, 4), beta=(9, 4), S0=(2, 4, 32, 32), starts=(3,),
               ws=(8,), out=(9, 4, 32), S_out=(2, 4, 32, 32))
ACCEPT = dict(p=(2, 3, 7), tokens=(2, 3), parent=(2, 3), u=(2, 3), noise=(2, 7), q=(2, 3, 7), lengths=(2,), err=(1,))
INTS = {"err", "starts", "tokens", "parent", "lengths"}


@pytest.mark.parametrize("call,shapes", [("step", STEP), ("prefill", PREFILL), ("accept", ACCEPT)])
def test_a_tensor_on_another_device_is_refused(canopy, no_calls, call, shapes):
    def tensors(elsewhere=None):
        return {n: on(int(n == elsewhere), *s, dtype=torch.uint8 if n == "ws" else torch.int32 if n in INTS
                      else torch.float32) for n, s in shapes.items()}

    with pytest.raises(Exception) as e:  # all on one device: through the checks, up to the device that is not there
        getattr(canopy, call)(**tensors())
    assert not isinstance(e.value, canopy.CanopyError)
    for name in shapes:
        if name in ("q", "p") and name == next(iter(shapes)):
            continue  # the device that the others are compared with
        with pytest.raises(canopy.CanopyError, match="same device"):
            getattr(canopy, call)(**tensors(name))
