"""Sizes that do not fit the library's ints are refused, not cut down to their
lower 32 bits.  On tensors without memory that say they are on a GPU; the
library's entry points are replaced by ones that record their sizes."""

import pytest
import torch

from gated_deltanet_linear_tree_gb300 import build
from tests.test_serving_devices import INTS, ACCEPT, PREFILL, STEP, OnGpu

BIG = 2 ** 32 + 2  # its lower 32 bits are a size that is fine


@pytest.fixture(scope="module")
def canopy():
    build.build()
    from gated_deltanet_linear_tree_gb300 import canopy
    canopy.load()
    return canopy


@pytest.mark.parametrize("call,shapes,small", [("accept", ACCEPT, 7), ("accept", ACCEPT, 3), ("accept", ACCEPT, 2),
                                               ("step", STEP, 4), ("prefill", PREFILL, 9), ("prefill", PREFILL, 4)])
def test_sizes_beyond_32_bits_are_refused(canopy, monkeypatch, call, shapes, small):
    lib = type("Lib", (), {"canopy_prefill_workspace_bytes": staticmethod(lambda *a: 8)})
    monkeypatch.setattr(canopy, "load", lambda: lib)

    def at(name, shape):
        t = torch.empty(*[BIG if n == small else n for n in shape], device="meta",
                        dtype=torch.uint8 if name == "ws" else torch.int32 if name in INTS else torch.float32)
        t = t.as_subclass(OnGpu)
        t.index = 0
        return t

    args = {n: at(n, s) for n, s in shapes.items()}
    with pytest.raises(canopy.CanopyError, match="sizes"):
        getattr(canopy, call)(**args)
