"""An output that does not fit raises torch's own error from either side of
the binding, and the next call works."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_out_of_memory(lib, monkeypatch):
    B, HV, d = 64, 32, 128
    q, v = torch.randn(B, HV, d, device="cuda"), torch.randn(B, HV, d, device="cuda")
    g, beta = torch.rand(B, HV, device="cuda") + 0.1, torch.rand(B, HV, device="cuda")
    S = torch.randn(B, HV, d, d, device="cuda")  # 134 MB, and as much for the new state
    lib.step(q, q, v, g, beta, S)
    stub = type("Stub", (), {"step": staticmethod(lambda *args: None)})
    for side in ("native", "python"):
        torch.cuda.empty_cache()
        total = torch.cuda.get_device_properties(0).total_memory
        torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (32 << 20)) / total)
        try:
            with pytest.raises(torch.OutOfMemoryError):
                lib.step(q, q, v, g, beta, S)
        finally:
            torch.cuda.set_per_process_memory_fraction(1.0)
        o, S1 = lib.step(q, q, v, g, beta, S)
        assert torch.isfinite(S1).all()
        del o, S1
        monkeypatch.setattr(lib, "_marshal", stub)
