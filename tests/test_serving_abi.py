"""The serving-loop entry points without a GPU: sizes, plans, and arguments
that are refused on the host before any CUDA call."""

import ctypes

import pytest
import torch

from gated_deltanet_linear_tree_gb300 import build


@pytest.fixture(scope="module")
def canopy():
    build.build()
    from gated_deltanet_linear_tree_gb300 import canopy
    canopy.load()
    return canopy


def test_prefill_plan(canopy):
    """bf16 at d = 128 goes in chunks from a mean length on that falls with
    the number of states; everything else token by token."""
    plan = canopy.prefill_plan
    assert plan(16384, 1, 16, 32, True, 128) == "chunked"
    assert plan(37, 1, 16, 16, True, 128) == "scan"
    assert plan(64, 1, 16, 16, True, 128) == "chunked"
    assert plan(47, 1, 16, 32, True, 128) == "scan"
    assert plan(48, 1, 16, 32, True, 128) == "chunked"
    assert plan(26 * 64, 64, 16, 32, True, 128) == "chunked"
    assert plan(25 * 64, 64, 16, 32, True, 128) == "scan"
    assert plan(16384, 1, 16, 32, False, 128) == "scan"
    assert plan(16384, 1, 16, 32, True, 32) == "scan"
    assert plan(3, 1, 16, 32, True, 128, force="chunked") == "chunked"
    assert plan(16384, 1, 16, 32, True, 128, force="scan") == "scan"
    for bad in ((0, 1, 1, 1), (8, 0, 1, 1), (8, 1, 2, 3), (8, 1, 0, 1), (8, 70000, 1, 1)):
        assert plan(*bad, True, 128) == "none"
    assert plan(8, 1, 1, 1, True, 64) == "none"
    assert plan(8, 1, 1, 1, False, 128, force="chunked") == "none"


def test_prefill_workspace(canopy):
    """48 KiB and 768 bytes per chunk and value head, at most N / 64 + B chunks."""
    size = canopy.load().canopy_prefill_workspace_bytes
    per = 49152 + 768
    assert size(1, 1, 1, 128, 128) >= per
    assert size(6400, 3, 4, 128, 128) - size(6400, 2, 4, 128, 128) == 4 * per
    assert size(6464, 3, 4, 128, 128) - size(6400, 3, 4, 128, 128) == 4 * per
    assert 0 < size(6400, 3, 4, 32, 32) < per
    for bad in ((0, 1, 1, 128, 128), (8, 0, 1, 128, 128), (8, 1, 0, 128, 128), (8, 1, 1, 64, 64), (8, 1, 1, 128, 32)):
        assert size(*bad) == 0


def test_refused_on_the_host(canopy):
    """Fake pointers are never followed."""
    lib = canopy.load()
    p = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(10)]
    odd = ctypes.c_void_p(0x10004)

    def prefill(q=p[0], S0=p[5], starts=p[6], N=8, HV=4, d=128, scale=1.0, flags=0, o_dt=0):
        return lib.canopy_prefill(q, p[1], p[2], 1, p[3], p[4], S0, starts, N, 2, 2, HV, d, d, scale, p[7], o_dt,
                                  p[8], p[9], flags, None)

    assert prefill(q=odd) == 1 and prefill(S0=odd) == 1 and prefill(starts=None) == 1 and prefill(N=-1) == 1
    assert prefill(HV=5) == 1 and prefill(scale=float("inf")) == 1 and prefill(flags=8) == 1 and prefill(o_dt=3) == 1
    assert prefill(d=64) == 3

    def step(S=p[5], S_new=p[6], B=2, scale=1.0, err=None):
        return lib.canopy_step(p[0], p[1], p[2], 0, p[3], p[4], S, S_new, B, 2, 4, 128, 128, scale, p[7], 1, err, None)

    assert step(S=odd) == 1 and step(S_new=None) == 1 and step(B=-1) == 1 and step(scale=float("nan")) == 1
    assert step(err=ctypes.c_void_p(0x10001)) == 1 and step(B=1 << 20) == 3

    def accept(p_=p[0], noise=p[4], T=4, V=9, counts=p[7]):
        return lib.canopy_accept(p_, None, 0, p[1], p[2], None, p[3], noise, T, 2, V, p[5], p[6], counts, None, None)

    assert accept(p_=odd) == 1 and accept(noise=None) == 1 and accept(counts=None) == 1 and accept(T=0) == 1
    assert accept(T=257) == 3 and accept(V=1 << 25) == 3


def test_binding_refuses_what_is_not_on_a_gpu(canopy):
    """The native side turns it down and the Python side says why."""
    x = torch.zeros(2, 4, 128)
    with pytest.raises(canopy.CanopyError, match="CUDA"):
        canopy.step(x, x, x, torch.ones(2, 4), torch.ones(2, 4), torch.zeros(2, 4, 128, 128))
    with pytest.raises(canopy.CanopyError):
        canopy.step(None, x, x, torch.ones(2, 4), torch.ones(2, 4), torch.zeros(2, 4, 128, 128))
    with pytest.raises(canopy.CanopyError, match="CUDA"):
        canopy.prefill(x, x, x, x[..., 0], x[..., 0], None, torch.zeros(2, dtype=torch.int32),
                       torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(canopy.CanopyError):
        canopy.accept(torch.zeros(2, 3), None, None, None, None)
    with pytest.raises(canopy.CanopyError, match="CUDA"):
        canopy.accept(torch.zeros(1, 2, 5), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32),
                      torch.zeros(1, 2), torch.ones(1, 5))
    with pytest.raises(KeyError):
        canopy.prefill_plan(8, 1, 1, 1, True, 128, force="other")
