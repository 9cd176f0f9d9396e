"""Packed sequences whose starts are out of order or out of range, and
workspaces that hold anything: the prefill over the starts as they are read,
against the float64 recurrence.

Starts are read as s_i, the largest of starts[0 .. i] after each is brought
into [0, N].  The bound is the one of the other prefill tests: 1e-4 of the
rms, fp32 sums of 128 terms with a factor of ten to spare."""

import numpy as np
import pytest
import torch

import oracle
from tests import serving_cases as sc
from tests.test_gpu_serving import PATHS, close

pytestmark = pytest.mark.gpu

INT_MAX, INT_MIN = 2 ** 31 - 1, -2 ** 31


def check(lib, starts, N, H, HV, force, bf16, d, seed):
    x = sc.layer_inputs([N], H, HV, d, bf16, seed=seed, kind="rates")
    B = len(starts) - 1
    rng = np.random.default_rng(seed)
    x["S0"] = (0.1 * rng.standard_normal((B, HV, d, d))).astype(np.float32)
    x["starts"] = np.array(starts, np.int32)
    read = np.maximum.accumulate(np.clip(np.array(starts, np.int64), 0, N))
    o_ref, S_ref = oracle.serving.recurrence(**dict(x, starts=read))
    t = sc.to_cuda(x, bf16)
    o = torch.full((N, HV, d), 7.0, device="cuda")
    ws = lib.prefill_workspace(N, B, HV, d)
    ws[256:] = 255  # NaN in every type
    _, S = lib.prefill(t["q"], t["k"], t["v"], t["g"], t["beta"], t["S0"], t["starts"], ws, force=force, out=o)
    assert lib.read_device_error(ws) == (0 if np.array_equal(read, starts) else lib.DEVERR_LENGTH)
    assert (o[:read[0]] == 7).all() and (o[read[-1]:] == 7).all()
    close(o[read[0]:read[-1]], o_ref[read[0]:read[-1]])
    close(S, S_ref)


@pytest.mark.parametrize("force,bf16,d", PATHS)
@pytest.mark.parametrize("starts", [
    [0, 384, 64, 512], [0, 130, 70, 10, 200, 190, 300], [40, 10, 300, 0, 310], [0, INT_MAX, 100, 512],
    [INT_MIN, 64, INT_MIN, 200, INT_MAX], [500, 0], [600, 100, 512], [0, 200, 200, 100, 200, 512, 511]],
    ids=lambda s: "_".join(map(str, s)))
def test_starts_out_of_order(lib, starts, force, bf16, d):
    check(lib, starts, 512, 1, 2, force, bf16, d, seed=len(starts))


@pytest.mark.parametrize("starts,HV", [([0, 384, 64, 512], 39), ([0, 500, 40, 100, 505, 512], 13)])
def test_starts_out_of_order_many_states(lib, starts, HV):
    """Enough states for a walk that is planned from the lengths."""
    check(lib, starts, 512, 1, HV, "chunked", True, 128, seed=HV)


@pytest.mark.parametrize("force,bf16,d", [("chunked", True, 128), ("scan", True, 128), ("scan", False, 32)])
@pytest.mark.parametrize("B", [31, 127, 128, 129, 1025, 2500])
@pytest.mark.parametrize("ordered", [True, False])
def test_many_sequences(lib, B, ordered, force, bf16, d):
    """Around the numbers from which the walk is not planned and the starts are
    ordered ahead."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 3, B)
    lens[B // 2] = 200
    starts = np.concatenate([[0], np.cumsum(lens)])
    if not ordered:
        starts[rng.integers(1, B, 9)] = rng.integers(-9, starts[-1] // 2, 9)
        starts[B // 3] = starts[B // 3 + 20]
    check(lib, starts.tolist(), int(lens.sum()), 1, 1, force, bf16, d, seed=B)


def test_one_workspace_for_calls_of_other_sizes(lib):
    """A workspace for the largest sizes, NaN beyond the error word at first, then whatever the calls leave."""
    HV = 3
    ws = lib.prefill_workspace(900, 1100, HV, 128)
    ws[256:] = 255
    for i, lens in enumerate([[300, 0, 65], [900], [1] * 5, [64, 128, 3], [0] * 1099 + [70], [30, 500, 2], [0, 0], [65]]):
        lens = lens if sum(lens) else lens + [1]
        x = sc.layer_inputs(lens, HV, HV, 128, True, seed=i, kind="rates")
        o_ref, S_ref = oracle.serving.recurrence(**x)
        t = sc.to_cuda(x, True)
        for force in ("chunked", "scan", "chunked"):
            o, S = lib.prefill(t["q"], t["k"], t["v"], t["g"], t["beta"], t["S0"], t["starts"], ws, force=force)
            close(o, o_ref)
            close(S, S_ref)
    assert lib.read_device_error(ws) == 0
