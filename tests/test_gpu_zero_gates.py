"""Gates of zero (what exp(-x) leaves in fp32 from x = 104 on) in the prefill
and the step: the state before the token is forgotten and the token written,
as the recurrence in float64 says.  Bound: 1e-4 of the rms (fp32 sums)."""

import numpy as np
import pytest
import torch

import oracle
from tests import serving_cases as sc
from tests.test_gpu_serving import PATHS, close, prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("force,bf16,d", PATHS)
@pytest.mark.parametrize("at", [[0], [31], [32], [63], [64], [149], [15, 16, 17, 100, 127], list(range(150))],
                         ids=lambda x: f"{x[0]}x{len(x)}")
def test_prefill_zero_gates(lib, force, bf16, d, at):
    """At the ends of a chunk and of its halves, in a row, and throughout; one head's gates only."""
    x = sc.layer_inputs([150, 70], 2, 4, d, bf16, seed=at[0], kind="rates")
    x["g"][at, 1] = 0.0
    x["g"][150 + np.array(at[:1]) % 70, 2] = -0.0
    o_ref, S_ref = oracle.serving.recurrence(**x)
    o, S, err = prefill(lib, sc.to_cuda(x, bf16), force, d)
    assert err == 0
    close(o, o_ref)
    close(S, S_ref)


def test_prefill_zero_gates_many_states(lib):
    x = sc.layer_inputs([300, 64, 65, 1], 13, 39, 128, True, seed=1, kind="rates")
    x["g"][np.random.default_rng(2).random(x["g"].shape) < 0.02] = 0.0
    o_ref, S_ref = oracle.serving.recurrence(**x)
    o, S, err = prefill(lib, sc.to_cuda(x, True), "chunked", 128)
    assert err == 0
    close(o, o_ref)
    close(S, S_ref)


@pytest.mark.parametrize("bf16,d", [(True, 128), (False, 128), (False, 32)])
def test_step_zero_gates(lib, bf16, d):
    x = sc.layer_inputs([1] * 5, 2, 4, d, bf16, seed=3)
    x["g"][[0, 2, 4], [1, 3, 0]] = 0.0
    o_ref, S_ref = oracle.serving.recurrence(scale=0.3, **x)
    t = sc.to_cuda(x, bf16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, S = lib.step(*[t[n] for n in ("q", "k", "v", "g", "beta")], t["S0"], scale=0.3, err=err)
    assert int(err) == 0
    close(o, o_ref)
    close(S, S_ref)


@pytest.mark.parametrize("force,bf16,d", PATHS)
@pytest.mark.parametrize("bad", [-0.5, np.nan, np.inf])
def test_gates_that_are_still_refused(lib, force, bf16, d, bad):
    """Reported, and read with the write strength as g = 1, beta = 0."""
    x = sc.layer_inputs([40, 50], 2, 2, d, bf16, seed=6)
    t = sc.to_cuda(x, bf16)
    t["g"][41, 1] = bad
    o, S, err = prefill(lib, t, force, d)
    assert err == lib.DEVERR_GATE
    x["g"][41, 1], x["beta"][41, 1] = 1.0, 0.0
    o_ref, S_ref = oracle.serving.recurrence(**x)
    close(o, o_ref)
    close(S, S_ref)
    one = {n: t[n][41:42].clone() for n in ("q", "k", "v", "g", "beta")}
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, S1 = lib.step(*one.values(), t["S0"][:1], err=word)
    assert int(word) == lib.DEVERR_GATE and torch.equal(S1[0, 1], t["S0"][0, 1])
