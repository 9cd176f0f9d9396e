"""A prompt's o and S do not depend on the prompts beside it, bit for bit:
whether four blocks share a state of it, two or one, and wherever it starts,
the same products are formed of the same parts in the same order."""

import numpy as np
import pytest
import torch

from tests import serving_cases as sc

pytestmark = pytest.mark.gpu


def run(lib, t, starts):
    N, HV, B = t["v"].shape[0], t["v"].shape[1], len(starts) - 1
    ws = lib.prefill_workspace(N, B, HV, 128)
    o, S = lib.prefill(t["q"], t["k"], t["v"], t["g"], t["beta"], t["S0"],
                       torch.tensor(starts, dtype=torch.int32, device="cuda"), ws, force="chunked", scale=0.3)
    assert lib.read_device_error(ws) == 0
    return o, S


@pytest.mark.parametrize("kind", ["plain", "aligned", "forget", "rates"])
@pytest.mark.parametrize("length,others,H,HV", [
    (500, [64] * 47, 2, 2), (500, [700] * 30, 1, 2), (500, [130, 64, 1], 13, 13), (640, [600, 3, 0, 64] * 3, 2, 6),
    (77, [900] * 5, 3, 9), (1300, [70, 64, 1], 13, 26), (333, [300] * 200, 1, 1), (250, [250] * 39, 4, 16)])
def test_a_prompt_alone_and_beside_others(lib, length, others, H, HV, kind):
    lens = others[:1] + [length] + others[1:]
    x = sc.layer_inputs(lens, H, HV, 128, True, seed=length + HV, kind=kind)
    starts = x.pop("starts")
    t = sc.to_cuda(x, True)
    o, S = run(lib, t, starts.tolist())
    lo, hi = int(starts[1]), int(starts[2])
    for shift in (0, 1):  # alone, and as the second sequence behind one row
        pad = {n: torch.cat([t[n][:shift], t[n][lo:hi]]) for n in ("q", "k", "v", "g", "beta")}
        pad["S0"] = torch.cat([t["S0"][:shift], t["S0"][1:2]])
        o1, S1 = run(lib, pad, list(range(shift + 1)) + [shift + length])
        assert torch.equal(o1[shift:], o[lo:hi])
        assert torch.equal(S1[shift], S[1])
