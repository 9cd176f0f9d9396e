"""Step, prefill and accept on a stream other than the default one, behind
work that is still running there, and in a captured graph that is replayed
with other inputs: the results of plain calls, bit for bit."""

import pytest
import torch

from tests import serving_cases as sc

pytestmark = pytest.mark.gpu


def inputs(seed):
    lens = [130, 0, 70, 1]
    x = sc.to_cuda(sc.layer_inputs(lens, 2, 4, 128, True, seed=seed, kind="rates"), True)
    a = {n: torch.from_numpy(v).cuda() for n, v in sc.accept_inputs(3, 12, 9001, seed=seed, kind="wide").items()
         if v is not None}
    return {**x, **{"a_" + n: v for n, v in a.items()}}


LAYER = ("q", "k", "v", "g", "beta")


def loop(lib, x, ws):
    """Prompts either way, a step from the states they leave, an acceptance."""
    out = []
    for force in ("chunked", "scan"):
        o, S = lib.prefill(*[x[n] for n in LAYER], x["S0"], x["starts"], ws, force=force)
        o1, S1 = lib.step(*[x[n][:4] for n in LAYER], S, o_dtype=torch.bfloat16)
        out += [o, S, o1, S1]
    return out + list(lib.accept(*[x["a_" + n] for n in ("p", "tokens", "parent", "u", "noise")], q=x["a_q"]))


def equal(got, ref):
    return len(got) == len(ref) and all(torch.equal(y, r) for y, r in zip(got, ref))


def test_on_another_stream(lib):
    ws = lib.prefill_workspace(201, 4, 4, 128)
    first, second = inputs(1), inputs(2)
    ref = loop(lib, second, ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some 10 ms: what follows waits on this stream only
        for n in first:
            first[n].copy_(second[n])
        got = loop(lib, first, ws)
    side.synchronize()
    assert equal(got, ref)
    assert lib.read_device_error(ws) == 0


def test_in_a_captured_graph(lib):
    ws = lib.prefill_workspace(201, 4, 4, 128)
    x = inputs(3)
    for _ in range(2):
        loop(lib, x, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = loop(lib, x, ws)
    for seed in (3, 4, 5):
        other = inputs(seed)
        for n in x:
            x[n].copy_(other[n])
        graph.replay()
        torch.cuda.synchronize()
        assert equal(got, loop(lib, other, ws))
    assert lib.read_device_error(ws) == 0
