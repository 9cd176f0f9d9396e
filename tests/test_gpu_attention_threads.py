"""The attention layers' calls from several threads at once, each on a stream and a workspace of its own, and captured
graphs that share a workspace and are replayed by turns: the results of plain calls, bit for bit."""

import threading

import pytest
import torch

from test_gpu_attention_streams import equal, inputs, layer, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bf16", [True, False])
def test_threads(lib, bf16):
    seeds = (1, 2, 3, 4)
    ref = {s: layer(lib, inputs(s, bf16), workspace(lib)) for s in seeds}
    xs = {s: [inputs(s, bf16) for _ in range(6)] for s in seeds}
    spaces = {s: workspace(lib) for s in seeds}
    torch.cuda.synchronize()
    out, failed = {s: [] for s in seeds}, []

    def work(s):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for x in xs[s]:
                    out[s].append(layer(lib, x, spaces[s]))
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in seeds]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for s in seeds:
        assert len(out[s]) == 6 and all(equal(o, ref[s]) for o in out[s])
        assert lib.read_device_error(spaces[s]) == 0


@pytest.mark.parametrize("bf16", [True, False])
def test_graphs_that_share_a_workspace(lib, bf16):
    ws, seeds = workspace(lib), (5, 6)
    ref = {s: layer(lib, inputs(s, bf16), workspace(lib)) for s in seeds}
    xs, graphs, got = {s: inputs(s, bf16) for s in seeds}, {}, {}
    torch.cuda.synchronize()
    for s in seeds:
        graphs[s] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[s]):
            got[s] = layer(lib, xs[s], ws)
    for _ in range(3):
        for s in seeds:
            for n, t in inputs(s, bf16).items():
                xs[s][n].copy_(t)
        for s in seeds:  # behind one another on one stream
            graphs[s].replay()
        torch.cuda.synchronize()
        assert all(equal(got[s], ref[s]) for s in seeds)
    assert lib.read_device_error(ws) == 0
