"""The ends of what the attention layers' calls take: the most streams, the deepest trees, pages larger than any
context, rows before the first sequence, trees of one node, and a first call that is captured."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
from attention_cases import TREES, U16, attend_case, cache, check_attend, rounded, tensor

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("tree", ["chain", "random", "wide"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 3)])
def test_largest_trees(lib, tree, window, sinks, bf16):
    check_attend(lib, attend_case(1, [256, 255, 225], [70, 0, 31], 4, 2, 64, 16, bf16, T=256, tree=TREES[tree]), window,
                 sinks)
    check_attend(lib, attend_case(2, [256], [33], 2, 1, 128, 64, bf16, T=256, tree=TREES[tree]), window, sinks)


@pytest.mark.parametrize("bf16", [True, False])
def test_trees_of_one_node(lib, bf16):
    check_attend(lib, attend_case(3, [1, 0, 1, 1], [0, 9, 64, 200], 8, 2, 128, 16, bf16, T=1, tree=TREES["chain"]))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("page", [512, 4096])
@pytest.mark.parametrize("HQ,HKV,d", [(8, 2, 128), (4, 4, 64)])
def test_large_pages(lib, page, HQ, HKV, d, bf16):
    check_attend(lib, attend_case(4, [1] * 3, [3, 600, 4500], HQ, HKV, d, page, bf16, T=1))
    check_attend(lib, attend_case(5, [300, 40], [10, 4090], HQ, HKV, d, page, bf16), 200, 5)


@pytest.mark.parametrize("bf16", [True, False])
def test_rows_before_the_first_sequence(lib, bf16):
    """starts[0] > 0: those rows belong to no stream and stay as they were, as do those behind the last."""
    rng = np.random.RandomState(6)
    HQ, HKV, d, page, lens, ctxs = 8, 2, 64, 16, [40, 1, 90], np.array([20, 300, 7], np.int32)
    c = attend_case(6, lens, ctxs, HQ, HKV, d, page, bf16)
    front, back, N = 13, 5, sum(lens)
    total = front + N + back
    x = {n: tensor(rounded(rng.standard_normal((total, H, d)), bf16), bf16) for n, H in (("q", HQ), ("k", HKV), ("v", HKV))}
    starts = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32, device="cuda")
    ws = lib.attend_workspace(total, 3, HQ, HKV, d)
    out = []
    for lo, hi, s in ((front, front + N, starts), (0, total, starts + front)):
        k, v, err = tensor(c["k"], bf16), tensor(c["v"], bf16), torch.zeros(1, dtype=torch.int32, device="cuda")
        args = dict(page_table=tensor(c["table"]), context=tensor(ctxs), starts=s)
        rows = [x[n][lo:hi].contiguous() for n in "qkv"]
        q, _ = lib.qk_prep(*rows, k_cache=k, v_cache=v, q_out=torch.full_like(rows[0], 7.0), err=err, **args)
        o = lib.attend(q, k, v, ws=ws, out=torch.full_like(q, 7.0), **args)
        assert int(err) == 0 and lib.read_device_error(ws) == 0
        out.append((q, o, k, v))
    for i in (0, 1):
        whole = out[1][i]
        assert (whole[:front] == 7).all() and (whole[front + N:] == 7).all()
        out[1] = (*out[1][:i], whole[front:front + N], *out[1][i + 1:])
    for a, b in zip(out[0][:1] + out[0][2:], out[1][:1] + out[1][2:]):
        assert torch.equal(a, b)
    # pieces may be cut elsewhere: weights and outputs are rounded once in either
    step = U16 if bf16 else 2.0 ** -16
    assert (out[0][1].float() - out[1][1].float()).abs().max() <= 4 * step * float(out[0][3].abs().max())


@pytest.mark.parametrize("bf16", [True, False])
def test_the_most_streams(lib, bf16):
    """65,535 streams of one token, in packed rows and as rows of their own: each sees itself and one token before."""
    B, HQ, HKV, d, page = 65535, 2, 1, 64, 16
    dt = torch.bfloat16 if bf16 else torch.float32
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    k_cache, v_cache = (torch.randn(B, HKV, page, d, device="cuda", generator=gen).to(dt) for _ in range(2))
    table = torch.randperm(B, device="cuda", generator=gen).int().view(B, 1)
    q, k, v = (torch.randn(B, H, d, device="cuda", generator=gen).to(dt) for H in (HQ, HKV, HKV))
    context = torch.ones(B, dtype=torch.int32, device="cuda")
    ws = lib.attend_workspace(B, B, HQ, HKV, d)
    got = []
    for starts in (None, torch.arange(B + 1, dtype=torch.int32, device="cuda")):
        kc, vc = k_cache.clone(), v_cache.clone()
        args = dict(k_cache=kc, v_cache=vc, page_table=table, context=context)
        qp, _ = lib.qk_prep(q, k, v, starts=starts, **args)
        got.append((qp, kc, vc, lib.attend(qp, ws=ws, starts=starts, **args)))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    qp, kc, vc, o = got[0]
    assert lib.read_device_error(ws) == 0
    at = table[:, 0].long()
    assert torch.equal(vc[at, :, 1], v) and torch.equal(vc[at, :, 0], v_cache[at, :, 0])
    K, V = kc[at, 0, :2].double(), vc[at, 0, :2].double()
    p = torch.softmax(d ** -0.5 * torch.einsum("bhd,bjd->bhj", qp.double(), K), -1)
    ref, weight = torch.einsum("bhj,bjd->bhd", p, V), torch.einsum("bhj,bjd->bhd", p, V.abs())
    # the scores, of sums of magnitudes below 40, are off by 40 (d + 4) half steps of fp32; weights and outputs are rounded
    bound = (2 * 40 * 68 * 2.0 ** -24 + 2.0 ** -20 + (U16 if bf16 else 0)) * weight + \
        (1.01 * U16 if bf16 else 2.0 ** -23) * ref.abs()
    assert ((o.double() - ref).abs() <= bound).all()
    parent = torch.full((B, 1), -1, dtype=torch.int32, device="cuda")
    accepted = torch.zeros(B, dtype=torch.int32, device="cuda")
    before = kc.clone()
    new = lib.cache_commit(accepted, parent, kc, vc, table, context)
    assert (new == 2).all() and torch.equal(kc, before)


FIRST = """
import torch
from gated_deltanet_linear_tree_gb300 import canopy
bf16, T = {bf16}, {T}
dt = torch.bfloat16 if bf16 else torch.float32
torch.manual_seed(0)
q, k, v = (torch.randn(2, T, H, 64, device="cuda").to(dt) for H in (4, 2, 2))
kc, vc = (torch.randn(40, 2, 16, 64, device="cuda").to(dt) for _ in range(2))
table = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
context = torch.tensor([100, 37], dtype=torch.int32, device="cuda")
parent = torch.arange(-1, T - 1, dtype=torch.int32, device="cuda").expand(2, T).contiguous()
accepted = torch.full((2,), T - 1, dtype=torch.int32, device="cuda")
ws = canopy.attend_workspace(2 * T, 2, 4, 2, 64)
args = dict(k_cache=kc, v_cache=vc, page_table=table)
def calls():
    p, _ = canopy.qk_prep(q, k, v, context=context, **args)
    o = canopy.attend(p, ws=ws, context=context, parent=parent, **args)
    return p, o, canopy.cache_commit(accepted, parent, context=context, **args)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
ref = calls()
assert all(torch.equal(a, b) for a, b in zip(got, ref))
assert canopy.read_device_error(ws) == 0
print("same")
"""


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T", [2, 40])
def test_first_calls_captured(lib, T, bf16):
    r = subprocess.run([sys.executable, "-c", FIRST.format(bf16=bf16, T=T)], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("lead", [(3, 5), (3, 1), (1, 5), (1, 1), (400, 3), (7,), (1,), (2500,)])
@pytest.mark.parametrize("native", [True, False])
def test_slices_of_a_projection(lib, lead, native, bf16, monkeypatch):
    """Queries, keys and values side by side in one buffer, with a gap behind them: the results of dense ones."""
    lib.load()
    if not native:
        monkeypatch.setattr(lib, "_marshal", type("Stub", (), {"qk_prep": staticmethod(lambda *a: None)}))
    HQ, HKV, d, page = 6, 2, 64, 16
    dt = torch.bfloat16 if bf16 else torch.float32
    torch.manual_seed(len(lead) + lead[0])
    wide = torch.randn(*lead, HQ + 2 * HKV + 1, d, device="cuda").to(dt)
    q, k, v, _ = wide.split([HQ, HKV, HKV, 1], -2)
    B, T = lead if len(lead) == 2 else (lead[0], 1)
    pages = -(-(T + 20) // page)
    caches = torch.randn(2, B * pages, HKV, page, d, device="cuda").to(dt)
    table = torch.randperm(B * pages, device="cuda").int().view(B, pages)
    context = torch.randint(0, 20, (B,), dtype=torch.int32, device="cuda")
    freqs = torch.rand(16, device="cuda")
    out = []
    for rows in ((q, k, v), [x.contiguous() for x in (q, k, v)]):
        mine = caches.clone()
        args = dict(lengths=torch.full((B,), max(1, T - 1), dtype=torch.int32, device="cuda")) if len(lead) == 2 else {}
        p, _ = lib.qk_prep(*rows, freqs=freqs, k_cache=mine[0], v_cache=mine[1], page_table=table, context=context,
                           q_out=torch.full((*lead, HQ, d), 7.0, device="cuda", dtype=dt), **args)
        out.append([p, mine, *lib.qk_prep(*rows[:2], norm="l2")])
    assert all(torch.equal(a, b) for a, b in zip(*out))
    assert not torch.equal(out[0][1], caches)
