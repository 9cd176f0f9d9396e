"""qk_prep, attend and cache_commit on another stream behind work that is still running there, in a captured graph
that is replayed with other inputs, and through the Python side of the binding: the results of plain calls, bit for
bit; sequences without rows; two calls at once."""

import numpy as np
import pytest
import torch

from attention_cases import TREES, cache, rounded, tensor

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, T, PAGE = 5, 8, 2, 128, 20, 16


def inputs(seed, bf16=True):
    rng = np.random.RandomState(seed)
    lens = np.array([60, 0, 131, 1, 9])
    ctx = np.array([0, 40, 300, 17, 64]) + seed
    k, v = (rounded(rng.standard_normal((280, HKV, PAGE, D)), bf16) for _ in range(2))
    new = lambda n, H: tensor(rounded(rng.standard_normal((n, H, D)), bf16), bf16)  # noqa: E731
    x = {"k_cache": tensor(k, bf16), "v_cache": tensor(v, bf16)}
    order = rng.permutation(280)[:B * 50].reshape(B, 50).astype(np.int32)
    x.update(page_table=tensor(np.pad(order, ((0, 0), (0, 10)), constant_values=-1)), context=tensor(ctx.astype(np.int32)),
             starts=tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)))
    for n, rows in (("p", int(lens.sum())), ("t", B * T), ("s", B)):
        for name, H in (("q", HQ), ("k", HKV), ("v", HKV)):
            x[n + name] = new(rows, H) if n != "t" else new(rows, H).view(B, T, H, D)
    x["parent"] = tensor(np.stack([TREES["random"](T, rng) for _ in range(B)]).astype(np.int32))
    x["lengths"] = tensor(np.array([T, 0, 7, T, 1], np.int32))
    x["accepted"] = tensor(np.array([T - 1, -1, 6, 3, 0], np.int32))
    x["w"] = tensor((1 + 0.1 * rng.standard_normal(D)).astype(np.float32))
    x["freqs"] = tensor((1e4 ** (-np.arange(32) / 32)).astype(np.float32))
    return x


def layer(lib, x, ws):
    """Prompts, a tree and its commit, single tokens; window on the way."""
    cached = {n: x[n] for n in ("k_cache", "v_cache", "page_table")}
    args = dict(q_weight=x["w"], k_weight=x["w"], freqs=x["freqs"], **cached)
    q, _ = lib.qk_prep(x["pq"], x["pk"], x["pv"], context=x["context"], starts=x["starts"], **args)
    out = [q, lib.attend(q, *cached.values(), x["context"], ws, starts=x["starts"])]
    out.append(lib.attend(q, *cached.values(), x["context"], ws, starts=x["starts"], window=50, sinks=3))
    filled = {"q_out": torch.zeros_like(x["tq"])}
    q, _ = lib.qk_prep(x["tq"], x["tk"], x["tv"], context=x["context"], lengths=x["lengths"], **args, **filled)
    out += [q, lib.attend(q, *cached.values(), x["context"], ws, parent=x["parent"], lengths=x["lengths"],
                          out=torch.zeros_like(q))]
    ctx = lib.cache_commit(x["accepted"], x["parent"], *cached.values(), x["context"], lengths=x["lengths"])
    q, _ = lib.qk_prep(x["sq"], x["sk"], x["sv"], context=ctx, **args)
    out += [ctx, q, lib.attend(q, *cached.values(), ctx, ws)]
    out += list(lib.qk_prep(x["tq"], x["tk"], norm="l2"))
    return out + [x["k_cache"].clone(), x["v_cache"].clone()]


def equal(got, ref):
    return len(got) == len(ref) and all(torch.equal(y, r) for y, r in zip(got, ref))


def workspace(lib):
    return lib.attend_workspace(201, B, HQ, HKV, D)


@pytest.mark.parametrize("bf16", [True, False])
def test_on_another_stream(lib, bf16):
    ws = workspace(lib)
    first, second = inputs(1, bf16), inputs(2, bf16)
    ref = layer(lib, inputs(2, bf16), ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some 10 ms: what follows waits on this stream only
        for n in first:
            first[n].copy_(second[n])
        got = layer(lib, first, ws)
    side.synchronize()
    assert equal(got, ref)
    assert lib.read_device_error(ws) == 0


@pytest.mark.parametrize("bf16", [True, False])
def test_in_a_captured_graph(lib, bf16):
    ws = workspace(lib)
    x = inputs(3, bf16)
    layer(lib, x, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(lib, x, ws)
    for seed in (3, 4, 5):
        other = inputs(seed, bf16)
        for n in x:
            x[n].copy_(other[n])
        graph.replay()
        torch.cuda.synchronize()
        assert equal(got, layer(lib, other, ws))
    assert lib.read_device_error(ws) == 0


def test_two_streams_at_once(lib):
    a, b, wa, wb = inputs(6), inputs(7), workspace(lib), workspace(lib)
    ref = [layer(lib, inputs(s), wa) for s in (6, 7)]
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        x, y = {n: t.clone() for n, t in a.items()}, {n: t.clone() for n, t in b.items()}
        torch.cuda.synchronize()
        with torch.cuda.stream(one):
            p = layer(lib, x, wa)
        with torch.cuda.stream(two):
            q = layer(lib, y, wb)
        torch.cuda.synchronize()
        assert equal(p, ref[0]) and equal(q, ref[1])


def test_native_and_python_marshalling_agree(lib, monkeypatch):
    ws = workspace(lib)
    native = layer(lib, inputs(8), ws)
    lib.load()
    stub = type("Stub", (), {n: staticmethod(lambda *args: None) for n in ("qk_prep", "attend", "cache_commit")})
    monkeypatch.setattr(lib, "_marshal", stub)
    assert equal(layer(lib, inputs(8), ws), native)


@pytest.mark.parametrize("rows,ctx", [(1, 2000), (130, 900), (700, 3000)])
def test_the_next_call_waits(lib, rows, ctx):
    """A call that overwrites what the one before it reads (its queries, its keys) comes after it, pieces cut or not."""
    rng = np.random.RandomState(rows)
    k, v, table = cache(rng, [ctx + rows], 1, D, 64, True)
    q0 = tensor(rounded(rng.standard_normal((rows, 2, D)), True), True)
    k0, v0 = tensor(k, True), tensor(v, True)
    td, cd = tensor(table), tensor(np.array([ctx], np.int32))
    starts = tensor(np.array([0, rows], np.int32))
    ws = lib.attend_workspace(rows, 1, 2, 1, D)
    ref = lib.attend(q0, k0, v0, td, cd, ws, starts=starts)
    new = torch.ones(rows, 1, D, device="cuda", dtype=torch.bfloat16)
    for _ in range(20):
        q, kd, vd = q0.clone(), k0.clone(), v0.clone()
        torch.cuda.synchronize()
        o = lib.attend(q, kd, vd, td, cd, ws, starts=starts)
        lib.qk_prep(q, new, new, norm="l2", q_out=q, k_cache=kd, v_cache=vd, page_table=td, context=cd, starts=starts)
        p = lib.attend(q, kd, vd, td, cd, ws, starts=starts)
        torch.cuda.synchronize()
        assert torch.equal(o, ref)
        assert torch.equal(p, lib.attend(q, kd, vd, td, cd, ws, starts=starts))


def test_no_rows_at_all(lib):
    """Sequences whose rows are all missing: nothing is written."""
    x, ws = inputs(9), workspace(lib)
    none, before = torch.zeros(B, dtype=torch.int32, device="cuda"), [x["k_cache"].clone(), x["v_cache"].clone()]
    cached = [x[n] for n in ("k_cache", "v_cache", "page_table")]
    out = torch.full_like(x["tq"], 3.0)
    lib.attend(x["tq"], *cached, x["context"], ws, parent=x["parent"], lengths=none, out=out)
    lib.attend(x["pq"], *cached, x["context"], ws, starts=torch.zeros(B + 1, dtype=torch.int32, device="cuda"),
               out=(o := torch.full_like(x["pq"], 3.0)))
    lib.qk_prep(x["tq"], x["tk"], x["tv"], context=x["context"], lengths=none, q_out=(q := torch.full_like(out, 3.0)),
                k_cache=cached[0], v_cache=cached[1], page_table=cached[2])
    assert (out == 3).all() and (o == 3).all() and (q == 3).all()
    assert torch.equal(before[0], x["k_cache"]) and torch.equal(before[1], x["v_cache"])
    assert lib.read_device_error(ws) == 0


def test_many_sequences(lib):
    """More sequences than the kernel for few rows plans by itself."""
    n, d = 700, 64
    rng = np.random.RandomState(0)
    ctx = rng.randint(0, 90, size=n)
    k, v, table = cache(rng, ctx + 1, 1, d, 16, True)
    q = tensor(rounded(rng.standard_normal((n, 3, d)), True), True)
    kd, vd, td, cd = tensor(k, True), tensor(v, True), tensor(table), tensor(ctx.astype(np.int32))
    ws = lib.attend_workspace(n, n, 3, 1, d)
    o = lib.attend(q, kd, vd, td, cd, ws)
    for i in range(0, n, 50):  # the same streams, fifty at a time
        part = slice(i, i + 50)
        w = lib.attend_workspace(50, 50, 3, 1, d)
        ref = lib.attend(q[part].contiguous(), kd, vd, td[part].contiguous(), cd[part].contiguous(), w)
        assert (o[part].float() - ref.float()).abs().max() <= 2 ** -6  # cut elsewhere: some weights' roundings
    assert lib.read_device_error(ws) == 0
