"""The serving-loop operators (prefill, step, accept) on the GPU against their
float64 definitions.

Tolerances.  The states, U and the products are fp32 with operands of 24 bits
on both paths, so that errors are those of fp32 sums of 128 (and 64) terms:
about sqrt(128) 2^-24 = 7e-7 of the result's rms for one product, and a few
times that through the three products of a chunk; the largest of up to 10^6
elements sits 5 standard deviations out.  1e-4 of the rms (the framework's
fp32 bound) leaves a factor of ten.  "aligned" inputs subtract terms of the
size of their sum at every token and have the same bound.  A bf16 output is
the fp32 output rounded once, bit for bit."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from tests import serving_cases as sc

pytestmark = pytest.mark.gpu

TOL = 1e-4


def close(x, ref):
    x = x.cpu().numpy().astype(np.float64)
    rms = np.sqrt((ref ** 2).mean()) if ref.size else 0.0
    assert (np.abs(x - ref) <= TOL * rms).all(), float(np.abs(x - ref).max() / max(rms, 1e-300))


# ---- step ------------------------------------------------------------------


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("B,H,HV,d", [(1, 1, 1, 128), (3, 2, 6, 128), (5, 4, 4, 32), (70, 3, 3, 128)])
def test_step(lib, B, H, HV, d, bf16):
    x = sc.layer_inputs([1] * B, H, HV, d, bf16, seed=B)
    o_ref, S_ref = oracle.serving.recurrence(scale=0.3, **x)
    t = sc.to_cuda(x, bf16)
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, S = lib.step(*args, t["S0"], scale=0.3, err=err)
    close(o, o_ref)
    close(S, S_ref)
    keep = t["S0"].clone()
    o16, S2 = lib.step(*args, keep, S_out=keep, scale=0.3, o_dtype=torch.bfloat16, err=err)  # in place
    assert torch.equal(o16, o.bfloat16())
    assert S2.data_ptr() == keep.data_ptr() and torch.equal(keep, S)
    assert int(err) == 0


def test_step_bad_gate_is_reported_and_contained(lib):
    x = sc.layer_inputs([1] * 4, 2, 2, 128, True, seed=9)
    good = sc.to_cuda(x, True)
    o0, S0 = lib.step(*[good[n] for n in ("q", "k", "v", "g", "beta")], good["S0"])
    x["g"][2, 1] = np.nan
    x["beta"][3, 0] = np.inf
    t = sc.to_cuda(x, True)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, S = lib.step(*[t[n] for n in ("q", "k", "v", "g", "beta")], t["S0"], err=err)
    assert int(err) == lib.DEVERR_GATE
    ok = torch.ones(4, 2, dtype=torch.bool, device="cuda")
    ok[2, 1] = ok[3, 0] = False
    assert torch.equal(S[ok], S0[ok]) and torch.equal(o[ok], o0[ok])
    assert torch.equal(S[~ok], t["S0"][~ok])  # read as g = 1, beta = 0


# ---- prefill ----------------------------------------------------------------

PATHS = [("chunked", True, 128), ("scan", True, 128), ("scan", False, 128), ("scan", False, 32), ("scan", True, 32)]
LENS = [[1], [37], [64], [65], [0, 5, 128, 0], [200, 1, 0, 63, 129], [16, 16, 17]]


def prefill(lib, t, force, d, **kw):
    N, B, HV = t["v"].shape[0], t["starts"].numel() - 1, t["v"].shape[1]
    ws = lib.prefill_workspace(N, B, HV, d)
    S0 = kw.pop("S0") if "S0" in kw else t["S0"]
    o, S = lib.prefill(t["q"], t["k"], t["v"], t["g"], t["beta"], S0, t["starts"], ws, force=force, **kw)
    return o, S, lib.read_device_error(ws)


@pytest.mark.parametrize("force,bf16,d", PATHS)
@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x)))
def test_prefill(lib, force, bf16, d, lens):
    H, HV = [(1, 1), (2, 6), (3, 3)][sum(lens) % 3]
    x = sc.layer_inputs(lens, H, HV, d, bf16, seed=sum(lens) + d)
    o_ref, S_ref = oracle.serving.recurrence(scale=0.3, **x)
    t = sc.to_cuda(x, bf16)
    o, S, err = prefill(lib, t, force, d, scale=0.3)
    assert err == 0
    close(o, o_ref)
    close(S, S_ref)
    o16, S16, _ = prefill(lib, t, force, d, scale=0.3, o_dtype=torch.bfloat16, S_out=t["S0"])  # in place
    assert torch.equal(o16, o.bfloat16())
    assert torch.equal(S16, S) and S16.data_ptr() == t["S0"].data_ptr()


@pytest.mark.parametrize("lens,H,HV", [([130, 1, 0, 64, 77, 191], 7, 14), ([320], 26, 78), ([3] * 140, 1, 1),
                                       ([200, 65, 0, 130], 8, 24), ([1, 127], 24, 72)])
def test_prefill_many_states(lib, lens, H, HV):
    """Enough (sequence, value head) pairs for two chains of value columns per block, and more sequences than
    are started by length."""
    x = sc.layer_inputs(lens, H, HV, 128, True, seed=HV, kind="rates")
    o_ref, S_ref = oracle.serving.recurrence(**x)
    o, S, err = prefill(lib, sc.to_cuda(x, True), "chunked", 128)
    assert err == 0
    close(o, o_ref)
    close(S, S_ref)


@pytest.mark.parametrize("lens,HV", [([1300, 70, 64, 1], 26), ([1300, 800, 70, 64, 10, 1], 17), ([3, 700], 51)])
@pytest.mark.parametrize("o_bf16", [False, True])
def test_prefill_uneven_batches(lib, lens, HV, o_bf16):
    """One prompt much longer than the rest, whose states are shared by two or four blocks."""
    x = sc.layer_inputs(lens, HV, HV, 128, True, seed=HV, kind="rates")
    o_ref, S_ref = oracle.serving.recurrence(**x)
    t = sc.to_cuda(x, True)
    o, S, err = prefill(lib, t, "chunked", 128)
    assert err == 0
    close(o, o_ref)
    close(S, S_ref)
    if o_bf16:
        rounded, S2, _ = prefill(lib, t, "chunked", 128, out=torch.empty_like(o, dtype=torch.bfloat16))
        assert torch.equal(rounded, o.bfloat16()) and torch.equal(S, S2)


@pytest.mark.parametrize("N,lo,hi,HV", [(2100, 0, 2100, 2), (2112, 70, 2001, 4), (2048, 0, 2048, 36),
                                        (2304, 1200, 2304, 26), (2100, 0, 10, 2), (2200, 2150, 2200, 30)])
def test_prefill_one_long_sequence(lib, N, lo, hi, HV):
    """A prompt of many chunks, or what is left of one, anywhere in rows that are otherwise NaN."""
    x = sc.layer_inputs([hi - lo], HV, HV, 128, True, seed=HV, kind="rates")
    o_ref, S_ref = oracle.serving.recurrence(**x)
    t = sc.to_cuda(x, True)
    y = {n: torch.full((N, *t[n].shape[1:]), float("nan"), dtype=t[n].dtype, device="cuda")
         for n in ("q", "k", "v", "g", "beta")}
    for n in y:
        y[n][lo:hi] = t[n]
    y["starts"] = torch.tensor([lo, hi], dtype=torch.int32, device="cuda")
    o = torch.full((N, HV, 128), 7.0, device="cuda")
    for again in range(3):  # the workspace's earlier contents do not matter, nor is a call in another's way
        S = t["S0"].clone()
        y["S0"] = S
        _, _, err = prefill(lib, y, "chunked", 128, out=o, S_out=S)
        assert err == 0
        close(o[lo:hi], o_ref)
        close(S, S_ref)
    assert (o[:lo] == 7).all() and (o[hi:] == 7).all()


@pytest.mark.parametrize("force,bf16,d", PATHS)
@pytest.mark.parametrize("kind", ["aligned", "forget", "rates"])
def test_prefill_hard_inputs(lib, force, bf16, d, kind):
    x = sc.layer_inputs([150, 90], 2, 4, d, bf16, seed=5, kind=kind)
    o_ref, S_ref = oracle.serving.recurrence(**x)
    o, S, err = prefill(lib, sc.to_cuda(x, bf16), force, d)
    assert err == 0
    close(o, o_ref)
    close(S, S_ref)


@pytest.mark.parametrize("force,bf16,d", PATHS)
def test_prefill_zero_states_and_split_prompts(lib, force, bf16, d):
    """S0 None is a zero state, and a prompt in two calls ends where one call ends."""
    x = sc.layer_inputs([100, 130], 2, 2, d, bf16, seed=8, kind="rates")
    zero = dict(x, S0=None)
    o_ref, S_ref = oracle.serving.recurrence(**zero)
    t = sc.to_cuda(x, bf16)
    o, S, _ = prefill(lib, t, force, d, S0=None)
    close(o, o_ref)
    close(S, S_ref)
    cut = 70  # the second prompt's first 70 tokens, then the rest
    part = {n: t[n][100:230].contiguous() for n in ("q", "k", "v", "g", "beta")}
    S1 = None
    outs = []
    for lo, hi in ((0, cut), (cut, 130)):
        y = {n: part[n][lo:hi].contiguous() for n in part}
        y["starts"] = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
        o1, S1, _ = prefill(lib, y, force, d, S0=S1)
        outs.append(o1)
    close(torch.cat(outs), o_ref[100:])
    close(S1[0], S_ref[1])


@pytest.mark.parametrize("force,bf16,d", PATHS)
def test_prefill_keeps_sequences_apart(lib, force, bf16, d):
    """NaN and infinities in one sequence, and in the packed rows of no
    sequence, leave the others' results alone, bit for bit."""
    lens = [30, 70, 45]
    x = sc.layer_inputs(lens, 2, 2, d, bf16, seed=4)
    t = sc.to_cuda(x, bf16)
    o0, S0, _ = prefill(lib, t, force, d)
    bad = {n: v.clone() for n, v in t.items()}
    bad["q"][30:100] = float("nan")
    bad["k"][30:100] = float("inf")
    bad["v"][30:100] = float("nan")
    bad["S0"][1] = float("nan")
    o1, S1, _ = prefill(lib, bad, force, d)
    for b, s in ((0, slice(0, 30)), (2, slice(100, 145))):
        assert torch.equal(o0[s], o1[s]) and torch.equal(S0[b], S1[b])
    # sequences that do not cover the packed rows: the others' rows of o stay as they were
    bad["starts"] = torch.tensor([3, 30, 30, 30], dtype=torch.int32, device="cuda")
    out = torch.full_like(o0, 7.0)
    prefill(lib, bad, force, d, out=out)
    assert (out[:3] == 7).all() and (out[30:] == 7).all() and not (out[3:30] == 7).all()


@pytest.mark.parametrize("force,bf16,d", PATHS)
def test_prefill_reports_bad_starts_and_gates(lib, force, bf16, d):
    x = sc.layer_inputs([40, 50], 2, 2, d, bf16, seed=6)
    t = sc.to_cuda(x, bf16)
    for starts in ([0, 95, 90], [-5, 40, 90], [0, 60, 40]):
        y = dict(t, starts=torch.tensor(starts, dtype=torch.int32, device="cuda"))
        assert prefill(lib, y, force, d)[2] == lib.DEVERR_LENGTH
    y = dict(t, g=t["g"].clone())
    y["g"][41, 1] = 0.0
    assert prefill(lib, y, force, d)[2] == lib.DEVERR_GATE
    x["g"][41, 1], x["beta"][41, 1] = 1.0, 0.0  # what it is read as
    o_ref, S_ref = oracle.serving.recurrence(**x)
    o, S, _ = prefill(lib, y, force, d)
    close(o, o_ref)
    close(S, S_ref)


# ---- accept -----------------------------------------------------------------


def run_accept(lib, x, bf16=False, err=None):
    dt = torch.bfloat16 if bf16 else torch.float32
    t = {n: None if v is None else torch.from_numpy(np.ascontiguousarray(v)).cuda() for n, v in x.items()}
    q = None if t["q"] is None else t["q"].to(dt)
    got = lib.accept(t["p"].to(dt), t["tokens"], t["parent"], t["u"], t["noise"], q=q, lengths=t["lengths"], err=err)
    return [y.cpu().numpy() for y in got]


def same(got, ref):
    for y, r in zip(got, ref):
        assert np.array_equal(y, r)


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("B,T,V,kind,ragged", [
    (1, 1, 1, "chain", False), (2, 2, 3, "chain", False), (3, 8, 1000, "chain", False), (5, 33, 777, "random", True),
    (4, 64, 4096, "wide", True), (2, 40, 5003, "star", False), (1, 256, 2048, "random", False),
    (2, 12, 50021, "random", False), (70, 9, 130, "random", True), (2, 7, 140001, "star", False)])
def test_accept(lib, B, T, V, kind, ragged, bf16, draft):
    for spread in (0.5, 4.0):
        x = sc.accept_inputs(B, T, V, seed=V + T, kind=kind, draft=draft, bf16=bf16, spread=spread, ragged=ragged)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        same(run_accept(lib, x, bf16, err), oracle.serving.accept(**x))
        assert int(err) == 0


@pytest.mark.parametrize("B,V", [(2, 70001), (9, 131072), (10, 131075), (1, 196608), (1, 196609), (3, 53249)])
def test_accept_slices(lib, B, V):
    """Vocabularies around the sizes from which a block's slice is held in part or not at all."""
    x = sc.accept_inputs(B, 6, V, seed=B + V, kind="star", draft=True)
    same(run_accept(lib, x), oracle.serving.accept(**x))


def test_accept_draft_equal_to_target(lib):
    """With p = q every first child is accepted (u < 1), down to a leaf."""
    x = sc.accept_inputs(6, 20, 999, seed=1)
    x["q"] = x["p"].copy()
    rng = np.random.default_rng(2)
    for b in range(6):
        for c in range(1, 20):
            x["tokens"][b, c] = np.argmax(x["q"][b, x["parent"][b, c]] / rng.exponential(size=999))
    got = run_accept(lib, x)
    same(got, oracle.serving.accept(**x))
    for b in range(6):
        assert not (x["parent"][b] == got[0][b]).any()


@pytest.mark.parametrize("draft", [True, False])
def test_accept_residual_zero_falls_back_to_the_target(lib, draft):
    """A row whose whole mass is refused: the next token comes from the row itself."""
    x = sc.accept_inputs(2, 3, 50, seed=2, kind="star", draft=draft)
    x["p"][:] = 0
    x["p"][:, :, 17] = 1
    x["tokens"][:] = 17
    x["u"][:] = 1.0  # outside [0, 1): refuses what has the whole mass
    if draft:
        x["q"] = x["p"].copy()
    got = run_accept(lib, x)
    same(got, oracle.serving.accept(**x))
    assert (got[0] == 0).all() and (got[1][:, 0] == 17).all() and (got[2] == 1).all()


def test_accept_ties_go_to_the_lowest_index(lib):
    x = sc.accept_inputs(3, 2, 5000, seed=3, kind="chain")
    x["p"][:] = np.float32(1 / 4096)
    x["p"][:, :, 4096:] = 0
    x["noise"][:] = 1
    x["noise"][:, [4000, 123, 2500]] = 0.5
    x["lengths"] = np.ones(3, np.int32)
    got = run_accept(lib, x)
    assert (got[1][:, 0] == 123).all()
    same(got, oracle.serving.accept(**x))


def test_accept_rows_past_the_length_are_not_looked_at(lib):
    x = sc.accept_inputs(4, 16, 600, seed=4, ragged=True)
    x["lengths"][:] = [0, 1, 9, 16]
    ref = oracle.serving.accept(**x)
    for b, n in enumerate(x["lengths"]):
        x["p"][b, n:] = np.nan
        x["q"][b, n:] = np.nan
        x["tokens"][b, n:] = -9
        x["parent"][b, n:] = 99
        x["u"][b, n:] = np.nan
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    same(run_accept(lib, x, err=err), ref)
    assert int(err) == 0


def test_accept_reports_bad_trees_tokens_and_lengths(lib):
    base = sc.accept_inputs(2, 8, 300, seed=5, kind="random")
    for change, bit in ((lambda x: x["parent"].__setitem__((0, 5), 6), lib.DEVERR_TREE),
                        (lambda x: x["tokens"].__setitem__((1, 3), 300), lib.DEVERR_TOKEN),
                        (lambda x: x["tokens"].__setitem__((1, 3), -1), lib.DEVERR_TOKEN),
                        (lambda x: x.__setitem__("lengths", np.array([8, 9], np.int32)), lib.DEVERR_LENGTH)):
        x = {n: None if v is None else v.copy() for n, v in base.items()}
        change(x)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = run_accept(lib, x, err=err)
        assert int(err) == bit
        assert ((got[0] >= 0) & (got[0] < 8)).all() and ((got[2] >= 1) & (got[2] <= 8)).all()
        run_accept(lib, x)  # and without an error word


# ---- together, and refusals --------------------------------------------------


def test_serving_loop(lib):
    """Prompts, then rounds of verify, accept and commit, then single steps:
    the state is the recurrence's over the prompt and the emitted tokens."""
    B, H, HV, d, T, V = 3, 2, 4, 128, 12, 400
    lens = [70, 5, 130]
    rng = np.random.default_rng(7)
    x = sc.layer_inputs(lens, H, HV, d, True, seed=7, kind="rates")
    _, S_ref = oracle.serving.recurrence(**x)
    _, S, _ = prefill(lib, sc.to_cuda(x, True), None, d)
    close(S, S_ref)
    ws = lib.workspace(B, T, HV, d)
    for rnd in range(3):
        y = sc.layer_inputs([T] * B, H, HV, d, True, seed=20 + rnd, kind="rates")
        a = sc.accept_inputs(B, T, V, seed=30 + rnd, ragged=rnd == 2)
        if a["lengths"] is not None:
            a["lengths"] = np.maximum(a["lengths"], 1)
        t = sc.to_cuda(y, True)
        tree = {n: t[n].reshape((B, T) + tuple(t[n].shape[1:])) for n in ("q", "k", "v", "g", "beta")}
        parent = torch.from_numpy(a["parent"]).cuda()
        lengths = None if a["lengths"] is None else torch.from_numpy(a["lengths"]).cuda()
        lib.verify(tree["q"], tree["k"], tree["v"], tree["g"], tree["beta"], S, parent, ws, lengths=lengths)
        u, noise = torch.from_numpy(a["u"]).cuda(), torch.from_numpy(a["noise"]).cuda()
        accepted, out, counts = lib.accept(torch.from_numpy(a["p"]).cuda(), torch.from_numpy(a["tokens"]).cuda(),
                                           parent, u, noise, q=torch.from_numpy(a["q"]).cuda(), lengths=lengths)
        S = lib.commit(accepted, S, tree["k"], parent, ws, lengths=lengths)
        ref = oracle.serving.accept(**a)
        same([z.cpu().numpy() for z in (accepted, out, counts)], ref)
        for b in range(B):
            path, n = [], int(ref[0][b])
            while n >= 0:
                path.insert(0, b * T + n)
                n = int(a["parent"][b, n])
            z = {m: y[m][path] for m in ("q", "k", "v", "g", "beta")}
            _, s1 = oracle.serving.recurrence(**z, S0=S_ref[b:b + 1], starts=[0, len(path)])
            S_ref[b] = s1[0]
        bound = 1e-2 * np.sqrt((S_ref ** 2).mean())  # the verify's own bf16-path bound
        assert (np.abs(S.cpu().numpy() - S_ref) <= bound).all()
    assert lib.read_device_error(ws) == 0


def test_refusals(lib):
    x = sc.to_cuda(sc.layer_inputs([4, 4], 2, 4, 128, True, seed=1), True)
    ws = lib.prefill_workspace(8, 2, 4, 128)
    E = lib.CanopyError

    def pre(**kw):
        y = {**x, "ws": ws, **kw}
        return lib.prefill(y["q"], y["k"], y["v"], y["g"], y["beta"], y["S0"], y["starts"], y["ws"],
                           **{n: y[n] for n in ("out", "S_out", "force", "scale") if n in y})

    pre()
    for kw in (dict(q=x["q"].half()), dict(q=x["q"].cpu()), dict(k=x["k"][:, :1]), dict(v=x["v"].float()),
               dict(v=x["v"][:, :3].contiguous(), g=x["g"][:, :3].contiguous(), beta=x["beta"][:, :3].contiguous(),
                    S0=x["S0"][:, :3].contiguous()),
               dict(q=x["q"].transpose(0, 1)), dict(g=x["g"].double()), dict(S0=x["S0"][:1]),
               dict(starts=x["starts"].long()), dict(starts=x["starts"][:1]), dict(ws=ws[:64]),
               dict(out=torch.empty(8, 4, 64, device="cuda")), dict(scale=float("nan")),
               dict(S_out=x["S0"].double())):
        with pytest.raises(E):
            pre(**kw)
    one = {n: x[n][:2].contiguous() for n in ("q", "k", "v", "g", "beta")}
    for kw in (dict(S=x["S0"].transpose(2, 3)), dict(q=one["q"][:1]), dict(v=one["v"][:, :3].contiguous()),
               dict(err=torch.zeros(1, device="cuda")), dict(scale=float("inf"))):
        y = {**one, "S": x["S0"], **kw}
        with pytest.raises(E):
            lib.step(y["q"], y["k"], y["v"], y["g"], y["beta"], y["S"],
                     **{n: y[n] for n in ("err", "scale") if n in y})
    a = sc.accept_inputs(2, 4, 32, seed=1)
    t = {n: torch.from_numpy(v).cuda() for n, v in a.items() if v is not None}
    good = dict(p=t["p"], tokens=t["tokens"], parent=t["parent"], u=t["u"], noise=t["noise"], q=t["q"])
    lib.accept(**good)
    for kw in (dict(p=t["p"].half()), dict(q=t["q"].bfloat16()), dict(q=t["q"][:, :2]),
               dict(tokens=t["tokens"].long()), dict(u=t["u"].double()), dict(noise=t["noise"][:1]),
               dict(lengths=torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(E):
            lib.accept(**dict(good, **kw))
    big = torch.zeros(1, 257, 4, device="cuda")
    with pytest.raises(E):
        lib.accept(big, *(torch.zeros(1, 257, dtype=torch.int32, device="cuda") for _ in range(2)),
                   torch.zeros(1, 257, device="cuda"), torch.ones(1, 4, device="cuda"))


def test_native_and_python_marshalling_agree(lib, monkeypatch):
    """The native side's calls and the Python side's give the same results,
    with given outputs and without; what the native side turns down (a whole
    number for scale) the Python side takes; a size that the library refuses
    raises from either."""
    x = sc.to_cuda(sc.layer_inputs([40, 30], 2, 4, 128, True, seed=3), True)
    a = {n: v if v is None else torch.from_numpy(v).cuda() for n, v in sc.accept_inputs(2, 9, 200, seed=3).items()}
    ws = lib.prefill_workspace(70, 2, 4, 128)
    one = [x[n][:2].contiguous() for n in ("q", "k", "v", "g", "beta")]
    layer = [x[n] for n in ("q", "k", "v", "g", "beta")]
    odd = torch.zeros(2, 4, 64, device="cuda")

    def calls(scale):
        out = []
        given = torch.empty(2, 4, 128, device="cuda", dtype=torch.bfloat16)
        for kw in (dict(), dict(out=given, S_out=torch.empty_like(x["S0"])), dict(o_dtype=torch.bfloat16)):
            out += lib.step(*one, x["S0"], scale=scale, **kw)
        assert out[2].data_ptr() == given.data_ptr()
        out += lib.prefill(*layer, x["S0"], x["starts"], ws, scale=scale)
        out += lib.prefill(*layer, None, x["starts"], ws, scale=scale, o_dtype=torch.bfloat16,
                           S_out=torch.empty_like(x["S0"]), force="scan")
        out += lib.accept(a["p"], a["tokens"], a["parent"], a["u"], a["noise"], q=a["q"])
        with pytest.raises(lib.CanopyError, match="unsupported"):
            lib.step(odd, odd, odd, torch.ones(2, 4, device="cuda"), torch.ones(2, 4, device="cuda"),
                     torch.zeros(2, 4, 64, 64, device="cuda"))
        return out

    lib.load()
    assert lib._marshal.step(*one, x["S0"], torch.float32, None, None, 2, None) is None
    native, mixed = calls(2.0), calls(2)
    stub = type("Stub", (), {n: staticmethod(lambda *args: None) for n in ("step", "prefill", "accept")})
    monkeypatch.setattr(lib, "_marshal", stub)
    python = calls(2.0)
    for y in (mixed, python):
        assert len(y) == len(native) and all(torch.equal(s, t) and s.dtype == t.dtype for s, t in zip(native, y))


def test_abi_argument_errors(lib):
    """Refused on the host before any CUDA call: the pointers are never followed."""
    L = lib.load()
    p = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(10)]

    def pre(q=p[0], N=8, B=2, H=2, HV=4, d=128, dt=1, flags=0, S0=p[5], ws=p[9]):
        return L.canopy_prefill(q, p[1], p[2], dt, p[3], p[4], S0, p[6], N, B, H, HV, d, d, 1.0, p[7], 0, p[8], ws,
                                flags, None)

    assert pre(q=None) == 1 and pre(ws=None) == 1 and pre(S0=ctypes.c_void_p(0x10004)) == 1
    assert pre(N=0) == 1 and pre(B=0) == 1 and pre(HV=3) == 1 and pre(dt=5) == 1 and pre(flags=4) == 1
    assert pre(flags=3) == 1 and pre(d=64) == 3 and pre(dt=0, flags=2) == 3 and pre(d=32, flags=2) == 3
    assert pre(B=70000) == 3
    assert lib.prefill_plan(8, 2, 2, 4, False, 128) == "scan"
    assert lib.prefill_plan(8, 2, 2, 3, False, 128) == "none"
    assert lib.prefill_plan(8, 2, 2, 4, True, 128, force="scan") == "scan"
    assert L.canopy_prefill_workspace_bytes(0, 1, 1, 128, 128) == 0
    assert L.canopy_prefill_workspace_bytes(8, 1, 1, 64, 64) == 0

    def st(S=p[5], B=2, H=2, HV=4, d=128, dt=1, err=None):
        return L.canopy_step(p[0], p[1], p[2], dt, p[3], p[4], S, p[6], B, H, HV, d, d, 1.0, p[7], 0, err, None)

    assert st(S=None) == 1 and st(B=0) == 1 and st(HV=3) == 1 and st(dt=2) == 1 and st(d=64) == 3
    assert st(err=ctypes.c_void_p(0x10002)) == 1 and st(B=65536) == 3

    def ac(x=p[0], T=4, B=2, V=9, dt=0, q=None, lengths=None):
        return L.canopy_accept(x, q, dt, p[1], p[2], lengths, p[3], p[4], T, B, V, p[5], p[6], p[7], None, None)

    assert ac(x=None) == 1 and ac(T=0) == 1 and ac(V=0) == 1 and ac(dt=3) == 1 and ac(T=257) == 3
    assert ac(V=(1 << 24) + 1) == 3 and ac(q=ctypes.c_void_p(0x10004)) == 1
    assert ac(lengths=ctypes.c_void_p(0x10004)) == 1
