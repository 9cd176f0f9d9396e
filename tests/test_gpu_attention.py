"""The attention layers' operators on the GPU against their definitions in 64 bits."""

import numpy as np
import pytest
import torch

import oracle
from attention_cases import (TREES, U16, U32, attend_bound, attend_case, attend_reference, cache, check_attend,
                             rounded, run_attend, tensor)

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------- qk_prep


def prep_inputs(seed, N, HQ, HKV, d, bf16, rot=0, axes=1, norm="rms", far=5000):
    rng = np.random.RandomState(seed)
    size = np.exp(rng.standard_normal((N, 1, 1)))
    x = {n: rounded(size * rng.standard_normal((N, H, d)), bf16) for n, H in (("q", HQ), ("k", HKV), ("v", HKV))}
    x["wq"], x["wk"] = ((1 + 0.2 * rng.standard_normal(d)).astype(np.float32) for _ in range(2))
    if norm != "rms":
        x["wq"] = x["wk"] = None
    x["freqs"] = x["positions"] = x["axis"] = None
    if rot:
        x["freqs"] = (1e4 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)
        x["positions"] = rng.randint(0, far, size=(axes, N)).astype(np.int32)
        x["axis"] = rng.randint(0, axes, size=rot // 2).astype(np.int32) if axes > 1 else None
    return x


def prep_bound(x, ref, weight, bf16, d):
    """Off by: the norm's sum of d squares, the root, the quotient and the two products, (d / 2 + 8) half steps of
    the row's largest value (a pair mixes two columns); the angle, 2e-7; the type's rounding."""
    top = np.abs(ref).max(-1, keepdims=True)
    return ((d / 2 + 8) * U32 + 2e-7) * 2 * top + (U16 if bf16 else U32) * np.abs(ref) + 1e-30


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("N,HQ,HKV,d,norm,rot,axes,pairs", [
    (1, 16, 4, 128, "rms", 64, 1, "half"), (3, 5, 5, 64, "rms", 64, 1, "adjacent"), (37, 7, 1, 128, "l2", 0, 1, "half"),
    (500, 28, 4, 128, "rms", 128, 3, "half"), (129, 6, 2, 64, "none", 24, 2, "adjacent"),
    (65, 3, 3, 128, "l2", 8, 1, "half"), (2000, 32, 8, 128, "rms", 96, 3, "half"), (700, 16, 16, 64, "none", 0, 1, "half")])
def test_prep_without_a_cache(lib, N, HQ, HKV, d, norm, rot, axes, pairs, bf16):
    x = prep_inputs(N + rot, N, HQ, HKV, d, bf16, rot, axes, norm)
    opt = lambda a: None if a is None else tensor(a)  # noqa: E731
    positions = None if x["positions"] is None else x["positions"][0] if axes == 1 else x["positions"]
    q, k = lib.qk_prep(tensor(x["q"], bf16), tensor(x["k"], bf16), norm=norm, q_weight=opt(x["wq"]),
                       k_weight=opt(x["wk"]), freqs=opt(x["freqs"]), positions=opt(positions), axis=opt(x["axis"]),
                       pairs=pairs)
    for y, src, w in ((q, "q", "wq"), (k, "k", "wk")):
        ref = oracle.attention.prep(x[src], norm, x[w], 1e-6, x["freqs"], x["positions"], x["axis"], pairs)
        off = np.abs(y.double().cpu().numpy() - ref)
        assert (off <= prep_bound(x[src], ref, x[w], bf16, d)).all()


@pytest.mark.parametrize("how", ["expanded", "transposed", "spaced"])
def test_prep_positions_of_any_layout(lib, how, monkeypatch):
    """Axes that are alike by expansion, axes last in memory, tokens apart: the results of dense positions."""
    x = prep_inputs(4, 60, 4, 2, 64, False, 32, 3, "none")
    q, k = tensor(x["q"]).view(5, 12, 4, 64), tensor(x["k"]).view(5, 12, 2, 64)
    dense = tensor(x["positions"]).view(3, 5, 12)
    if how == "expanded":
        laid = dense[1].expand(3, 5, 12)
        dense = laid.contiguous()
    elif how == "transposed":
        laid = dense.permute(1, 2, 0).contiguous().permute(2, 0, 1)
    else:
        laid = torch.zeros(3, 5, 12, 2, dtype=torch.int32, device="cuda")[..., 0]
        laid.copy_(dense)
    assert not laid.is_contiguous()
    args = dict(norm="none", freqs=tensor(x["freqs"]), axis=tensor(x["axis"]))
    ref = lib.qk_prep(q, k, positions=dense, **args)
    got = lib.qk_prep(q, k, positions=laid, **args)
    monkeypatch.setattr(lib, "_marshal", type("Stub", (), {"qk_prep": staticmethod(lambda *a: None)}))
    py = lib.qk_prep(q, k, positions=laid, **args)
    for a, b, c in zip(ref, got, py):
        assert torch.equal(a, b) and torch.equal(a, c)
    with pytest.raises(lib.CanopyError, match="distance"):
        lib.qk_prep(q, k, positions=torch.zeros(3, 5, 24, dtype=torch.int32, device="cuda")[..., :12], **args)


def test_prep_far_positions(lib):
    """Angles of positions near 2^31 and of negative ones keep their precision."""
    x = prep_inputs(3, 64, 2, 2, 128, False, 128, 1, "none")
    x["positions"][0, :32] = np.random.RandomState(1).randint(2 ** 30, 2 ** 31 - 1, size=32)
    x["positions"][0, 32:] = -x["positions"][0, 32:]
    q, _ = lib.qk_prep(tensor(x["q"]), tensor(x["k"]), norm="none", freqs=tensor(x["freqs"]),
                       positions=tensor(x["positions"][0]))
    ref = oracle.attention.prep(x["q"], "none", None, 0, x["freqs"], x["positions"])
    # the oracle's float64 product is off by up to 2^31 * 2^-53 = 2.4e-7 itself
    bound = prep_bound(x["q"], ref, None, False, 128) + 4 * 2.4e-7 * np.abs(ref).max()
    assert (np.abs(q.double().cpu().numpy() - ref) <= bound).all()


def test_prep_zero_rows_and_in_place(lib):
    """A row of zeros stays zeros; q_out and k_out may be q and k; tokens may lie apart."""
    qkv = torch.randn(50, 12, 128, device="cuda", dtype=torch.bfloat16)
    qkv[7] = 0
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    a, b = lib.qk_prep(q, k, norm="l2")
    c, d = q.contiguous(), k.contiguous()
    e, f = lib.qk_prep(c, d, norm="l2", q_out=c, k_out=d)
    assert e is c and f is d and torch.equal(a, c) and torch.equal(b, d)
    assert (a[7] == 0).all() and (b[7] == 0).all()
    ref = torch.nn.functional.normalize(q.double(), dim=-1)
    keep = torch.arange(50) != 7
    assert ((a.double() - ref)[keep].abs() <= 1.02 * U16 * ref[keep].abs() + 1e-7).all()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("kind", ["packed", "trees", "tokens"])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_prep_into_the_cache(lib, kind, page, bf16):
    """Rows at their places, every other slot of the caches and row of q_out as it was."""
    rng = np.random.RandomState(page)
    HQ, HKV, d, T = 6, 3, 64, 9
    ctxs = np.array([0, 15, 300, 64, 17], np.int32)
    lens = np.array([33, 0, 1, 70, 5] if kind == "packed" else [9, 0, 1, 4, 9] if kind == "trees" else [1] * 5, np.int32)
    behind = 3 if kind == "packed" else 0  # rows behind the last sequence
    N = 5 * T if kind == "trees" else int(lens.sum()) + behind
    x = prep_inputs(5, N, HQ, HKV, d, bf16, 32)
    kc, vc, table = cache(rng, ctxs + lens, HKV, d, page, bf16)
    first = np.arange(5) * T if kind == "trees" else np.concatenate([[0], np.cumsum(lens)])[:-1]
    lead = (5, T) if kind == "trees" else (N,)
    q, k, v = (tensor(x[n], bf16).view(*lead, -1, d) for n in "qkv")
    q_out = torch.full_like(q, 7.0)
    kd, vd, err = tensor(kc, bf16), tensor(vc, bf16), torch.zeros(1, dtype=torch.int32, device="cuda")
    starts = tensor(np.concatenate([first, [lens.sum()]]).astype(np.int32)) if kind == "packed" else None
    lib.qk_prep(q, k, v, q_weight=tensor(x["wq"]), k_weight=tensor(x["wk"]), freqs=tensor(x["freqs"]), k_cache=kd,
                v_cache=vd, page_table=tensor(table), context=tensor(ctxs), starts=starts, q_out=q_out,
                lengths=tensor(lens) if kind == "trees" else None, err=err)
    assert int(err) == 0
    pos = np.zeros((1, N), np.int64)
    for b in range(5):
        pos[0, first[b]:first[b] + lens[b]] = ctxs[b] + np.arange(lens[b])
    qr = oracle.attention.prep(x["q"], "rms", x["wq"], 1e-6, x["freqs"], pos)
    kr = oracle.attention.prep(x["k"], "rms", x["wk"], 1e-6, x["freqs"], pos)
    k_ref, v_ref, written = kc.astype(np.float64), vc.astype(np.float64), np.zeros(kc.shape, bool)
    mine = np.zeros(N, bool)
    for b in range(5):
        for i in range(lens[b]):
            at = int(ctxs[b]) + i
            to = (table[b, at // page], slice(None), at % page)
            k_ref[to], v_ref[to], written[to] = kr[first[b] + i], x["v"][first[b] + i], True
            mine[first[b] + i] = True
    got_q = q_out.view(N, HQ, d).double().cpu().numpy()
    assert (got_q[~mine] == 7.0).all()
    assert (np.abs(got_q - qr) <= prep_bound(None, qr, None, bf16, d))[mine].all()
    got_k, got_v = kd.double().cpu().numpy(), vd.double().cpu().numpy()
    assert (got_v == v_ref).all()
    assert (got_k == k_ref)[~written].all()
    assert (np.abs(got_k - k_ref) <= prep_bound(None, k_ref, None, bf16, d)).all()


# --------------------------------------------------------------------------- attend


HEADS = [(16, 4, 128), (8, 8, 64), (7, 1, 128), (32, 2, 64), (12, 4, 128), (5, 5, 64)]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("HQ,HKV,d", HEADS)
@pytest.mark.parametrize("page", [16, 64, 256])
def test_single_tokens(lib, HQ, HKV, d, page, bf16):
    ctxs = [0, 1, 63, 64, 65, 127, 128, 700]
    check_attend(lib, attend_case(1, [1] * 8, ctxs, HQ, HKV, d, page, bf16, T=1))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("HQ,HKV,d", HEADS)
@pytest.mark.parametrize("T,tree", [(2, "random"), (33, "random"), (64, "wide"), (64, "chain"), (200, "random")])
def test_trees(lib, HQ, HKV, d, T, tree, bf16):
    ctxs = [0, 100, 129]
    check_attend(lib, attend_case(T, [T, 0, T - T // 3], ctxs, HQ, HKV, d, 32, bf16, T=T, tree=TREES[tree]))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,lens", [(3, [3, 1, 0]), (70, [70, 0, 41])])
def test_rows_of_streams_without_a_tree(lib, T, lens, bf16):
    check_attend(lib, attend_case(T, lens, [0, 100, 129], 8, 4, 128, 32, bf16, T=T))


@pytest.mark.parametrize("bf16", [True, False])
def test_far_pages(lib, bf16):
    """Pages beyond 2^31 elements and 2^32 bytes of the caches: prepared, attended and moved as near ones are."""
    HQ, HKV, d, page, pages, T = 8, 8, 128, 64, 40000, 12
    dt = torch.bfloat16 if bf16 else torch.float32
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    small = [torch.randn(9, HKV, page, d, device="cuda", generator=gen).to(dt) for _ in range(2)]
    big = [torch.empty(pages, HKV, page, d, device="cuda", dtype=dt) for _ in range(2)]
    for x, y in zip(small, big):
        y[-9:] = x
    near = torch.tensor([[0, 5, 2, 7], [1, 3, 8, 4]], dtype=torch.int32, device="cuda")
    context = torch.tensor([150, 70], dtype=torch.int32, device="cuda")
    parent = torch.tensor([[-1] + [(i - 1) // 2 for i in range(1, T)]] * 2, dtype=torch.int32, device="cuda")
    accepted = torch.tensor([T - 1, 6], dtype=torch.int32, device="cuda")
    x = [torch.randn(2, T, H, d, device="cuda", generator=gen).to(dt) for H in (HQ, HKV, HKV)]
    one = torch.randn(2, HQ, d, device="cuda", generator=gen).to(dt)
    ws = lib.attend_workspace(2 * T, 2, HQ, HKV, d)
    out = []
    for (k, v), table in ((small, near), (big, near + pages - 9)):
        q, _ = lib.qk_prep(*x, norm="l2", k_cache=k, v_cache=v, page_table=table, context=context)
        o = lib.attend(q, k, v, table, context, ws, parent=parent)
        c = lib.cache_commit(accepted, parent, k, v, table, context)
        out.append([q, o, c, lib.attend(one, k, v, table, c, ws), k[-9:], v[-9:]])
    assert all(torch.equal(a, b) for a, b in zip(*out))
    assert lib.read_device_error(ws) == 0


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("HQ,HKV,d", HEADS)
@pytest.mark.parametrize("lens,ctxs", [([1], [0]), ([300], [0]), ([5, 0, 130, 64, 1], [0, 9, 128, 250, 513]),
                                       ([17, 257], [600, 31])])
def test_packed(lib, HQ, HKV, d, lens, ctxs, bf16):
    check_attend(lib, attend_case(len(lens), lens, ctxs, HQ, HKV, d, 64, bf16))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("kind", ["tokens", "trees", "packed"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (50, 0), (128, 1), (200, 130), (100000, 3)])
def test_windows(lib, kind, window, sinks, bf16):
    ctxs = [0, 3, 129, 700]
    if kind == "tokens":
        c = attend_case(5, [1] * 4, ctxs, 8, 2, 128, 16, bf16, T=1)
    elif kind == "trees":
        c = attend_case(6, [70, 9, 70, 33], ctxs, 8, 2, 64, 64, bf16, T=70, tree=TREES["chain" if sinks else "random"])
    else:
        c = attend_case(7, [300, 1, 77, 160], ctxs, 8, 2, 128, 32, bf16)
    check_attend(lib, c, window, sinks)


@pytest.mark.parametrize("bf16", [True, False])
def test_long_cache_split(lib, bf16):
    """Work split along the cache and joined, in runs of the same workspace that differ in size; twice the same."""
    ws = lib.attend_workspace(40, 3, 8, 2, 128)
    a = attend_case(8, [1], [20011], 8, 2, 128, 128, bf16, T=1)
    x = check_attend(lib, a, ws=ws)
    check_attend(lib, attend_case(9, [7, 3], [5000, 33], 8, 2, 128, 16, bf16), ws=ws)
    assert np.array_equal(x, check_attend(lib, a, ws=ws))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("kind", ["tokens", "trees", "packed"])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_hidden_places_hold_anything(lib, kind, bad, bf16):
    """NaN and infinities in places that no row sees (behind the end, out of the window, in pages of no stream)
    and, in a row's keys and values, that it does not see itself."""
    window, sinks, ctxs = (40, 2, [90, 130]) if kind != "trees" else (0, 0, [90, 130])
    if kind == "tokens":
        c = attend_case(1, [1, 1], ctxs, 4, 2, 64, 16, bf16, T=1)
    elif kind == "trees":
        c = attend_case(2, [20, 31], ctxs, 4, 2, 64, 16, bf16, T=31, tree=TREES["random"])
    else:
        c = attend_case(3, [40, 150], ctxs, 4, 2, 64, 16, bf16)
    ref, weight = attend_reference(c, window, sinks)
    seen = np.zeros(c["k"].shape[:1] + c["k"].shape[2:3], bool)
    for b in range(2):
        lo = max(sinks, c["ctxs"][b] - window + 1) if window else 0
        for i in [*range(min(sinks, c["ctxs"][b])), *range(lo, c["ctxs"][b] + c["lens"][b])]:
            seen[c["table"][b, i // 16], i % 16] = True
    hide = np.broadcast_to(~seen[:, None, :, None], c["k"].shape)
    c["k"], c["v"] = np.where(hide, bad, c["k"]).astype(np.float32), np.where(hide, bad, c["v"]).astype(np.float32)
    gone = np.array([[window and (j + 1) * 16 <= c["ctxs"][b] - window + 1 and j * 16 >= sinks
                      for j in range(c["table"].shape[1])] for b in range(2)], bool)
    c["table"] = np.where(gone, -7, c["table"]).astype(np.int32)
    # the last new row's own key and value: it alone sees them (trees: no node stands below the last)
    poisoned = []
    if kind != "tokens":
        for b in range(2):
            at = int(c["ctxs"][b] + c["lens"][b]) - 1
            c["v"][c["table"][b, at // 16], 0, at % 16, 5] = bad
            poisoned.append(c["rows"][b][int(c["lens"][b]) - 1])
    o, err = run_attend(lib, c, window, sinks)
    assert err == 0
    mine = np.setdiff1d(np.concatenate([np.asarray(r, int) for r in c["rows"]])[:], poisoned)
    mine = mine[[i for i, r in enumerate(mine) if not np.isnan(ref[r]).any()]]
    clean = dict(c, k=np.nan_to_num(c["k"], nan=0, posinf=0, neginf=0))
    assert (np.abs(o[mine] - ref[mine]) <= attend_bound(clean, ref[mine], weight[mine], 300)).all()
    for r in poisoned:
        assert not np.isfinite(o[r, :2, 5]).any()
        assert np.isfinite(o[r, 2:]).all()


def test_bad_data_sets_bits(lib):
    """Pages out of range, places beyond the table, contexts below zero, bad trees and starts: an error bit and no fault."""
    c = attend_case(1, [5, 40], [60, 100], 4, 2, 64, 16, True)
    for change, bit in (("page", lib.DEVERR_PAGE), ("room", lib.DEVERR_PAGE), ("context", lib.DEVERR_LENGTH)):
        d = dict(c, table=c["table"].copy(), ctxs=c["ctxs"].copy())
        if change == "page":
            d["table"][0, 1] = len(c["k"])
            d["table"][1, 2] = -1
        elif change == "room":
            d["ctxs"][1] = 2 ** 31 - 1
        else:
            d["ctxs"][0] = -5
        assert run_attend(lib, d)[1] == bit
    t = attend_case(2, [9, 9], [60, 100], 4, 2, 64, 16, True, T=9, tree=TREES["random"])
    t["parent"][1, 4] = 4
    assert run_attend(lib, t)[1] == lib.DEVERR_TREE
    t = attend_case(2, [9, 9], [60, 100], 4, 2, 64, 16, True, T=9, tree=TREES["random"])
    t["lens"][0] = 10
    assert run_attend(lib, t)[1] == lib.DEVERR_LENGTH


# --------------------------------------------------------------------------- cache_commit


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,tree", [(1, "chain"), (8, "chain"), (33, "wide"), (64, "random"), (256, "random"),
                                    (256, "chain")])
@pytest.mark.parametrize("page,HKV,d", [(16, 2, 64), (64, 5, 128)])
def test_commit(lib, T, tree, page, HKV, d, bf16):
    rng = np.random.RandomState(T + page)
    ctxs = np.array([0, 15, 300, 64], np.int32)
    lens = np.array([T, T, max(1, T // 2), T], np.int32)
    parent = np.stack([TREES[tree](T, rng) for _ in range(4)]).astype(np.int32)
    accepted = np.array([T - 1, -1, lens[2] - 1, rng.randint(T)], np.int32)
    k, v, table = cache(rng, ctxs + lens, HKV, d, page, bf16)
    kd, vd, err = tensor(k, bf16), tensor(v, bf16), torch.zeros(1, dtype=torch.int32, device="cuda")
    new = lib.cache_commit(tensor(accepted), tensor(parent), kd, vd, tensor(table), tensor(ctxs),
                           lengths=tensor(lens), err=err)
    kr, vr, cr = oracle.attention.commit(accepted, parent, k, v, table, ctxs)
    assert int(err) == 0 and np.array_equal(new.cpu().numpy(), cr)
    for got, ref, old in ((kd, kr, k), (vd, vr, v)):
        got = got.float().cpu().numpy()
        for b in range(4):  # places behind the new length keep whatever the tree left there
            for i in range(int(cr[b])):
                at = (table[b, i // page], slice(None), i % page)
                assert np.array_equal(got[at], ref[at])
        used = {int(p) for b in range(4) for p in table[b, :-(-(ctxs[b] + lens[b]) // page)]}
        free = [p for p in range(len(k)) if p not in used]
        assert np.array_equal(got[free], old[free])


def test_commit_bad_data(lib):
    rng = np.random.RandomState(0)
    k, v, table = cache(rng, [20, 20], 2, 64, 16, False)
    parent = np.stack([TREES["chain"](8, rng)] * 2).astype(np.int32)

    def bits(accepted=(7, 7), ctxs=(5, 5), table=table, parent=parent):
        kd, vd, err = tensor(k), tensor(v), torch.zeros(1, dtype=torch.int32, device="cuda")
        new = lib.cache_commit(tensor(np.array(accepted, np.int32)), tensor(parent), kd, vd, tensor(table),
                               tensor(np.array(ctxs, np.int32)), err=err)
        return int(err), new.tolist(), np.array_equal(kd.cpu().numpy(), k) and np.array_equal(vd.cpu().numpy(), v)

    assert bits() == (0, [13, 13], True)  # a chain's path lies where it is already
    assert bits(accepted=(8, -2)) == (lib.DEVERR_ACCEPTED, [5, 5], True)
    assert bits(ctxs=(2 ** 31 - 9, 5))[0] == lib.DEVERR_PAGE
    assert bits(ctxs=(-1, 5))[0] == lib.DEVERR_LENGTH
    t = table.copy()
    t[0, 0] = 99
    assert bits(table=t)[0] == lib.DEVERR_PAGE
    p = parent.copy()
    p[1, 3] = 5
    assert bits(parent=p)[0] == lib.DEVERR_TREE


# --------------------------------------------------------------------------- together


@pytest.mark.parametrize("bf16", [True, False])
def test_a_round(lib, bf16):
    """Prompts, a tree, its accepted path and a single token through a layer: the last token's output is that of
    the layer run over exactly the tokens that stay."""
    rng = np.random.RandomState(11)
    B, HQ, HKV, d, T, page = 3, 8, 2, 64, 12, 16
    lens = np.array([40, 3, 75], np.int32)
    kc, vc, table = cache(rng, lens + T + 1, HKV, d, page, bf16)
    kd, vd, td = tensor(kc, bf16), tensor(vc, bf16), tensor(table)
    freqs = tensor((1e4 ** (-np.arange(16) / 16)).astype(np.float32))
    w = tensor(np.ones(d, np.float32))
    new = lambda n, H: tensor(rounded(rng.standard_normal((n, H, d)), bf16), bf16)  # noqa: E731
    args = dict(q_weight=w, k_weight=w, freqs=freqs, k_cache=kd, v_cache=vd, page_table=td)
    N = int(lens.sum())
    starts = tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    x = [new(N, H) for H in (HQ, HKV, HKV)]
    kept = [[[y[starts[b]:starts[b + 1]] for y in x]] for b in range(B)]
    q, _ = lib.qk_prep(*x, context=zero, starts=starts, **args)
    ws = lib.attend_workspace(N, B, HQ, HKV, d)
    lib.attend(q, kd, vd, td, zero, ws, starts=starts)
    context = tensor(lens)
    parent = tensor(np.stack([TREES["random"](T, rng) for _ in range(B)]).astype(np.int32))
    x = [new(B * T, H).view(B, T, H, d) for H in (HQ, HKV, HKV)]
    depth = np.stack([oracle.depths(p) for p in parent.cpu().numpy()])
    positions = tensor((lens[:, None] + depth).astype(np.int32))
    q, _ = lib.qk_prep(*x, context=context, positions=positions, **args)
    lib.attend(q, kd, vd, td, context, ws, parent=parent)
    accepted = [T - 1, 5, 8]
    context = lib.cache_commit(tensor(np.array(accepted, np.int32)), parent, kd, vd, td, context)
    for b in range(B):
        path = oracle.root_path(parent[b].tolist(), accepted[b])
        kept[b].append([y[b, path] for y in x])
    x = [new(B, H) for H in (HQ, HKV, HKV)]
    q, _ = lib.qk_prep(*x, context=context, **args)
    o = lib.attend(q, kd, vd, td, context, ws)
    assert lib.read_device_error(ws) == 0
    kd, vd = kd.float().cpu().numpy(), vd.float().cpu().numpy()
    qs = np.zeros((B, HQ, d), np.float32)
    for b in range(B):
        kept[b].append([y[b:b + 1] for y in x])
        y = [torch.cat(z).contiguous() for z in zip(*kept[b])]
        at = torch.arange(len(y[0]), dtype=torch.int32, device="cuda")
        qb, kb = lib.qk_prep(y[0], y[1], q_weight=w, k_weight=w, freqs=freqs, positions=at)
        for i in range(len(at)):  # the places hold the kept tokens, bit for bit
            assert np.array_equal(oracle.attention.place(kd, table, b, i), kb[i].float().cpu().numpy())
            assert np.array_equal(oracle.attention.place(vd, table, b, i), y[2][i].float().cpu().numpy())
        qs[b] = qb[-1].float().cpu().numpy()
    c = dict(q=qs, k=kd, v=vd, table=table, ctxs=context.cpu().numpy(), rows=[[b] for b in range(B)], parent=None,
             bf16=bf16, scale=d ** -0.5)
    ref, size = attend_reference(c)
    assert (np.abs(o.double().cpu().numpy() - ref) <= attend_bound(c, ref, size, 100)).all()
