"""Values that are not finite and what a row that sees them gets: the definition's infinities and NaN in their
columns, finite sums in all others, wherever tiles and pieces end."""

import numpy as np
import pytest
import torch

from attention_cases import TREES, attend_bound, attend_case, attend_reference, run_attend

pytestmark = pytest.mark.gpu

# kind -> plan, rows of the sequences, contexts, heads, T, tree
CASES = {
    "few_chains": ("few", [4, 2, 3], [90, 0, 61], (8, 2, 64), 4, "chain"),
    "few_trees": ("few", [4, 4, 1], [700, 60, 5], (12, 4, 128), 4, "random"),
    "few_packed": ("few", [1] * 30 + [40], [3 * i for i in range(31)], (8, 2, 128), None, None),
    "tiles_trees": ("tiles", [31, 20], [90, 130], (4, 2, 64), 31, "random"),
    "tiles_packed": ("tiles", [150, 40, 1], [130, 0, 900], (8, 2, 128), None, None),
    "tiles_wide": ("tiles", [70, 33], [400, 81], (7, 1, 128), 70, "wide"),
}


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 2)])
@pytest.mark.parametrize("kind", CASES)
def test_values_that_are_not_finite_stay_in_their_columns(lib, kind, window, sinks, bf16):
    plan, lens, ctxs, (HQ, HKV, d), T, tree = CASES[kind]
    c = attend_case(len(kind), lens, ctxs, HQ, HKV, d, 16, bf16, T=T, tree=TREES[tree] if tree else None, sharp=0.5)
    assert lib.attend_plan(len(c["q"]), len(lens), HQ, HKV, bf16, d) == (plan if bf16 else "fp32")
    # a few new rows of every sequence, the last and ones in the middle, each with bad values in some columns
    rng = np.random.RandomState(3)
    for b, n in enumerate(lens):
        for i in {n - 1, n // 2, n // 3} - {0} if n > 1 else {0}:
            at = int(ctxs[b] + i)
            place = c["v"][c["table"][b, at // 16], :, at % 16]
            for bad in (np.inf, -np.inf, np.nan):
                place[rng.randint(HKV), rng.randint(d)] = bad
        if ctxs[b] > 5:  # and a place that all of its rows see
            at = int(ctxs[b]) - 5
            c["v"][c["table"][b, at // 16], rng.randint(HKV), at % 16, rng.randint(d)] = np.inf
    with np.errstate(invalid="ignore"):
        ref, _ = attend_reference(c, window, sinks)
        clean = dict(c, v=np.where(np.isfinite(c["v"]), c["v"], 0).astype(np.float32))
        plain, weight = attend_reference(clean, window, sinks)
    o, err = run_attend(lib, c, window, sinks)
    assert err == 0
    mine = np.concatenate([np.asarray(r, int) for r in c["rows"]])
    o, ref, plain, weight = o[mine], ref[mine], plain[mine], weight[mine]
    assert 0 < (~np.isfinite(ref)).sum() < ref.size / 4
    hit = ~np.isfinite(ref)
    assert np.array_equal(np.isnan(o), np.isnan(ref))
    assert np.array_equal(o[hit & ~np.isnan(ref)], ref[hit & ~np.isnan(ref)])
    # the other columns' sums are those of the values without the bad ones, which have no part in them
    off = np.abs(o - plain)[~hit]
    assert (off <= attend_bound(c, plain, weight, int((c["ctxs"] + c["lens"]).max()))[~hit]).all()


@pytest.mark.parametrize("kind", ["window", "trees", "tokens"])
def test_caches_of_nothing_but_nan(lib, kind):
    """Every row sees such values in every tile: NaN throughout, and no wait gives up."""
    d, HKV, page = 128, 2, 64
    B, n, ctx = (2, 1500, 3000) if kind == "window" else (6, 64 if kind == "trees" else 1, 1000)
    pages = -(-(n + ctx) // page)
    k = torch.randn(B * pages, HKV, page, d, device="cuda").bfloat16()
    v = torch.full_like(k, float("nan"))
    table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
    context = torch.full((B,), ctx, dtype=torch.int32, device="cuda")
    q = torch.randn(B, n, 4 * HKV, d, device="cuda").bfloat16()
    ws = lib.attend_workspace(B * n, B, 4 * HKV, HKV, d)
    args = dict(parent=torch.arange(-1, n - 1, dtype=torch.int32, device="cuda").expand(B, n).contiguous()) \
        if kind == "trees" else dict(window=700, sinks=70)
    assert lib.attend(q, k, v, table, context, ws, **args).isnan().all()
    assert lib.read_device_error(ws) == 0
