"""The documented calls of an attention layer, run as they stand there: after them the cache and the last outputs are
those of the tokens that stay, prompts and accepted paths."""

import pathlib
import re

import numpy as np
import pytest
import torch

import oracle
from attention_cases import TREES, attend_bound, attend_reference, cache, rounded, tensor
from gated_deltanet_linear_tree_gb300 import canopy

pytestmark = pytest.mark.gpu


def example():
    root = pathlib.Path(__file__).resolve().parent.parent
    blocks = [b for p in sorted(root.glob("*.md")) for b in re.findall(r"```python\n(.*?)```", p.read_text(), re.S)]
    mine = [b for b in blocks if b.startswith("# an attention layer between")]
    assert len(mine) == 1
    return mine[0]


@pytest.mark.parametrize("before", [[0, 0, 0], [5, 0, 37]])
def test_the_example_runs_and_keeps_the_tokens(lib, before):
    rng = np.random.RandomState(4)
    B, T, HQ, HKV, d, page = 3, 9, 8, 2, 128, 16
    lens = np.array([40, 3, 20])
    kc, vc, table = cache(rng, np.array(before) + lens + T + 1, HKV, d, page, True)
    x = {n: {k: tensor(rounded(rng.standard_normal((*lead, H, d)), True), True)
             for k, H in (("q", HQ), ("k", HKV), ("v", HKV))}
         for n, lead in (("prompt", (int(lens.sum()),)), ("tree", (B, T)), ("token", (B,)))}
    parent = np.stack([TREES["random"](T, rng) for _ in range(B)]).astype(np.int32)
    accepted = np.array([T - 1, 4, 6], np.int32)
    names = dict(canopy=canopy, N=int(lens.sum()), B=B, T=T, HQ=HQ, HKV=HKV, k_cache=tensor(kc, True),
                 v_cache=tensor(vc, True), page_table=tensor(table), context=tensor(np.array(before, np.int32)),
                 starts=tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)),
                 wq=tensor((1 + 0.1 * rng.standard_normal(d)).astype(np.float32)),
                 wk=tensor((1 + 0.1 * rng.standard_normal(d)).astype(np.float32)),
                 freqs=tensor((1e4 ** (-np.arange(32) / 32)).astype(np.float32)), parent=tensor(parent),
                 depth=tensor(np.stack([oracle.depths(p) for p in parent]).astype(np.int32)),
                 accepted=tensor(accepted))
    for n, prefix in (("prompt", ""), ("tree", "tree_"), ("token", "token_")):
        names.update({prefix + k: y for k, y in x[n].items()})
    exec(example(), names)
    assert lib.read_device_error(names["ws"]) == 0
    kd, vd, o = (names[n].float().cpu().numpy() for n in ("k_cache", "v_cache", "o"))
    starts = np.concatenate([[0], np.cumsum(lens)])
    ends, qs = [], np.zeros((B, HQ, d), np.float32)
    for b in range(B):
        path = oracle.root_path(parent[b], int(accepted[b]))
        kept = [torch.cat([x["prompt"][k][starts[b]:starts[b + 1]], x["tree"][k][b, sorted(path)],
                           x["token"][k][b:b + 1]]).contiguous() for k in "qkv"]
        at = torch.arange(before[b], before[b] + len(kept[0]), dtype=torch.int32, device="cuda")
        qb, kb = lib.qk_prep(kept[0], kept[1], q_weight=names["wq"], k_weight=names["wk"], freqs=names["freqs"],
                             positions=at)
        for i, p in enumerate(at.tolist()):
            assert np.array_equal(oracle.attention.place(kd, table, b, p), kb[i].float().cpu().numpy())
            assert np.array_equal(oracle.attention.place(vd, table, b, p), kept[2][i].float().cpu().numpy())
        qs[b] = qb[-1].float().cpu().numpy()
        ends.append(before[b] + len(kept[0]) - 1)
    assert names["context"].tolist() == ends
    c = dict(q=qs, k=kd, v=vd, table=table, ctxs=np.array(ends), rows=[[b] for b in range(B)], parent=None, bf16=True,
             scale=d ** -0.5)
    ref, size = attend_reference(c)
    assert (np.abs(o.astype(np.float64) - ref) <= attend_bound(c, ref, size, 100)).all()
