"""A context below zero in qk_prep: reported, and nothing is written to the caches for that stream, whose tokens stay
as they are; its queries, and the other streams, are those of the call without it."""

import numpy as np
import pytest
import torch

import oracle
from attention_cases import cache, rounded, tensor
from test_gpu_attention import prep_bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("kind", ["packed", "packed_many", "trees", "tokens"])
@pytest.mark.parametrize("below", [-1, -7, -2 ** 31])
@pytest.mark.parametrize("report", [True, False])
def test_a_negative_context_writes_nothing(lib, kind, below, bf16, report):
    rng = np.random.RandomState(1)
    B, HQ, HKV, d, page = 3, 6, 2, 64, 16
    lens = {"packed": [5, 9, 3], "packed_many": [700, 1500, 300], "trees": [9, 9, 9], "tokens": [1, 1, 1]}[kind]
    ctxs, N = np.array([20, 33, 7], np.int32), sum(lens)
    kc, vc, table = cache(rng, ctxs + np.array(lens), HKV, d, page, bf16)
    lead = (B, 9) if kind == "trees" else (N,)
    x = {n: rounded(rng.standard_normal((N, H, d)), bf16) for n, H in (("q", HQ), ("k", HKV), ("v", HKV))}
    freqs = (1e4 ** (-np.arange(16) / 16)).astype(np.float32)
    starts = tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)) if "packed" in kind else None

    def run(ctxs):
        kd, vd, err = tensor(kc, bf16), tensor(vc, bf16), torch.zeros(1, dtype=torch.int32, device="cuda")
        q, _ = lib.qk_prep(*(tensor(x[n], bf16).view(*lead, -1, d) for n in "qkv"), freqs=tensor(freqs), k_cache=kd,
                           v_cache=vd, page_table=tensor(table), context=tensor(ctxs), starts=starts,
                           err=err if report else None)
        return q.view(N, HQ, d), kd, vd, int(err)

    q0, k0, v0, none = run(ctxs)
    bad = ctxs.copy()
    bad[1] = below
    q1, k1, v1, bits = run(bad)
    assert none == 0 and bits == (lib.DEVERR_LENGTH if report else 0)
    pages = torch.from_numpy(table[1][table[1] >= 0].astype(np.int64)).cuda()
    for good, got, before in ((k0, k1, kc), (v0, v1, vc)):
        want = good.clone()
        want[pages] = tensor(before, bf16)[pages]
        assert torch.equal(got, want)
    mine = slice(lens[0], lens[0] + lens[1])
    rest = np.setdiff1d(np.arange(N), np.arange(N)[mine])
    assert torch.equal(q0[rest], q1[rest])
    ref = oracle.attention.prep(x["q"][mine], "rms", None, 1e-6, freqs, np.arange(lens[1])[None])  # read as zero
    assert (np.abs(q1[mine].double().cpu().numpy() - ref) <= prep_bound(None, ref, None, bf16, d)).all()
