"""Outputs that lie over inputs, or over one another, are refused on the host (fake pointers, never followed); next to
them, or in place where that is allowed, they are not."""

import ctypes

import pytest
import torch

from gated_deltanet_linear_tree_gb300 import build


@pytest.fixture(scope="module")
def canopy():
    build.build()
    from gated_deltanet_linear_tree_gb300 import canopy
    canopy.load()
    return canopy


AT = [0x100000 * (i + 1) for i in range(20)]


def P(x):
    return ctypes.c_void_p(x)


@pytest.mark.parametrize("es", [2, 4])
def test_attend(canopy, es):
    rows, cache = 8 * 4 * 128 * es, 3 * 2 * 16 * 128 * es

    def call(q=AT[0], kc=AT[1], vc=AT[2], o=AT[6]):
        return canopy.load().canopy_attend(P(q), int(es == 2), P(kc), P(vc), P(AT[3]), 3, 16, 4, P(AT[4]), None, None,
                                           None, 8, 2, 4, 2, 128, 0, 0, 1.0, P(o), P(AT[7]), None)

    for o in (AT[0], AT[0] + 16, AT[0] + rows - 16, AT[0] - rows + 16, AT[1], AT[1] + cache - 16, AT[2] - rows + 16):
        assert call(o=o) == 1


@pytest.mark.parametrize("es", [2, 4])
def test_qk_prep(canopy, es):
    N, HQ, HKV, d = 8, 4, 2, 128
    nq, nk, cache = N * HQ * d * es, N * HKV * d * es, 3 * 2 * 16 * 128 * es

    def call(q=AT[0], k=AT[1], v=AT[2], ldq=HQ * d, ldk=HKV * d, ldv=HKV * d, qo=AT[6], ko=None, kc=AT[7], vc=AT[8]):
        bare = kc is None
        return canopy.load().canopy_qk_prep(
            P(q), P(k), None if bare else P(v), int(es == 2), ldq, ldk, ldv, 1, None, None, 1e-6, None, 0, None, 1, 0, 1,
            None, 0, N, 0 if bare else 2, HQ, HKV, d, P(qo), None if ko is None else P(ko), None if bare else P(kc),
            None if bare else P(vc), None if bare else P(AT[9]), 3, 16, 4, None if bare else P(AT[10]), None, None, None,
            None)

    # in place, but the tokens lie apart; a row later; over keys and values, before or behind
    for kw in (dict(qo=AT[0], ldq=6 * d), dict(qo=AT[0] + 16), dict(qo=AT[0] + HQ * d * es), dict(qo=AT[1] - nq + 16),
               dict(qo=AT[1] + nk - 16), dict(qo=AT[2]), dict(qo=AT[0] + (N - 1) * 9 * d * es, ldq=9 * d),
               dict(vc=AT[7]), dict(vc=AT[7] + cache - 16), dict(kc=AT[0]), dict(vc=AT[2] + nk - 16),
               dict(kc=AT[1] - cache + 16), dict(qo=AT[7]), dict(qo=AT[8] + cache - 16)):
        assert call(**kw) == 1, kw
    bare = dict(kc=None, vc=None, ko=AT[11])
    for kw in (dict(ko=AT[1], ldk=3 * d), dict(ko=AT[1] + 16), dict(ko=AT[0]), dict(ko=AT[6]),
               dict(ko=AT[6] + nq - 16), dict(qo=AT[1])):
        assert call(**{**bare, **kw}) == 1, kw


def test_cache_commit(canopy):
    B, T, cache = 3, 8, 3 * 2 * 16 * 128 * 2

    def call(acc=AT[0], parent=AT[1], lengths=AT[2], kc=AT[3], vc=AT[4], ctx=AT[5], new=AT[6]):
        return canopy.load().canopy_cache_commit(P(acc), P(parent), P(lengths), P(kc), P(vc), 1, P(AT[7]), 3, 16, 4,
                                                 P(ctx), T, B, 2, 128, P(new), None, None)

    for kw in (dict(new=AT[5]), dict(new=AT[5] + 8), dict(new=AT[5] - 8), dict(new=AT[0]), dict(new=AT[2] + 4),
               dict(new=AT[1] + 4 * B * T - 4), dict(vc=AT[3]), dict(vc=AT[3] + cache - 16)):
        assert call(**kw) == 1, kw


@pytest.mark.gpu
@pytest.mark.parametrize("bf16", [True, False])
def test_next_to_the_inputs(lib, bf16):
    """One piece of memory, shared without a gap; queries in place beside keys that go to the cache."""
    dt = torch.bfloat16 if bf16 else torch.float32
    torch.manual_seed(0)
    B, HQ, HKV, d = 3, 4, 2, 64
    all_rows = torch.randn(2 * HQ + 2 * HKV, B, d, device="cuda").to(dt)
    q, k, v, out = (x.view(B, -1, d) for x in all_rows.split([HQ, HKV, HKV, HQ]))
    caches = torch.randn(2, 9, HKV, 16, d, device="cuda").to(dt)
    other = caches.clone()
    table = torch.arange(9, dtype=torch.int32, device="cuda").view(3, 3)
    context = torch.tensor([0, 20, 47], dtype=torch.int32, device="cuda")
    ws = lib.attend_workspace(B, B, HQ, HKV, d)
    ref, _ = lib.qk_prep(q, k, v, k_cache=other[0], v_cache=other[1], page_table=table, context=context)
    o = lib.attend(ref, *other, table, context, ws)
    got, _ = lib.qk_prep(q, k, v, q_out=q, k_cache=caches[0], v_cache=caches[1], page_table=table, context=context)
    assert got is q and torch.equal(q, ref) and torch.equal(caches, other)
    assert torch.equal(lib.attend(q, *caches, table, context, ws, out=out), o) and torch.equal(out, o)
    with pytest.raises(lib.CanopyError):
        lib.attend(q, *caches, table, context, ws, out=q)
    one = torch.randn(1, HQ + 2 * HKV, d, device="cuda").to(dt)  # a token's slices are dense
    q, k, v = one.split([HQ, HKV, HKV], 1)
    args = dict(k_cache=caches[0], v_cache=caches[1], page_table=table[:1], context=context[:1])
    want, _ = lib.qk_prep(q, k, v, **args)
    lib.qk_prep(q, k, v, q_out=q, **args)
    assert torch.equal(q, want)
