"""The attention layers' entry points without a GPU: plans, workspaces, and arguments that are refused on the
host before any CUDA call.  Fake pointers are never followed."""

import ctypes

import pytest
import torch

from gated_deltanet_linear_tree_gb300 import build
from tests.test_serving_devices import OnGpu, on

BIG = 2 ** 32 + 2  # its lower 32 bits are a size that is fine


@pytest.fixture(scope="module")
def canopy():
    build.build()
    from gated_deltanet_linear_tree_gb300 import canopy
    canopy.load()
    return canopy


P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(20)]
ODD4, ODD16 = ctypes.c_void_p(0x10002), ctypes.c_void_p(0x10008)


def test_plans(canopy):
    """Up to 16 rows (tokens by query heads of a key head) a sequence on average are few."""
    plan = canopy.attend_plan
    assert plan(1, 1, 16, 4, True, 128) == "few"
    assert plan(4, 1, 16, 4, True, 128) == "few" and plan(5, 1, 16, 4, True, 128) == "tiles"
    assert plan(64, 64, 32, 2, True, 64) == "few" and plan(64, 64, 34, 2, True, 64) == "tiles"
    assert plan(1024, 16, 16, 4, True, 128) == "tiles"
    assert plan(1, 1, 16, 4, False, 128) == plan(4096, 1, 16, 4, False, 64) == "fp32"
    for bad in ((0, 1, 4, 4, 128), (4, 0, 4, 4, 128), (4, 1, 4, 3, 128), (4, 1, 4, 0, 128), (4, 1, 4, 4, 32),
                (4, 1, 130, 2, 128), (4, 70000, 4, 4, 128), (2 ** 30, 1, 4, 4, 128)):
        assert plan(*bad[:4], True, bad[4]) == "none"
        assert canopy.load().canopy_attend_workspace_bytes(*bad) == 0


def test_workspace_grows_with_rows_and_sequences(canopy):
    size = canopy.load().canopy_attend_workspace_bytes
    last = 0
    for N in (1, 2, 4, 5, 16, 17, 33, 65, 1000, 100000):
        n = size(N, 1, 16, 4, 128)
        assert n >= last > -1
        last = n
        assert size(N, 2, 16, 4, 128) >= n
    assert size(1, 1, 16, 4, 128) >= 4096 + 608 * 16 * 130 * 4
    assert size(1000, 1, 16, 4, 128) >= 4096 + 304 * 256 * 130 * 4


def test_attend_refused(canopy):
    lib = canopy.load()

    def call(q=P[0], dt=1, kc=P[1], vc=P[2], table=P[3], pages=9, ps=64, most=4, ctx=P[4], starts=P[5], parent=None,
             lengths=None, N=8, B=2, HQ=4, HKV=2, d=128, window=0, sinks=0, scale=1.0, o=P[6], ws=P[7]):
        return lib.canopy_attend(q, dt, kc, vc, table, pages, ps, most, ctx, starts, parent, lengths, N, B, HQ, HKV, d,
                                 window, sinks, scale, o, ws, None)

    for kw in (dict(q=None), dict(q=ODD16), dict(kc=None), dict(vc=ODD16), dict(table=None), dict(table=ODD4),
               dict(ctx=None), dict(o=None), dict(ws=None), dict(dt=2), dict(pages=0), dict(ps=0), dict(most=0),
               dict(N=0), dict(B=0), dict(HKV=3), dict(window=-1), dict(sinks=-1, window=4), dict(sinks=4),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(parent=P[8]), dict(lengths=P[8]), dict(starts=None, N=9), dict(starts=ODD4)):
        assert call(**kw) == 1, kw
    for kw in (dict(d=32), dict(d=256), dict(ps=8), dict(ps=48), dict(HQ=130), dict(B=70000),
               dict(most=2 ** 25, ps=64), dict(pages=2 ** 30, HKV=2), dict(starts=None, parent=P[8], N=514),
               dict(N=2 ** 30)):
        assert call(**kw) == 3, kw


def test_qk_prep_refused(canopy):
    lib = canopy.load()

    def call(q=P[0], k=P[1], v=P[2], dt=1, ldq=512, ldk=256, ldv=256, norm=1, qw=P[3], kw=P[4], eps=1e-6, freqs=P[5],
             R=64, positions=None, axes=1, steps=(8, 1), axis=None, pairs=0, N=8, B=2, HQ=4, HKV=2, d=128, qo=P[6],
             ko=None,
             kc=P[7], vc=P[8], table=P[9], pages=9, ps=64, most=4, ctx=P[10], starts=P[11], lengths=None, err=None):
        return lib.canopy_qk_prep(q, k, v, dt, ldq, ldk, ldv, norm, qw, kw, eps, freqs, R, positions, axes, *steps,
                                  axis,
                                  pairs, N, B, HQ, HKV, d, qo, ko, kc, vc, table, pages, ps, most, ctx, starts,
                                  lengths, err, None)

    bare = dict(v=None, B=0, ko=P[12], kc=None, vc=None, table=None, ctx=None, starts=None, positions=P[13])
    for kw in (dict(q=None), dict(k=ODD16), dict(v=None), dict(qo=None), dict(vc=None), dict(table=None),
               dict(ctx=None), dict(ko=P[12]), dict(dt=2), dict(norm=3), dict(norm=0), dict(pairs=2), dict(eps=-1.0),
               dict(eps=float("nan")), dict(R=-8), dict(R=136), dict(R=0), dict(freqs=None), dict(axis=P[13]),
               dict(positions=P[13], axes=0), dict(positions=P[13], steps=(-1, 1)),
               dict(positions=P[13], steps=(8, -1)), dict(ldq=504), dict(ldk=260), dict(ldv=255), dict(qw=ODD16),
               dict(lengths=P[13]), dict(starts=None, N=9), dict(N=0), dict(HKV=3), dict(err=ODD4),
               dict(R=0, freqs=None, positions=P[13]), dict(bare, ko=None), dict(bare, v=P[2]), dict(bare, starts=P[3]),
               dict(bare, positions=None), dict(bare, B=1)):
        assert call(**kw) == 1, kw
    for kw in (dict(R=60), dict(d=32, ldq=512, R=8), dict(ps=8), dict(ps=48), dict(B=70000),
               dict(HQ=130, ldq=130 * 128)):
        assert call(**kw) == 3, kw


def test_cache_commit_refused(canopy):
    lib = canopy.load()

    def call(acc=P[0], parent=P[1], lengths=None, kc=P[2], vc=P[3], dt=1, table=P[4], pages=9, ps=64, most=4, ctx=P[5],
             T=8, B=2, HKV=2, d=128, new=P[6], err=None):
        return lib.canopy_cache_commit(acc, parent, lengths, kc, vc, dt, table, pages, ps, most, ctx, T, B, HKV, d,
                                       new, err, None)

    for kw in (dict(acc=None), dict(acc=ODD4), dict(parent=None), dict(kc=None), dict(vc=ODD16), dict(dt=3),
               dict(table=None), dict(ctx=None), dict(new=None), dict(new=P[5]), dict(T=0), dict(B=0), dict(HKV=0),
               dict(pages=0), dict(err=ODD4), dict(lengths=ODD4)):
        assert call(**kw) == 1, kw
    for kw in (dict(T=257), dict(d=32), dict(ps=24), dict(B=70000)):
        assert call(**kw) == 3, kw


# name -> shape; one token of two streams, or trees of three nodes
CACHE = dict(k_cache=(5, 2, 16, 64), v_cache=(5, 2, 16, 64), page_table=(2, 3), context=(2,))
ATTEND = dict(q=(2, 3, 4, 64), **CACHE, ws=(8,), parent=(2, 3), lengths=(2,), out=(2, 3, 4, 64))
PREP = dict(q=(2, 3, 4, 64), k=(2, 3, 2, 64), v=(2, 3, 2, 64), q_weight=(64,), k_weight=(64,), freqs=(16,),
            positions=(2, 2, 3), axis=(16,), q_out=(2, 3, 4, 64), **CACHE, lengths=(2,), err=(1,))
COMMIT = dict(accepted=(2,), parent=(2, 3), **CACHE, lengths=(2,), err=(1,))
INTS = {"page_table", "context", "parent", "lengths", "accepted", "positions", "axis", "err"}
CALLS = [("attend", ATTEND), ("qk_prep", PREP), ("cache_commit", COMMIT)]


def dtype_of(name):
    return torch.uint8 if name == "ws" else torch.int32 if name in INTS else torch.float32


@pytest.fixture
def no_calls(canopy, monkeypatch):
    lib = type("Lib", (), {"canopy_attend_workspace_bytes": staticmethod(lambda *a: 8)})  # no entry point to call
    monkeypatch.setattr(canopy, "load", lambda: lib)


@pytest.mark.parametrize("call,shapes", CALLS)
def test_a_tensor_on_another_device_is_refused(canopy, no_calls, call, shapes):
    def tensors(elsewhere=None):
        return {n: on(int(n == elsewhere), *s, dtype=dtype_of(n)) for n, s in shapes.items()}

    with pytest.raises(Exception) as e:  # all on one device: through the checks, up to the device that is not there
        getattr(canopy, call)(**tensors())
    assert not isinstance(e.value, canopy.CanopyError)
    for name in shapes:
        if (call, name) in (("attend", "q"), ("qk_prep", "q"), ("cache_commit", "k_cache")):
            continue  # the device that the others are compared with
        with pytest.raises(canopy.CanopyError, match="same device"):
            getattr(canopy, call)(**tensors(name))


@pytest.mark.parametrize("call,shapes", CALLS)
def test_a_tensor_of_another_shape_is_refused(canopy, no_calls, call, shapes):
    for name, shape in shapes.items():
        if name in ("ws", "freqs"):
            continue
        for i in range(len(shape)):
            odd = tuple(n + (7 if j == i else 0) for j, n in enumerate(shape))
            if (name, i) in (("positions", 0), ("page_table", 1)) or name == "k_cache" and i in (0, 2) or \
                    (call, name, i) == ("cache_commit", "parent", 1):
                continue  # sizes of its own (the caches' are compared with each other)
            args = {n: on(0, *(odd if n == name else s), dtype=dtype_of(n)) for n, s in shapes.items()}
            with pytest.raises(canopy.CanopyError):
                getattr(canopy, call)(**args)


@pytest.mark.parametrize("call,shapes,small", [("attend", ATTEND, 4), ("attend", ATTEND, 5), ("qk_prep", PREP, 4),
                                               ("cache_commit", COMMIT, 5), ("cache_commit", COMMIT, 3)])
def test_sizes_beyond_32_bits_are_refused(canopy, no_calls, call, shapes, small):
    def at(name, shape):
        t = torch.empty(*[BIG if n == small else n for n in shape], device="meta", dtype=dtype_of(name))
        t = t.as_subclass(OnGpu)
        t.index = 0
        return t

    with pytest.raises(canopy.CanopyError, match="sizes"):
        getattr(canopy, call)(**{n: at(n, s) for n, s in shapes.items()})


def test_combinations_that_are_refused(canopy, no_calls):
    a = {n: on(0, *s, dtype=dtype_of(n)) for n, s in ATTEND.items()}
    starts = on(0, 3, dtype=torch.int32)
    packed = on(0, 9, 4, 64)
    for kw in (dict(starts=starts), dict(q=packed, out=None), dict(q=packed, out=None, starts=starts),
               dict(q=packed, out=None, parent=None, starts=starts),
               dict(q=packed, out=None, parent=None, lengths=None),
               dict(q=a["q"].half()), dict(k_cache=a["k_cache"].bfloat16()), dict(ws=on(0, 4, dtype=torch.uint8)),
               dict(window=2 ** 31)):
        with pytest.raises(canopy.CanopyError):
            canopy.attend(**{**a, **kw})
    p = {n: on(0, *s, dtype=dtype_of(n)) for n, s in PREP.items()}
    for kw in (dict(k_out=p["k"]), dict(v=None), dict(k_cache=None), dict(starts=starts),
               dict(positions=on(0, 2, 2, dtype=torch.int32)),
               dict(q=p["q"].transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(canopy.CanopyError):
            canopy.qk_prep(**{**p, **kw})


def test_oracle_of_the_attention_layers():
    """The oracle's own pins: rotations keep lengths and differences of positions, equal keys average the values."""
    import numpy as np

    import oracle
    rng = np.random.RandomState(0)
    x, y = rng.standard_normal((2, 5, 1, 32))
    f = 0.1 ** np.arange(8)
    rot = lambda z, p: oracle.attention.prep(z, "none", freqs=f, positions=np.array([p] * 1))  # noqa: E731
    a, b = rot(x, [3, 4, 5, 6, 7]), rot(y, [1, 1, 9, 2, 0])
    c, d = rot(x, [103, 104, 105, 106, 107]), rot(y, [101, 101, 109, 102, 100])
    assert np.allclose((a * b).sum(-1), (c * d).sum(-1)) and np.allclose((a ** 2).sum(), (x ** 2).sum())
    n = oracle.attention.prep(x, "l2", eps=0)
    assert np.allclose((n ** 2).sum(-1), 1)
    assert np.allclose(oracle.attention.prep(x, "rms", eps=0), n * 32 ** 0.5)
    k, v = np.ones((3, 1, 4, 8)), rng.standard_normal((3, 1, 4, 8))
    table = np.array([[2, 0]])
    o, w = oracle.attention.attend(rng.standard_normal((2, 2, 8)), k, v, table, [5], [range(2)])
    seen = np.concatenate([v[2, 0], v[0, 0]])
    assert np.allclose(o[0], seen[:6].mean(0)) and np.allclose(o[1, 1], seen[:7].mean(0)) and (w >= np.abs(o)).all()
    o, _ = oracle.attention.attend(rng.standard_normal((2, 1, 8)), k, v, table, [5], [range(2)], np.array([[-1, 0]]),
                                   window=2, sinks=1)
    assert np.allclose(o[1, 0], seen[[0, 5, 6]].mean(0))
    kn, vn, ctx = oracle.attention.commit([3], np.array([[-1, 0, 0, 2]]), k, v, table, np.array([4]))
    assert ctx.tolist() == [7] and np.allclose(vn[0, 0, :3], v[0, 0][[0, 2, 3]]) and np.allclose(vn[2], v[2])
