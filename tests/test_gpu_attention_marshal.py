"""The native side of the binding turns down integers that do not fit, before it lets other Python threads run, and
leaves no error behind."""

import pytest
import torch

pytestmark = pytest.mark.gpu

BIG = [2 ** 31, -2 ** 31 - 1, 2 ** 63, 2 ** 200, -2 ** 200]


@pytest.fixture
def native(lib):
    lib.load()
    if isinstance(lib._marshal, lib._NoMarshal):
        pytest.skip("the native side is not built here")
    return lib._marshal


@pytest.mark.parametrize("big", BIG)
def test_norm_and_pairs(native, big):
    q, k = torch.randn(2, 3, 2, 64, device="cuda").unbind()
    out, plain = torch.full_like(q, 7), [q, k, None, 1, None, None, 1e-6, None, None, None, 0, None, None] + [None] * 7
    assert native.qk_prep(*plain) is not None
    for at in (3, 10):
        a = list(plain)
        a[11], a[at] = out, big
        assert native.qk_prep(*a) is None
    assert (out == 7).all()


@pytest.mark.parametrize("big", BIG)
def test_window_and_sinks(lib, native, big):
    q, (k, v) = torch.randn(1, 2, 64, device="cuda"), torch.randn(2, 1, 2, 16, 64, device="cuda").unbind()
    table, context = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((1, 1), (1,)))
    ws, out = lib.attend_workspace(1, 1, 2, 2, 64), torch.full_like(q, 7)
    plain = [q, k, v, table, context, ws, None, None, None, 4, 2, None, None]
    assert native.attend(*plain) is not None
    for at in (9, 10):
        a = list(plain)
        a[12], a[at] = out, big
        assert native.attend(*a) is None
    assert (out == 7).all()
