"""Up to 64 query heads on a key head: every row tile, slot and join that these sizes take, in both types."""

import numpy as np
import pytest

from attention_cases import TREES, attend_case, check_attend

pytestmark = pytest.mark.gpu

HEADS = [(17, 1, 64), (34, 2, 128), (24, 1, 128), (96, 2, 64), (48, 1, 128), (64, 1, 64), (128, 2, 128)]


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("HQ,HKV,d", HEADS)
def test_single_tokens(lib, HQ, HKV, d, bf16):
    check_attend(lib, attend_case(1, [1] * 5, [0, 1, 80, 130, 700], HQ, HKV, d, 32, bf16, T=1))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("HQ,HKV,d", HEADS)
def test_one_token(lib, HQ, HKV, d, bf16):
    check_attend(lib, attend_case(2, [1], [3000], HQ, HKV, d, 16, bf16, T=1))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("HQ,HKV,d", HEADS)
@pytest.mark.parametrize("T,tree", [(2, "chain"), (7, "random"), (33, "random")])
def test_trees(lib, HQ, HKV, d, T, tree, bf16):
    check_attend(lib, attend_case(T, [T, 0, T - T // 3], [0, 100, 129], HQ, HKV, d, 16, bf16, T=T, tree=TREES[tree]))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("HQ,HKV,d", HEADS)
def test_packed(lib, HQ, HKV, d, bf16):
    check_attend(lib, attend_case(3, [5, 0, 70, 11, 1], [0, 9, 128, 250, 513], HQ, HKV, d, 64, bf16))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("HQ,HKV,d", HEADS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (50, 3), (200, 130)])
def test_windows(lib, HQ, HKV, d, window, sinks, bf16):
    check_attend(lib, attend_case(4, [1] * 3, [3, 129, 700], HQ, HKV, d, 16, bf16, T=1), window, sinks)
    check_attend(lib, attend_case(5, [40, 1, 90], [3, 129, 300], HQ, HKV, d, 32, bf16), window, sinks)
    check_attend(lib, attend_case(6, [9, 20], [129, 300], HQ, HKV, d, 64, bf16, T=20, tree=TREES["random"]), window,
                 sinks)


@pytest.mark.parametrize("g", [1, 4, 7, 16])
def test_one_long_sequence_among_single_tokens(lib, g):
    """Row tiles follow one another in a sequence of the kernel for few rows."""
    lens = [1] * 40 + [{1: 500, 4: 100, 7: 40}[g]] if g < 16 else [1] * 30 + [0] * 30 + [29]
    c = attend_case(g, lens, [(37 * i) % 300 for i in range(len(lens))], 2 * g, 2, 128, 16, True)
    assert lib.attend_plan(len(c["q"]), len(lens), 2 * g, 2, True, 128) == "few" and len(c["q"]) == sum(lens)
    check_attend(lib, c)
    check_attend(lib, c, 30, 2)
    rest = dict(c, lens=c["lens"][::-1].copy(), ctxs=c["ctxs"][::-1].copy(), table=c["table"][::-1].copy())
    first = np.concatenate([[0], np.cumsum(rest["lens"])])
    rest["rows"] = [range(int(f), int(f) + int(n)) for f, n in zip(first, rest["lens"])]
    check_attend(lib, rest)
