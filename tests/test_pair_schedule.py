"""The order in which the dense block's CTA pairs take their items, without a GPU, compiled from
the kernel's own header: every item once, in ascending order a pair, the long ones first."""
import ctypes as C
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def after(tmp_path_factory):
    d = tmp_path_factory.mktemp("schedule")
    src, so = d / "schedule.cpp", d / "schedule.so"
    src.write_text('#include "pair_schedule.h"\nextern "C" int next(int pairs, int n, int ahead, int pair, int item) '
                   "{ return moe::PairSchedule(pairs, n, ahead).next(pair, item); }\n")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", f"-I{ROOT}/fp4_weight_grouped_gb300/csrc", str(src), "-o",
                    str(so)], check=True)
    return getattr(C.CDLL(str(so)), 'next')


def taken(after, pairs, long_items, ahead, items):
    """The items of each pair, as the kernel's loops take them."""
    out = []
    for pair in range(pairs):
        mine, i = [], pair
        while i < items:
            mine.append(i)
            i = after(pairs, long_items, ahead, pair, i)
        assert mine == sorted(set(mine))
        out.append(mine)
    return out


@pytest.mark.parametrize("seed", range(200))
def test_every_item_once(after, seed):
    rng = random.Random(seed)
    pairs = rng.choice([1, 2, 3, 7, 76])
    long_items = rng.randint(0, pairs - 1)
    ahead = rng.randint(1, 40) if long_items else 0
    items = long_items + rng.randint(0 if long_items else 1, 400)
    got = taken(after, pairs, long_items, ahead, items)
    assert sorted(sum(got, [])) == list(range(items))
    for pair in range(long_items):
        assert got[pair][0] == pair
        # nobody takes a short item after a long one while the others still have rounds ahead
        assert all(i >= long_items + ahead * (pairs - long_items) for i in got[pair][1:])


def test_without_long_items_it_goes_round(after):
    assert taken(after, 3, 0, 0, 8) == [[0, 3, 6], [1, 4, 7], [2, 5]]
