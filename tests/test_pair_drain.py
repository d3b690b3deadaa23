"""The end of a CTA pair of the dense block in which a wait gave up, without a GPU: a model of
the stage barriers, and what is made up for compiled from the kernel's own header.

A stage's barrier completes when the even producer has arrived (expecting both CTAs' bytes)
and the bytes that it expects have landed.  Either producer stops at any stage within a
ring's length of what has been consumed; copies may still be under way then.  The pair may
leave only when every issued copy has landed, and it learns of that from those barriers."""
import ctypes as C
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("pair")
    src, so = d / "pair.cpp", d / "pair.so"
    src.write_text('#include "pair_drain.h"\nextern "C" void fix(uint32_t i, uint32_t n0, uint32_t n1, uint32_t bytes, uint32_t *o) '
                   "{ moe::PairFix f = moe::pair_fix(i, n0, n1, bytes); o[0] = f.arrive; o[1] = f.expect; o[2] = f.complete; }\n"
                   'extern "C" uint32_t first(uint32_t n0, uint32_t n1, uint32_t s) { return moe::pair_first(n0, n1, s); }\n')
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", f"-I{ROOT}/fp4_weight_grouped_gb300/csrc", str(src), "-o",
                    str(so)], check=True)
    lib = C.CDLL(str(so))

    def fix(i, n0, n1, b):
        o = (C.c_uint32 * 3)()
        lib.fix(i, n0, n1, b, o)
        return bool(o[0]), o[1], o[2]
    return fix, lib.first


class Barriers:
    def __init__(self, n):
        self.n, self.pending, self.tx, self.phase = n, [1] * n, [0] * n, [0] * n

    def settle(self, s):
        if self.pending[s] == 0 and self.tx[s] == 0:
            self.phase[s] += 1
            self.pending[s] = 1

    def arrive(self, s, expect):
        assert self.pending[s] == 1, "one arrival too many"
        self.tx[s] += expect
        self.pending[s] = 0
        self.settle(s)

    def land(self, s, n):
        self.tx[s] -= n
        self.settle(s)

    def done(self, i):
        return self.phase[i % self.n] > i // self.n


@pytest.mark.parametrize("seed", range(300))
def test_every_issued_copy_has_landed(rule, seed):
    fix, first = rule
    rng = random.Random(seed)
    n = rng.randint(2, 11)
    even, odd = rng.randint(1, 9) * 1024, rng.randint(1, 9) * 1024
    consumed = rng.randint(0, 40)
    # a producer is at most a ring past what is consumed; both have issued what is consumed
    n0, n1 = consumed + rng.randint(0, n), consumed + rng.randint(0, n)
    b, flying = Barriers(n), []
    for i in range(max(n0, n1)):
        copies = []
        if i < n0:
            b.arrive(i % n, even + odd)
            copies.append(even)
        if i < n1:
            copies.append(odd)
        for c in copies:
            if i < consumed or rng.random() < 0.4:
                b.land(i % n, c)
            else:
                flying.append((i, c))
    rng.shuffle(flying)
    for i in range(first(n0, n1, n), max(n0, n1)):
        if b.done(i):
            continue
        arrive, expect, complete = fix(i, n0, n1, odd)
        if arrive:
            b.arrive(i % n, expect)
        if complete:
            b.land(i % n, complete)
        # the wait: copies land in any order until this stage's barrier completes
        while not b.done(i):
            assert flying, "a barrier that never completes"
            j, c = flying.pop()
            b.land(j % n, c)
        assert not [f for f in flying if f[0] == i], "left with a copy under way"
    assert not flying
