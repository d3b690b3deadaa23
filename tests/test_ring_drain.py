"""The end of a W4A4 CTA in which a wait gave up, without a GPU: a model of the ring's
barriers, and the count of missing arrivals compiled from the kernels' own header.

A stage's barrier completes when the producer, the four converter warps of the stage's set
and (in the even CTA of a pair) the relay have arrived and its copies have landed.  Everyone
goes through the stages in order and stops at any point; a copy may still be under way then.
The CTA may leave only when every issued copy has landed, and it learns of that from those
barriers.
"""
import ctypes as C
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def missing(tmp_path_factory):
    d = tmp_path_factory.mktemp("drain")
    src, so = d / "drain.cpp", d / "drain.so"
    src.write_text('#include "ring_drain.h"\nextern "C" uint32_t missing(uint32_t s, uint32_t from, uint32_t n, uint32_t k, '
                   "const uint32_t *at, const uint32_t *relay) { return moe::missing_arrivals(s, from, n, k, at, relay); }\n")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", f"-I{ROOT}/fp4_weight_grouped_gb300/csrc", str(src), "-o",
                    str(so)], check=True)
    f = C.CDLL(str(so)).missing
    words = C.POINTER(C.c_uint32)
    f.argtypes, f.restype = [C.c_uint32] * 4 + [words, words], C.c_uint32
    return lambda stage, start, r: f(stage, start, r.n, r.k, (C.c_uint32 * 8)(*[a % (2 * r.n) for a in r.at]),
                                     (C.c_uint32 * 1)(r.relayed % (2 * r.n)) if r.relay else None)


class Ring:
    def __init__(self, rng, n_stages, k_stages, items, relay):
        self.rng, self.n, self.k, self.total, self.relay = rng, n_stages, k_stages, items * k_stages, relay
        self.count = 5 + relay
        self.pending = [self.count] * n_stages       # arrivals that a slot's phase waits for
        self.copies = [0] * n_stages                 # copies under way
        self.phase = [0] * n_stages
        self.used = 0                                # stages whose MMAs are done
        self.issued = 0
        self.at = [self.first(w // 4, 0) for w in range(8)]    # next stage of each converter warp
        self.relayed = 0

    def first(self, s, stage):
        """The first stage at or after `stage` of set s."""
        while stage < self.total and stage % self.k % 2 != s:
            stage += 1
        return stage

    def arrive(self, slot):
        assert self.pending[slot] > 0, "one arrival too many"
        self.pending[slot] -= 1
        self.complete(slot)

    def complete(self, slot):
        if self.pending[slot] == 0 and self.copies[slot] == 0:
            self.phase[slot] += 1
            self.pending[slot] = self.count

    def done(self, stage):
        return self.phase[stage % self.n] > stage // self.n

    def land(self):
        slots = [s for s in range(self.n) if self.copies[s]]
        if slots:
            s = self.rng.choice(slots)
            self.copies[s] = 0
            self.complete(s)

    def step(self, who):
        if who == "copy":
            self.land()
        elif who == "produce" and self.issued < min(self.total, self.used + self.n):
            slot = self.issued % self.n
            self.copies[slot] = 1
            self.issued += 1
            self.arrive(slot)
        elif who == "mma" and self.used < self.issued and self.done(self.used):
            self.used += 1
        elif who == "relay" and self.relay and self.relayed < min(self.total, self.used + self.n):
            self.arrive(self.relayed % self.n)
            self.relayed += 1
        elif isinstance(who, int) and self.at[who] < min(self.total, self.used + self.n):
            self.arrive(self.at[who] % self.n)
            self.at[who] = self.first(who // 4, self.at[who] + 1)


def window(r):
    return range(max(0, r.issued - r.n), r.issued)


def stopped(seed):
    """A ring that ran for a while, most of whose parts then stopped one by one."""
    rng = random.Random(seed)
    r = Ring(rng, rng.randint(3, 5), rng.randint(1, 7), rng.randint(1, 6), rng.random() < 0.5)
    who = ["copy", "produce", "mma", "relay", *range(8)]
    for _ in range(rng.randint(0, 400)):
        r.step(rng.choice(who))
    for w in rng.sample(who, len(who)):
        for _ in range(rng.randint(0, 6)):
            r.step(w)
    return r


def test_waiting_alone_is_not_enough():
    """With every copy landed, some barriers of issued stages still never complete."""
    stuck = 0
    for seed in range(200):
        r = stopped(seed)
        for _ in range(r.n):
            r.land()
        stuck += any(not r.done(i) for i in window(r))
    assert stuck


def test_missing_arrivals_complete_every_issued_stage(missing):
    late = 0
    for seed in range(3000):
        r = stopped(seed)
        start = next((i for i in window(r) if not r.done(i)), r.issued)
        for i in range(start, r.issued):
            assert r.phase[i % r.n] >= i // r.n, "the phase before is complete"
            for _ in range(missing(i, start, r)):
                r.arrive(i % r.n)
            late += r.copies[i % r.n]
            assert r.done(i) == (r.copies[i % r.n] == 0), "only the copies are waited for"
        for _ in range(r.n):
            r.land()
        assert all(r.done(i) for i in window(r))
    assert late > 1000
