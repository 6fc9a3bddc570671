"""How decoding behind a prefix divides the SMs between its two attention kernels
(a host rule, asked through its self-test entry): in bounds, and near the best
division under the model that the rule is made from."""

import random

import pytest

from exact_attention_104_b200 import FAError, binding
from exact_attention_104_b200.build import build

SMS = 148
# SM time in us: a key tile and a unit's start and end of the prefix's kernel, a step of the other's
TILE, UNIT, STEP = {64: 1.3, 128: 1.8, 256: 3.2}, {64: 4, 128: 4, 256: 6}, {64: 0.15, 128: 0.28, 256: 0.33}
HBM = 6554.2e3  # bytes a us


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


class Model:
    """Time of the two kernels side by side: caches two thirds full, read no faster
    than HBM gives."""

    def __init__(self, B, Hq, Hkv, Nq, Np, Ncap, d):
        self.d, self.row_tiles = d, -(-B * (Hq // Hkv) * Nq // 128)
        self.units, self.unit_tiles = Hkv * self.row_tiles, -(-Np // 128)
        keys = 16 if d == 256 else 32
        steps = B * Hkv * -(-Ncap // keys) * 2 / 3
        self.own_us, self.hbm_us = STEP[d] * steps, steps * keys * d * 4 / HBM

    def time(self, n, split):
        if split:
            tiles, units = -(-self.unit_tiles // split), 1
        else:
            tiles = -(-self.units * self.unit_tiles // n)
            units = (tiles + self.unit_tiles - 2) // self.unit_tiles + 1
        return max(tiles * TILE[self.d] + units * UNIT[self.d], self.own_us / (SMS - n), self.hbm_us)

    def best(self):
        equal = min(self.time(n, 0) for n in range(1, SMS))
        steps = [self.time(s * self.units, s) for s in range(1, SMS) if self.row_tiles > 1 and s * self.units < SMS]
        return min([equal, *steps])


def _check(c):
    n, split = binding.fa_selftest_cache_share(*c)
    m = Model(*c)
    assert 1 <= n <= SMS - 16 and n <= m.units * m.unit_tiles
    assert split == 0 or (m.row_tiles > 1 and n == split * m.units)
    # the bounds on the division cost up to SMS / (SMS - 16), going in step may cost a
    # tenth; equal runs are whole tiles, and of a unit more than the average
    allowed = 1.1 * SMS / (SMS - 16) * m.best() + TILE[m.d] + 2 * UNIT[m.d]
    assert m.time(n, split) <= allowed, (c, n, split, m.time(n, split), m.best())


# (B, Hq, Hkv, Nq, Np, Ncap, d)
@pytest.mark.parametrize("c", [
    (240, 64, 8, 1, 128, 1500, 128),    # 120 units of one tile beside large caches
    (240, 64, 8, 1, 500, 1500, 128),
    (160, 64, 8, 1, 20001, 100, 128),   # 80 units: twice as many do not fit
    (160, 64, 8, 1, 8192, 64, 128),
    (200, 32, 8, 1, 2000, 300, 64),
    (24, 16, 8, 5, 20001, 1500, 256),
    (32, 32, 8, 1, 8192, 1024, 128),
    (17, 8, 8, 1, 1, 65536, 128),       # one tile a unit, eight in all
    (60000, 1, 1, 1, 1, 1, 64),
], ids=lambda c: "b{}_hq{}_hkv{}_nq{}_np{}_cap{}_d{}".format(*c))
def test_division_is_near_the_best(c):
    _check(c)


def test_division_over_random_sizes():
    rng, log = random.Random(7), lambda r, lo, hi: round(lo * (hi / lo) ** r.random())
    for _ in range(2000):
        Hkv, G, d = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        Nq = rng.randint(1, 16 // G)
        B = log(rng, 16 // (G * Nq) + 1, 600)
        _check((B, Hkv * G, Hkv, Nq, log(rng, 1, 65536), log(rng, 1, 32768), d))


def test_in_step_where_it_was_measured_faster():
    # 24 x 5 rows behind 20001 keys: six CTAs for each of the 16 units
    assert binding.fa_selftest_cache_share(24, 16, 8, 5, 20001, 1500, 256) == (96, 6)


def test_no_division_where_one_kernel_runs():
    for c in ((2, 4, 2, 1, 500, 100, 64),      # few rows: the split kernel takes both
              (8, 4, 2, 20, 500, 100, 64),     # more than 16 rows a sequence: the other takes both
              (32, 32, 8, 1, 500, 0, 64), (32, 32, 8, 1, 0, 500, 64), (0, 4, 2, 1, 500, 100, 64)):
        assert binding.fa_selftest_cache_share(*c) == (0, 0)
    for c in ((2, 3, 2, 1, 500, 100, 64), (2, 4, 2, 1, 500, 100, 96), (2, 4, 2, 1, -1, 100, 64)):
        with pytest.raises(FAError):
            binding.fa_selftest_cache_share(*c)


@pytest.mark.parametrize("d,most", [(64, 32), (128, 32), (256, 64)])
def test_scores_are_stored_only_while_they_are_few(d, most):
    """17 to 64 query rows against a sequence's keys: more than `most` MB of scores
    would take longer than reading the keys again, so the workspace has no room for
    them; up to 16 rows, or no more than `most` MB, it has."""
    def workspace(B, G, Nq, n):
        return binding.fa_decode_weights_workspace_bytes(B, 8 * G, 8, Nq, n, d)

    for B, G, Nq in ((8, 8, 8), (1, 4, 8), (2, 3, 6)):
        row = B * 8 * G * Nq * 4  # bytes of one key's scores
        n = (most << 20) // row // 128 * 128
        assert workspace(B, G, Nq, n) >= n * row
        assert workspace(B, G, Nq, n + 128) < workspace(B, G, Nq, n)
    assert workspace(8, 16, 1, 32768) >= 8 * 8 * 16 * 32768 * 4
