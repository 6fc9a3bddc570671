"""The work list of the key-weights kernel, restated: every CTA's run of steps
covers each visible (query row, key) pair exactly once, reads rows in bounds,
and writes its sums to slots of its own within the workspace."""

import random

import numpy as np
import pytest

N_CTAS = 148


class Seq:
    def __init__(self, n, Nq, G, causal, keys, bn, row_tiles):
        self.len, self.keys, self.bn, self.G, self.row_tiles = n, keys, bn, G, row_tiles
        self.units = -(-n // keys) if n > 0 and row_tiles > 0 else 0
        self.kb = -(-n // bn)
        self.whole = self.units
        if causal and keys == 256:
            self.whole = min(self.units, -(-(n - Nq) // keys)) if n > Nq else 0

    def head_tiles(self, u):
        return self.kb - self.keys // self.bn * u

    def steps(self, u):
        return self.row_tiles if u < self.whole else self.G * self.head_tiles(u)

    def total(self):
        m = self.units - self.whole
        return self.whole * self.row_tiles + self.G * (
            m * self.kb - self.keys // self.bn * (m * (self.whole + self.units - 1) // 2))


def _run(B, G, Hkv, Nq, Ncap, lens, causal, bn, nres):
    row_tiles = -(-G * Nq // bn)
    keys = 128 if row_tiles <= nres else 256
    seqs = [Seq(n, Nq, G, causal, keys, bn, row_tiles) for n in lens]
    for s in seqs:
        assert s.total() == sum(s.steps(u) for u in range(s.units))
    steps = [(b, h, u, s) for b in range(B) for h in range(Hkv) for u in range(seqs[b].units)
             for s in range(seqs[b].steps(u))]
    assert len(steps) == Hkv * sum(s.total() for s in seqs)
    per = -(-len(steps) // N_CTAS)
    units_max = -(-Ncap // keys)
    slots = {}
    seen = [[np.zeros((G * Nq, Ncap), int) for _ in range(Hkv)] for _ in range(B)]
    for x, (b, hkv, u, s) in enumerate(steps):
        q, n = seqs[b], lens[b]
        cta, unit = x // per, (b * Hkv + hkv) * units_max + u
        assert slots.setdefault(unit + cta, (unit, cta)) == (unit, cta)
        assert unit + cta < B * Hkv * units_max + N_CTAS
        if u < q.whole:
            row0, rows = s * bn, min(bn, G * Nq - s * bn)
        else:
            h, t = divmod(s, q.head_tiles(u))
            row0, rows = h * Nq + u * keys - (n - Nq) + t * bn, min(bn, n - u * keys - t * bn)
            assert row0 // Nq == (row0 + rows - 1) // Nq == h
        assert rows > 0 and 0 <= row0 and row0 + rows <= G * Nq
        r = np.arange(row0, row0 + rows)
        k = np.arange(u * keys, min(n, (u + 1) * keys))
        vis = (r % Nq)[:, None] >= k[None] - (n - Nq) if causal else np.ones((rows, len(k)), bool)
        seen[b][hkv][np.ix_(r, k)] += vis
    for b in range(B):
        i, k = np.arange(G * Nq) % max(Nq, 1), np.arange(Ncap)
        want = (k[None] < lens[b]) & ((k[None] <= lens[b] - Nq + i[:, None]) | (not causal))
        for hkv in range(Hkv):
            assert (seen[b][hkv] == want).all()


@pytest.mark.parametrize("seed", range(60))
def test_key_weights_work_list(seed):
    rng = random.Random(seed)
    bn, nres = rng.choice([(128, 4), (128, 2), (64, 2)])
    B, G, Hkv, Ncap = rng.randint(1, 4), rng.choice([1, 2, 3, 4]), rng.randint(1, 3), rng.randint(1, 900)
    Nq = Ncap if rng.random() < 0.4 else rng.randint(0, 300)
    lens = [rng.choice([rng.randint(0, Ncap), Ncap, -1]) for _ in range(B)]
    _run(B, G, Hkv, Nq, Ncap, [max(n, 0) for n in lens], rng.random() < 0.7, bn, nres)
