"""The work lists of the cache kernels, restated: the CTAs' runs cover each
visible (query row, key) pair of the key weights, and each key tile of the cache
attention, exactly once, read rows in bounds, and write to slots of their own
within the workspace.  And the mbarrier protocol of the key-weights kernel as a
randomised model (see test_barrier_protocols)."""

import random

import numpy as np
import pytest

from test_barrier_protocols import _Bar, _run as _drive, _waiter

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


def _cache_runs(p_units, p_rt, np_keys, Hkv, own_rt, lens, keys, n_ctas, cta):
    """CacheRuns restated: yields (unit, prefix, b, hkv, rt, t0, t1, tiles)."""
    tiles_of = lambda n: -(-n // keys) if n > 0 else 0  # noqa: E731
    in_prefix = p_units * tiles_of(np_keys)
    own = [Hkv * own_rt * tiles_of(n) for n in lens]
    total = in_prefix + sum(own)
    per = -(-total // n_ctas)
    x = per * cta
    if x >= total:
        return
    left = min(total, x + per) - x
    if x < in_prefix:
        prefix, tiles = True, tiles_of(np_keys)
        unit, t0 = divmod(x, tiles)
        b, (hkv, rt) = 0, divmod(unit, p_rt)
    else:
        x -= in_prefix
        prefix, b = False, 0
        while x >= own[b]:
            x -= own[b]
            b += 1
        tiles = tiles_of(lens[b])
        u, t0 = divmod(x, tiles)
        hkv, rt = divmod(u, own_rt)
        unit = p_units + (b * Hkv + hkv) * own_rt + rt
    while True:
        t1 = min(tiles, t0 + left)
        yield unit, prefix, b, hkv, rt, t0, t1, tiles
        left -= t1 - t0
        if left <= 0:
            return
        t0 = 0
        if prefix and unit + 1 < p_units:
            unit += 1
            hkv, rt = divmod(unit, p_rt)
            continue
        if prefix:
            prefix, b, hkv, rt = False, -1, Hkv - 1, own_rt - 1
        rt += 1
        if rt == own_rt:
            rt, hkv = 0, hkv + 1
            if hkv == Hkv:
                hkv, b = 0, b + 1
                while tiles_of(lens[b]) == 0:
                    b += 1
                tiles = tiles_of(lens[b])
        unit = p_units + (b * Hkv + hkv) * own_rt + rt


@pytest.mark.parametrize("units,tiles,n_ctas", [(16, 157, 96), (6, 1, 148), (24, 3, 144), (5, 7, 25), (2, 300, 148)])
def test_cache_work_list_of_a_prefix_in_step(units, tiles, n_ctas):
    """The same number of CTAs for every unit: every tile once, no gap between a
    unit's first and last CTA, slots of their own."""
    split = n_ctas // units
    per, seen, slots, ctas = -(-tiles // split), set(), set(), {}
    for cta in range(n_ctas):
        unit = cta // split
        t0 = (cta - unit * split) * per
        if unit >= units or t0 >= tiles:
            continue
        for t in range(t0, min(tiles, t0 + per)):
            assert (unit, t) not in seen
            seen.add((unit, t))
        assert unit + cta not in slots
        slots.add(unit + cta)
        ctas.setdefault(unit, []).append(cta)
    assert len(seen) == units * tiles and max(slots) < units + n_ctas
    assert all(c == list(range(c[0], c[-1] + 1)) for c in ctas.values())


@pytest.mark.parametrize("seed", range(60))
def test_cache_work_list(seed):
    rng = random.Random(seed)
    keys, n_ctas = rng.choice([(128, 148), (16, 592), (32, 1184)])
    B, Hkv, own_rt = rng.randint(1, 40), rng.randint(1, 4), rng.choice([0, 1, 1, 2])
    p_rt = rng.choice([0, 1, 3]) if own_rt else 1
    np_keys = rng.choice([rng.randint(1, 300), rng.randint(1, 30000)])
    lens = [rng.choice([0, -1, rng.randint(0, 400), rng.randint(0, 5000)]) for _ in range(B)] if own_rt else [0] * B
    p_units, seen, slots, ranges = Hkv * p_rt, {}, {}, {}
    for cta in range(n_ctas):
        for unit, prefix, b, hkv, rt, t0, t1, tiles in _cache_runs(p_units, p_rt, np_keys, Hkv, own_rt, lens, keys,
                                                                 n_ctas, cta):
            assert 0 <= t0 < t1 <= tiles
            n = np_keys if prefix else lens[b]
            assert (tiles - 1) * keys < n <= tiles * keys
            assert unit == (hkv * p_rt + rt if prefix else p_units + (b * Hkv + hkv) * own_rt + rt)
            for t in range(t0, t1):
                assert (unit, t) not in seen
                seen[unit, t] = cta
            assert (unit + cta) not in slots
            slots[unit + cta] = unit
            first, _ = ranges.get(unit, (None, None))
            ranges[unit] = (cta if t0 == 0 else first, cta if t1 == tiles else None)
    want = Hkv * p_rt * -(-np_keys // keys) + Hkv * own_rt * sum(-(-n // keys) for n in lens if n > 0)
    assert len(seen) == want
    assert all(s < p_units + B * Hkv * own_rt + n_ctas for s in slots)
    for unit, (c0, c1) in ranges.items():  # every CTA between the two has a slot of the unit
        assert c0 is not None and c1 is not None
        assert all(slots[unit + c] == unit for c in range(c0, c1 + 1))


def _simulate(units, resident, nk, nq, nbuf, nl, seed, heads=2, nwg=4):
    """One CTA's run: `units` row-tile counts of consecutive units (resident: all
    the same; `heads` splits them into kv heads).  The 4 warps of each of the `nwg`
    reading warpgroups are roles of their own."""
    rnd = random.Random(seed)
    ku = 1 if resident else 2
    # (unit, step in unit, unit ends, head starts, head ends)
    per_head = max(1, len(units) // heads)
    steps = [(u, s, s == n - 1, s == 0 and u % per_head == 0, s == n - 1 and (u + 1) % per_head == 0)
             for u, n in enumerate(units) for s in range(n)]
    steps[-1] = (*steps[-1][:2], True, steps[-1][3], True)
    bars = {}
    for name, n, count in (("kf", nk, 1), ("ke", nk, 1), ("qf", nq, 1), ("qe", nq, 1), ("sf", nbuf, 1),
                           ("se", nbuf, 4), ("lf", nl, 1), ("le", nl, 4 * ku)):
        for i in range(n):
            bars[f"{name}{i}"] = _Bar(count)
    wait = _waiter(bars)
    tma, pipe = [], []
    kslot, qslot, sbuf, lbuf = [None] * nk, [None] * nq, [None] * nbuf, [None] * nl
    done = {}

    def tma_done(item):
        slots, i, what, bar = item
        slots[i] = what
        bars[bar].arrive()

    def pipe_done(item):
        if item[0] == "commit":
            bars[item[1]].arrive()
            return
        _, x, sub, k, kwhat, q, qwhat = item
        assert kslot[k] == kwhat and qslot[q] == qwhat and sbuf[x] is None
        sbuf[x] = sub

    def producer():
        kseq = qseq = 0
        for i, (u, s, ends, head, _) in enumerate(steps):
            todo = []
            if resident and head:
                todo += [("q", (u // per_head, t)) for t in range(units[u])]
            if s == 0:
                todo += [("k", (u, k)) for k in range(ku)]
            if not resident:
                todo.append(("q", i))
            for kind, what in todo:
                seq, n, slots = (kseq, nk, kslot) if kind == "k" else (qseq, nq, qslot)
                if seq >= n:
                    yield from wait(f"{kind}e{seq % n}", seq // n - 1)
                tma.append((slots, seq % n, what, f"{kind}f{seq % n}"))
                kseq, qseq = kseq + (kind == "k"), qseq + (kind == "q")
            yield

    def mma():
        kseq = qseq = sub = 0
        for i, (u, s, ends, head, head_ends) in enumerate(steps):
            if resident and head:
                for t in range(units[u]):
                    yield from wait(f"qf{(qseq + t) % nq}", (qseq + t) // nq)
            if s == 0:
                for k in range(ku):
                    yield from wait(f"kf{(kseq + k) % nk}", (kseq + k) // nk)
            if not resident:
                yield from wait(f"qf{qseq % nq}", qseq // nq)
            q, qwhat = ((qseq + s) % nq, (u // per_head, s)) if resident else (qseq % nq, i)
            for k in range(ku):
                x = sub % nbuf
                if sub >= nbuf:
                    yield from wait(f"se{x}", sub // nbuf - 1)
                pipe.append(("mma", x, sub, (kseq + k) % nk, (u, k), q, qwhat))
                pipe.append(("commit", f"sf{x}"))
                sub += 1
            if not resident:
                pipe.append(("commit", f"qe{qseq % nq}"))
                qseq += 1
            elif head_ends:
                pipe.extend(("commit", f"qe{(qseq + t) % nq}") for t in range(units[u]))
                qseq += units[u]
            if ends:
                pipe.extend(("commit", f"ke{(kseq + k) % nk}") for k in range(ku))
                kseq += ku
            yield

    def filler(w):
        for q in range(w, len(steps), 2):
            if q >= nl:
                yield from wait(f"le{q % nl}", q // nl - 1)
            yield
            lbuf[q % nl] = q
            bars[f"lf{q % nl}"].arrive()

    def reader(grp):
        for sub in range(grp, len(steps) * ku, nwg):
            q, x = sub // ku, sub % nbuf
            yield from wait(f"lf{q % nl}", q // nl)
            assert lbuf[q % nl] == q
            yield from wait(f"sf{x}", sub // nbuf)
            assert sbuf[x] == sub
            yield
            assert sbuf[x] == sub and lbuf[q % nl] == q
            done[sub] = done.get(sub, 0) + 1
            if done[sub] == 4:
                sbuf[x] = None
            bars[f"se{x}"].arrive()
            bars[f"le{q % nl}"].arrive()

    gens = {"producer": producer(), "mma": mma(), "fill0": filler(0), "fill1": filler(1)}
    gens.update({f"wg{g}w{w}": reader(g) for g in range(nwg) for w in range(4)})
    _drive(gens, {"tma": (tma, tma_done), "pipe": (pipe, pipe_done)}, rnd, max_steps=2_000_000)
    assert done == {sub: 4 for sub in range(len(steps) * ku)}


# (resident, K slots, Q slots, TMEM buffers) of d = 64, 128, 256
_SHAPES = [(True, 8, 4, 4), (True, 4, 2, 4), (True, 2, 2, 8), (False, 4, 8, 4), (False, 2, 4, 4), (False, 2, 2, 8)]


def _units(resident, nq, rng):
    if resident:
        return [rng.randint(1, nq)] * rng.randint(1, 12)
    return [rng.randint(1, 7) for _ in range(rng.randint(1, 8))]


@pytest.mark.parametrize("shape", _SHAPES)
def test_key_weights_protocol(shape):
    resident, nk, nq, nbuf = shape
    for seed in range(12):
        rng = random.Random(seed)
        _simulate(_units(resident, nq, rng), resident, nk, nq, nbuf, 8, seed)


def test_key_weights_model_catches_a_ring_whose_readers_change():
    # four buffers for two fillers and three readers in turn: a reader waits for
    # a phase of a buffer whose phase before is not filled yet
    with pytest.raises(AssertionError):
        for seed in range(60):
            _simulate([1] * 24, True, 4, 2, 8, 4, seed, nwg=3)
