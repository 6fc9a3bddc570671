"""The barriers of fa_cache_tc_kernel as a randomised model (see
test_barrier_protocols): one CTA's runs of key tiles, with the K/V ring, the two
buffers that scores and weights share, the Q tile's space that also stages O, the
exchange of row maxima through two halves, and O in TMEM across units."""

import random

import pytest

from test_barrier_protocols import _Bar, _run, _waiter

WARPS = [(wg, quarter) for wg in range(2) for quarter in range(4)]


def _unit_k(j):
    return 0 if j == 0 else 2 * j - 1


def _unit_v(j, n):
    return 2 * n - 1 if j == n - 1 else 2 * j + 2


def _decode(u, n):
    """(is V, tile) of the u-th of a run's 2n loads."""
    if u == 0:
        return False, 0
    if u == 2 * n - 1:
        return True, n - 1
    return (False, (u + 1) // 2) if u & 1 else (True, u // 2 - 1)


def _simulate(runs, nslot, nch, seed, mistake=None):
    """runs: key tiles of the CTA's consecutive units."""
    rnd = random.Random(seed)
    starts = [sum(runs[:r]) for r in range(len(runs))]  # number of a run's first tile
    bars = {"q": _Bar(8)}
    for i in range(nslot):
        bars[f"kf{i}"], bars[f"ke{i}"] = _Bar(1), _Bar(1)
    for x in range(2):
        bars[f"s{x}"], bars[f"p{x}"], bars[f"o{x}"] = _Bar(1), _Bar(8), _Bar(1)
    named = {"all": _Bar(8), **{quarter: _Bar(2) for quarter in range(4)}}
    wait, wait_named = _waiter(bars), _waiter(named)
    tma, pipe = [], []
    slot = [None] * nslot
    scores = [None, None]                        # tile whose scores or weights a buffer holds
    read, weights = {}, {}                       # warps that have read a tile's scores, written its weights
    q_tile, staging = {w: None for w in WARPS}, set()  # run whose Q each warp wrote; warps whose O is staged
    s_done, pv_done = set(), set()
    o_read = {w: 0 for w in WARPS}               # runs whose O the warp has taken
    maxima = {}                                  # (half, wg, quarter) -> [content, read by the other warpgroup]
    rescales = random.Random(seed + 1)
    rescaled = [[rescales.random() < 0.3 for _ in range(4)] for _ in range(sum(runs))]  # by tile and quarter

    def tma_done(item):
        s, what = item
        slot[s] = what
        bars[f"kf{s}"].arrive()

    def pipe_done(item):
        if item[0] == "commit":
            bars[item[1]].arrive()
        elif item[0] == "s":
            _, run, j, slots = item
            tile = starts[run] + j
            assert all(slot[s] == (run, False, j, c) for c, s in enumerate(slots))
            assert all(r == run for r in q_tile.values()) and not staging
            assert tile < 2 or tile - 2 in pv_done
            scores[tile & 1] = tile
            s_done.add(tile)
        else:
            _, run, j, slots = item
            tile = starts[run] + j
            assert all(slot[s] == (run, True, j, c) for c, s in enumerate(slots))
            assert scores[tile & 1] == tile and weights[tile] == set(WARPS)
            if j == 0:
                assert all(n == run for n in o_read.values())
            pv_done.add(tile)

    def producer():
        seq = 0
        for run, n in enumerate(runs):
            for u in range(2 * n):
                is_v, j = _decode(u, n)
                for c in range(nch):
                    s = seq % nslot
                    if seq >= nslot:
                        yield from wait(f"ke{s}", seq // nslot - 1)
                    tma.append((s, (run, is_v, j, c)))
                    seq += 1
                    yield

    def mma():
        seq0 = 0
        for run, n in enumerate(runs):
            slots = lambda u: [(seq0 + u * nch + c) % nslot for c in range(nch)]  # noqa: B023, E731

            def arrived(u):
                for c in range(nch):
                    s = seq0 + u * nch + c  # noqa: B023
                    yield from wait(f"kf{s % nslot}", s // nslot)

            def product(kind, u, j):
                pipe.append((kind, run, j, slots(u)))  # noqa: B023
                pipe.append(("commit", f"{'s' if kind == 's' else 'o'}{(starts[run] + j) & 1}"))  # noqa: B023
                pipe.extend(("commit", f"ke{s}") for s in slots(u))  # noqa: B023

            yield from wait("q", run)
            for j in range(min(2, n)):
                yield from arrived(_unit_k(j))
                product("s", _unit_k(j), j)
            for j in range(n):
                tile = starts[run] + j
                yield from arrived(_unit_v(j, n))
                yield from wait(f"p{tile & 1}", tile >> 1)
                product("pv", _unit_v(j, n), j)
                if j + 2 < n:
                    yield from arrived(_unit_k(j + 2))
                    product("s", _unit_k(j + 2), j + 2)
            seq0 += 2 * n * nch

    def put(key, what):
        assert key not in maxima or maxima[key][1], "overwritten before it was read"
        maxima[key] = [what, False]

    def take(key, what):
        assert maxima[key][0] == what
        maxima[key][1] = True

    def softmax(warp):
        wg, quarter = warp
        met = {"all": 0, quarter: 0}

        def meet(name):
            if mistake == "no_all" and name == "all":
                return
            k = met[name]
            met[name] += 1
            named[name].arrive()
            yield from wait_named(name, k)

        for run, n in enumerate(runs):
            yield from meet("all")
            assert run == 0 or all(starts[run] - 1 - i in s_done for i in range(runs[run - 1]))
            assert not staging, "Q over an O that is still staged"
            q_tile[warp] = run
            yield
            bars["q"].arrive()
            for j in range(n):
                tile = starts[run] + j
                x = tile & 1
                yield from wait(f"s{x}", tile >> 1)
                assert scores[x] == tile
                yield
                assert scores[x] == tile and not weights.get(tile, set()) & {(0, quarter), (1, quarter)}
                read.setdefault(tile, set()).add(warp)
                put((x, wg, quarter), tile)
                if mistake != "no_meeting":
                    yield from meet(quarter)
                take((x, wg ^ 1, quarter), tile)
                yield
                if j > 0 and rescaled[tile][quarter]:
                    if mistake != "no_odone":
                        yield from wait(f"o{(tile - 1) & 1}", (tile - 1) >> 1)
                    assert tile - 1 in pv_done and tile not in pv_done
                    yield
                assert read[tile] >= {(0, quarter), (1, quarter)}
                weights.setdefault(tile, set()).add(warp)
                bars[f"p{x}"].arrive()
            tile = starts[run] + n - 1
            yield from wait(f"o{tile & 1}", tile >> 1)
            if wg == 1:
                put(((tile & 1) ^ 1, 1, quarter), ("l", run))
            yield from meet(quarter)
            if wg == 0:
                take(((tile & 1) ^ 1, 1, quarter), ("l", run))
            assert all(starts[run] + i in s_done for i in range(n))
            for _ in range(2):
                staging.add(warp)
                yield
                assert tile in pv_done and tile + 1 not in pv_done
                staging.discard(warp)
            o_read[warp] += 1

    gens = {"producer": producer(), "mma": mma(), **{w: softmax(w) for w in WARPS}}
    _run(gens, {"tma": (tma, tma_done), "pipe": (pipe, pipe_done)}, rnd, max_steps=2_000_000)
    assert pv_done == set(range(sum(runs))) and all(n == len(runs) for n in o_read.values())


def _runs(seed):
    rng = random.Random(seed)
    return [rng.choice([1, 1, 2, 3, 5, 9]) for _ in range(rng.randint(1, 7))]


@pytest.mark.parametrize("nslot,nch", [(8, 1), (5, 1), (5, 2)], ids=["d64", "d128", "d256"])
def test_cache_tc_protocol(nslot, nch):
    for seed in range(25):
        _simulate(_runs(seed), nslot, nch, seed)


@pytest.mark.parametrize("mistake", ["no_all", "no_meeting", "no_odone"])
def test_cache_tc_model_catches_a_missing_wait(mistake):
    with pytest.raises((AssertionError, KeyError)):
        for seed in range(60):
            _simulate([3, 2, 4], 5, 1, seed, mistake)
