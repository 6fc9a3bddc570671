"""GPU parity of the cache operators (decoding behind a shared prefix, decoding
with key weights, key weights of known queries, eviction) against their fp64
definitions, with the bounds of _cache_oracle.  What a cache holds behind a
sequence's length is NaN throughout."""

import math

import numpy as np
import pytest
import torch

import _cache_oracle as ref
from exact_attention_104_b200 import (attention_decode, attention_decode_prefix, attention_decode_weights,
                                      attention_forward, attention_key_weights, binding, cache_evict, lib)

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _short_waits():
    lib().fa_set_wait_cap(1 << 28)
    yield
    lib().fa_set_wait_cap(0)


def _ok():
    torch.cuda.synchronize()
    assert binding.fa_device_status() == binding.FA_OK


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF16)


def _lengths(lens):
    return None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")


def _cache(g, B, Hkv, cap, d, lens, std=1.0):
    """A cache whose rows behind the lengths are NaN."""
    x = _normal(g, B, Hkv, cap, d, std=std)
    for b in range(B):
        if lens is not None and lens[b] >= 0:
            x[b, :, lens[b]:] = math.nan
    return x


# ------------------------------------------------------------------ prefix
def _check_prefix(B, Hq, Hkv, Nq, Np, cap, d, causal, lens, seed=0, std=1.0):
    g = _gen(seed)
    q = _normal(g, B, Hq, Nq, d, std=std)
    kp, vp = _normal(g, Hkv, Np, d, std=std), _normal(g, Hkv, Np, d)
    k, v = _cache(g, B, Hkv, cap, d, lens, std), _cache(g, B, Hkv, cap, d, lens)
    o, lse = attention_decode_prefix(q, kp, vp, k, v, _lengths(lens), causal=causal)
    _ok()
    for b in range(B):
        n = cap if lens is None else lens[b]
        r = ref.attention(q[b], torch.cat([kp, k[b, :, :n]], 1), torch.cat([vp, v[b, :, :n]], 1), causal,
                          1 / math.sqrt(d))
        ref.check_o_lse(o[b], lse[b], r, Np + n, (b, n))


# (B, Hq, Hkv, Nq, Np, cap, d, causal, lens)
PREFIX = [
    (1, 1, 1, 1, 1, 1, 64, True, None),
    (1, 1, 1, 1, 1, 0, 128, True, None),                      # the prefix alone
    (2, 4, 2, 1, 0, 100, 128, True, [100, 37]),               # ragged caches, no prefix
    (3, 4, 2, 2, 0, 40, 64, True, [0, 1, 40]),                # nothing, less than Nq, full
    (3, 4, 2, 4, 5, 40, 64, True, [0, 1, 40]),                # rows that sit inside the prefix
    (3, 4, 2, 9, 5, 40, 128, True, [0, 2, 40]),               # rows before the first key, prefix too short
    (3, 4, 2, 9, 5, 40, 128, False, [0, 2, 40]),
    (4, 8, 2, 1, 500, 64, 64, True, [1, 22, 43, 64]),
    (5, 16, 2, 3, 129, 200, 256, True, [200, 1, 31, 32, 33]),
    (7, 8, 8, 1, 4097, 130, 128, True, [0, 1, 127, 128, 129, 130, 64]),
    (16, 32, 4, 1, 1000, 300, 128, True, [300 - 17 * b for b in range(16)]),   # 128 rows a kv head
    (9, 16, 2, 5, 777, 90, 256, True, [90 - 9 * b for b in range(9)]),         # 360 rows
    (3, 6, 2, 256, 300, 260, 64, True, [260, 3, 256]),        # the largest Nq
    (2, 2, 1, 17, 20001, 700, 128, False, [700, 350]),
    (33, 4, 1, 2, 640, 70, 128, True, [70 - 2 * b for b in range(33)]),
]


@pytest.mark.parametrize("c", PREFIX, ids=lambda c: "b{}_hq{}_hkv{}_nq{}_np{}_cap{}_d{}_{}".format(*c[:7], "c" if c[7] else "nc"))
def test_prefix_matches_definition(c):
    _check_prefix(*c)


@pytest.mark.parametrize("std", [4.0, 0.01])
def test_prefix_with_peaked_and_flat_softmax(std):
    # at std 4 scores reach some 2^9: the running maximum moves, most weights vanish
    _check_prefix(3, 8, 2, 4, 700, 300, 128, True, [300, 5, 150], seed=5, std=std)


def test_prefix_with_scores_that_grow_along_the_keys():
    # every run's maximum passes the one before: the running rescale in earnest
    d, Np, cap = 64, 1500, 500
    q = torch.ones(1, 2, 1, d, dtype=BF16, device="cuda")
    ramp = torch.linspace(0, 30, Np + cap, device="cuda")[:, None].expand(-1, d).to(BF16)
    v = _normal(_gen(3), Np + cap, d)
    args = [x.contiguous() for x in (ramp[None, :Np], v[None, :Np], ramp[None, None, Np:], v[None, None, Np:])]
    o, lse = attention_decode_prefix(q, *args, scale=0.5)
    _ok()
    ref.check_o_lse(o[0], lse[0], ref.attention(q[0], ramp[None], v[None], False, 0.5), Np + cap, "ramp")


def test_prefix_without_prefix_is_plain_decoding():
    g = _gen(8)
    q, k, v = _normal(g, 2, 8, 2, 128), _normal(g, 2, 2, 700, 128), _normal(g, 2, 2, 700, 128)
    none = torch.empty(2, 0, 128, dtype=BF16, device="cuda")
    o, lse = attention_decode_prefix(q, none, none, k, v, causal=True)
    o2, lse2 = attention_decode(q, k, v, causal=True)
    _ok()
    for b in range(2):
        r = ref.attention(q[b], k[b], v[b], True, 1 / math.sqrt(128))
        ref.check_o_lse(o[b], lse[b], r, 700, "prefix")
    assert (o.float() - o2.float()).abs().max() <= 2e-2 and (lse - lse2).abs().max() <= 1e-3


def test_prefix_seeded_random_shapes():
    rng = np.random.default_rng(314)
    for i in range(40):
        d, Hkv = int(rng.choice([64, 128, 256])), int(rng.integers(1, 4))
        G, B = int(rng.choice([1, 2, 3, 4, 8])), int(rng.integers(1, 12))
        Nq = int(rng.choice([1, 1, 1, 2, 3, 5, 8, 20]))
        Np, cap = int(rng.integers(0, 3000)), int(rng.integers(1, 600))
        lens = [int(x) for x in rng.integers(0, cap + 1, B)]
        _check_prefix(B, Hkv * G, Hkv, Nq, Np, cap, d, bool(rng.integers(0, 2)), lens, seed=i)


# ---------------------------------------------------------- decode weights
def _weights(g, B, Hkv, cap, lens):
    w = (torch.randn(B, Hkv, cap, generator=g, device="cuda") * 2).exp()
    for b in range(B):
        if lens is not None and lens[b] >= 0:
            w[b, :, lens[b]:] = math.nan
    return w


def _check_decode_weights(B, Hq, Hkv, Nq, cap, d, causal, lens, seed=0, std=1.0, known=True, inplace=False):
    g = _gen(seed)
    q = _normal(g, B, Hq, Nq, d, std=std)
    k, v = _cache(g, B, Hkv, cap, d, lens, std), _cache(g, B, Hkv, cap, d, lens)
    w = _weights(g, B, Hkv, cap, lens) if known else None
    before = w.clone() if known else torch.zeros(B, Hkv, cap, device="cuda")
    o, lse, wo = attention_decode_weights(q, k, v, w, _lengths(lens), causal=causal, weights_out=w if inplace else None)
    _ok()
    if inplace:
        assert wo is w
    for b in range(B):
        n = cap if lens is None else lens[b]
        r = ref.attention(q[b], k[b, :, :n], v[b, :, :n], causal, 1 / math.sqrt(d))
        ref.check_o_lse(o[b], lse[b], r, n, (b, n))
        ref.check_weights(wo[b], before[b], r, n, False, (b, n))
        if w is not None and not inplace:
            assert torch.equal(w[b].view(torch.int32), before[b].view(torch.int32))


# (B, Hq, Hkv, Nq, cap, d, causal, lens)
DECODE_W = [
    (1, 1, 1, 1, 1, 64, True, None),
    (1, 8, 2, 1, 700, 64, True, None),
    (2, 4, 4, 1, 33, 128, True, [33, 1]),
    (3, 8, 2, 3, 40, 128, True, [0, 2, 40]),              # an empty cache, rows before the first key
    (3, 8, 2, 3, 40, 256, False, [0, 2, 40]),
    (2, 16, 2, 8, 1500, 128, True, [1500, 1031]),         # 64 rows a kv head
    (2, 32, 1, 5, 600, 256, True, [600, 64]),             # 160 rows
    (1, 4, 1, 256, 300, 64, True, [299]),                 # the largest Nq
    (4, 8, 8, 1, 5000, 128, True, [5000, 4097, 1025, 1024]),
    (1, 4, 1, 1, 32768, 128, True, [32767]),
]


@pytest.mark.parametrize("c", DECODE_W, ids=lambda c: "b{}_hq{}_hkv{}_nq{}_cap{}_d{}_{}".format(*c[:6], "c" if c[6] else "nc"))
def test_decode_weights_matches_definition(c):
    _check_decode_weights(*c)


@pytest.mark.parametrize("known,inplace", [(False, False), (True, True)])
def test_decode_weights_from_zero_and_in_place(known, inplace):
    _check_decode_weights(3, 8, 2, 2, 300, 128, True, [300, 0, 170], seed=2, known=known, inplace=inplace)


@pytest.mark.parametrize("std", [4.0, 0.01])
def test_decode_weights_with_peaked_and_flat_softmax(std):
    _check_decode_weights(2, 8, 2, 4, 700, 128, True, [700, 5], seed=3, std=std)


def test_decode_weights_without_queries_or_keys():
    g = _gen(4)
    k, v, w = _normal(g, 2, 2, 50, 64), _normal(g, 2, 2, 50, 64), _weights(g, 2, 2, 50, None)
    q = torch.empty(2, 4, 0, 64, dtype=BF16, device="cuda")
    _, _, wo = attention_decode_weights(q, k, v, w, _lengths([50, 3]))
    _ok()
    assert torch.equal(wo, w)
    q = _normal(g, 2, 4, 1, 64)
    none, wn = torch.empty(2, 2, 0, 64, dtype=BF16, device="cuda"), torch.empty(2, 2, 0, device="cuda")
    o, lse, _ = attention_decode_weights(q, none, none, wn)
    _ok()
    assert (o == 0).all() and (lse == -math.inf).all()


def test_decode_weights_seeded_random_shapes():
    rng = np.random.default_rng(2718)
    for i in range(40):
        d, Hkv = int(rng.choice([64, 128, 256])), int(rng.integers(1, 4))
        G, B = int(rng.choice([1, 2, 3, 4, 8])), int(rng.integers(1, 5))
        Nq, cap = int(rng.choice([1, 1, 1, 2, 3, 5, 8, 20])), int(rng.integers(1, 4000))
        lens = [int(x) for x in rng.integers(0, cap + 1, B)]
        _check_decode_weights(B, Hkv * G, Hkv, Nq, cap, d, bool(rng.integers(0, 2)), lens, seed=i)


# ------------------------------------------------------------- key weights
def _check_key_weights(B, Hq, Hkv, Nq, cap, d, causal, lens, seed=0, std=1.0, known=True, inplace=False):
    g = _gen(seed)
    q, k = _normal(g, B, Hq, Nq, d, std=std), _cache(g, B, Hkv, cap, d, lens, std)
    w = _weights(g, B, Hkv, cap, lens) if known else None
    before = w.clone() if known else torch.zeros(B, Hkv, cap, device="cuda")
    refs, lse = [], torch.empty(B, Hq, Nq, device="cuda")
    for b in range(B):
        n = cap if lens is None else lens[b]
        refs.append((n, ref.attention(q[b], k[b, :, :n], None, causal, 1 / math.sqrt(d))))
        lse[b] = refs[b][1][1].float()
        if causal and n < Nq:  # rows before the sequence: whatever they hold
            lse[b, :, :Nq - n] = math.nan
            q[b, :, :Nq - n] = math.nan
    wo = attention_key_weights(q, k, lse, w, _lengths(lens), causal=causal, weights_out=w if inplace else None)
    _ok()
    for b, (n, r) in enumerate(refs):
        ref.check_weights(wo[b], before[b], r, n, True, (b, n))


# (B, Hq, Hkv, Nq, cap, d, causal, lens)
KEY_W = [
    (1, 1, 1, 1, 1, 64, True, None),
    (1, 4, 2, 1, 300, 128, True, None),
    (3, 4, 2, 64, 300, 128, True, [300, 0, 129]),
    (3, 4, 2, 64, 300, 64, True, [300, 30, 64]),           # a sequence shorter than the window
    (3, 4, 2, 64, 300, 64, False, [300, 30, 1]),
    (2, 4, 2, 257, 257, 128, True, None),                  # whole prompts
    (2, 4, 2, 257, 257, 128, False, None),
    (2, 3, 1, 300, 300, 256, True, [300, 211]),            # a padded batch of prompts
    (1, 8, 1, 128, 128, 256, True, None),
    (1, 2, 2, 1030, 1030, 64, True, None),
    (1, 16, 2, 64, 5000, 128, True, [4999]),
    (1, 4, 1, 1500, 4000, 128, True, [3999]),              # the last part of a prompt
]


@pytest.mark.parametrize("c", KEY_W, ids=lambda c: "b{}_hq{}_hkv{}_nq{}_cap{}_d{}_{}".format(*c[:6], "c" if c[6] else "nc"))
def test_key_weights_match_definition(c):
    _check_key_weights(*c)


@pytest.mark.parametrize("known,inplace", [(False, False), (True, True)])
def test_key_weights_from_zero_and_in_place(known, inplace):
    _check_key_weights(3, 8, 2, 200, 300, 128, True, [300, 0, 170], seed=2, known=known, inplace=inplace)


@pytest.mark.parametrize("std", [4.0, 0.01])
def test_key_weights_with_peaked_and_flat_softmax(std):
    _check_key_weights(2, 8, 2, 140, 700, 128, True, [700, 500], seed=3, std=std)


def test_key_weights_without_queries_and_with_rows_that_see_nothing():
    g = _gen(6)
    k, w = _normal(g, 2, 2, 50, 64), _weights(g, 2, 2, 50, None)
    wo = attention_key_weights(torch.empty(2, 4, 0, 64, dtype=BF16, device="cuda"), k,
                               torch.empty(2, 4, 0, device="cuda"), w)
    _ok()
    assert torch.equal(wo, w)
    # LSE -inf (no key visible): no weight, even where the mask shows keys
    lse = torch.full((2, 4, 3), -math.inf, device="cuda")
    wo = attention_key_weights(_normal(g, 2, 4, 3, 64), k, lse, w)
    _ok()
    assert torch.equal(wo, w)


def test_key_weights_agree_with_the_decoding_call():
    g = _gen(7)
    q, k, v = _normal(g, 2, 8, 6, 128), _normal(g, 2, 2, 900, 128), _normal(g, 2, 2, 900, 128)
    lens = _lengths([900, 411])
    _, lse, w = attention_decode_weights(q, k, v, lengths=lens, causal=True)
    w2 = attention_key_weights(q, k, lse, lengths=lens, causal=True)
    _ok()
    for b, n in enumerate([900, 411]):
        r = ref.attention(q[b], k[b, :, :n], None, True, 1 / math.sqrt(128))
        zero = torch.zeros_like(w[b])
        ref.check_weights(w[b], zero, r, n, False, "decode")
        ref.check_weights(w2[b], zero, r, n, False, "prompt")


def test_key_weights_seeded_random_shapes():
    rng = np.random.default_rng(1618)
    for i in range(40):
        d, Hkv = int(rng.choice([64, 128, 256])), int(rng.integers(1, 4))
        G, B = int(rng.choice([1, 2, 3, 4, 8])), int(rng.integers(1, 4))
        cap = int(rng.integers(1, 2000))
        Nq = cap if rng.random() < 0.4 else int(rng.integers(1, 257))
        lens = [int(x) for x in rng.integers(0, cap + 1, B)]
        _check_key_weights(B, Hkv * G, Hkv, Nq, cap, d, bool(rng.integers(0, 2)), lens, seed=i)


# ---------------------------------------------------------------- eviction
def _check_evict(w, lens, budget, recent, d, out_cap=None, seed=0):
    """w: fp32 [B, Hkv, cap] on the GPU; K, V random with NaN behind the lengths."""
    B, Hkv, cap = w.shape
    g = _gen(seed)
    k, v = _cache(g, B, Hkv, cap, d, lens), _cache(g, B, Hkv, cap, d, lens)
    size = budget if out_cap is None else out_cap
    ko, vo = _normal(g, B, Hkv, size, d), _normal(g, B, Hkv, size, d)
    wo = torch.randn(B, Hkv, size, generator=g, device="cuda")
    io = torch.full((B, Hkv, size), 77, dtype=torch.int32, device="cuda")
    old = [t.clone() for t in (ko, vo, wo, io)]
    ko, vo, wo, io, lo = cache_evict(k, v, w, budget, recent, _lengths(lens), out_cap=out_cap, k_out=ko, v_out=vo,
                                     weights_out=wo, index=io)
    _ok()
    for b in range(B):
        n = cap if lens is None else lens[b]
        count = min(n, budget)
        assert lo[b].item() == count
        for h in range(Hkv):
            want = ref.evict(w[b, h].tolist(), n, budget, recent)
            assert io[b, h, :count].tolist() == want, (b, h)
            idx = torch.tensor(want, dtype=torch.long, device="cuda")
            for got, src in ((ko, k), (vo, v)):
                assert torch.equal(got[b, h, :count].view(torch.int16), src[b, h, idx].view(torch.int16))
                assert (got[b, h, count:budget].float() == 0).all()
            assert torch.equal(wo[b, h, :count].view(torch.int32), w[b, h, idx].view(torch.int32))
            assert (wo[b, h, count:budget] == 0).all() and (io[b, h, count:budget] == -1).all()
    for got, was in zip((ko, vo, wo, io), old):
        assert torch.equal(got[:, :, budget:], was[:, :, budget:])


# (B, Hkv, cap, budget, recent, lens, out_cap, d)
EVICT = [
    (1, 1, 1, 1, 0, None, None, 64),
    (1, 2, 10, 1, 1, None, None, 64),
    (2, 2, 10, 20, 3, [10, 0], None, 128),                  # all stay, room beyond the cache
    (3, 2, 1000, 256, 32, [1000, 256, 257], None, 64),
    (3, 2, 1000, 256, 256, [1000, 100, 257], 300, 128),     # only recent ones
    (3, 2, 1000, 255, 0, [1000, 999, 1], 300, 256),         # only heavy ones
    (2, 3, 5000, 777, 100, [4999, 1025], None, 128),
    (1, 2, 70000, 9000, 1, [69999], None, 64),
    (40, 8, 300, 64, 8, [300 - 5 * b for b in range(40)], 70, 64),
]


@pytest.mark.parametrize("c", EVICT, ids=lambda c: "b{}_hkv{}_cap{}_budget{}_recent{}_d{}".format(*c[:5], c[7]))
def test_evict_matches_definition(c):
    B, Hkv, cap, budget, recent, lens, out_cap, d = c
    w = _weights(_gen(cap), B, Hkv, cap, None).masked_fill(
        torch.rand(B, Hkv, cap, generator=_gen(1), device="cuda") < 0.05, 0.0)
    for b in range(B):
        if lens is not None:
            w[b, :, lens[b]:] = math.inf  # never taken
    _check_evict(w, lens, budget, recent, d, out_cap)


@pytest.mark.parametrize("cap", [300, 3000, 20000])
@pytest.mark.parametrize("kind", ["equal", "zeros", "few", "special", "rising", "falling", "one_bit"])
def test_evict_ties_and_special_weights(kind, cap):
    g = _gen(11)
    j = torch.arange(cap, device="cuda", dtype=F32)
    w = {"equal": torch.full((cap,), 0.75, device="cuda"), "zeros": torch.zeros(cap, device="cuda"),
         "few": torch.randint(0, 3, (cap,), generator=g, device="cuda").float(),
         "special": torch.tensor([math.nan, -math.inf, -1.0, -0.0, 0.0, 1e-45, 1.0, math.inf, -math.nan],
                                 device="cuda")[torch.randint(0, 9, (cap,), generator=g, device="cuda")],
         "rising": j, "falling": -j,
         # values that differ in the last bit only: every digit of the radix matters
         "one_bit": (torch.full((cap,), 1.0, device="cuda").view(torch.int32)
                     + torch.randint(0, 2, (cap,), generator=g, device="cuda").int()).view(F32)}[kind]
    _check_evict(w[None, None].contiguous(), None, cap // 3, cap // 20, 64)


def test_evict_seeded_random_shapes():
    rng = np.random.default_rng(55)
    for i in range(40):
        d, B, Hkv = int(rng.choice([64, 128, 256])), int(rng.integers(1, 4)), int(rng.integers(1, 4))
        cap = int(rng.integers(1, 4000))
        budget = int(rng.integers(1, cap + 20))
        lens = [int(x) for x in rng.integers(0, cap + 1, B)]
        w = torch.randint(0, 400, (B, Hkv, cap), generator=_gen(i), device="cuda").float() / 16
        _check_evict(w, lens, budget, int(rng.integers(0, budget + 1)), d,
                     budget + int(rng.integers(0, 30)), seed=i)


# ------------------------------------------------------------ used together
def test_serving_run_with_a_bounded_cache():
    """A padded batch of prompts, their key weights, eviction, decoding steps that
    append to the cut caches behind a shared prefix of weights, and a second
    eviction: each step against its definition on what the step before left."""
    B, Hq, Hkv, N, d, budget, recent, steps = 2, 8, 2, 400, 128, 100, 20, 12
    scale, g = 1 / math.sqrt(d), _gen(21)
    q, k, v = _normal(g, B, Hq, N, d), _normal(g, B, Hkv, N, d), _normal(g, B, Hkv, N, d)
    _, lse = attention_forward(q, k, v, causal=True)
    w = attention_key_weights(q, k, lse, causal=True)
    room = budget + steps
    k, v, w, index, lens = cache_evict(k, v, w, budget, recent, out_cap=room)
    _ok()
    assert lens.tolist() == [budget] * B and (index[:, :, :budget].diff(dim=-1) > 0).all()
    for t in range(steps):
        new_k, new_v = _normal(g, B, Hkv, d), _normal(g, B, Hkv, d)
        k[:, :, budget + t], v[:, :, budget + t], w[:, :, budget + t] = new_k, new_v, 0.0
        lens += 1
        qt, before = _normal(g, B, Hq, 1, d), w.clone()
        o, lse, w = attention_decode_weights(qt, k, v, w, lens, causal=True, weights_out=w)
        _ok()
        for b in range(B):
            n = budget + t + 1
            r = ref.attention(qt[b], k[b, :, :n], v[b, :, :n], True, scale)
            ref.check_o_lse(o[b], lse[b], r, n, (t, b))
            ref.check_weights(w[b], before[b], r, n, False, (t, b))
    _check_evict(w, lens.tolist(), budget, recent, d)
    # the same caches behind a prefix
    kp, vp, qt = _normal(g, Hkv, 300, d), _normal(g, Hkv, 300, d), _normal(g, B, Hq, 1, d)
    o, lse = attention_decode_prefix(qt, kp, vp, k, v, lens, causal=True)
    _ok()
    for b in range(B):
        r = ref.attention(qt[b], torch.cat([kp, k[b]], 1), torch.cat([vp, v[b]], 1), True, scale)
        ref.check_o_lse(o[b], lse[b], r, 300 + room, b)


def _all_calls(seed):
    """One call of each operator as closures over their inputs and outputs."""
    g = _gen(seed)
    B, Hq, Hkv, d, cap = 3, 8, 2, 128, 700 + seed
    lens = _lengths([cap, 0, cap // 2 + seed])
    q, k, v = _normal(g, B, Hq, 2, d), _normal(g, B, Hkv, cap, d), _normal(g, B, Hkv, cap, d)
    kp, vp, w = _normal(g, Hkv, 900, d), _normal(g, Hkv, 900, d), _weights(g, B, Hkv, cap, None)
    qw = _normal(g, B, Hq, 150, d)
    _, lse_w = attention_decode_prefix(qw, kp[:, :0].contiguous(), vp[:, :0].contiguous(), k, v, lens, causal=True)
    torch.cuda.synchronize()
    return [lambda: attention_decode_prefix(q, kp, vp, k, v, lens, causal=True),
            lambda: attention_decode_weights(q, k, v, w, lens, causal=True),
            lambda: (attention_key_weights(qw, k, lse_w, w, lens, causal=True),),
            lambda: cache_evict(k, v, w, 200, 30, lens)]


def _same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


def test_same_bits_every_time_and_on_two_streams_at_once():
    calls = _all_calls(1) + _all_calls(2)
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[] for _ in calls]
    for _ in range(5):
        for i, c in enumerate(calls):
            with torch.cuda.stream(streams[i // 4]):
                got[i].append(c())
    _ok()
    for w, gs in zip(want, got):
        assert all(_same(w, x) for x in gs)


def test_captured_and_replayed_with_other_lengths():
    g = _gen(31)
    B, Hq, Hkv, d, cap = 2, 8, 2, 128, 600
    lens = _lengths([600, 600])
    q, k, v = _normal(g, B, Hq, 1, d), _normal(g, B, Hkv, cap, d), _normal(g, B, Hkv, cap, d)
    kp, vp, w = _normal(g, Hkv, 333, d), _normal(g, Hkv, 333, d), _weights(g, B, Hkv, cap, None)
    lse_q = torch.zeros(B, Hq, 1, device="cuda")

    def step():
        return [*attention_decode_prefix(q, kp, vp, k, v, lens, causal=True),
                *attention_decode_weights(q, k, v, w, lens, causal=True),
                attention_key_weights(q, k, lse_q, w, lens, causal=True), *cache_evict(k, v, w, 100, 10, lens)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        outs = step()
    for ns in ([600, 600], [0, 77], [599, 1]):
        lens.copy_(torch.tensor(ns))
        q.normal_(generator=g)
        graph.replay()
        got = [t.clone() for t in outs]
        assert _same(got, step())
    _ok()


def test_call_on_a_stream_of_its_own():
    g = _gen(41)
    q, k, v = _normal(g, 1, 4, 1, 64), _normal(g, 1, 2, 500, 64), _normal(g, 1, 2, 500, 64)
    want = attention_decode_weights(q, k, v)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream, 0):
        got = attention_decode_weights(q, k, v, stream=stream)
        torch.cuda.synchronize()
        assert _same(want, got)
    _ok()


def test_more_than_32_sequences_and_none_with_a_key():
    lens = [(37 * b) % 150 for b in range(70)]
    for some in (lens, [0] * 70):
        _check_prefix(70, 4, 2, 1, 200, 150, 64, True, some, seed=91)
        _check_prefix(70, 4, 2, 9, 0, 150, 64, True, some, seed=92)
        _check_decode_weights(70, 4, 2, 2, 150, 64, True, some, seed=93)
        _check_decode_weights(70, 8, 1, 9, 150, 128, True, some, seed=94)
        _check_key_weights(70, 4, 2, 150, 150, 64, True, some, seed=95)
        _check_key_weights(70, 4, 2, 20, 150, 128, True, some, seed=96)


@pytest.mark.parametrize("shift", [0, 1, 2, 3])
@pytest.mark.parametrize("n", [40, 41])
def test_weights_at_any_4_byte_boundary(shift, n):
    g = _gen(101)
    q, k, v = _normal(g, 2, 4, 3, 64), _normal(g, 2, 2, n, 64), _normal(g, 2, 2, n, 64)
    lens = _lengths([n, 7])
    buf = torch.rand(2 * 2 * n + 4, generator=g, device="cuda")
    w = buf[shift:shift + 4 * n].view(2, 2, n)
    aligned = w.clone()
    o, lse, want = attention_decode_weights(q, k, v, aligned, lens, causal=True)
    want2 = attention_key_weights(q, k, lse, aligned, lens, causal=True)
    got2 = attention_key_weights(q, k, lse, w, lens, causal=True)
    ev = cache_evict(k, v, aligned, 20, 3, lens), cache_evict(k, v, w, 20, 3, lens)
    around = buf.clone()
    _, _, got = attention_decode_weights(q, k, v, w, lens, causal=True, weights_out=w)
    _ok()
    assert torch.equal(got, want) and torch.equal(got2, want2) and _same(*ev)
    assert torch.equal(buf[:shift], around[:shift]) and torch.equal(buf[shift + 4 * n:], around[shift + 4 * n:])


def test_workspace_given_and_used_again():
    g = _gen(71)
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")  # its contents do not matter
    for B, Nq, n in ((2, 1, 300), (3, 9, 77), (2, 1, 300)):
        q, k, v = _normal(g, B, 4, Nq, 64), _normal(g, B, 2, n, 64), _normal(g, B, 2, n, 64)
        kp = _normal(g, 2, 200, 64)
        for call in (lambda **kw: attention_decode_prefix(q, kp, kp, k, v, causal=True, **kw),
                     lambda **kw: attention_decode_weights(q, k, v, causal=True, **kw)):
            want = call()
            assert _same(want, call(workspace=ws))
            ws.random_(generator=g)
    _ok()


def test_cache_of_more_than_2_to_31_elements():
    # the last kv head lies behind element 2^31; the others hold zeros
    Hkv, n, d, budget, recent = 5, 2_000_003, 256, 1000, 100
    g = _gen(81)
    k = torch.zeros(1, Hkv, n, d, dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    assert k.numel() - n * d < 2 ** 31 < k.numel()
    k[0, -1], v[0, -1] = _normal(g, n, d), _normal(g, n, d)
    q = _normal(g, 1, 2 * Hkv, 1, d, std=4.0)
    o, lse, w = attention_decode_weights(q, k, v, causal=True)
    kp = _normal(g, Hkv, 40, d)
    o2, lse2 = attention_decode_prefix(q, kp, kp, k, v, causal=True)
    w2 = attention_key_weights(q, k, lse, causal=True)
    ev = cache_evict(k, v, w, budget, recent)
    _ok()
    for got_o, got_lse, keys, values in ((o, lse, k[0, -1:], v[0, -1:]),
                                         (o2, lse2, torch.cat([kp[-1:], k[0, -1:]], 1),
                                          torch.cat([kp[-1:], v[0, -1:]], 1))):
        r = ref.attention(q[0, -2:], keys, values, True, 1 / math.sqrt(d))
        ref.check_o_lse(got_o[0, -2:], got_lse[0, -2:], r, keys.shape[1], "last head")
        if got_o is o:
            zero = torch.zeros(1, n, device="cuda")
            ref.check_weights(w[0, -1:], zero, r, n, False, "decode")
            ref.check_weights(w2[0, -1:], zero, r, n, True, "key weights")
        del r
    order = torch.sort(w[0, -1, :n - recent], descending=True, stable=True).indices[:budget - recent]
    want = torch.cat([order.sort().values, torch.arange(n - recent, n, device="cuda")])
    assert torch.equal(ev[3][0, -1].long(), want)
    assert torch.equal(ev[0][0, -1], k[0, -1, want]) and torch.equal(ev[1][0, -1], v[0, -1, want])


# ------------------------------------------------------- refusals, bad data
@pytest.mark.parametrize("bad", [-1, 301, 2 ** 31 - 1, -2 ** 31])
def test_lengths_out_of_range_are_reported(bad):
    g = _gen(51)
    B, Hq, Hkv, d, cap = 3, 4, 2, 64, 300
    q, k, v = _normal(g, B, Hq, 1, d), _normal(g, B, Hkv, cap, d), _normal(g, B, Hkv, cap, d)
    kp, vp, w = _normal(g, Hkv, 200, d), _normal(g, Hkv, 200, d), _weights(g, B, Hkv, cap, None)
    lse_q = torch.zeros(B, Hq, 1, device="cuda")
    good = _lengths([300, 5, 120])
    lens = _lengths([300, bad, 120])

    def outputs():
        new = lambda *shape, dtype=BF16: torch.full(shape, 7, dtype=dtype, device="cuda")  # noqa: E731
        return dict(out=new(B, Hq, 1, d), lse=new(B, Hq, 1, dtype=F32), weights_out=new(B, Hkv, cap, dtype=F32))

    def ev(n):
        new = lambda *shape, dtype=BF16: torch.full(shape, 7, dtype=dtype, device="cuda")  # noqa: E731
        return cache_evict(k, v, w, 50, 10, n, k_out=new(B, Hkv, 50, d), v_out=new(B, Hkv, 50, d),
                           weights_out=new(B, Hkv, 50, dtype=F32), index=new(B, Hkv, 50, dtype=torch.int32),
                           lengths_out=new(B, dtype=torch.int32))

    calls = [lambda n, o: attention_decode_prefix(q, kp, vp, k, v, n, out=o["out"], lse=o["lse"]),
             lambda n, o: attention_decode_weights(q, k, v, w, n, **o),
             lambda n, o: (attention_key_weights(q, k, lse_q, w, n, weights_out=o["weights_out"]),),
             lambda n, o: ev(n)]
    for call in calls:
        want = call(good, outputs())
        _ok()
        got = call(lens, outputs())
        torch.cuda.synchronize()
        assert binding.fa_device_status() == binding.FA_ERR_INVALID_ARG
        assert binding.fa_device_status() == binding.FA_OK
        for x, y in zip(want, got):
            assert torch.equal(x[0], y[0]) and torch.equal(x[2], y[2])
            assert (y[1].float() == 7).all()


def test_wrong_arguments_are_refused():
    g = _gen(61)
    B, Hq, Hkv, d, cap = 2, 4, 2, 64, 30
    q, k, v = _normal(g, B, Hq, 1, d), _normal(g, B, Hkv, cap, d), _normal(g, B, Hkv, cap, d)
    kp, w, n = _normal(g, Hkv, 20, d), _weights(g, B, Hkv, cap, None), _lengths([30, 30])
    lse = torch.zeros(B, Hq, 1, device="cuda")
    half = torch.float16
    refused = [
        lambda: attention_decode_prefix(q, kp, kp, k, v.to(half), n),
        lambda: attention_decode_prefix(q, kp, kp[:, :10], k, v, n),
        lambda: attention_decode_prefix(q, kp[:1], kp[:1], k, v, n),
        lambda: attention_decode_prefix(q, kp, kp, k, v, n.long()),
        lambda: attention_decode_prefix(q, kp, kp, k, v, n.cpu()),
        lambda: attention_decode_prefix(q, kp, kp, k, v, n[:1]),
        lambda: attention_decode_prefix(q[:, :3].contiguous(), kp, kp, k, v, n),       # Hq % Hkv
        lambda: attention_decode_prefix(q, kp, kp, k.transpose(1, 2).contiguous().transpose(1, 2), v, n),
        lambda: attention_decode_prefix(q, kp, kp, k, v, n, out=q),                    # output over an input
        lambda: attention_decode_prefix(q, kp, kp, k, v, n, scale=0.0),
        lambda: attention_decode_prefix(q.expand(B, Hq, 1, d).repeat(1, 1, 257, 1), kp, kp, k, v, n),
        lambda: attention_decode_prefix(q, kp, kp, k, v, n,
                                        workspace=torch.empty(256, dtype=torch.uint8, device="cuda")),
        lambda: attention_decode_prefix(q[..., :32].contiguous(), kp[..., :32].contiguous(),
                                        kp[..., :32].contiguous(), k[..., :32].contiguous(),
                                        v[..., :32].contiguous(), n),
        lambda: attention_decode_weights(q, k, v, w.double(), n),
        lambda: attention_decode_weights(q, k, v, w[..., :20], n),
        lambda: attention_decode_weights(q, k, v, w, n, out=q),
        lambda: attention_key_weights(q, k, lse[..., 0], w, n),
        lambda: attention_key_weights(q, k, lse.to(half), w, n),
        lambda: attention_key_weights(q.cpu(), k, lse, w, n),
        lambda: attention_key_weights(q, k, lse, w, n, scale=math.inf),
        lambda: cache_evict(k, v, w, 0, 0, n),
        lambda: cache_evict(k, v, w, 10, 11, n),
        lambda: cache_evict(k, v, w, 10, -1, n),
        lambda: cache_evict(k, v, w, 10, 1, n, out_cap=9),
        lambda: cache_evict(k, v, w[:, :1].contiguous(), 10, 1, n),
        lambda: cache_evict(k, v, w, 30, 1, n, k_out=k),                               # output over an input
    ]
    for i, call in enumerate(refused):
        with pytest.raises(binding.FAError):
            call()
            pytest.fail(f"call {i} was accepted")
    _ok()
