"""GPU tests of the cache operators' workspaces (of exactly the size asked for,
with guard bytes on both sides), of both sides of the limit on stored scores, of
prompts of different lengths taken from a forward pass over a padded batch, and of
eviction against the order of its weights."""

import math

import numpy as np
import pytest
import torch

import _cache_oracle as ref
from exact_attention_104_b200 import (attention_decode_prefix, attention_decode_weights, attention_forward,
                                      attention_key_weights, binding, cache_evict, lib)

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
GUARD = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def _short_waits():
    lib().fa_set_wait_cap(1 << 28)
    yield
    lib().fa_set_wait_cap(0)


def _ok():
    torch.cuda.synchronize()
    assert binding.fa_device_status() == binding.FA_OK


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(BF16)


def _same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


def _guarded(call, need, g):
    """The call with a workspace of `need` bytes between two guards of random bytes."""
    assert need % 256 == 0 and need > 0
    buf = torch.randint(0, 256, (need + 2 * GUARD,), generator=g, device="cuda", dtype=torch.uint8)
    assert buf.data_ptr() % 256 == 0
    before = buf.clone()
    want = call()
    got = call(workspace=buf[GUARD:GUARD + need])
    _ok()
    assert _same(want, got)
    assert torch.equal(buf[:GUARD], before[:GUARD]) and torch.equal(buf[GUARD + need:], before[GUARD + need:])
    with pytest.raises(binding.FAError):
        call(workspace=buf[GUARD:GUARD + need - 256])


@pytest.mark.parametrize("seed", range(24))
def test_workspace_of_exactly_the_size_asked_for(seed):
    rng, g = np.random.default_rng(seed), torch.Generator("cuda").manual_seed(seed)
    d, Hkv, G = int(rng.choice([64, 128, 256])), int(rng.integers(1, 9)), int(rng.choice([1, 2, 3, 4, 8]))
    B, Nq = int(rng.choice([1, 2, 5, 9, 40])), int(rng.choice([1, 1, 2, 5, 8, 20]))
    Np, cap = int(rng.integers(1, 3000)), int(rng.integers(1, 1500))
    causal = bool(rng.integers(0, 2))
    n = torch.tensor([int(x) for x in rng.integers(0, cap + 1, B)], dtype=torch.int32, device="cuda")
    q, kp, vp = _normal(g, B, Hkv * G, Nq, d), _normal(g, Hkv, Np, d), _normal(g, Hkv, Np, d)
    k, v, w = _normal(g, B, Hkv, cap, d), _normal(g, B, Hkv, cap, d), torch.rand(B, Hkv, cap, device="cuda")
    for lens in (n, None):
        _guarded(lambda **kw: attention_decode_prefix(q, kp, vp, k, v, lens, causal=causal, **kw),
                 binding.fa_decode_prefix_workspace_bytes(B, Hkv * G, Hkv, Nq, Np, cap, d), g)
        _guarded(lambda **kw: attention_decode_weights(q, k, v, w, lens, causal=causal, **kw),
                 binding.fa_decode_weights_workspace_bytes(B, Hkv * G, Hkv, Nq, cap, d), g)
    Nq = cap if cap < 600 else int(rng.integers(1, 400))
    q = _normal(g, B, Hkv * G, Nq, d)
    lse = torch.full((B, Hkv * G, Nq), math.log(cap) + 0.5, device="cuda")
    for lens in (n, None):
        _guarded(lambda **kw: (attention_key_weights(q, k, lse, w, lens, causal=causal, **kw),),
                 binding.fa_key_weights_workspace_bytes(B, Hkv * G, Hkv, Nq, cap, d), g)


# 17 to 64 rows: up to 32 MB of scores are stored (64 MB at d = 256), beyond that the keys are read again
@pytest.mark.parametrize("B,Hkv,G,Nq,n,d", [(1, 8, 8, 8, 16384, 64), (1, 8, 8, 8, 16385, 64), (1, 8, 6, 4, 43647, 128),
                                            (1, 8, 6, 4, 43900, 128), (2, 4, 8, 8, 32768, 256),
                                            (2, 4, 8, 8, 32999, 256)])
def test_weights_on_both_sides_of_the_limit_on_scores(B, Hkv, G, Nq, n, d):
    g = torch.Generator("cuda").manual_seed(n)
    q, k, v = _normal(g, B, Hkv * G, Nq, d), _normal(g, B, Hkv, n, d), _normal(g, B, Hkv, n, d)
    w = torch.rand(B, Hkv, n, generator=g, device="cuda")
    lens = [n - 1000 * b for b in range(B)]
    o, lse, wo = attention_decode_weights(q, k, v, w, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                          causal=True)
    _ok()
    for b in range(B):
        for h in range(0, Hkv, 3):
            heads, m = slice(h * G, (h + 1) * G), lens[b]
            r = ref.attention(q[b, heads], k[b, h:h + 1, :m], v[b, h:h + 1, :m], True, d ** -0.5)
            ref.check_o_lse(o[b, heads], lse[b, heads], r, m, (b, h))
            ref.check_weights(wo[b, h:h + 1], w[b, h:h + 1], r, m, False, (b, h))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompts_of_different_lengths_from_a_padded_forward_pass(d):
    """fa_fwd on a right-padded batch leaves row i at position i; the key weights
    want each sequence's rows to end with it: rows 0 .. n-1 moved to N-n .. N-1."""
    B, Hq, Hkv, N = 4, 4, 2, 401
    lens, g = [401, 77, 1, 290], torch.Generator("cuda").manual_seed(d)
    q, k, v = _normal(g, B, Hq, N, d), _normal(g, B, Hkv, N, d), _normal(g, B, Hkv, N, d)
    _, lse = attention_forward(q, k, v, causal=True)
    q_end, lse_end = torch.full_like(q, math.nan), torch.full_like(lse, math.nan)
    for b, n in enumerate(lens):
        q_end[b, :, N - n:], lse_end[b, :, N - n:] = q[b, :, :n], lse[b, :, :n]
    w = attention_key_weights(q_end, k, lse_end, lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                              causal=True)
    _ok()
    for b, n in enumerate(lens):
        _, lse_ref, p, _, tol_s = ref.attention(q[b, :, :n], k[b, :, :n], None, True, d ** -0.5)
        # the definition with the LSE that the call was given
        given = lse[b, :, :n].double()
        p = p * torch.exp(lse_ref - given)[..., None]
        ref.check_weights(w[b], torch.zeros_like(w[b]), (None, given, p, None, tol_s), n, True, (b, n))


@pytest.mark.parametrize("cap,budget,recent", [(900, 100, 0), (9000, 1000, 77), (40000, 1, 0), (40000, 39999, 5)])
def test_eviction_by_the_order_of_its_weights(cap, budget, recent):
    """No dropped key weighs more than a kept one, nor as much with a lower index."""
    g = torch.Generator("cuda").manual_seed(cap)
    B, Hkv, d = 2, 2, 64
    k, v = _normal(g, B, Hkv, cap, d), _normal(g, B, Hkv, cap, d)
    w = torch.randint(0, 50, (B, Hkv, cap), generator=g, device="cuda").float() * 2.0 ** -40
    _, _, wo, index, count = cache_evict(k, v, w, budget, recent)
    _ok()
    assert count.tolist() == [budget] * B
    for wb, ib, ob in zip(w.flatten(0, 1), index.flatten(0, 1).long(), wo.flatten(0, 1)):
        assert (ib.diff() > 0).all() and torch.equal(ob, wb[ib])
        assert ib[budget - recent:].tolist() == list(range(cap - recent, cap))
        kept = torch.zeros(cap, dtype=torch.bool, device="cuda")
        kept[ib[:budget - recent]] = True
        old = torch.arange(cap, device="cuda") < cap - recent
        least = wb[kept].min()
        assert not (wb[old & ~kept] > least).any()
        equal = (old & (wb == least)).nonzero().flatten()
        assert kept[equal].int().diff().le(0).all()  # of those, the first ones stay
