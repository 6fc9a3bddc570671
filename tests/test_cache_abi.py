"""Argument checks of the cache operators that need no GPU: the C ABI rejects
invalid arguments before touching CUDA, and the binding refuses CPU tensors."""

import pytest
import torch

from exact_attention_104_b200 import (FAError, attention_decode_prefix, attention_decode_weights,
                                      attention_key_weights, binding, cache_evict)
from exact_attention_104_b200.build import build

FAKE = 1 << 20  # an aligned, non-null address; validation must reject before any use
INV, UNS, OK = binding.FA_ERR_INVALID_ARG, binding.FA_ERR_UNSUPPORTED, binding.FA_OK


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def _prefix(**kw):
    a = dict(q=FAKE, kp=FAKE * 2, vp=FAKE * 3, k=FAKE * 4, v=FAKE * 5, lengths=FAKE * 6, o=FAKE * 7, lse=FAKE * 8,
             B=2, Hq=4, Hkv=2, Nq=1, Np=300, Ncap=100, d=128, causal=1, scale=0.088, ws=FAKE * 9, wsb=1 << 20)
    a.update(kw)
    return binding.fa_fwd_decode_prefix(*[a[n] for n in (
        "q", "kp", "vp", "k", "v", "lengths", "o", "lse", "B", "Hq", "Hkv", "Nq", "Np", "Ncap", "d", "causal",
        "scale", "ws", "wsb")], 0)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=0), INV), (dict(kp=0), INV), (dict(v=0), INV), (dict(o=0), INV), (dict(lse=0), INV), (dict(ws=0), INV),
    (dict(k=FAKE * 4 + 8), INV),                       # misaligned
    (dict(lengths=FAKE * 6 + 2), INV),
    (dict(ws=FAKE * 9 + 16), INV),                     # workspace not 256-aligned
    (dict(wsb=100), INV),                              # workspace too small
    (dict(o=FAKE), INV), (dict(o=FAKE * 2), INV),      # output over an input
    (dict(lse=FAKE * 7), INV),                         # outputs over each other
    (dict(ws=FAKE * 6), INV),                          # workspace over lengths
    (dict(Hq=3), INV), (dict(Np=-1), INV), (dict(Ncap=-1), INV), (dict(scale=float("nan")), INV),
    (dict(d=96), UNS), (dict(Nq=257), UNS), (dict(B=70000), UNS),
    (dict(Np=1 << 30, Hkv=2), UNS),                    # Hkv·Np reaches 2^31
    (dict(B=0), OK), (dict(Nq=0), OK),                 # empty problems: nothing to do
])
def test_prefix_argument_validation(kw, expect):
    assert _prefix(**kw) == expect


def _weights(**kw):
    a = dict(q=FAKE, k=FAKE * 2, v=FAKE * 3, lengths=FAKE * 4, w=FAKE * 5, wo=FAKE * 6, o=FAKE * 7, lse=FAKE * 8,
             B=2, Hq=4, Hkv=2, Nq=1, Nk=300, d=128, causal=1, scale=0.088, ws=FAKE * 9, wsb=1 << 20)
    a.update(kw)
    return binding.fa_fwd_decode_weights(*[a[n] for n in (
        "q", "k", "v", "lengths", "w", "wo", "o", "lse", "B", "Hq", "Hkv", "Nq", "Nk", "d", "causal", "scale", "ws",
        "wsb")], 0)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=0), INV), (dict(k=0), INV), (dict(wo=0), INV), (dict(ws=0), INV),
    (dict(wo=FAKE * 5 + 4), INV),                      # overlaps weights without being them
    (dict(wo=FAKE * 2), INV), (dict(wo=FAKE * 7), INV), (dict(w=FAKE * 5 + 2), INV),
    (dict(wsb=1000), INV), (dict(Hq=3), INV), (dict(Nk=-1), INV), (dict(scale=0.0), INV),
    (dict(d=32), UNS), (dict(Nq=257), UNS), (dict(B=40000, Hkv=2, Nk=4), UNS),
    (dict(B=0), OK), (dict(Nq=0, Nk=0), OK),
])
def test_decode_weights_argument_validation(kw, expect):
    assert _weights(**kw) == expect


def _keyw(**kw):
    a = dict(q=FAKE, k=FAKE * 2, lse=FAKE * 3, lengths=FAKE * 4, w=FAKE * 5, wo=FAKE * 6, B=2, Hq=4, Hkv=2, Nq=300,
             Nk=300, d=128, causal=1, scale=0.088, ws=FAKE * 9, wsb=1 << 20)
    a.update(kw)
    return binding.fa_key_weights(*[a[n] for n in (
        "q", "k", "lse", "lengths", "w", "wo", "B", "Hq", "Hkv", "Nq", "Nk", "d", "causal", "scale", "ws", "wsb")], 0)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=0), INV), (dict(k=0), INV), (dict(lse=0), INV), (dict(wo=0), INV), (dict(ws=0), INV),
    (dict(wo=FAKE), INV), (dict(wo=FAKE * 5 + 4), INV), (dict(lse=FAKE * 3 + 2), INV), (dict(k=FAKE * 2 + 8), INV),
    (dict(ws=FAKE * 9 + 16), INV), (dict(Hq=3), INV), (dict(Nq=-1), INV), (dict(scale=float("inf")), INV),
    (dict(d=96), UNS), (dict(B=40000, Hkv=2, Nk=4), UNS), (dict(B=60000, Hq=60000, Hkv=1, Nq=300), UNS),
    (dict(B=0), OK), (dict(Nk=0), OK),
])
def test_key_weights_argument_validation(kw, expect):
    assert _keyw(**kw) == expect


def _evict(**kw):
    a = dict(k=FAKE, v=FAKE * 2, w=FAKE * 3, lengths=FAKE * 4, ko=FAKE * 5, vo=FAKE * 6, wo=FAKE * 7, index=FAKE * 8,
             lo=FAKE * 9, B=2, Hkv=2, Nk=300, out_cap=120, budget=100, recent=10, d=128)
    a.update(kw)
    return binding.fa_cache_evict(*[a[n] for n in (
        "k", "v", "w", "lengths", "ko", "vo", "wo", "index", "lo", "B", "Hkv", "Nk", "out_cap", "budget", "recent",
        "d")], 0)


@pytest.mark.parametrize("kw,expect", [
    (dict(k=0), INV), (dict(w=0), INV), (dict(ko=0), INV), (dict(index=0), INV), (dict(lo=0), INV),
    (dict(budget=0), INV), (dict(budget=121), INV), (dict(recent=-1), INV), (dict(recent=101), INV),
    (dict(ko=FAKE), INV), (dict(vo=FAKE * 5), INV), (dict(wo=FAKE * 3), INV), (dict(lo=FAKE * 4), INV),
    (dict(ko=FAKE * 5 + 8), INV), (dict(index=FAKE * 8 + 2), INV),
    (dict(d=96), UNS), (dict(B=40000), UNS), (dict(Nk=1 << 30), UNS), (dict(out_cap=1 << 30), UNS),
    (dict(B=0), OK),
])
def test_evict_argument_validation(kw, expect):
    assert _evict(**kw) == expect


def test_workspace_bytes():
    # 256-byte rounded, 0 for sizes that the call refuses, more with scores to keep
    ws, ww, wk = (binding.fa_decode_prefix_workspace_bytes, binding.fa_decode_weights_workspace_bytes,
                  binding.fa_key_weights_workspace_bytes)
    assert ws(4, 8, 2, 1, 500, 64, 64) % 256 == 0 and ws(4, 8, 2, 1, 500, 64, 64) > 0
    assert ws(4, 7, 2, 1, 500, 64, 64) == 0 and ws(4, 8, 2, 257, 500, 64, 64) == 0 and ws(4, 8, 2, 1, 5, 6, 96) == 0
    assert ww(1, 8, 2, 1, 700, 64) >= 8 * 700 * 4 and ww(40000, 8, 2, 1, 7, 64) == 0
    assert wk(1, 4, 2, 300, 300, 128) % 256 == 0 and wk(1, 3, 2, 300, 300, 128) == 0
    assert ws(0, 8, 2, 1, 500, 64, 64) == 256 and wk(1, 4, 2, 300, 0, 128) == 256


def test_cpu_tensors_are_refused():
    q, k = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    w, lse = torch.zeros(1, 2, 8), torch.zeros(1, 2, 1)
    for call in (lambda: attention_decode_prefix(q, k[0], k[0], k, k), lambda: attention_decode_weights(q, k, k, w),
                 lambda: attention_key_weights(q, k, lse, w), lambda: cache_evict(k, k, w, 4),
                 lambda: cache_evict(None, k, w, 4)):
        with pytest.raises(FAError):
            call()
