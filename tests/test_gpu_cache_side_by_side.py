"""GPU parity of decoding behind a prefix where its two attention kernels run side
by side (at most 16 query rows a sequence, more than 16 in the batch): divisions of
the SMs of every kind, several streams, capture and replay."""

import math

import pytest
import torch

import _cache_oracle as ref
from exact_attention_104_b200 import attention_decode_prefix, binding, lib

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _short_waits():
    lib().fa_set_wait_cap(1 << 28)
    yield
    lib().fa_set_wait_cap(0)


def _ok():
    torch.cuda.synchronize()
    assert binding.fa_device_status() == binding.FA_OK


def _lengths(lens):
    return torch.tensor(lens, dtype=torch.int32, device="cuda")


def _inputs(B, Hq, Hkv, Nq, Np, cap, d, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    return (normal(B, Hq, Nq, d), normal(Hkv, Np, d), normal(Hkv, Np, d), normal(B, Hkv, cap, d),
            normal(B, Hkv, cap, d))


def _check(inputs, lens, o, lse, some):
    """Against the definition, for the sequences `some`."""
    q, kp, vp, k, v = inputs
    for b in some:
        n = lens[b]
        r = ref.attention(q[b], torch.cat([kp, k[b, :, :n]], 1), torch.cat([vp, v[b, :, :n]], 1), True,
                          1 / math.sqrt(q.shape[-1]))
        ref.check_o_lse(o[b], lse[b], r, kp.shape[1] + n, (b, n))


# (B, Hq, Hkv, Nq, Np, cap, d): one row tile; in step; a unit a CTA; units of one tile; more units than CTAs
SHAPES = [
    (6, 8, 2, 1, 900, 150, 128),
    (5, 8, 2, 1, 1, 40, 64),
    (40, 16, 2, 1, 2100, 70, 128),
    (24, 16, 8, 5, 1300, 90, 256),
    (200, 32, 8, 1, 700, 60, 64),
    (240, 64, 8, 1, 128, 500, 128),
    (160, 64, 8, 1, 1500, 30, 128),
    (600, 16, 8, 2, 130, 17, 64),
]


@pytest.mark.parametrize("c", SHAPES, ids=lambda c: "b{}_hq{}_hkv{}_nq{}_np{}_cap{}_d{}".format(*c))
def test_side_by_side_matches_definition(c):
    B, cap = c[0], c[5]
    n_ctas, _ = binding.fa_selftest_cache_share(*c)
    assert n_ctas > 0
    inputs = _inputs(*c)
    lens = [(7 * b) % (cap + 1) for b in range(B)]
    lens[-1] = cap
    o, lse = attention_decode_prefix(*inputs, _lengths(lens), causal=True)
    _ok()
    _check(inputs, lens, o, lse, sorted({0, 1, 2, B // 3, B // 2, B - 2, B - 1}))


@pytest.mark.parametrize("c", [SHAPES[0], SHAPES[2], SHAPES[3], SHAPES[5]],
                         ids=lambda c: "b{}_hq{}_hkv{}_nq{}_np{}_cap{}_d{}".format(*c))
def test_side_by_side_captured_and_replayed_with_other_lengths(c):
    B, cap = c[0], c[5]
    inputs, lens = _inputs(*c), _lengths([cap] * B)
    g = torch.Generator("cuda").manual_seed(3)
    call = lambda: attention_decode_prefix(*inputs, lens, causal=True)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        first = call()
        second = call()  # behind it, in a workspace that the first may have used
    for ns in ([cap] * B, [0] * B, [(11 * b) % (cap + 1) for b in range(B)]):
        lens.copy_(torch.tensor(ns))
        inputs[0].normal_(generator=g)
        graph.replay()
        graph.replay()  # at once behind the first: its kernels overwrite what that one's read
        got = [t.clone() for t in (*first, *second)]
        want = call()
        _ok()
        for x, y in zip(got, (*want, *want)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        _check(inputs, ns, *want, (0, B // 2, B - 1))


def test_side_by_side_on_two_streams_at_once():
    sets = [(_inputs(*c, seed=i), _lengths([(5 * b) % (c[5] + 1) for b in range(c[0])]))
            for i, c in enumerate((SHAPES[2], SHAPES[3]))]
    want = [attention_decode_prefix(*x, n, causal=True) for x, n in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(20):
        for i, (x, n) in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                got[i].append(attention_decode_prefix(*x, n, causal=True))
    _ok()
    for w, outs in zip(want, got):
        for o in outs:
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(w, o))
