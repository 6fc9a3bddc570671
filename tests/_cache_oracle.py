"""Plain fp64 definitions of the cache operators, and bounds of what fp32
arithmetic on bf16 inputs may differ from them.

Bounds.  A score is a sum of d products, exact in fp32, added in fp32: each of
its d additions is off by one step at most (2^-23 of the partial sum, cut or
rounded), so by delta = d 2^-23 scale sum|q k|; turning it to log2 units and
subtracting the maximum adds three roundings of 2^-24 |S| each.  An exponential of
a number off by t has the relative error t, and the hardware's 2^x another 2^-22.
Sums of n positive terms in a chain are off by n 2^-24 of themselves; the longest
chain of a row's keys is ceil(keys / 16) in a lane, plus the merges (64 is more
than there are)."""

import math

import torch

U24 = 2.0 ** -24


def lens_of(lengths, B, cap):
    return [cap] * B if lengths is None else [int(x) for x in lengths.cpu()]


def last_visible(n, Nq, causal):
    """Index of the last key each of Nq rows sees out of n (-1: none)."""
    i = torch.arange(Nq)
    return (n - Nq + i).clamp(min=-1) if causal else torch.full((Nq,), n - 1)


def attention(q, keys, values, causal, scale):
    """One sequence: q [Hq, Nq, d], keys, values [Hkv, n, d].  Returns o, lse, p
    [Hq, Nq, n], sum p|v| and the bound on a score's error (all fp64)."""
    Hq, Nq, d = q.shape
    Hkv, n, _ = keys.shape
    G = Hq // Hkv
    q, keys = q.double(), keys.double().repeat_interleave(G, 0)
    last = last_visible(n, Nq, causal).to(q.device)
    seen = torch.arange(n, device=q.device)[None] <= last[:, None]
    s = (scale * (q @ keys.transpose(1, 2))).masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1) if n else torch.full((Hq, Nq), -math.inf, dtype=torch.float64, device=q.device)
    p = torch.exp(s - lse[..., None]).nan_to_num(0.0)
    mag = scale * (q.abs() @ keys.abs().transpose(1, 2))
    top = (mag * seen).amax(-1) if n else torch.zeros(Hq, Nq, dtype=torch.float64, device=q.device)
    smax = s.abs().nan_to_num(0.0, posinf=0.0).amax(-1) if n else top
    tol_s = d * 2 * U24 * top + 3 * U24 * smax
    if values is None:
        return None, lse, p, None, tol_s
    v = values.double().repeat_interleave(G, 0)
    return p @ v, lse, p, p @ v.abs(), tol_s


def sum_tol(n):
    return (-(-n // 16) + 64) * U24 + 2.0 ** -22


def check_o_lse(o, lse, ref, n, where):
    """o, lse of one sequence against attention()'s result over its n keys.  P
    enters the second product as two bf16 parts (2^-16 off)."""
    o_ref, lse_ref, _, absv, tol_s = ref
    rel = 2 * tol_s + 2 * sum_tol(n) + 2.0 ** -16
    tol = o_ref.abs() * 2.0 ** -8 + rel[..., None] * absv + 1e-30
    bad = (o.double() - o_ref).abs() > tol
    assert not bad.any(), (where, "O", ((o.double() - o_ref).abs() / tol).max().item())
    empty = lse_ref == -math.inf
    assert torch.equal(lse == -math.inf, empty), (where, "empty rows")
    tol = tol_s + sum_tol(n) + 2 * U24 * lse_ref.abs().masked_fill(empty, 0.0)
    err = (lse.double() - lse_ref).masked_fill(empty, 0.0).abs()
    assert not (err > tol).any(), (where, "LSE", (err / tol).max().item())


def weight_sum(p, tol_s, lse_tol, Hkv):
    """Sum of the weights over the rows of each kv head's group, and its bound:
    each weight is off by the score's, the LSE's and the exponential's error;
    the chain is the rows."""
    Hq, Nq, n = p.shape
    rel = tol_s + lse_tol + 2.0 ** -22 + (Hq // Hkv * Nq + 2) * U24
    group = lambda x: x.reshape(Hkv, Hq // Hkv * Nq, n).sum(1)  # noqa: E731
    return group(p), group(p * rel[..., None])


def check_weights(got, before, ref, n, lse_known, where):
    """got, before: [Hkv, cap] of one sequence; what lies at or behind n must
    be what it was, bit for bit."""
    _, lse, p, _, tol_s = ref
    assert torch.equal(got[:, n:].view(torch.int32), before[:, n:].view(torch.int32)), (where, "behind the end")
    finite = lse.masked_fill(lse == -math.inf, 0.0).abs()
    # lse known: its product with log2 e and the subtraction round twice; else it is computed as in check_o_lse
    lse_tol = 3 * U24 * finite + (0.0 if lse_known else tol_s + sum_tol(n))
    add, tol = weight_sum(p, tol_s, lse_tol, got.shape[0])
    want = before[:, :n].double() + add
    tol = tol + U24 * want.abs() + 1e-30
    err = (got[:, :n].double() - want).abs()
    assert not (err > tol).any(), (where, "weights", (err / tol).max().item())


def evict(weights, n, budget, recent):
    """Kept slots of one sequence and kv head, in order; weights: list."""
    if n <= budget:
        return list(range(n))
    rank = [-math.inf if math.isnan(x) else x for x in weights[:n - recent]]
    nan = [math.isnan(x) for x in weights[:n - recent]]
    best = sorted(range(n - recent), key=lambda j: (nan[j], -rank[j], j))[:budget - recent]
    return sorted(best) + list(range(n - recent, n))
