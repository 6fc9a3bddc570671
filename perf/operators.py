"""Cases and plain forms of the operators for serving from a bounded key/value cache.

Four operators, each through the package's Python entry point:

prefix          attention_decode_prefix: decoding for a batch that shares a long prefix
decode_weights  attention_decode_weights: decoding that adds up the attention weight of every key
key_weights     attention_key_weights: the same weights for a prompt, or for its last queries
evict           cache_evict: the cache cut down to the recent keys and those of greatest weight

``run`` computes the plain form, or with ``own`` set makes the package's call.
Every sequence b has ``lengths[b]`` keys in a cache with room for more; what the
cache holds behind them is left over from earlier use.  The Nq query rows of a
head are the last Nq positions of the sequence.
"""

import math

import torch

own = False

DTYPE = torch.bfloat16


# ------------------------------------------------------------------ cases
def listed():
    return [
        # four short chats behind one system prompt, small heads: latency
        dict(name="prefix_small_b4_np500_d64", op="prefix", B=4, Hq=8, Hkv=2, Nq=1, Np=500, cap=64, low=1, d=64,
             causal=True),
        # a serving batch behind a long system prompt, one token a step
        dict(name="prefix_batch_b32_np8192_d128", op="prefix", B=32, Hq=32, Hkv=8, Nq=1, Np=8192, cap=1024, low=64,
             d=128, causal=True),
        # five drafted tokens a sequence over a shared document of odd length, wide heads
        dict(name="prefix_draft_b24_nq5_np20001_d256", op="prefix", B=24, Hq=16, Hkv=8, Nq=5, Np=20001, cap=1500,
             low=700, d=256, causal=True),
        # one sequence, one token, short cache: latency
        dict(name="decode_weights_small_n700_d64", op="decode_weights", B=1, Hq=8, Hkv=2, Nq=1, cap=700, low=700, d=64,
             causal=True),
        # one decoding step of eight sequences with full 32k-token caches
        dict(name="decode_weights_long_b8_n32768_d128", op="decode_weights", B=8, Hq=32, Hkv=8, Nq=1, cap=32768,
             low=32768, d=128, causal=True),
        # eight drafted tokens a sequence, ragged caches of odd lengths
        dict(name="decode_weights_draft_b4_nq8_n10007_d128", op="decode_weights", B=4, Hq=16, Hkv=2, Nq=8, cap=10007,
             low=3001, d=128, causal=True),
        # the last 64 queries of four prompts weigh the keys of the whole prompt
        dict(name="key_weights_window_b4_nq64_n16384_d128", op="key_weights", B=4, Hq=32, Hkv=8, Nq=64, cap=16384,
             low=9000, d=128, causal=True),
        # every query of short prompts, no multiple of the tile, small heads
        dict(name="key_weights_prompt_b2_n2001_d64", op="key_weights", B=2, Hq=16, Hkv=16, Nq=2001, cap=2001, low=2001,
             d=64, causal=True),
        # every query of one long prompt
        dict(name="key_weights_prompt_b1_n8192_d128", op="key_weights", B=1, Hq=16, Hkv=4, Nq=8192, cap=8192, low=8192,
             d=128, causal=True),
        # one short cache cut to a quarter: latency
        dict(name="evict_small_n1000_d64", op="evict", B=1, Hkv=2, cap=1000, low=1000, d=64, budget=256, recent=32),
        # a batch of ragged caches, some within the budget already
        dict(name="evict_batch_b16_n8192_d128", op="evict", B=16, Hkv=8, cap=8192, low=1500, d=128, budget=2048,
             recent=256),
        # long caches cut to an eighth
        dict(name="evict_long_b4_n65536_d128", op="evict", B=4, Hkv=8, cap=65536, low=60001, d=128, budget=8192,
             recent=1024),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges: sizes spread over their logarithm, no
    more bytes or operations than the costliest listed case of its operator."""
    op = rng.choice(["prefix", "decode_weights", "key_weights", "evict"])
    peers = [c for c in listed() if c["op"] == op]
    most = {key: max(work(c)[key] for c in peers) for key in ("bytes", "flops")}
    while True:
        d = rng.choice([64, 128, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        c = dict(op=op, B=_log_int(rng, 1, 32), Hkv=Hkv, d=d)
        if op == "evict":
            c["cap"] = _log_int(rng, 1000, 65536)
            c["budget"] = _log_int(rng, 128, max(129, c["cap"] // 2))
            c["recent"] = rng.randint(0, c["budget"] // 2)
        else:
            c["Hq"] = Hkv * rng.choice([1, 2, 4, 8])
            c["causal"] = rng.random() < 0.75
            if op == "key_weights":
                c["cap"] = _log_int(rng, 1000, 16384)
                c["Nq"] = c["cap"] if rng.random() < 0.5 and c["cap"] <= 8192 else _log_int(rng, 16, 256)
            else:
                c["Nq"] = 1 if rng.random() < 0.6 else rng.randint(2, 8)
                c["cap"] = _log_int(rng, 64, 1500) if op == "prefix" else _log_int(rng, 700, 32768)
                if op == "prefix":
                    c["Np"] = _log_int(rng, 500, 20001)
        prompt = op == "key_weights" and c["Nq"] == c["cap"]
        c["low"] = c["cap"] if prompt else rng.randint(max(1, c.get("Nq", 1), c["cap"] // 8), c["cap"])
        w = work(c)
        # the plain form's score matrix stays within that of the largest listed prompt
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"] and _pairs_stored(c) <= 16 * 8192 * 8192:
            return c


def _lengths(c):
    """The sequences' lengths: spread evenly over low .. cap, not in order."""
    B, low, cap = c["B"], c["low"], c["cap"]
    if B == 1:
        return [cap]
    step = next(s for s in (7, 5, 11, 13, 17, 3, 1) if math.gcd(s, B) == 1)
    return [low + ((b * step) % B) * (cap - low) // (B - 1) for b in range(B)]


def _pairs_stored(c):
    return c["B"] * c.get("Hq", 0) * c.get("Nq", 0) * (c["cap"] + c.get("Np", 0))


def work(c):
    lens, d, Hkv = _lengths(c), c["d"], c["Hkv"]
    if c["op"] == "evict":
        kept = sum(min(n, c["budget"]) for n in lens)
        # weights of all keys; kept rows in and out; kept weights and indices out
        return dict(bytes=Hkv * (4 * sum(lens) + kept * (8 * d + 8)), flops=Hkv * sum(lens))
    B, Hq, Nq, Np = c["B"], c["Hq"], c["Nq"], c.get("Np", 0)
    seen = 0
    for n in lens:
        total = Np + n
        seen += sum(max(0, min(total, total - Nq + i + 1)) for i in range(Nq)) if c["causal"] else total * Nq
    rows, keys = B * Hq * Nq, sum(lens)
    if c["op"] == "prefix":
        return dict(bytes=4 * Hkv * d * (Np + keys) + rows * (4 * d + 4), flops=4 * d * Hq * seen)
    if c["op"] == "decode_weights":
        return dict(bytes=Hkv * keys * (4 * d + 8) + rows * (4 * d + 4), flops=4 * d * Hq * seen)
    return dict(bytes=Hkv * keys * (2 * d + 8) + rows * (2 * d + 4), flops=2 * d * Hq * seen)


# ----------------------------------------------------------------- inputs
def _logsumexp_rows(q, k, lens, scale, causal):
    """fp32 log-sum-exp of every row's visible scores, one head at a time."""
    B, Hq, Nq, _ = q.shape
    Hkv, cap = k.shape[1], k.shape[2]
    out = torch.empty(B, Hq, Nq, device=q.device)
    for b in range(B):
        seen = _visible(lens[b:b + 1], Nq, cap, causal)[0]
        for h in range(Hq):
            s = (q[b, h].float() @ k[b, h * Hkv // Hq].float().T) * scale
            out[b, h] = torch.logsumexp(s.masked_fill_(~seen, -math.inf), dim=-1)
    return out


def prepare(c, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    lens = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")
    B, Hkv, cap, d = c["B"], c["Hkv"], c["cap"], c["d"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(DTYPE)

    def weights():
        # sums of attention weights: a few keys hold most of it, some hold nothing yet
        w = torch.randn(B, Hkv, cap, generator=g, device="cuda").mul_(2.0).exp_()
        return w.masked_fill_(torch.rand(B, Hkv, cap, generator=g, device="cuda") < 0.05, 0.0)

    st = dict(c, lengths=lens, k=normal(B, Hkv, cap, d))
    if c["op"] == "evict":
        return dict(st, v=normal(B, Hkv, cap, d), weights=weights())
    st.update(q=normal(B, c["Hq"], c["Nq"], d), scale=1.0 / math.sqrt(d))
    if c["op"] == "prefix":
        return dict(st, v=normal(B, Hkv, cap, d), k_prefix=normal(Hkv, c["Np"], d), v_prefix=normal(Hkv, c["Np"], d))
    st["weights"] = weights()
    if c["op"] == "decode_weights":
        st["v"] = normal(B, Hkv, cap, d)
    else:
        st["lse"] = _logsumexp_rows(st["q"], st["k"], lens, st["scale"], c["causal"])
    return st


# ------------------------------------------------------------ plain forms
def _visible(lens, Nq, cap, causal, Np=0):
    """[B, Nq, Np + cap] truth values: the keys that each query row sees."""
    key = torch.arange(Np + cap, device=lens.device)
    total = lens.long()[:, None, None] + Np
    seen = (key < total).expand(-1, Nq, -1)
    if causal:
        seen = seen & (key <= total - Nq + torch.arange(Nq, device=lens.device)[:, None])
    return seen


def _softmax_rows(s):
    """Weights and log-sum-exp of the rows of s; a row of -inf has weights 0."""
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, torch.ones_like(total))
    return p, (top + torch.log(total)).squeeze(-1)


def _grouped(q, Hkv):
    """[B, Hq, Nq, d] in 32 bits as [B, Hkv, G*Nq, d]."""
    B, Hq, Nq, d = q.shape
    return q.float().reshape(B, Hkv, Hq // Hkv * Nq, d)


def _rows_mask(seen, G):
    """[B, Nq, keys] as [B, 1, G*Nq, keys]: row g*Nq + i is query i."""
    return seen.repeat(1, G, 1)[:, None]


def _plain_prefix(st):
    q, lens, Np, cap, Hkv = st["q"], st["lengths"], st["Np"], st["cap"], st["Hkv"]
    seen = _rows_mask(_visible(lens, st["Nq"], cap, st["causal"], Np), st["Hq"] // Hkv)
    qg = _grouped(q, Hkv)
    own_keys = (torch.arange(cap, device=q.device) < lens[:, None])[:, None, :, None]
    s = torch.cat([qg @ st["k_prefix"].float().transpose(-1, -2), qg @ st["k"].float().transpose(-1, -2)], -1)
    p, lse = _softmax_rows((s * st["scale"]).masked_fill(~seen, -math.inf))
    o = p[..., :Np] @ st["v_prefix"].float() + p[..., Np:] @ st["v"].float().masked_fill(~own_keys, 0.0)
    return o.reshape(q.shape).to(DTYPE), lse.reshape(q.shape[:-1])


def _plain_decode_weights(st):
    q, lens, cap, Hkv = st["q"], st["lengths"], st["cap"], st["Hkv"]
    seen = _rows_mask(_visible(lens, st["Nq"], cap, st["causal"]), st["Hq"] // Hkv)
    own_keys = (torch.arange(cap, device=q.device) < lens[:, None])[:, None, :, None]
    s = _grouped(q, Hkv) @ st["k"].float().transpose(-1, -2) * st["scale"]
    p, lse = _softmax_rows(s.masked_fill(~seen, -math.inf))
    o = p @ st["v"].float().masked_fill(~own_keys, 0.0)
    return o.reshape(q.shape).to(DTYPE), lse.reshape(q.shape[:-1]), st["weights"] + p.sum(-2)


def _plain_key_weights(st):
    q, Hkv = st["q"], st["Hkv"]
    seen = _rows_mask(_visible(st["lengths"], st["Nq"], st["cap"], st["causal"]), st["Hq"] // Hkv)
    qg = _grouped(q, Hkv)
    s = qg @ st["k"].float().transpose(-1, -2) * st["scale"]
    p = torch.exp(s - st["lse"].reshape(qg.shape[:-1])[..., None]).masked_fill(~seen, 0.0)
    return st["weights"] + p.sum(-2)


def _plain_evict(st):
    w, lens, budget, recent = st["weights"], st["lengths"].long()[:, None, None], st["budget"], st["recent"]
    cap, d = st["cap"], st["d"]
    slot = torch.arange(cap, device=w.device)
    # order of keeping: the recent keys, then the others by weight, then what is no key
    rank = w.masked_fill(slot >= lens - recent, math.inf).masked_fill(slot >= lens, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    count = lens.clamp(max=budget)
    first = torch.arange(min(budget, cap), device=w.device) < count
    kept = torch.sort(order[..., :budget].masked_fill(~first, cap), dim=-1).values
    src = kept.clamp(max=cap - 1)
    rows = src[..., None].expand(-1, -1, -1, d)
    first = first.expand_as(kept)
    k = torch.gather(st["k"], 2, rows).masked_fill(~first[..., None], 0.0)
    v = torch.gather(st["v"], 2, rows).masked_fill(~first[..., None], 0.0)
    w = torch.gather(w, 2, src).masked_fill(~first, 0.0)
    return k, v, w, kept.masked_fill(~first, -1).int(), count[:, 0, 0].int()


_PLAIN = dict(prefix=_plain_prefix, decode_weights=_plain_decode_weights, key_weights=_plain_key_weights,
              evict=_plain_evict)


def _own_run(st):
    import exact_attention_104_b200 as fa

    if st["op"] == "prefix":
        return fa.attention_decode_prefix(st["q"], st["k_prefix"], st["v_prefix"], st["k"], st["v"], st["lengths"],
                                          causal=st["causal"])
    if st["op"] == "decode_weights":
        return fa.attention_decode_weights(st["q"], st["k"], st["v"], st["weights"], st["lengths"],
                                           causal=st["causal"])
    if st["op"] == "key_weights":
        return fa.attention_key_weights(st["q"], st["k"], st["lse"], st["weights"], st["lengths"],
                                        causal=st["causal"])
    return fa.cache_evict(st["k"], st["v"], st["weights"], st["budget"], st["recent"], st["lengths"])


def run(state):
    if own:
        return _own_run(state)
    return _PLAIN[state["op"]](state)


# ------------------------------------------------- definition in 64 bits
def _exact_rows(q, keys, values, last, scale):
    """O and LSE of rows q [n, d] that see the keys 0 .. last[row], in 64 bits."""
    s = scale * torch.einsum("nd,kd->nk", q, keys)
    s[torch.arange(keys.shape[0], device=q.device)[None] > last[:, None]] = -math.inf
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[:, None]).nan_to_num_(0.0)
    return None if values is None else p @ values, lse, p


def _exact_attention(st):
    q, lens = st["q"].double(), st["lengths"].tolist()
    B, Hq, Nq, d = q.shape
    Hkv, Np = st["Hkv"], st.get("Np", 0)
    G = Hq // Hkv
    o, lse = torch.zeros_like(q), torch.zeros(B, Hq, Nq, dtype=torch.float64, device=q.device)
    w = st["weights"].double().clone() if "weights" in st else None
    for b in range(B):
        n = Np + lens[b]
        last = torch.full((Nq,), n - 1, device=q.device)
        if st["causal"]:
            last = n - Nq + torch.arange(Nq, device=q.device)
        for g in range(Hkv):
            keys, values = st["k"][b, g, :lens[b]].double(), st["v"][b, g, :lens[b]].double()
            if Np:
                keys = torch.cat([st["k_prefix"][g].double(), keys])
                values = torch.cat([st["v_prefix"][g].double(), values])
            heads = slice(g * G, (g + 1) * G)
            oo, ll, p = _exact_rows(q[b, heads].reshape(G * Nq, d), keys, values, last.repeat(G), st["scale"])
            o[b, heads], lse[b, heads] = oo.reshape(G, Nq, d), ll.reshape(G, Nq)
            if w is not None:
                w[b, g, :lens[b]] += p.sum(0)
    return (o, lse) if w is None else (o, lse, w)


def _exact_key_weights(st):
    q, lens = st["q"].double(), st["lengths"].tolist()
    B, Hq, Nq, d = q.shape
    G = Hq // st["Hkv"]
    w = st["weights"].double().clone()
    for b in range(B):
        n = lens[b]
        for h in range(Hq):
            s = st["scale"] * torch.einsum("id,jd->ij", q[b, h], st["k"][b, h // G, :n].double())
            p = torch.exp(s - st["lse"][b, h].double()[:, None])
            if st["causal"]:
                p = p.tril(n - Nq)
            w[b, h // G, :n] += p.sum(0)
    return w


def _exact_evict(st):
    k, v, w = st["k"].double(), st["v"].double(), st["weights"].double()
    B, Hkv, cap, d = k.shape
    size = min(st["budget"], cap)
    ko, vo = torch.zeros(B, Hkv, size, d).to(k), torch.zeros(B, Hkv, size, d).to(k)
    wo, index = torch.zeros(B, Hkv, size).to(k), torch.full((B, Hkv, size), -1, dtype=torch.int32, device=k.device)
    counts = []
    for b, n in enumerate(st["lengths"].tolist()):
        count = min(n, st["budget"])
        counts.append(count)
        for h in range(Hkv):
            recent = min(st["recent"], n) if n > st["budget"] else n
            values = w[b, h, :n - recent].tolist()
            best = sorted(range(n - recent), key=lambda j: (-values[j], j))[:count - recent]
            chosen = torch.tensor(sorted(best) + list(range(n - recent, n)), dtype=torch.long, device=k.device)
            ko[b, h, :count], vo[b, h, :count] = k[b, h, chosen], v[b, h, chosen]
            wo[b, h, :count], index[b, h, :count] = w[b, h, chosen], chosen.int()
    return ko, vo, wo, index, torch.tensor(counts, dtype=torch.int32, device=k.device)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(st)
    if case["op"] == "key_weights":
        return _exact_key_weights(st)
    return _exact_attention(st)
