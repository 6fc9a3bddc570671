"""Run a few attention calls on one synthetic shape, for a profiler to capture.

    python -m exact_attention_104_b200.profile_run fwd B H N d causal qk_std [calls]
    python -m exact_attention_104_b200.profile_run bwd B H N d causal qk_std [calls]
    python -m exact_attention_104_b200.profile_run prefix B Hq Hkv Nq Np Ncap d [calls]
    python -m exact_attention_104_b200.profile_run decode_weights B Hq Hkv Nq Nk d [calls]
    python -m exact_attention_104_b200.profile_run key_weights B Hq Hkv Nq Nk d [calls]
    python -m exact_attention_104_b200.profile_run evict B Hkv Nk budget recent d [calls]

``fwd`` runs ``calls`` forward calls (default 4); ``bwd`` runs one forward and
``calls`` backward calls (default 3).  Inputs are the seeded standard-normal
tensors of ``workloads.make_inputs`` (Q and K times qk_std), one kv head per
query head.  The cache operators run ``calls`` causal calls (default 3) on full
caches of seeded standard-normal tensors.  Exits non-zero if a call or the device
status reports an error.
"""

import sys

import torch

from . import binding
from .workloads import Workload, make_inputs

CACHE_ARGS = {"prefix": 7, "decode_weights": 6, "key_weights": 6, "evict": 6}


def run_cache(kind, a, calls):
    g = torch.Generator("cuda").manual_seed(777)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    if kind == "evict":
        B, Hkv, Nk, budget, recent, d = a
        k, v, w = normal(B, Hkv, Nk, d), normal(B, Hkv, Nk, d), normal(B, Hkv, Nk, dtype=torch.float32).exp()
        call = lambda: binding.cache_evict(k, v, w, budget, recent)  # noqa: E731
    elif kind == "prefix":
        B, Hq, Hkv, Nq, Np, Ncap, d = a
        q, kp, vp = normal(B, Hq, Nq, d), normal(Hkv, Np, d), normal(Hkv, Np, d)
        k, v = normal(B, Hkv, Ncap, d), normal(B, Hkv, Ncap, d)
        call = lambda: binding.attention_decode_prefix(q, kp, vp, k, v, causal=True)  # noqa: E731
    else:
        B, Hq, Hkv, Nq, Nk, d = a
        q, k = normal(B, Hq, Nq, d), normal(B, Hkv, Nk, d)
        if kind == "decode_weights":
            v = normal(B, Hkv, Nk, d)
            call = lambda: binding.attention_decode_weights(q, k, v, causal=True)  # noqa: E731
        else:
            lse = torch.full((B, Hq, Nq), 8.0, device="cuda")  # of the size that a few thousand keys give
            call = lambda: binding.attention_key_weights(q, k, lse, causal=True)  # noqa: E731
    for _ in range(calls):
        call()


def main(argv):
    kind = argv[0] if argv else ""
    if kind in CACHE_ARGS:
        n = CACHE_ARGS[kind]
        if len(argv) < 1 + n:
            print(__doc__)
            return 2
        run_cache(kind, [int(x) for x in argv[1:1 + n]], int(argv[1 + n]) if len(argv) > 1 + n else 3)
    else:
        if kind not in ("fwd", "bwd") or len(argv) < 7:
            print(__doc__)
            return 2
        B, H, N, d = (int(x) for x in argv[1:5])
        causal = argv[5] in ("1", "true", "True")
        qk_std = float(argv[6])
        calls = int(argv[7]) if len(argv) > 7 else (4 if kind == "fwd" else 3)
        w = Workload("profile", B, H, H, N, d, causal, qk_std, 777)
        q, k, v, do = make_inputs(w, "cuda")
        if kind == "fwd":
            for _ in range(calls):
                binding.attention_forward(q, k, v, causal=causal, scale=w.scale)
        else:
            o, lse = binding.attention_forward(q, k, v, causal=causal, scale=w.scale)
            for _ in range(calls):
                binding.attention_backward(q, k, v, o, lse, do, causal=causal, scale=w.scale)
    torch.cuda.synchronize()
    status = binding.fa_device_status()
    if status != binding.FA_OK:
        print("device status", status)
        return 1
    print("ok")
    return 0


if __name__ == "__main__":
    sys.exit(main(sys.argv[1:]))
