"""ctypes binding for libfa_b200.so (argument marshalling only).

Every function here forwards to the C ABI declared in ``include/fa.h``; all
arithmetic runs in the library's CUDA kernels.  There is no fallback: if the
library is missing or the device is unsupported, calls raise ``FAError``.
"""

from __future__ import annotations

import ctypes
import functools
import math
import os

import torch

# FA_B200_DEBUG=1 selects the debug build (device-side checks, -DFA_DEBUG)
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)),
                        "libfa_b200_debug.so" if os.environ.get("FA_B200_DEBUG") == "1" else "libfa_b200.so")

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT, FA_ERR_DEVICE_CHECK = range(6)

_lib = None


class FAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {fa_status_string(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """Load the shared library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise FAError(FA_ERR_UNSUPPORTED, f"{LIB_PATH} is missing; build it with "
                      "`python -m exact_attention_104_b200.build`"
                      + (" --debug" if LIB_PATH.endswith("_debug.so") else ""))
    L = ctypes.CDLL(LIB_PATH)
    vp, i, f, z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, vp]
    L.fa_fwd.restype = i
    L.fa_fwd_pair.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, vp]
    L.fa_fwd_pair.restype = i
    L.fa_bwd_workspace_bytes.argtypes = [i, i, i, i, i]
    L.fa_bwd_workspace_bytes.restype = z
    L.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, vp, z, vp]
    L.fa_bwd.restype = i
    L.fa_device_status.argtypes = [vp]
    L.fa_device_status.restype = i
    L.fa_status_string.argtypes = [i]
    L.fa_status_string.restype = ctypes.c_char_p
    L.fa_set_wait_cap.argtypes = [ctypes.c_longlong]
    L.fa_set_wait_cap.restype = i
    L.fa_profile_next.argtypes = [vp, vp]
    L.fa_profile_next.restype = i
    L.fa_selftest_wait_timeout.argtypes = [ctypes.c_longlong, vp]
    L.fa_selftest_wait_timeout.restype = i
    L.fa_selftest_exp2.argtypes = [vp, vp, ctypes.c_longlong, i, vp]
    L.fa_selftest_exp2.restype = i
    L.fa_selftest_cache_share.argtypes = [i, i, i, i, i, i, i, ctypes.POINTER(i)]
    L.fa_selftest_cache_share.restype = i
    L.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, f, vp]
    L.fa_bwd_noalloc.restype = i
    L.fa_decode_workspace_bytes.argtypes = [i, i, i, i, i, i]
    L.fa_decode_workspace_bytes.restype = z
    L.fa_fwd_decode.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp, z, vp]
    L.fa_fwd_decode.restype = i
    L.fa_fwd_varlen_workspace_bytes.argtypes = [i, i, i, i, i, i]
    L.fa_fwd_varlen_workspace_bytes.restype = z
    L.fa_bwd_varlen_workspace_bytes.argtypes = [i, i, i, i, i, i]
    L.fa_bwd_varlen_workspace_bytes.restype = z
    L.fa_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp, z, vp]
    L.fa_fwd_varlen.restype = i
    L.fa_bwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp, z, vp]
    L.fa_bwd_varlen.restype = i
    L.fa_decode_prefix_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
    L.fa_decode_prefix_workspace_bytes.restype = z
    L.fa_fwd_decode_prefix.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, vp, z, vp]
    L.fa_fwd_decode_prefix.restype = i
    L.fa_decode_weights_workspace_bytes.argtypes = [i, i, i, i, i, i]
    L.fa_decode_weights_workspace_bytes.restype = z
    L.fa_fwd_decode_weights.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp, z, vp]
    L.fa_fwd_decode_weights.restype = i
    L.fa_key_weights_workspace_bytes.argtypes = [i, i, i, i, i, i]
    L.fa_key_weights_workspace_bytes.restype = z
    L.fa_key_weights.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp, z, vp]
    L.fa_key_weights.restype = i
    L.fa_cache_evict.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp]
    L.fa_cache_evict.restype = i
    _lib = L
    return L


def fa_status_string(status: int) -> str:
    try:
        return lib().fa_status_string(int(status)).decode()
    except FAError:
        return {0: "ok", 1: "invalid argument", 2: "unsupported configuration", 3: "CUDA error",
                4: "device wait timed out"}.get(int(status), "unknown status")


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, torch.Tensor):
        return x.data_ptr()
    return int(x)


def _stream_handle(stream) -> int | None:
    if stream is None:
        # the handle of torch.cuda.current_stream(), without building the object
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status: int, where: str):
    if status != FA_OK:
        raise FAError(status, where)


def fa_fwd(q, k, v, o, lse, B, Hq, Hkv, N, d, causal, scale, stream=None) -> int:
    """Raw C-ABI call; tensors or integer device pointers.  Returns the status."""
    return lib().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, N, d,
                        int(bool(causal)), float(scale), _stream_handle(stream))


def fa_fwd_pair(q, k, v, o, lse, B, Hq, Hkv, N, d, causal, scale, stream=None) -> int:
    """Raw C-ABI call of the forward pass on CTA pairs (d = 128).  Returns the
    status."""
    return lib().fa_fwd_pair(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, N, d,
                             int(bool(causal)), float(scale), _stream_handle(stream))


def fa_bwd_workspace_bytes(B, Hq, Hkv, N, d) -> int:
    return int(lib().fa_bwd_workspace_bytes(B, Hq, Hkv, N, d))


def fa_bwd(q, k, v, o, lse, do, dq, dk, dv, B, Hq, Hkv, N, d, causal, scale, workspace, workspace_bytes,
           stream=None) -> int:
    """Raw C-ABI call; tensors or integer device pointers.  Returns the status."""
    return lib().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv),
                        B, Hq, Hkv, N, d, int(bool(causal)), float(scale), _ptr(workspace),
                        int(workspace_bytes), _stream_handle(stream))


def fa_selftest_wait_timeout(cap_cycles: int, stream=None) -> int:
    return lib().fa_selftest_wait_timeout(int(cap_cycles), _stream_handle(stream))


def fa_selftest_cache_share(B, Hq, Hkv, Nq, Np, Ncap, d) -> tuple[int, int]:
    """SMs that decoding behind a prefix gives to the prefix, and CTAs of each of
    its units in step (see fa.h); no GPU is needed."""
    share = (ctypes.c_int * 2)()
    _check(lib().fa_selftest_cache_share(B, Hq, Hkv, Nq, Np, Ncap, d, share), "fa_selftest_cache_share")
    return share[0], share[1]


def fa_selftest_exp2(x, y, use_poly: bool, stream=None) -> int:
    return lib().fa_selftest_exp2(_ptr(x), _ptr(y), int(x.numel()), int(bool(use_poly)), _stream_handle(stream))


FA_NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024


def fa_bwd_noalloc(q, k, v, o, lse, do, dq, dk, dv, B, Hq, Hkv, N, d, causal, scale, stream=None) -> int:
    """Raw C-ABI call of the backward pass that uses the library's fixed
    device scratch array instead of a caller workspace (for callers that
    cannot allocate device memory).  Returns the status."""
    return lib().fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk),
                                _ptr(dv), B, Hq, Hkv, N, d, int(bool(causal)), float(scale),
                                _stream_handle(stream))


def fa_decode_workspace_bytes(B, Hq, Hkv, Nq, Nk, d) -> int:
    return lib().fa_decode_workspace_bytes(B, Hq, Hkv, Nq, Nk, d)


def fa_fwd_decode(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, d, causal, scale, workspace, workspace_bytes,
                  stream=None) -> int:
    """Raw C-ABI call of the decoding forward pass (Nq queries, the last
    positions of an Nk-long sequence).  Returns the status."""
    return lib().fa_fwd_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, Nk, d,
                               int(bool(causal)), float(scale), _ptr(workspace), int(workspace_bytes),
                               _stream_handle(stream))


def fa_fwd_varlen_workspace_bytes(nseq, Hq, Hkv, T, max_seqlen, d) -> int:
    return int(lib().fa_fwd_varlen_workspace_bytes(nseq, Hq, Hkv, T, max_seqlen, d))


def fa_bwd_varlen_workspace_bytes(nseq, Hq, Hkv, T, max_seqlen, d) -> int:
    return int(lib().fa_bwd_varlen_workspace_bytes(nseq, Hq, Hkv, T, max_seqlen, d))


def fa_fwd_varlen(q, k, v, o, lse, cu_seqlens, nseq, Hq, Hkv, T, max_seqlen, d, causal, scale, workspace,
                  workspace_bytes, stream=None) -> int:
    """Raw C-ABI call of the packed variable-length forward pass (sequences
    back to back along the token axis of [H, T, d] tensors, boundaries in the
    device int32 tensor cu_seqlens).  Returns the status."""
    return lib().fa_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(cu_seqlens), nseq, Hq, Hkv, T,
                               max_seqlen, d, int(bool(causal)), float(scale), _ptr(workspace),
                               int(workspace_bytes), _stream_handle(stream))


def fa_bwd_varlen(q, k, v, o, lse, do, dq, dk, dv, cu_seqlens, nseq, Hq, Hkv, T, max_seqlen, d, causal, scale,
                  workspace, workspace_bytes, stream=None) -> int:
    """Raw C-ABI call of the packed variable-length backward pass.  Returns
    the status."""
    return lib().fa_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk),
                               _ptr(dv), _ptr(cu_seqlens), nseq, Hq, Hkv, T, max_seqlen, d, int(bool(causal)),
                               float(scale), _ptr(workspace), int(workspace_bytes), _stream_handle(stream))


def fa_decode_prefix_workspace_bytes(B, Hq, Hkv, Nq, Np, Ncap, d) -> int:
    return int(lib().fa_decode_prefix_workspace_bytes(B, Hq, Hkv, Nq, Np, Ncap, d))


def fa_fwd_decode_prefix(q, k_prefix, v_prefix, k, v, lengths, o, lse, B, Hq, Hkv, Nq, Np, Ncap, d, causal, scale,
                         workspace, workspace_bytes, stream=None) -> int:
    """Raw C-ABI call of decoding for a batch that shares a prefix.  Returns
    the status."""
    return lib().fa_fwd_decode_prefix(_ptr(q), _ptr(k_prefix), _ptr(v_prefix), _ptr(k), _ptr(v), _ptr(lengths),
                                      _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, Np, Ncap, d, int(bool(causal)),
                                      float(scale), _ptr(workspace), int(workspace_bytes), _stream_handle(stream))


def fa_decode_weights_workspace_bytes(B, Hq, Hkv, Nq, Nk, d) -> int:
    return int(lib().fa_decode_weights_workspace_bytes(B, Hq, Hkv, Nq, Nk, d))


def fa_fwd_decode_weights(q, k, v, lengths, weights, weights_out, o, lse, B, Hq, Hkv, Nq, Nk, d, causal, scale,
                          workspace, workspace_bytes, stream=None) -> int:
    """Raw C-ABI call of decoding that adds up every key's attention weight.
    Returns the status."""
    return lib().fa_fwd_decode_weights(_ptr(q), _ptr(k), _ptr(v), _ptr(lengths), _ptr(weights), _ptr(weights_out),
                                       _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, Nk, d, int(bool(causal)), float(scale),
                                       _ptr(workspace), int(workspace_bytes), _stream_handle(stream))


def fa_key_weights_workspace_bytes(B, Hq, Hkv, Nq, Nk, d) -> int:
    return int(lib().fa_key_weights_workspace_bytes(B, Hq, Hkv, Nq, Nk, d))


def fa_key_weights(q, k, lse, lengths, weights, weights_out, B, Hq, Hkv, Nq, Nk, d, causal, scale, workspace,
                   workspace_bytes, stream=None) -> int:
    """Raw C-ABI call of the keys' attention weights from queries whose LSE is
    known.  Returns the status."""
    return lib().fa_key_weights(_ptr(q), _ptr(k), _ptr(lse), _ptr(lengths), _ptr(weights), _ptr(weights_out), B, Hq,
                                Hkv, Nq, Nk, d, int(bool(causal)), float(scale), _ptr(workspace),
                                int(workspace_bytes), _stream_handle(stream))


def fa_cache_evict(k, v, weights, lengths, k_out, v_out, weights_out, index, lengths_out, B, Hkv, Nk, out_cap, budget,
                   recent, d, stream=None) -> int:
    """Raw C-ABI call of the eviction by accumulated weight.  Returns the
    status."""
    return lib().fa_cache_evict(_ptr(k), _ptr(v), _ptr(weights), _ptr(lengths), _ptr(k_out), _ptr(v_out),
                                _ptr(weights_out), _ptr(index), _ptr(lengths_out), B, Hkv, Nk, out_cap, budget,
                                recent, d, _stream_handle(stream))


def fa_profile_next(start_event=None, stop_event=None) -> int:
    """Ask the next fa_fwd / fa_bwd call on this thread to record the given
    torch.cuda.Event objects around its attention kernel."""
    for ev in (start_event, stop_event):
        if ev is not None and not ev.cuda_event:
            ev.record()  # torch creates the underlying cudaEvent lazily
    s = start_event.cuda_event if start_event is not None else None
    e = stop_event.cuda_event if stop_event is not None else None
    return lib().fa_profile_next(s, e)


def fa_device_status(stream=None) -> int:
    return lib().fa_device_status(_stream_handle(stream))


def _shapes(q, k, v):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, H, N, d]")
    B, Hq, N, d = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[2] != N or k.shape[3] != d:
        raise ValueError(f"incompatible shapes q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)}")
    for t in (q, k, v):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous bf16 CUDA tensors")
    return B, Hq, k.shape[1], N, d


def attention_forward(q, k, v, causal=False, scale=None, out=None, lse=None, stream=None):
    """O, LSE = exact attention of bf16 [B,H,N,d] tensors on the current CUDA
    device (no CPU path).  Returns (o bf16 [B,Hq,N,d], lse fp32 [B,Hq,N])."""
    B, Hq, Hkv, N, d = _shapes(q, k, v)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, Hq, N, dtype=torch.float32, device=q.device)
    _check(fa_fwd(q, k, v, out, lse, B, Hq, Hkv, N, d, causal, scale, stream), "fa_fwd")
    return out, lse


def attention_backward(q, k, v, o, lse, do, causal=False, scale=None, dq=None, dk=None, dv=None,
                       workspace=None, stream=None):
    """dQ, dK, dV of exact attention given the forward outputs and dO."""
    B, Hq, Hkv, N, d = _shapes(q, k, v)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = fa_bwd_workspace_bytes(B, Hq, Hkv, N, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _check(fa_bwd(q, k, v, o, lse, do, dq, dk, dv, B, Hq, Hkv, N, d, causal, scale, workspace,
                  workspace.numel() * workspace.element_size(), stream), "fa_bwd")
    return dq, dk, dv


def attention_decode(q, k, v, causal=False, scale=None, out=None, lse=None, workspace=None, stream=None):
    """O, LSE of Nq queries q [B,Hq,Nq,d] against cached k, v [B,Hkv,Nk,d]; the
    queries are the last Nq positions of the sequence (see fa_fwd_decode)."""
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4 or k.shape != v.shape:
        raise FAError(FA_ERR_INVALID_ARG, "attention_decode: q, k, v must be [B,H,N,d] with k.shape == v.shape")
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if k.shape[0] != B or k.shape[3] != d:
        raise FAError(FA_ERR_INVALID_ARG, "attention_decode: batch or head dimension mismatch")
    for t in (q, k, v):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise FAError(FA_ERR_INVALID_ARG, "attention_decode: inputs must be contiguous bf16 CUDA tensors")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, Hq, Nq, dtype=torch.float32, device=q.device)
    need = fa_decode_workspace_bytes(B, Hq, Hkv, Nq, Nk, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _check(fa_fwd_decode(q, k, v, out, lse, B, Hq, Hkv, Nq, Nk, d, causal, scale, workspace,
                         workspace.numel() * workspace.element_size(), stream), "fa_fwd_decode")
    return out, lse


def _varlen_shapes(q, k, v, cu_seqlens):
    if q.dim() != 3 or k.dim() != 3 or k.shape != v.shape:
        raise FAError(FA_ERR_INVALID_ARG, "varlen: q must be [Hq, T, d] and k, v [Hkv, T, d]")
    Hq, T, d = q.shape
    if k.shape[1] != T or k.shape[2] != d:
        raise FAError(FA_ERR_INVALID_ARG, "varlen: token or head dimension mismatch")
    for t in (q, k, v):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise FAError(FA_ERR_INVALID_ARG, "varlen: q, k, v must be contiguous bf16 CUDA tensors")
    if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda or cu_seqlens.dim() != 1:
        raise FAError(FA_ERR_INVALID_ARG, "varlen: cu_seqlens must be a 1-D int32 CUDA tensor")
    return Hq, k.shape[0], T, d, cu_seqlens.numel() - 1


def attention_forward_varlen(q, k, v, cu_seqlens, max_seqlen, causal=False, scale=None, out=None, lse=None,
                             workspace=None, stream=None):
    """O, LSE of a packed batch: q [Hq, T, d], k, v [Hkv, T, d] bf16 with the
    sequences back to back along T (boundaries in the int32 CUDA tensor
    cu_seqlens); each sequence attends only to itself.  max_seqlen bounds
    every length.  Returns (o bf16 [Hq, T, d], lse fp32 [Hq, T])."""
    Hq, Hkv, T, d, nseq = _varlen_shapes(q, k, v, cu_seqlens)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(Hq, T, dtype=torch.float32, device=q.device)
    need = fa_fwd_varlen_workspace_bytes(nseq, Hq, Hkv, T, max_seqlen, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _check(fa_fwd_varlen(q, k, v, out, lse, cu_seqlens, nseq, Hq, Hkv, T, max_seqlen, d, causal, scale, workspace,
                         workspace.numel() * workspace.element_size(), stream), "fa_fwd_varlen")
    return out, lse


def attention_backward_varlen(q, k, v, o, lse, do, cu_seqlens, max_seqlen, causal=False, scale=None, dq=None,
                              dk=None, dv=None, workspace=None, stream=None):
    """dQ, dK, dV of a packed batch given the forward outputs and dO."""
    Hq, Hkv, T, d, nseq = _varlen_shapes(q, k, v, cu_seqlens)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = fa_bwd_varlen_workspace_bytes(nseq, Hq, Hkv, T, max_seqlen, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _check(fa_bwd_varlen(q, k, v, o, lse, do, dq, dk, dv, cu_seqlens, nseq, Hq, Hkv, T, max_seqlen, d, causal,
                         scale, workspace, workspace.numel() * workspace.element_size(), stream), "fa_bwd_varlen")
    return dq, dk, dv


# ------------------------------------------------------- bounded key/value caches
class _CacheCall:
    """Where one cache call runs: every tensor lies on the device of the first,
    the call runs with that device current, and on ``stream`` (or that device's
    current stream), from whose memory pool the tensors it allocates come.
    ``scope`` is None where that is the state already."""

    __slots__ = ("where", "first", "index", "scope")

    def __init__(self, where, first, stream):
        self.where = where
        self.first = first
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            self.refuse("inputs must be CUDA tensors")
        self.index = first.get_device()
        self.scope = None
        if stream is not None:
            # tensors of a stream given as a handle belong to that stream's pool too
            if not isinstance(stream, torch.cuda.Stream):
                stream = (torch.cuda.ExternalStream(int(stream), device=self.device) if int(stream)
                          else torch.cuda.default_stream(self.device))
            if stream.device != self.device:
                self.refuse("the stream belongs to another device")
            self.scope = torch.cuda.stream(stream)
        elif torch._C._cuda_getDevice() != self.index:
            self.scope = torch.cuda.device(self.device)

    @property
    def device(self):
        return self.first.device

    def refuse(self, why):
        raise FAError(FA_ERR_INVALID_ARG, f"{self.where}: {why}")

    def check(self, name, t, shape, dtype):
        if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == self.index and t.shape == shape
                and t.is_contiguous()):
            return
        if not isinstance(t, torch.Tensor) or t.get_device() != self.index:
            self.refuse(f"{name} must be a tensor on {self.device}")
        self.refuse(f"{name} must be contiguous {dtype} {list(shape)}, got {t.dtype} {list(t.shape)} "
                    f"with strides {list(t.stride())}")

    def scratch(self, t, need):
        """The caller's workspace, or a new one of the size needed."""
        if t is None:
            return self.first.new_empty(max(need, 256), dtype=torch.uint8)
        if not isinstance(t, torch.Tensor) or t.get_device() != self.index or not t.is_contiguous():
            self.refuse(f"workspace must be a contiguous tensor on {self.device}")
        return t

    def dims(self, q, k):
        if q.dim() != 4 or not isinstance(k, torch.Tensor) or k.dim() != 4:
            self.refuse("q and k must be [B, H, N, d]")
        return (*q.shape, k.shape[1], k.shape[2])

    def run(self, body):
        if self.scope is None:
            return body(torch._C._cuda_getCurrentRawStream(self.index))
        with self.scope:
            return body(torch._C._cuda_getCurrentRawStream(self.index))


@functools.lru_cache(maxsize=256)
def _workspace_bytes(name, *sizes):
    """A workspace query, a pure function of the sizes."""
    return getattr(lib(), name)(*sizes)


def attention_decode_prefix(q, k_prefix, v_prefix, k, v, lengths=None, causal=False, scale=None, out=None, lse=None,
                            workspace=None, stream=None):
    """O, LSE of Nq queries q [B,Hq,Nq,d] in a batch that shares a prefix: the
    keys of sequence b are k_prefix [Hkv,Np,d] followed by the first lengths[b]
    rows of k[b] ([B,Hkv,Ncap,d]; lengths None: all of them); the queries are
    its last Nq positions (see fa_fwd_decode_prefix).  Np and Ncap may be 0.
    Returns (o bf16 [B,Hq,Nq,d], lse fp32 [B,Hq,Nq])."""
    call = _CacheCall("attention_decode_prefix", q, stream)
    B, Hq, Nq, d, Hkv, Ncap = call.dims(q, k)
    if not isinstance(k_prefix, torch.Tensor) or k_prefix.dim() != 3:
        call.refuse("k_prefix must be [Hkv, Np, d]")
    Np = k_prefix.shape[1]
    check, own, pre = call.check, (B, Hkv, Ncap, d), (Hkv, Np, d)
    check("q", q, (B, Hq, Nq, d), torch.bfloat16)
    check("k", k, own, torch.bfloat16)
    check("v", v, own, torch.bfloat16)
    check("k_prefix", k_prefix, pre, torch.bfloat16)
    check("v_prefix", v_prefix, pre, torch.bfloat16)
    if lengths is not None:
        check("lengths", lengths, (B,), torch.int32)

    def body(handle):
        o = torch.empty_like(q) if out is None else out
        ls = q.new_empty((B, Hq, Nq), dtype=torch.float32) if lse is None else lse
        if out is not None:
            check("out", out, (B, Hq, Nq, d), torch.bfloat16)
        if lse is not None:
            check("lse", lse, (B, Hq, Nq), torch.float32)
        ws = call.scratch(workspace, _workspace_bytes("fa_decode_prefix_workspace_bytes", B, Hq, Hkv, Nq, Np, Ncap, d))
        _check(lib().fa_fwd_decode_prefix(
            q.data_ptr(), k_prefix.data_ptr(), v_prefix.data_ptr(), k.data_ptr(), v.data_ptr(),
            None if lengths is None else lengths.data_ptr(), o.data_ptr(), ls.data_ptr(), B, Hq, Hkv, Nq, Np, Ncap, d,
            1 if causal else 0, d ** -0.5 if scale is None else scale, ws.data_ptr(), ws.nbytes,
            handle), "fa_fwd_decode_prefix")
        return o, ls

    return call.run(body)


def attention_decode_weights(q, k, v, weights=None, lengths=None, causal=False, scale=None, out=None, lse=None,
                             weights_out=None, workspace=None, stream=None):
    """O, LSE of Nq queries q [B,Hq,Nq,d] against the first lengths[b] rows of
    the caches k, v [B,Hkv,Nk,d], and the attention weight that every key
    received, added to weights (fp32 [B,Hkv,Nk]; None: zero).  Passing the same
    tensor as weights and weights_out updates it in place (see
    fa_fwd_decode_weights).  Returns (o, lse, weights_out)."""
    call = _CacheCall("attention_decode_weights", q, stream)
    B, Hq, Nq, d, Hkv, Nk = call.dims(q, k)
    check, own = call.check, (B, Hkv, Nk, d)
    check("q", q, (B, Hq, Nq, d), torch.bfloat16)
    check("k", k, own, torch.bfloat16)
    check("v", v, own, torch.bfloat16)
    if weights is not None:
        check("weights", weights, (B, Hkv, Nk), torch.float32)
    if lengths is not None:
        check("lengths", lengths, (B,), torch.int32)

    def body(handle):
        o = torch.empty_like(q) if out is None else out
        ls = q.new_empty((B, Hq, Nq), dtype=torch.float32) if lse is None else lse
        wo = q.new_empty((B, Hkv, Nk), dtype=torch.float32) if weights_out is None else weights_out
        if out is not None:
            check("out", out, (B, Hq, Nq, d), torch.bfloat16)
        if lse is not None:
            check("lse", lse, (B, Hq, Nq), torch.float32)
        if weights_out is not None:
            check("weights_out", weights_out, (B, Hkv, Nk), torch.float32)
        ws = call.scratch(workspace, _workspace_bytes("fa_decode_weights_workspace_bytes", B, Hq, Hkv, Nq, Nk, d))
        _check(lib().fa_fwd_decode_weights(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), None if lengths is None else lengths.data_ptr(),
            None if weights is None else weights.data_ptr(), wo.data_ptr(), o.data_ptr(), ls.data_ptr(), B, Hq, Hkv,
            Nq, Nk, d, 1 if causal else 0, d ** -0.5 if scale is None else scale, ws.data_ptr(), ws.nbytes,
            handle), "fa_fwd_decode_weights")
        return o, ls, wo

    return call.run(body)


def attention_key_weights(q, k, lse, weights=None, lengths=None, causal=False, scale=None, weights_out=None,
                          workspace=None, stream=None):
    """The attention weight that every key of the caches k [B,Hkv,Nk,d] receives
    from the queries q [B,Hq,Nq,d] (the last Nq positions of each sequence)
    whose lse [B,Hq,Nq] is known, added to weights (fp32 [B,Hkv,Nk]; None:
    zero); see fa_key_weights, also for prompts of different lengths, whose rows
    have to end with them.  Returns weights_out."""
    call = _CacheCall("attention_key_weights", q, stream)
    B, Hq, Nq, d, Hkv, Nk = call.dims(q, k)
    check = call.check
    check("q", q, (B, Hq, Nq, d), torch.bfloat16)
    check("k", k, (B, Hkv, Nk, d), torch.bfloat16)
    check("lse", lse, (B, Hq, Nq), torch.float32)
    if weights is not None:
        check("weights", weights, (B, Hkv, Nk), torch.float32)
    if lengths is not None:
        check("lengths", lengths, (B,), torch.int32)

    def body(handle):
        wo = q.new_empty((B, Hkv, Nk), dtype=torch.float32) if weights_out is None else weights_out
        if weights_out is not None:
            check("weights_out", weights_out, (B, Hkv, Nk), torch.float32)
        ws = call.scratch(workspace, _workspace_bytes("fa_key_weights_workspace_bytes", B, Hq, Hkv, Nq, Nk, d))
        _check(lib().fa_key_weights(
            q.data_ptr(), k.data_ptr(), lse.data_ptr(), None if lengths is None else lengths.data_ptr(),
            None if weights is None else weights.data_ptr(), wo.data_ptr(), B, Hq, Hkv, Nq, Nk, d,
            1 if causal else 0, d ** -0.5 if scale is None else scale, ws.data_ptr(), ws.nbytes,
            handle), "fa_key_weights")
        return wo

    return call.run(body)


def cache_evict(k, v, weights, budget, recent=0, lengths=None, out_cap=None, k_out=None, v_out=None, weights_out=None,
                index=None, lengths_out=None, stream=None):
    """Cuts the caches k, v [B,Hkv,Nk,d] with the accumulated weights fp32
    [B,Hkv,Nk] down to budget keys a kv head: the last ``recent`` ones and, of
    the others, those of greatest weight, in their order (see fa_cache_evict).
    The outputs have out_cap slots (None: budget; more leaves room to decode
    into, and is not written).  Returns (k_out, v_out, weights_out, index int32
    [B,Hkv,out_cap], lengths_out int32 [B])."""
    call = _CacheCall("cache_evict", k, stream)
    if k.dim() != 4:
        call.refuse("k must be [B, Hkv, Nk, d]")
    B, Hkv, Nk, d = k.shape
    check = call.check
    check("k", k, (B, Hkv, Nk, d), torch.bfloat16)
    check("v", v, (B, Hkv, Nk, d), torch.bfloat16)
    check("weights", weights, (B, Hkv, Nk), torch.float32)
    if lengths is not None:
        check("lengths", lengths, (B,), torch.int32)
    cap = budget if out_cap is None else out_cap
    if not 1 <= budget <= cap or not 0 <= recent <= budget:
        call.refuse("budget must be in 1 .. out_cap and recent in 0 .. budget")
    rows, slots = (B, Hkv, cap, d), (B, Hkv, cap)

    def given_or_new(name, t, shape, dtype):
        if t is None:
            return k.new_empty(shape, dtype=dtype)
        check(name, t, shape, dtype)
        return t

    def body(handle):
        ko = given_or_new("k_out", k_out, rows, torch.bfloat16)
        vo = given_or_new("v_out", v_out, rows, torch.bfloat16)
        wo = given_or_new("weights_out", weights_out, slots, torch.float32)
        io = given_or_new("index", index, slots, torch.int32)
        lo = given_or_new("lengths_out", lengths_out, (B,), torch.int32)
        _check(lib().fa_cache_evict(
            k.data_ptr(), v.data_ptr(), weights.data_ptr(), None if lengths is None else lengths.data_ptr(),
            ko.data_ptr(), vo.data_ptr(), wo.data_ptr(), io.data_ptr(), lo.data_ptr(), B, Hkv, Nk, cap, budget, recent,
            d, handle), "fa_cache_evict")
        return ko, vo, wo, io, lo

    return call.run(body)
