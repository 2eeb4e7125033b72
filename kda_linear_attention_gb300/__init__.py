"""KDA (Kimi Delta Attention) recurrence for NVIDIA GB300 (sm_103a).

Thin Python binding of ``libkda_gb300.so`` (the C ABI in ``include/kda.h``):
it checks and marshals torch tensors into pointers and sizes and calls the
library on torch's current CUDA stream.  Every step of the computation runs
in the library's CUDA kernels; there is no CPU or PyTorch fallback, and the
calls raise if the library has not been built.

    o, S_out = prefill_chunked(q, k, v, g, beta, cu_seqlens, S0=None, chunk=64)
    o, S_out = prefill_chunked_noalloc(...)      # same, no device allocation
    ws = torch.empty(prefill_workspace_bytes(N, T, H), dtype=torch.uint8, device="cuda")
    o, S_out = prefill_chunked(..., workspace=ws) # same, in a workspace the caller owns
    o = decode_step(q, k, v, g, beta, S)          # S updated in place

The layer around the recurrence (conv1d + SiLU + L2 norm before it, gated
RMSNorm after it):

    q, k, v, conv_out = conv_prologue(xq, xk, xv, conv_w, cu_seqlens, conv_in=None)
    out, S_out = prefill_chunked_gated(q, k, v, g, beta, cu_seqlens, gate, norm_w)
    out, S_out, conv_out = prefill_layer(xq, xk, xv, conv_w, g, beta, gate, norm_w, cu_seqlens)
    out = decode_layer_step(xq, xk, xv, conv_w, conv_pool, g, beta, gate, norm_w, S_pool)

The hybrid model's other token mixer, latent attention over a paged cache
(bf16 rows of 512 latent + 64 shared key channels, [P, page, 576]):

    latent_append(x, cache, block_table, seq_lens, cu_seqlens, norm_w=w)   # new tokens' rows
    o, lse = latent_decode(q, cache, block_table, seq_lens, cu_seqlens)    # absorbed, over the pages
    rows = latent_gather(cache, block_table, cu_seqlens_k, total)          # rows back, to expand
    o, lse = latent_prefill(q, kv, k_pe, cu_seqlens_q, cu_seqlens_k)       # expanded, causal

Shapes of the recurrence (token-major): q, k, g [T, H, 128]; v [T, H, 128]; beta [T, H];
S [N, H, 128, 128] fp32; q/k/v bf16 or fp32, g/beta fp32.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Tuple

import torch

__all__ = ["prefill_chunked", "prefill_chunked_noalloc", "prefill_chunked_events",
           "prefill_workspace_bytes", "decode_step",
           "decode_step_pool", "conv_prologue", "prefill_chunked_gated", "prefill_layer",
           "decode_layer_step", "latent_append", "latent_gather", "latent_decode",
           "latent_decode_workspace_bytes", "latent_prefill", "latent_prefill_workspace_bytes",
           "device_error", "lib",
           "KDAError", "KDA_BF16", "KDA_F32", "library_path"]

_PKG = os.path.dirname(os.path.abspath(__file__))
# KDA_GB300_DEBUG=1 loads the debug build (python -m kda_linear_attention_gb300.build
# --debug): the same kernels with index checks that flag bit 3 of the device
# error word instead of touching memory outside a buffer.
_LIB_PATH = os.path.join(_PKG, "libkda_gb300_debug.so" if os.environ.get("KDA_GB300_DEBUG") == "1"
                         else "libkda_gb300.so")
_lib = None

KDA_BF16 = 0
KDA_F32 = 1
DK = 128
DV = 128


class KDAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s failed with status %d (%s)" % (what, status,
                                                            lib().kda_status_string(status).decode()))


def library_path() -> str:
    return _LIB_PATH


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                "%s is not built (python -m kda_linear_attention_gb300.build%s); "
                "this package has no CPU fallback"
                % (os.path.basename(_LIB_PATH), " --debug" if "debug" in _LIB_PATH else ""))
        L = ctypes.CDLL(_LIB_PATH)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        L.kda_version.argtypes = []
        L.kda_version.restype = i32
        L.kda_status_string.argtypes = [i32]
        L.kda_status_string.restype = ctypes.c_char_p
        L.kda_prefill_chunked.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                          i32, i64, i32, i32, i32, i32, i32, vp]
        L.kda_prefill_chunked.restype = i32
        L.kda_prefill_chunked_noalloc.argtypes = L.kda_prefill_chunked.argtypes
        L.kda_prefill_chunked_noalloc.restype = i32
        L.kda_prefill_chunked_events.argtypes = L.kda_prefill_chunked.argtypes + [
            ctypes.POINTER(ctypes.c_void_p)]
        L.kda_prefill_chunked_events.restype = i32
        L.kda_prefill_chunked_ws.argtypes = L.kda_prefill_chunked.argtypes[:-1] + [
            vp, ctypes.c_size_t, vp]
        L.kda_prefill_chunked_ws.restype = i32
        L.kda_prefill_workspace_bytes.argtypes = [i32, i64, i32, i32, i32, i32, i32]
        L.kda_prefill_workspace_bytes.restype = ctypes.c_size_t
        L.kda_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]
        L.kda_decode_step.restype = i32
        L.kda_decode_step_pool.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, i32, vp, i32, i32,
                                           i32, i32, i32, vp]
        L.kda_decode_step_pool.restype = i32
        f32 = ctypes.c_float
        L.kda_conv_prologue.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32,
                                        f32, f32, vp]
        L.kda_conv_prologue.restype = i32
        L.kda_prefill_chunked_gated.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, f32, vp, vp, vp,
                                                i32, i64, i32, i32, i32, i32, i32, vp]
        L.kda_prefill_chunked_gated.restype = i32
        L.kda_layer_prefill.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, f32, f32, f32,
                                        vp, vp, vp, i32, i64, i32, i32, i32, vp]
        L.kda_layer_prefill.restype = i32
        L.kda_decode_layer_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, i32,
                                            vp, i32, i32, i32, i32, f32, f32, f32, vp]
        L.kda_decode_layer_step.restype = i32
        L.kda_latent_append.argtypes = [vp, vp, vp, vp, vp, vp, f32, i32, i64, i64, i32, i32, i32,
                                        i32, vp]
        L.kda_latent_append.restype = i32
        L.kda_latent_gather.argtypes = [vp, vp, vp, vp, i32, i64, i64, i32, i32, i32, i32, vp]
        L.kda_latent_gather.restype = i32
        L.kda_latent_decode.argtypes = [vp, vp, vp, vp, vp, f32, vp, vp, i32, i64, i32, i64, i32,
                                        i32, i32, i32, vp, ctypes.c_size_t, vp]
        L.kda_latent_decode.restype = i32
        L.kda_latent_decode_workspace_bytes.argtypes = [i32, i64, i32, i32, i32]
        L.kda_latent_decode_workspace_bytes.restype = ctypes.c_size_t
        L.kda_latent_prefill.argtypes = [vp, vp, vp, i64, vp, vp, f32, i32, vp, vp, i32, i64, i64,
                                         i32, i32, i32, i32, vp, ctypes.c_size_t, vp]
        L.kda_latent_prefill.restype = i32
        L.kda_latent_prefill_workspace_bytes.argtypes = [i32, i64, i64, i32, i32, i32, i32]
        L.kda_latent_prefill_workspace_bytes.restype = ctypes.c_size_t
        L.kda_workspace_release.argtypes = []
        L.kda_workspace_release.restype = i32
        L.kda_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint), i32]
        L.kda_device_error.restype = i32
        _lib = L
    return _lib


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _qkv_dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError("q, k, v must be bfloat16 or float32, got %s" % t.dtype)


def _check(name: str, t: torch.Tensor, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _stream(device: torch.device, stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream(device) if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _prefill(fn_name: str, q, k, v, g, beta, cu_seqlens, S0, chunk, o, S_out, stream, extra=(),
             gated=None, ws=None):
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    T, H = q.shape[0], q.shape[1]
    N = cu_seqlens.numel() - 1
    dt = _qkv_dtype(q)
    _check("q", q, q.dtype, (T, H, DK), dev)
    _check("k", k, q.dtype, (T, H, DK), dev)
    _check("v", v, q.dtype, (T, H, DV), dev)
    _check("g", g, torch.float32, (T, H, DK), dev)
    _check("beta", beta, torch.float32, (T, H), dev)
    _check("cu_seqlens", cu_seqlens, torch.int32, (N + 1,), dev)
    if S0 is not None:
        _check("S0", S0, torch.float32, (N, H, DK, DV), dev)
    if o is None:
        o = torch.empty((T, H, DV), dtype=torch.float32, device=dev)
    if S_out is None:
        S_out = torch.empty((N, H, DK, DV), dtype=torch.float32, device=dev)
    _check("o", o, torch.float32, (T, H, DV), dev)
    _check("S_out", S_out, torch.float32, (N, H, DK, DV), dev)
    if gated is not None:
        gate, norm_w, eps = gated
        rc = getattr(lib(), fn_name)(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(S0), _p(gate),
                                     _p(norm_w), float(eps), _p(o), _p(S_out), _p(cu_seqlens), N,
                                     T, H, DK, DV, int(chunk), dt, _stream(dev, stream))
    elif ws is not None:
        rc = getattr(lib(), fn_name)(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(S0), _p(o),
                                     _p(S_out), _p(cu_seqlens), N, T, H, DK, DV, int(chunk), dt,
                                     ws[0], ctypes.c_size_t(ws[1]), _stream(dev, stream))
    else:
        rc = getattr(lib(), fn_name)(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(S0), _p(o),
                                     _p(S_out), _p(cu_seqlens), N, T, H, DK, DV, int(chunk), dt,
                                     _stream(dev, stream), *extra)
    if rc != 0:
        raise KDAError(rc, fn_name)
    return o, S_out


def prefill_workspace_bytes(N: int, T: int, H: int, chunk: int = 64, dtype: int = None) -> int:
    """Bytes of workspace ``prefill_chunked(..., workspace=...)`` needs
    (``kda_prefill_workspace_bytes``); 0 where the call needs none."""
    dt = KDA_BF16 if dtype is None else int(dtype)
    return int(lib().kda_prefill_workspace_bytes(int(N), int(T), int(H), DK, DV, int(chunk), dt))


def prefill_chunked(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                    beta: torch.Tensor, cu_seqlens: torch.Tensor,
                    S0: Optional[torch.Tensor] = None, chunk: int = 64,
                    o: Optional[torch.Tensor] = None, S_out: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None,
                    workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Chunked KDA prefill over packed varlen sequences (``kda_prefill_chunked``).

    Returns (o [T, H, 128] fp32, S_out [N, H, 128, 128] fp32).  ``S_out`` may
    be ``S0`` itself to update the states in place.  With ``workspace`` (a
    contiguous CUDA tensor of at least ``prefill_workspace_bytes`` bytes) the
    call runs in that buffer (``kda_prefill_chunked_ws``) instead of the
    library's own pool.
    """
    if workspace is not None:
        if workspace.device != q.device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the inputs' device")
        nbytes = workspace.numel() * workspace.element_size()
        return _prefill("kda_prefill_chunked_ws", q, k, v, g, beta, cu_seqlens, S0, chunk, o,
                        S_out, stream, ws=(_p(workspace), nbytes))
    return _prefill("kda_prefill_chunked", q, k, v, g, beta, cu_seqlens, S0, chunk, o, S_out,
                    stream)


def prefill_chunked_events(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                           beta: torch.Tensor, cu_seqlens: torch.Tensor, events,
                           S0: Optional[torch.Tensor] = None,
                           o: Optional[torch.Tensor] = None, S_out: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None
                           ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Tensor-core ``prefill_chunked`` (bf16, chunk 64) that also records four
    ``torch.cuda.Event`` (timing enabled) around its kernels: before the chunk
    plan, before the intra-chunk kernel, before the state pass, after it
    (``kda_prefill_chunked_events``)."""
    if len(events) != 4:
        raise ValueError("need four events")
    s = torch.cuda.current_stream(q.device) if stream is None else stream
    for e in events:
        if not e.cuda_event:          # torch creates the CUDA event at its first record
            e.record(s)
    evs = [ctypes.c_void_p(e.cuda_event) for e in events]
    arr = (ctypes.c_void_p * 4)(*evs)
    return _prefill("kda_prefill_chunked_events", q, k, v, g, beta, cu_seqlens, S0, 64, o, S_out,
                    stream, extra=(ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p)),))


def prefill_chunked_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                            beta: torch.Tensor, cu_seqlens: torch.Tensor,
                            S0: Optional[torch.Tensor] = None, chunk: int = 64,
                            o: Optional[torch.Tensor] = None, S_out: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None
                            ) -> Tuple[torch.Tensor, torch.Tensor]:
    """``prefill_chunked`` through ``kda_prefill_chunked_noalloc``: the library
    allocates nothing (its fixed scratch array bounds the input size; pass
    ``o`` and ``S_out`` to keep this binding from allocating them either)."""
    return _prefill("kda_prefill_chunked_noalloc", q, k, v, g, beta, cu_seqlens, S0, chunk, o,
                    S_out, stream)


def decode_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                beta: torch.Tensor, S: torch.Tensor, o: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One decode token per sequence (``kda_decode_step``); ``S`` is updated in place.

    q, k, g [B, H, 128]; v [B, H, 128]; beta [B, H]; S [B, H, 128, 128] fp32.
    Returns o [B, H, 128] fp32.
    """
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    B, H = q.shape[0], q.shape[1]
    dt = _qkv_dtype(q)
    _check("q", q, q.dtype, (B, H, DK), dev)
    _check("k", k, q.dtype, (B, H, DK), dev)
    _check("v", v, q.dtype, (B, H, DV), dev)
    _check("g", g, torch.float32, (B, H, DK), dev)
    _check("beta", beta, torch.float32, (B, H), dev)
    _check("S", S, torch.float32, (B, H, DK, DV), dev)
    if o is None:
        o = torch.empty((B, H, DV), dtype=torch.float32, device=dev)
    _check("o", o, torch.float32, (B, H, DV), dev)
    rc = lib().kda_decode_step(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(S), _p(o), B, H, DK, DV,
                               dt, _stream(dev, stream))
    if rc != 0:
        raise KDAError(rc, "kda_decode_step")
    return o


def decode_step_pool(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                     beta: torch.Tensor, S_pool: torch.Tensor,
                     state_indices: Optional[torch.Tensor] = None,
                     o: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One decode token per sequence on a state pool (``kda_decode_step_pool``).

    S_pool [P, H, 128, 128] fp32 or bf16 is updated in place at rows
    ``state_indices`` ([B] int32; negative = padding, o row zero), or at rows
    0..B-1 when it is None.  Returns o [B, H, 128] fp32.
    """
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    B, H = q.shape[0], q.shape[1]
    dt = _qkv_dtype(q)
    _check("q", q, q.dtype, (B, H, DK), dev)
    _check("k", k, q.dtype, (B, H, DK), dev)
    _check("v", v, q.dtype, (B, H, DV), dev)
    _check("g", g, torch.float32, (B, H, DK), dev)
    _check("beta", beta, torch.float32, (B, H), dev)
    if S_pool.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("S_pool must be float32 or bfloat16")
    P = S_pool.shape[0]
    _check("S_pool", S_pool, S_pool.dtype, (P, H, DK, DV), dev)
    if state_indices is not None:
        _check("state_indices", state_indices, torch.int32, (B,), dev)
    if o is None:
        o = torch.empty((B, H, DV), dtype=torch.float32, device=dev)
    _check("o", o, torch.float32, (B, H, DV), dev)
    sdt = KDA_BF16 if S_pool.dtype == torch.bfloat16 else KDA_F32
    rc = lib().kda_decode_step_pool(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(S_pool), sdt,
                                    _p(state_indices), P, _p(o), B, H, DK, DV, dt,
                                    _stream(dev, stream))
    if rc != 0:
        raise KDAError(rc, "kda_decode_step_pool")
    return o


# ------------------------------------------------------------ the layer
CONV_K = 4
Q_SCALE = DK ** -0.5          # the pages' q scale, 1/sqrt(head width)
L2_EPS = 1e-6
NORM_EPS = 1e-6


def conv_prologue(xq: torch.Tensor, xk: torch.Tensor, xv: torch.Tensor, conv_w: torch.Tensor,
                  cu_seqlens: torch.Tensor, conv_in: Optional[torch.Tensor] = None,
                  conv_out: Optional[torch.Tensor] = None, q_scale: float = Q_SCALE,
                  eps: float = L2_EPS, q=None, k=None, v=None,
                  stream: Optional[torch.cuda.Stream] = None):
    """conv1d + SiLU + L2 norm of the raw projections (``kda_conv_prologue``).

    xq, xk, xv [T, H, 128] bf16; conv_w [3, H, 128, 4] fp32; conv_in / conv_out
    [N, 3, 3, H, 128] bf16 windows (conv_in None = zeros; conv_out allocated
    if None).  Returns (q, k, v [T, H, 128] bf16, conv_out).
    """
    dev = xq.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    T, H = xq.shape[0], xq.shape[1]
    N = cu_seqlens.numel() - 1
    bf = torch.bfloat16
    for n, t in (("xq", xq), ("xk", xk), ("xv", xv)):
        _check(n, t, bf, (T, H, DK), dev)
    _check("conv_w", conv_w, torch.float32, (3, H, DK, CONV_K), dev)
    _check("cu_seqlens", cu_seqlens, torch.int32, (N + 1,), dev)
    wshape = (N, 3, CONV_K - 1, H, DK)
    if conv_in is not None:
        _check("conv_in", conv_in, bf, wshape, dev)
    if conv_out is None:
        conv_out = torch.empty(wshape, dtype=bf, device=dev)
    _check("conv_out", conv_out, bf, wshape, dev)
    q = torch.empty((T, H, DK), dtype=bf, device=dev) if q is None else q
    k = torch.empty((T, H, DK), dtype=bf, device=dev) if k is None else k
    v = torch.empty((T, H, DV), dtype=bf, device=dev) if v is None else v
    for n, t in (("q", q), ("k", k), ("v", v)):
        _check(n, t, bf, (T, H, DK), dev)
    rc = lib().kda_conv_prologue(_p(xq), _p(xk), _p(xv), _p(conv_w), _p(conv_in), _p(conv_out),
                                 _p(q), _p(k), _p(v), _p(cu_seqlens), N, T, H, DK,
                                 float(q_scale), float(eps), _stream(dev, stream))
    if rc != 0:
        raise KDAError(rc, "kda_conv_prologue")
    return q, k, v, conv_out


def prefill_chunked_gated(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                          beta: torch.Tensor, cu_seqlens: torch.Tensor, gate: torch.Tensor,
                          norm_w: torch.Tensor, S0: Optional[torch.Tensor] = None,
                          chunk: int = 64, eps: float = NORM_EPS,
                          out: Optional[torch.Tensor] = None, S_out: Optional[torch.Tensor] = None,
                          stream: Optional[torch.cuda.Stream] = None
                          ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Chunked prefill whose output is RMSNorm(o) * norm_w * sigmoid(gate)
    (``kda_prefill_chunked_gated``).  gate [T, H, 128] bf16, norm_w [128] fp32.
    Returns (out [T, H, 128] fp32, S_out)."""
    dev = q.device
    T, H = q.shape[0], q.shape[1]
    _check("gate", gate, torch.bfloat16, (T, H, DV), dev)
    _check("norm_w", norm_w, torch.float32, (DV,), dev)
    return _prefill("kda_prefill_chunked_gated", q, k, v, g, beta, cu_seqlens, S0, chunk, out,
                    S_out, stream, gated=(gate, norm_w, eps))


def prefill_layer(xq, xk, xv, conv_w, g, beta, gate, norm_w, cu_seqlens,
                  conv_in: Optional[torch.Tensor] = None, S0: Optional[torch.Tensor] = None,
                  q_scale: float = Q_SCALE, l2_eps: float = L2_EPS, norm_eps: float = NORM_EPS,
                  out: Optional[torch.Tensor] = None, S_out: Optional[torch.Tensor] = None,
                  conv_out: Optional[torch.Tensor] = None, one_call: bool = True,
                  stream: Optional[torch.cuda.Stream] = None):
    """The layer's prefill from raw projections in one C call
    (``kda_layer_prefill``: the conv + SiLU + L2-norm prologue, then the
    gated prefill, q, k, v in the library's workspace).  one_call=False runs
    the same layer as the two public calls, ``conv_prologue`` (q, k, v in
    tensors of this binding) then ``prefill_chunked_gated``.  Returns
    (out [T, H, 128] fp32, S_out [N, H, 128, 128] fp32,
    conv_out [N, 3, 3, H, 128] bf16)."""
    if not one_call:
        q, k, v, conv_out = conv_prologue(xq, xk, xv, conv_w, cu_seqlens, conv_in=conv_in,
                                          conv_out=conv_out, q_scale=q_scale, eps=l2_eps,
                                          stream=stream)
        out, S_out = prefill_chunked_gated(q, k, v, g, beta, cu_seqlens, gate, norm_w, S0=S0,
                                           eps=norm_eps, out=out, S_out=S_out, stream=stream)
        return out, S_out, conv_out
    dev = xq.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    T, H = xq.shape[0], xq.shape[1]
    N = cu_seqlens.numel() - 1
    bf = torch.bfloat16
    for n, t in (("xq", xq), ("xk", xk), ("xv", xv), ("gate", gate)):
        _check(n, t, bf, (T, H, DK), dev)
    _check("conv_w", conv_w, torch.float32, (3, H, DK, CONV_K), dev)
    _check("g", g, torch.float32, (T, H, DK), dev)
    _check("beta", beta, torch.float32, (T, H), dev)
    _check("norm_w", norm_w, torch.float32, (DV,), dev)
    _check("cu_seqlens", cu_seqlens, torch.int32, (N + 1,), dev)
    wshape = (N, 3, CONV_K - 1, H, DK)
    if conv_in is not None:
        _check("conv_in", conv_in, bf, wshape, dev)
    if conv_out is None:
        conv_out = torch.empty(wshape, dtype=bf, device=dev)
    _check("conv_out", conv_out, bf, wshape, dev)
    if S0 is not None:
        _check("S0", S0, torch.float32, (N, H, DK, DV), dev)
    if out is None:
        out = torch.empty((T, H, DV), dtype=torch.float32, device=dev)
    if S_out is None:
        S_out = torch.empty((N, H, DK, DV), dtype=torch.float32, device=dev)
    _check("out", out, torch.float32, (T, H, DV), dev)
    _check("S_out", S_out, torch.float32, (N, H, DK, DV), dev)
    rc = lib().kda_layer_prefill(_p(xq), _p(xk), _p(xv), _p(conv_w), _p(conv_in), _p(conv_out),
                                 _p(g), _p(beta), _p(S0), _p(gate), _p(norm_w), float(q_scale),
                                 float(l2_eps), float(norm_eps), _p(out), _p(S_out),
                                 _p(cu_seqlens), N, T, H, DK, DV, _stream(dev, stream))
    if rc != 0:
        raise KDAError(rc, "kda_layer_prefill")
    return out, S_out, conv_out


def decode_layer_step(xq: torch.Tensor, xk: torch.Tensor, xv: torch.Tensor, conv_w: torch.Tensor,
                      conv_pool: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                      gate: torch.Tensor, norm_w: torch.Tensor, S_pool: torch.Tensor,
                      state_indices: Optional[torch.Tensor] = None, q_scale: float = Q_SCALE,
                      l2_eps: float = L2_EPS, norm_eps: float = NORM_EPS,
                      out: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One token of the whole layer per sequence (``kda_decode_layer_step``):
    conv windows (conv_pool [P, 3, 3, H, 128] bf16) and states (S_pool
    [P, H, 128, 128] fp32 or bf16) updated in place at rows state_indices.
    Returns out [B, H, 128] fp32."""
    dev = xq.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    B, H = xq.shape[0], xq.shape[1]
    bf = torch.bfloat16
    for n, t in (("xq", xq), ("xk", xk), ("xv", xv), ("gate", gate)):
        _check(n, t, bf, (B, H, DK), dev)
    _check("conv_w", conv_w, torch.float32, (3, H, DK, CONV_K), dev)
    _check("g", g, torch.float32, (B, H, DK), dev)
    _check("beta", beta, torch.float32, (B, H), dev)
    _check("norm_w", norm_w, torch.float32, (DV,), dev)
    if S_pool.dtype not in (torch.float32, bf):
        raise TypeError("S_pool must be float32 or bfloat16")
    P = S_pool.shape[0]
    _check("S_pool", S_pool, S_pool.dtype, (P, H, DK, DV), dev)
    _check("conv_pool", conv_pool, bf, (P, 3, CONV_K - 1, H, DK), dev)
    if state_indices is not None:
        _check("state_indices", state_indices, torch.int32, (B,), dev)
    if out is None:
        out = torch.empty((B, H, DV), dtype=torch.float32, device=dev)
    _check("out", out, torch.float32, (B, H, DV), dev)
    sdt = KDA_BF16 if S_pool.dtype == bf else KDA_F32
    rc = lib().kda_decode_layer_step(_p(xq), _p(xk), _p(xv), _p(conv_w), _p(conv_pool), _p(g),
                                     _p(beta), _p(gate), _p(norm_w), _p(S_pool), sdt,
                                     _p(state_indices), P, _p(out), B, H, DK, DV, float(q_scale),
                                     float(l2_eps), float(norm_eps), _stream(dev, stream))
    if rc != 0:
        raise KDAError(rc, "kda_decode_layer_step")
    return out


# ------------------------------------------------------------ latent attention
LATENT = 512                  # latent width of a cached row
LATENT_PE = 64                # its key part shared by the heads
LATENT_ROW = LATENT + LATENT_PE
LATENT_SCALE = (DK + LATENT_PE) ** -0.5   # 1/sqrt(expanded key width)


# The calls below run once a layer and step with kernels of a few
# microseconds, so a call that is right passes one chain of cheap comparisons
# (a shape is asked for once and compared as numbers); one that is not goes
# through _check for the error's words.
_Tensor, _BF16, _F32, _I32 = torch.Tensor, torch.bfloat16, torch.float32, torch.int32


def _device(t) -> int:
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise ValueError("inputs must be CUDA tensors")
    return t.get_device()


def _plain(t, dtype, dev) -> bool:
    """Dense, of the type, on the device (an index)."""
    return t.dtype is dtype and t.get_device() == dev and t.is_contiguous()


def _refuse(dev, *tensors):
    """The first of (name, tensor, dtype, shape) that _check refuses; -1 in a
    shape stands for any size."""
    device = torch.device("cuda", dev)
    for name, t, dtype, shape in tensors:
        if t is None:
            continue
        if not isinstance(t, _Tensor) or t.dim() != len(shape):
            raise ValueError("%s must be a tensor of %d dimensions" % (name, len(shape)))
        _check(name, t, dtype, [n if m < 0 else m for n, m in zip(t.shape, shape)], device)
    raise ValueError("unsupported arguments")


# torch's inner names of what its public calls wrap; a torch without them is
# served by the public ones.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
                       or (lambda dev: torch.cuda.current_stream(dev).cuda_stream))


def _raw_stream(dev, stream):
    return _current_raw_stream(dev) if stream is None else stream.cuda_stream


def _empty(shape, dtype, like, stream):
    """Memory on the tensor's device, of the stream that uses it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


# A call's own workspace comes from torch's caching allocator without a tensor
# around it (10 MB as a tensor add 7 us to a call's host time, as plain memory
# 2 us).  It belongs to the stream (or to the graph being captured on it), so
# that giving it back right after the launches is safe: what the stream does
# later may have it next.  (A torch without these names gives a tensor.)
_raw_alloc = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None)
_raw_free = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None)


def _take_workspace(nbytes, like, stream, raw_stream):
    """(address, what holds it) of a call's own workspace, for _give_back."""
    if not nbytes:
        return None, None
    if _raw_alloc is None or _raw_free is None:
        t = _empty((nbytes,), torch.uint8, like, stream)
        return t.data_ptr(), t
    p = _raw_alloc(nbytes, raw_stream)
    return p, p


def _give_back(own):
    if type(own) is int:          # a tensor goes with its last name
        _raw_free(own)


def _given_workspace(t, dev):
    """(address, bytes) of the caller's workspace."""
    if not isinstance(t, _Tensor) or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return t.data_ptr(), t.numel() * t.element_size()


def latent_append(x: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                  seq_lens: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                  norm_w: Optional[torch.Tensor] = None, eps: float = NORM_EPS,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Write new tokens' rows into the paged latent cache (``kda_latent_append``).

    x [T, 576] bf16; cache [P, page, 576] bf16, updated in place; block_table
    [N, max_pages], seq_lens [N] (the new tokens counted in) and cu_seqlens
    [N + 1] int32 (None: one new token a sequence).  With norm_w [512] fp32
    the latent part is RMS-normalised.  Returns cache.
    """
    dev = _device(x)
    if dev != _current_device():       # a launch goes to the current device
        with torch.cuda.device(dev):
            return latent_append(x, cache, block_table, seq_lens, cu_seqlens, norm_w, eps, stream)
    N, xs, cs, ts = seq_lens.numel(), x.shape, cache.shape, block_table.shape
    if not (len(xs) == 2 and xs[1] == LATENT_ROW and _plain(x, _BF16, dev)
            and len(cs) == 3 and cs[2] == LATENT_ROW and _plain(cache, _BF16, dev)
            and len(ts) == 2 and ts[0] == N and _plain(block_table, _I32, dev)
            and seq_lens.dim() == 1 and _plain(seq_lens, _I32, dev)
            and (cu_seqlens is None or cu_seqlens.shape == (N + 1,) and _plain(cu_seqlens, _I32, dev))
            and (norm_w is None or norm_w.shape == (LATENT,) and _plain(norm_w, _F32, dev))):
        _refuse(dev, ("x", x, _BF16, (-1, LATENT_ROW)), ("cache", cache, _BF16, (-1, -1, LATENT_ROW)),
                ("block_table", block_table, _I32, (N, -1)), ("seq_lens", seq_lens, _I32, (N,)),
                ("cu_seqlens", cu_seqlens, _I32, (N + 1,)), ("norm_w", norm_w, _F32, (LATENT,)))
    rc = lib().kda_latent_append(
        x.data_ptr(), cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
        None if cu_seqlens is None else cu_seqlens.data_ptr(), None if norm_w is None else norm_w.data_ptr(),
        eps, N, xs[0], cs[0], cs[1], ts[1], LATENT, LATENT_PE, _raw_stream(dev, stream))
    if rc != 0:
        raise KDAError(rc, "kda_latent_append")
    return cache


def latent_gather(cache: torch.Tensor, block_table: torch.Tensor, cu_seqlens: torch.Tensor,
                  total: Optional[int] = None, out: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Read every sequence's first rows back, packed by cu_seqlens
    (``kda_latent_gather``).  total: the packed length cu_seqlens[N] (where
    ``out`` [total, 576] bf16 is not given).  Returns out."""
    dev = _device(cache)
    if dev != _current_device():       # a launch goes to the current device
        with torch.cuda.device(dev):
            return latent_gather(cache, block_table, cu_seqlens, total, out, stream)
    if out is None:
        if total is None:
            raise ValueError("give the packed length (total) or the output (out)")
        out = _empty((total, LATENT_ROW), _BF16, cache, stream)
    N, os, cs, ts = cu_seqlens.numel() - 1, out.shape, cache.shape, block_table.shape
    if not (len(os) == 2 and os[1] == LATENT_ROW and _plain(out, _BF16, dev)
            and len(cs) == 3 and cs[2] == LATENT_ROW and _plain(cache, _BF16, dev)
            and len(ts) == 2 and ts[0] == N and _plain(block_table, _I32, dev)
            and cu_seqlens.dim() == 1 and _plain(cu_seqlens, _I32, dev)):
        _refuse(dev, ("cache", cache, _BF16, (-1, -1, LATENT_ROW)), ("block_table", block_table, _I32, (N, -1)),
                ("cu_seqlens", cu_seqlens, _I32, (N + 1,)), ("out", out, _BF16, (-1, LATENT_ROW)))
    rc = lib().kda_latent_gather(cache.data_ptr(), block_table.data_ptr(), cu_seqlens.data_ptr(), out.data_ptr(),
                                 N, os[0], cs[0], cs[1], ts[1], LATENT, LATENT_PE, _raw_stream(dev, stream))
    if rc != 0:
        raise KDAError(rc, "kda_latent_gather")
    return out


@functools.lru_cache(maxsize=1024)
def latent_decode_workspace_bytes(N: int, T: int, H: int) -> int:
    """Bytes of workspace of ``latent_decode`` (``kda_latent_decode_workspace_bytes``)."""
    return int(lib().kda_latent_decode_workspace_bytes(int(N), int(T), int(H), LATENT, LATENT_PE))


def latent_decode(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                  seq_lens: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                  scale: float = LATENT_SCALE, o: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None
                  ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Absorbed attention of one or a few new tokens a sequence over the paged
    cache that holds them already (``kda_latent_decode``).

    q [T, H, 576] bf16; cache [P, page, 576] bf16; block_table [N, max_pages],
    seq_lens [N] and cu_seqlens [N + 1] int32 (None: one token a sequence; for
    65 to 512 heads faster than offsets that say the same).
    Returns (o [T, H, 512] bf16, lse [T, H] fp32); a query row of NaN or
    infinities has o = NaN where it sees anything.  The workspace
    (``latent_decode_workspace_bytes``) comes from torch's allocator unless
    one is given.
    """
    dev = _device(q)
    if dev != _current_device():       # a launch goes to the current device
        with torch.cuda.device(dev):
            return latent_decode(q, cache, block_table, seq_lens, cu_seqlens, scale, o, lse, workspace, stream)
    N, qs, cs, ts = seq_lens.numel(), q.shape, cache.shape, block_table.shape
    if not (len(qs) == 3 and qs[2] == LATENT_ROW and _plain(q, _BF16, dev)
            and len(cs) == 3 and cs[2] == LATENT_ROW and _plain(cache, _BF16, dev)
            and len(ts) == 2 and ts[0] == N and _plain(block_table, _I32, dev)
            and seq_lens.dim() == 1 and _plain(seq_lens, _I32, dev)
            and (cu_seqlens is None or cu_seqlens.shape == (N + 1,) and _plain(cu_seqlens, _I32, dev))):
        _refuse(dev, ("q", q, _BF16, (-1, -1, LATENT_ROW)), ("cache", cache, _BF16, (-1, -1, LATENT_ROW)),
                ("block_table", block_table, _I32, (N, -1)), ("seq_lens", seq_lens, _I32, (N,)),
                ("cu_seqlens", cu_seqlens, _I32, (N + 1,)))
    T, H, _ = qs
    if o is None:
        o = _empty((T, H, LATENT), _BF16, q, stream)
    elif not (o.shape == (T, H, LATENT) and _plain(o, _BF16, dev)):
        _refuse(dev, ("o", o, _BF16, (T, H, LATENT)))
    if lse is None:
        lse = _empty((T, H), _F32, q, stream)
    elif not (lse.shape == (T, H) and _plain(lse, _F32, dev)):
        _refuse(dev, ("lse", lse, _F32, (T, H)))
    s, own = _raw_stream(dev, stream), None
    if workspace is not None:
        ws, nbytes = _given_workspace(workspace, dev)
    else:
        nbytes = latent_decode_workspace_bytes(N, T, H)
        ws, own = _take_workspace(nbytes, q, stream, s)
    try:
        rc = lib().kda_latent_decode(
            q.data_ptr(), cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
            None if cu_seqlens is None else cu_seqlens.data_ptr(), scale, o.data_ptr(), lse.data_ptr(),
            N, T, H, cs[0], cs[1], ts[1], LATENT, LATENT_PE, ws, nbytes, s)
    finally:
        _give_back(own)
    if rc != 0:
        raise KDAError(rc, "kda_latent_decode")
    return o, lse


@functools.lru_cache(maxsize=1024)
def latent_prefill_workspace_bytes(N: int, Tq: int, Tk: int, H: int) -> int:
    """Bytes of workspace of ``latent_prefill`` (``kda_latent_prefill_workspace_bytes``)."""
    return int(lib().kda_latent_prefill_workspace_bytes(int(N), int(Tq), int(Tk), int(H), DK, LATENT_PE, DV))


def latent_prefill(q: torch.Tensor, kv: torch.Tensor, k_pe: torch.Tensor, cu_seqlens: torch.Tensor,
                   cu_seqlens_k: Optional[torch.Tensor] = None, scale: float = LATENT_SCALE,
                   causal: bool = True, o: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Expanded attention of new tokens over their sequence's keys and values
    (``kda_latent_prefill``).

    q [Tq, H, 192] bf16; kv [Tk, H, 256] bf16 (key 128 | value 128); k_pe
    [Tk, 64] bf16, its rows any multiple of 8 elements apart (so that
    ``rows[:, 512:]`` of gathered cache rows is taken as it is); cu_seqlens
    and cu_seqlens_k [N + 1] int32 (None: the same).  The queries of a
    sequence are its last tokens.  Returns (o [Tq, H, 128] bf16, lse [Tq, H]
    fp32); a query row of NaN or infinities has o = NaN where it sees
    anything.  The workspace (``latent_prefill_workspace_bytes``, often none)
    comes from torch's allocator unless one is given.
    """
    dev = _device(q)
    if dev != _current_device():       # a launch goes to the current device
        with torch.cuda.device(dev):
            return latent_prefill(q, kv, k_pe, cu_seqlens, cu_seqlens_k, scale, causal, o, lse, workspace, stream)
    if cu_seqlens_k is None:
        cu_seqlens_k = cu_seqlens
    N, qs, ks, ps = cu_seqlens.numel() - 1, q.shape, kv.shape, k_pe.shape
    if not (len(qs) == 3 and qs[2] == DK + LATENT_PE and _plain(q, _BF16, dev)
            and len(ks) == 3 and ks[1] == qs[1] and ks[2] == DK + DV and _plain(kv, _BF16, dev)
            and cu_seqlens.dim() == 1 and _plain(cu_seqlens, _I32, dev)
            and cu_seqlens_k.shape == (N + 1,) and _plain(cu_seqlens_k, _I32, dev)):
        H = qs[1] if len(qs) > 1 else -1
        _refuse(dev, ("q", q, _BF16, (-1, -1, DK + LATENT_PE)), ("kv", kv, _BF16, (-1, H, DK + DV)),
                ("cu_seqlens", cu_seqlens, _I32, (N + 1,)), ("cu_seqlens_k", cu_seqlens_k, _I32, (N + 1,)))
    Tq, H, _ = qs
    Tk = ks[0]
    if not (k_pe.get_device() == dev and k_pe.dtype is _BF16 and ps == (Tk, LATENT_PE)
            and (Tk == 0 or k_pe.stride(1) == 1)):
        raise ValueError("k_pe must be [%d, %d] bfloat16 on %s with dense rows"
                         % (Tk, LATENT_PE, q.device))
    # the stride of a dimension of one row means nothing
    pe_stride = k_pe.stride(0) if Tk > 1 else LATENT_PE
    if o is None:
        o = _empty((Tq, H, DV), _BF16, q, stream)
    elif not (o.shape == (Tq, H, DV) and _plain(o, _BF16, dev)):
        _refuse(dev, ("o", o, _BF16, (Tq, H, DV)))
    if lse is None:
        lse = _empty((Tq, H), _F32, q, stream)
    elif not (lse.shape == (Tq, H) and _plain(lse, _F32, dev)):
        _refuse(dev, ("lse", lse, _F32, (Tq, H)))
    s, own = _raw_stream(dev, stream), None
    if workspace is not None:
        ws, nbytes = _given_workspace(workspace, dev)
    else:
        nbytes = latent_prefill_workspace_bytes(N, Tq, Tk, H)
        ws, own = _take_workspace(nbytes, q, stream, s)
    try:
        rc = lib().kda_latent_prefill(
            q.data_ptr(), kv.data_ptr(), k_pe.data_ptr(), pe_stride, cu_seqlens.data_ptr(),
            cu_seqlens_k.data_ptr(), scale, 1 if causal else 0, o.data_ptr(), lse.data_ptr(), N, Tq, Tk, H,
            DK, LATENT_PE, DV, ws, nbytes, s)
    finally:
        _give_back(own)
    if rc != 0:
        raise KDAError(rc, "kda_latent_prefill")
    return o, lse


def device_error(reset: bool = True) -> int:
    """The library's device-side error word (``kda_device_error``); nonzero if
    a bounded wait inside a kernel gave up since the last reset."""
    code = ctypes.c_uint(0)
    rc = lib().kda_device_error(ctypes.byref(code), int(reset))
    if rc != 0:
        raise KDAError(rc, "kda_device_error")
    return int(code.value)


def workspace_release() -> None:
    """Give the library's workspace pool memory on the current device back to
    the driver (``kda_workspace_release``); synchronise the streams that ran
    prefills first."""
    rc = lib().kda_workspace_release()
    if rc != 0:
        raise KDAError(rc, "kda_workspace_release")
