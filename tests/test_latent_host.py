"""Host-side checks of the latent-attention calls (no GPU): the C entries
refuse bad arguments before launching anything, calls without tokens are
no-ops, and the binding refuses tensors it cannot take."""
import ctypes

import pytest

GOOD = ctypes.c_void_p(0x10000)   # aligned, never dereferenced
OFF4 = ctypes.c_void_p(0x10004)


@pytest.fixture(scope="module")
def L():
    from kda_linear_attention_gb300 import build
    build.build()
    import kda_linear_attention_gb300 as kda
    return kda.lib()


CACHE = dict(N=2, T=2, P=8, page=64, max_pages=4, dl=512, dp=64)
BAD_CACHE = [(dict(dl=256), 2), (dict(dp=0), 2), (dict(N=0), 2), (dict(T=-1), 2), (dict(T=1 << 31), 2),
             (dict(P=0), 2), (dict(max_pages=0), 2), (dict(page=8), 2), (dict(page=48), 2),
             (dict(page=2048), 2), (dict(page=0), 2), (dict(P=1 << 25, page=64), 2), (dict(P=1 << 62), 2)]


def _append(L, **kw):
    a = dict(CACHE, x=GOOD, cache=GOOD, table=GOOD, lens=GOOD, cu=None, w=None, eps=1e-6)
    a.update(kw)
    return L.kda_latent_append(a["x"], a["cache"], a["table"], a["lens"], a["cu"], a["w"], a["eps"], a["N"],
                               a["T"], a["P"], a["page"], a["max_pages"], a["dl"], a["dp"], None)


def _gather(L, **kw):
    a = dict(CACHE, cache=GOOD, table=GOOD, cu=GOOD, out=GOOD)
    a.update(kw)
    return L.kda_latent_gather(a["cache"], a["table"], a["cu"], a["out"], a["N"], a["T"], a["P"], a["page"],
                               a["max_pages"], a["dl"], a["dp"], None)


def _decode(L, **kw):
    a = dict(CACHE, q=GOOD, cache=GOOD, table=GOOD, lens=GOOD, cu=None, scale=0.1, o=GOOD, lse=GOOD, H=4,
             ws=GOOD, nbytes=1 << 40)
    a.update(kw)
    return L.kda_latent_decode(a["q"], a["cache"], a["table"], a["lens"], a["cu"], a["scale"], a["o"], a["lse"],
                               a["N"], a["T"], a["H"], a["P"], a["page"], a["max_pages"], a["dl"], a["dp"],
                               a["ws"], a["nbytes"], None)


def _prefill(L, **kw):
    a = dict(q=GOOD, kv=GOOD, pe=GOOD, stride=64, cu=GOOD, cuk=GOOD, scale=0.1, causal=1, o=GOOD, lse=GOOD, N=1,
             Tq=3, Tk=5, H=2, dn=128, dp=64, dv=128, ws=GOOD, nbytes=1 << 40)
    a.update(kw)
    return L.kda_latent_prefill(a["q"], a["kv"], a["pe"], a["stride"], a["cu"], a["cuk"], a["scale"],
                                a["causal"], a["o"], a["lse"], a["N"], a["Tq"], a["Tk"], a["H"], a["dn"],
                                a["dp"], a["dv"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("kw,status", BAD_CACHE + [
    (dict(T=3), 2), (dict(eps=-1.0), 8), (dict(eps=float("nan")), 8),
    (dict(x=None), 1), (dict(cache=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(x=OFF4), 4), (dict(w=OFF4), 4), (dict(cu=OFF4), 4)])
def test_append_rejects_bad_arguments(L, kw, status):
    assert _append(L, **kw) == status


@pytest.mark.parametrize("kw,status", BAD_CACHE + [
    (dict(cache=None), 1), (dict(table=None), 1), (dict(cu=None), 1), (dict(out=None), 1), (dict(out=OFF4), 4)])
def test_gather_rejects_bad_arguments(L, kw, status):
    assert _gather(L, **kw) == status


@pytest.mark.parametrize("kw,status", BAD_CACHE + [
    (dict(T=3), 2), (dict(H=0), 2), (dict(H=1 << 30), 2), (dict(scale=0.0), 8), (dict(scale=-1.0), 8),
    (dict(scale=float("inf")), 8), (dict(scale=float("nan")), 8),
    (dict(q=None), 1), (dict(cache=None), 1), (dict(o=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(q=OFF4), 4), (dict(lse=OFF4), 4), (dict(o=OFF4), 4), (dict(ws=ctypes.c_void_p(0x10010)), 4)])
def test_decode_rejects_bad_arguments(L, kw, status):
    assert _decode(L, **kw) == status


def test_decode_workspace(L):
    need = L.kda_latent_decode_workspace_bytes(2, 2, 4, 512, 64)
    for bad in ((0, 2, 4, 512, 64), (2, 0, 4, 512, 64), (2, 2, 0, 512, 64), (2, 2, 4, 256, 64),
                (2, 1 << 30, 4, 512, 64)):
        assert L.kda_latent_decode_workspace_bytes(*bad) == 0
    if need > 0:
        assert _decode(L, ws=None, nbytes=need) == 6
        assert _decode(L, nbytes=need - 1) == 6


@pytest.mark.parametrize("kw,status", [
    (dict(dn=64), 2), (dict(dp=32), 2), (dict(dv=64), 2), (dict(N=0), 2), (dict(H=0), 2), (dict(Tq=-1), 2),
    (dict(Tk=-1), 2), (dict(Tq=1 << 30, H=2), 2), (dict(Tk=1 << 30, H=2), 2), (dict(stride=63), 2),
    (dict(stride=68), 2), (dict(stride=0), 2), (dict(scale=0.0), 8), (dict(scale=float("nan")), 8),
    (dict(causal=2), 8), (dict(ws=ctypes.c_void_p(0x10010)), 4), (dict(q=None), 1), (dict(kv=None), 1), (dict(pe=None), 1), (dict(cu=None), 1),
    (dict(cuk=None), 1), (dict(o=None), 1), (dict(q=OFF4), 4), (dict(pe=OFF4), 4), (dict(lse=OFF4), 4)])
def test_prefill_rejects_bad_arguments(L, kw, status):
    assert _prefill(L, **kw) == status


def test_prefill_workspace(L):
    """None with many work tiles (256 queries of a head each) or few keys; one
    for few queries over many keys."""
    for none in ((1, 4096, 4096, 96, 128, 64, 128), (1, 16, 16, 1, 128, 64, 128), (0, 16, 9000, 1, 128, 64, 128),
                 (1, 0, 9000, 1, 128, 64, 128), (1, 16, 9000, 1, 128, 64, 64), (1, 16, 0, 1, 128, 64, 128),
                 (1, 300, 600, 16, 128, 64, 128), (2, 2024, 18408, 32, 128, 64, 128)):
        assert L.kda_latent_prefill_workspace_bytes(*none) == 0
    need = L.kda_latent_prefill_workspace_bytes(1, 16, 9000, 2, 128, 64, 128)
    pieces = need // (16 * 2 * 129 * 4)
    assert need == pieces * 16 * 2 * 129 * 4 and 2 <= pieces <= 32
    big = dict(Tq=16, Tk=9000)
    assert _prefill(L, ws=None, nbytes=need, **big) == 6
    assert _prefill(L, nbytes=need - 1, **big) == 6


def test_calls_without_tokens_are_noops(L):
    assert _append(L, T=0, N=2, cu=GOOD, x=None) == 0
    assert _gather(L, T=0, out=None) == 0
    assert _decode(L, T=0, N=2, cu=GOOD, q=None, ws=None, nbytes=0) == 0
    assert _prefill(L, Tq=0, q=None) == 0


def test_binding_fails_loudly_without_cuda_tensors():
    torch = pytest.importorskip("torch")
    import kda_linear_attention_gb300 as kda
    bf = torch.bfloat16
    cache, table = torch.zeros(4, 16, 576, dtype=bf), torch.zeros(1, 4, dtype=torch.int32)
    lens, cu = torch.ones(1, dtype=torch.int32), torch.tensor([0, 1], dtype=torch.int32)
    with pytest.raises(ValueError):
        kda.latent_append(torch.zeros(1, 576, dtype=bf), cache, table, lens)
    with pytest.raises(ValueError):
        kda.latent_gather(cache, table, cu, total=1)
    with pytest.raises(ValueError):
        kda.latent_decode(torch.zeros(1, 2, 576, dtype=bf), cache, table, lens)
    with pytest.raises(ValueError):
        kda.latent_prefill(torch.zeros(1, 2, 192, dtype=bf), torch.zeros(1, 2, 256, dtype=bf),
                           torch.zeros(1, 64, dtype=bf), cu)


@pytest.mark.parametrize("T", [1 << 31, 1 << 33, 1 << 61, 1 << 62, (1 << 63) - 1])
def test_lengths_past_32_bits_are_refused(L, T):
    """Token counts whose product with the heads leaves 64 bits, too."""
    for H in (1, 2, 4, 8):
        assert _decode(L, T=T, H=H, cu=GOOD) == 2
        assert _prefill(L, Tq=T, H=H) == 2 and _prefill(L, Tk=T, H=H) == 2 and _prefill(L, Tq=T, Tk=T, H=H) == 2
        assert L.kda_latent_decode_workspace_bytes(2, T, H, 512, 64) == 0
        assert L.kda_latent_prefill_workspace_bytes(1, T, 9000, H, 128, 64, 128) == 0
        assert L.kda_latent_prefill_workspace_bytes(1, 16, T, H, 128, 64, 128) == 0


def test_binding_loads_in_a_torch_without_its_inner_names():
    """The names that the latent calls take from torch._C for speed have
    public stand-ins."""
    import os
    import subprocess
    import sys
    pytest.importorskip("torch")
    script = """
import torch
for n in ("_cuda_cudaCachingAllocator_raw_alloc", "_cuda_cudaCachingAllocator_raw_delete", "_cuda_getDevice",
          "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, n):
        delattr(torch._C, n)
import kda_linear_attention_gb300 as kda
assert kda._raw_alloc is None and kda._raw_free is None
assert kda._current_device is torch.cuda.current_device and callable(kda._current_raw_stream)
address, own = kda._take_workspace(100, torch.zeros(1), None, 0)
assert address == own.data_ptr() and own.numel() == 100 and own.dtype is torch.uint8
kda._give_back(own)
assert kda._take_workspace(0, torch.zeros(1), None, 0) == (None, None)
kda._give_back(None)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", script], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
