"""Host-side checks of the rotary and 4-bit cache calls (no GPU): the C entries
refuse bad arguments before launching anything, calls without tokens are
no-ops, the binding refuses tensors it cannot take, and the tables of turns are
the frequencies they stand for."""
import ctypes
import math

import numpy as np
import pytest

GOOD = ctypes.c_void_p(0x10000)   # aligned, never dereferenced
OFF4 = ctypes.c_void_p(0x10004)
OFF16 = ctypes.c_void_p(0x10010)  # not in whole sectors
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    from kda_linear_attention_gb300 import build
    build.build()
    import kda_linear_attention_gb300 as kda
    return kda.lib()


CACHE = dict(N=2, T=2, P=8, page=64, max_pages=4, dl=512, dp=64)
BAD_CACHE = [(dict(dl=256), 2), (dict(dp=0), 2), (dict(N=0), 2), (dict(T=-1), 2), (dict(T=1 << 31), 2),
             (dict(P=0), 2), (dict(max_pages=0), 2), (dict(page=8), 2), (dict(page=48), 2),
             (dict(page=2048), 2), (dict(P=1 << 25, page=64), 2), (dict(P=1 << 62), 2)]
BAD_ROTATION = [(dict(amp=NAN), 8), (dict(amp=INF), 8), (dict(layout=2), 8), (dict(layout=-1), 8)]
BAD_EXPONENT = [(dict(exponent=33), 8), (dict(exponent=-33), 8), (dict(exponent=1 << 30), 8)]


def _rotate(L, **kw):
    a = dict(x=GOOD, xt=256, xh=64, out=GOOD, ot=256, oh=64, turns=GOOD, lens=GOOD, cu=None, amp=1.0, layout=0,
             inverse=0, N=2, T=2, H=4, d=64, dtype=0)
    a.update(kw)
    return L.kda_latent_rotate(a["x"], a["xt"], a["xh"], a["out"], a["ot"], a["oh"], a["turns"], a["lens"], a["cu"],
                               a["amp"], a["layout"], a["inverse"], a["N"], a["T"], a["H"], a["d"], a["dtype"], None)


def _append_rotated(L, **kw):
    a = dict(CACHE, x=GOOD, cache=GOOD, table=GOOD, lens=GOOD, cu=None, w=None, eps=1e-6, turns=GOOD, amp=1.0, layout=0)
    a.update(kw)
    return L.kda_latent_append_rotated(a["x"], a["cache"], a["table"], a["lens"], a["cu"], a["w"], a["eps"],
                                       a["turns"], a["amp"], a["layout"], a["N"], a["T"], a["P"], a["page"],
                                       a["max_pages"], a["dl"], a["dp"], None)


def _append4(L, **kw):
    a = dict(CACHE, x=GOOD, cache=GOOD, table=GOOD, lens=GOOD, cu=None, w=None, eps=1e-6, turns=None, amp=1.0,
             layout=0, exponent=0)
    a.update(kw)
    return L.kda_latent4_append(a["x"], a["cache"], a["table"], a["lens"], a["cu"], a["w"], a["eps"], a["turns"],
                                a["amp"], a["layout"], a["exponent"], a["N"], a["T"], a["P"], a["page"],
                                a["max_pages"], a["dl"], a["dp"], None)


def _gather4(L, **kw):
    a = dict(CACHE, cache=GOOD, table=GOOD, cu=GOOD, out=GOOD, exponent=0)
    a.update(kw)
    return L.kda_latent4_gather(a["cache"], a["table"], a["cu"], a["out"], a["exponent"], a["N"], a["T"], a["P"],
                                a["page"], a["max_pages"], a["dl"], a["dp"], None)


def _decode4(L, **kw):
    a = dict(CACHE, q=GOOD, cache=GOOD, table=GOOD, lens=GOOD, cu=None, scale=0.1, exponent=0, o=GOOD, lse=GOOD, H=4,
             ws=GOOD, nbytes=1 << 40)
    a.update(kw)
    return L.kda_latent4_decode(a["q"], a["cache"], a["table"], a["lens"], a["cu"], a["scale"], a["exponent"], a["o"],
                                a["lse"], a["N"], a["T"], a["H"], a["P"], a["page"], a["max_pages"], a["dl"],
                                a["dp"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("kw,status", BAD_ROTATION + [
    (dict(dtype=2), 5), (dict(N=0), 2), (dict(T=-1), 2), (dict(T=1 << 31), 2), (dict(T=1 << 62), 2), (dict(T=3), 2),
    (dict(H=0), 2), (dict(H=(1 << 24) + 1), 2), (dict(T=1 << 30, H=4, cu=GOOD), 2), (dict(d=0), 2), (dict(d=24), 2),
    (dict(d=272), 2), (dict(xt=-8), 2), (dict(xt=4), 2), (dict(xh=1 << 31), 2), (dict(ot=100), 2), (dict(oh=-64), 2), (dict(ot=0), 2), (dict(oh=0), 2), (dict(oh=32), 2),
    (dict(dtype=1, xt=2), 2), (dict(inverse=2), 8), (dict(x=None), 1), (dict(out=None), 1), (dict(turns=None), 1),
    (dict(lens=None), 1), (dict(x=OFF4), 4), (dict(out=OFF4), 4), (dict(turns=OFF4), 4), (dict(cu=OFF4), 4)])
def test_rotate_rejects_bad_arguments(L, kw, status):
    assert _rotate(L, **kw) == status


@pytest.mark.parametrize("kw,status", BAD_CACHE + BAD_ROTATION + [
    (dict(T=3), 2), (dict(eps=-1.0), 8), (dict(eps=NAN), 8), (dict(x=None), 1), (dict(cache=None), 1),
    (dict(table=None), 1), (dict(lens=None), 1), (dict(turns=None), 1), (dict(x=OFF4), 4), (dict(w=OFF4), 4),
    (dict(turns=OFF4), 4)])
def test_append_rotated_rejects_bad_arguments(L, kw, status):
    assert _append_rotated(L, **kw) == status


@pytest.mark.parametrize("kw,status", BAD_CACHE + BAD_ROTATION + BAD_EXPONENT + [
    (dict(T=3), 2), (dict(eps=-1.0), 8), (dict(x=None), 1), (dict(cache=None), 1), (dict(table=None), 1),
    (dict(lens=None), 1), (dict(x=OFF4), 4), (dict(cache=OFF16), 4), (dict(turns=OFF4), 4)])
def test_append4_rejects_bad_arguments(L, kw, status):
    assert _append4(L, **kw) == status


@pytest.mark.parametrize("kw,status", BAD_CACHE + BAD_EXPONENT + [
    (dict(cache=None), 1), (dict(table=None), 1), (dict(cu=None), 1), (dict(out=None), 1), (dict(out=OFF4), 4),
    (dict(cache=OFF16), 4)])
def test_gather4_rejects_bad_arguments(L, kw, status):
    assert _gather4(L, **kw) == status


@pytest.mark.parametrize("kw,status", BAD_CACHE + BAD_EXPONENT + [
    (dict(T=3), 2), (dict(H=0), 2), (dict(H=1 << 30), 2), (dict(scale=0.0), 8), (dict(scale=-1.0), 8),
    (dict(scale=INF), 8), (dict(scale=NAN), 8), (dict(q=None), 1), (dict(cache=None), 1), (dict(o=None), 1),
    (dict(table=None), 1), (dict(lens=None), 1), (dict(q=OFF4), 4), (dict(lse=OFF4), 4), (dict(o=OFF4), 4),
    (dict(ws=OFF16), 4), (dict(cache=OFF16), 4)])
def test_decode4_rejects_bad_arguments(L, kw, status):
    assert _decode4(L, **kw) == status


def test_decode4_workspace(L):
    need = L.kda_latent4_decode_workspace_bytes(2, 2, 4, 512, 64)
    for bad in ((0, 2, 4, 512, 64), (2, 0, 4, 512, 64), (2, 2, 0, 512, 64), (2, 2, 4, 256, 64),
                (2, 1 << 30, 4, 512, 64), (2, 1 << 62, 4, 512, 64)):
        assert L.kda_latent4_decode_workspace_bytes(*bad) == 0
    if need > 0:
        assert _decode4(L, ws=None, nbytes=need) == 6
        assert _decode4(L, nbytes=need - 1) == 6


def test_calls_without_tokens_are_noops(L):
    assert _rotate(L, T=0, cu=GOOD, x=None, out=None) == 0
    assert _append_rotated(L, T=0, cu=GOOD, x=None) == 0
    assert _append4(L, T=0, cu=GOOD, x=None) == 0
    assert _gather4(L, T=0, out=None) == 0
    assert _decode4(L, T=0, cu=GOOD, q=None, ws=None, nbytes=0) == 0


def test_binding_fails_loudly_without_cuda_tensors():
    torch = pytest.importorskip("torch")
    import kda_linear_attention_gb300 as kda
    bf = torch.bfloat16
    cache, cache4 = torch.zeros(4, 16, 576, dtype=bf), torch.zeros(4, 16, 416, dtype=torch.uint8)
    table, lens, cu = torch.zeros(1, 4, dtype=torch.int32), torch.ones(1, dtype=torch.int32), torch.tensor([0, 1]).int()
    turns, _ = kda.rotary_turns(device="cpu")
    x = torch.zeros(1, 576, dtype=bf)
    for call in (lambda: kda.latent_rotate(torch.zeros(1, 2, 64, dtype=bf), turns, lens),
                 lambda: kda.latent_append_rotated(x, cache, table, lens, turns),
                 lambda: kda.latent4_append(x, cache4, table, lens),
                 lambda: kda.latent4_gather(cache4, table, cu, total=1),
                 lambda: kda.latent4_decode(torch.zeros(1, 2, 576, dtype=bf), cache4, table, lens)):
        with pytest.raises(ValueError):
            call()


def _radians(turns):
    return turns.numpy().astype(np.uint64).astype(np.float64) * 2.0 ** -64 * 2 * math.pi


WHOLE = 2 * math.pi * 2.0 ** -64     # a table counts whole 2^-64ths of a turn


def test_turns_are_the_frequencies():
    pytest.importorskip("torch")
    import kda_linear_attention_gb300 as kda
    t, amp = kda.rotary_turns(64, base=10000.0, device="cpu")
    f = 10000.0 ** (-np.arange(32) / 32)
    assert amp == 1.0 and t.shape == (32,) and np.allclose(_radians(t), f, rtol=2.0 ** -50, atol=WHOLE)
    t, amp = kda.rotary_turns(64, method="linear", factor=4.0, device="cpu")
    assert amp == 1.0 and np.allclose(_radians(t), f / 4, rtol=2.0 ** -50, atol=WHOLE)
    t, amp = kda.rotary_turns(64, method="ntk", factor=4.0, device="cpu")
    assert np.allclose(_radians(t), (10000.0 * 4.0 ** (64 / 62)) ** (-np.arange(32) / 32), rtol=2.0 ** -48, atol=WHOLE)
    assert np.isclose(_radians(t)[-1], f[-1] / 4, rtol=1e-12)        # the slowest pair as with "linear"
    # negative and large frequencies wrap: whole turns a position are none
    t, _ = kda.rotary_turns(4, frequencies=[-0.5, 2 * math.pi * 3 + 0.25], device="cpu")
    assert np.allclose(_radians(t), [2 * math.pi - 0.5, 0.25], rtol=0, atol=1e-14)


def test_yarn_keeps_fast_pairs_and_divides_slow_ones():
    pytest.importorskip("torch")
    import kda_linear_attention_gb300 as kda
    t, amp = kda.rotary_turns(64, method="yarn", factor=8.0, trained_length=4096, device="cpu")
    f = 10000.0 ** (-np.arange(32) / 32)
    got, turned = _radians(t), 4096 * f / (2 * math.pi)
    assert amp == pytest.approx(0.1 * math.log(8) + 1)
    # whole pairs outside the ramp, whose ends are rounded outwards
    fast, slow = np.flatnonzero(turned > 32)[:-1], np.flatnonzero(turned < 1)[1:]
    assert len(fast) and len(slow)
    assert np.allclose(got[fast], f[fast], rtol=1e-14) and np.allclose(got[slow], f[slow] / 8, rtol=1e-14)
    assert (np.diff(got) < 0).all() and (got <= f * (1 + 1e-14)).all() and (got >= f / 8 * (1 - 1e-14)).all()
    t, amp = kda.rotary_turns(64, method="yarn", factor=1.0, trained_length=4096, device="cpu")
    assert amp == 1.0 and np.allclose(_radians(t), f, rtol=1e-14)


@pytest.mark.parametrize("kw", [dict(d=0), dict(d=63), dict(d=258), dict(base=0.0), dict(base=NAN), dict(factor=0.0),
                                dict(factor=INF), dict(method="none"), dict(method="yarn"), dict(d=2, method="ntk"),
                                dict(method="yarn", trained_length=0), dict(d=4, frequencies=[1.0]),
                                dict(method="yarn", trained_length=10, beta_fast=1.0), dict(d=2, frequencies=[NAN]),
                                dict(d=2, frequencies=[1.0], method="linear")])
def test_turns_refuse_what_they_cannot_hold(kw):
    pytest.importorskip("torch")
    import kda_linear_attention_gb300 as kda
    with pytest.raises(ValueError):
        kda.rotary_turns(device="cpu", **kw)


@pytest.mark.parametrize("kw", [dict(method="yarn", trained_length=4096, base=0.5), dict(frequencies=[1e300] * 32),
                                dict(method="yarn", trained_length=INF), dict(method="ntk", factor=1e300, base=1e300),
                                dict(method="ntk", factor=1e305), dict(method="linear", factor=1e-305),
                                dict(method="yarn", trained_length=64, beta_fast=INF)])
def test_turns_refuse_what_is_out_of_range(kw):
    pytest.importorskip("torch")
    import kda_linear_attention_gb300 as kda
    with pytest.raises(ValueError):
        kda.rotary_turns(device="cpu", **kw)


@pytest.mark.parametrize("length", [1, 4, 6])
def test_yarn_divides_every_pair_of_a_context_below_a_turn(length):
    pytest.importorskip("torch")
    import kda_linear_attention_gb300 as kda
    t, _ = kda.rotary_turns(64, method="yarn", factor=8.0, trained_length=length, device="cpu")
    assert np.allclose(_radians(t), 10000.0 ** (-np.arange(32) / 32) / 8, rtol=1e-14, atol=WHOLE)


@pytest.mark.parametrize("kw,status", [
    (dict(ot=64), 2), (dict(ot=64, oh=64), 2), (dict(ot=248), 2), (dict(ot=64, oh=120), 2),
    (dict(xt=512), 8), (dict(xh=0), 8), (dict(ot=512), 8)])
def test_rotate_rejects_outputs_that_overlap(L, kw, status):
    assert _rotate(L, **kw) == status


def test_rotate_takes_strides_in_either_order(L):
    """Arguments that are right but for a pointer, which is looked at last."""
    assert _rotate(L, ot=64, oh=128, turns=None) == 8       # in place with other strides
    assert _rotate(L, xt=64, xh=128, ot=64, oh=128, turns=None) == 1
    assert _rotate(L, ot=256, oh=64, turns=None) == 1
    assert _rotate(L, xt=0, xh=0, T=1, N=1, H=1, turns=None) == 1


@pytest.mark.parametrize("which", ["x", "out", "view"])
def test_rotate_refuses_tensors_that_require_a_gradient(which):
    torch = pytest.importorskip("torch")
    import kda_linear_attention_gb300 as kda
    x, out = torch.zeros(1, 2, 64), torch.zeros(1, 2, 64)
    turns, lens = torch.zeros(32, dtype=torch.int64), torch.ones(1, dtype=torch.int32)
    if which == "view":
        x = torch.zeros(1, 2, 80, requires_grad=True)[..., 16:]
    else:
        {"x": x, "out": out}[which].requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        kda.latent_rotate(x, turns, lens, out=out)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):     # goes on to the next check
        kda.latent_rotate(x, turns, lens, out=out)


MOST = (1 << 31) - 1


@pytest.mark.parametrize("kw,status", [
    (dict(xt=MOST - 7), 2), (dict(ot=MOST - 7), 2), (dict(xt=MOST - 7, dtype=1), 2), (dict(xt=1 << 30), 2),
    (dict(xt=1 << 29), 1), (dict(ot=1 << 29), 1), (dict(xt=0), 1), (dict(T=1, xt=MOST - 7), 1),
    (dict(T=0, xt=MOST - 7), 0)])
def test_rotate_rejects_rows_past_2_to_the_60_elements(L, kw, status):
    """Two numbers below 2^31 can multiply to more bytes than 63 bits count; all is
    right but for that and a pointer, which is looked at later."""
    a = dict(dict(out=ctypes.c_void_p(0x20000), xt=64, xh=64, ot=64, oh=64, T=MOST, N=1, H=1, cu=GOOD, turns=None), **kw)
    assert _rotate(L, **a) == status
