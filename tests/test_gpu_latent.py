"""GPU parity of latent attention over the paged cache, through the public
calls, against the fp64 oracle: rows written (``latent_append``) and read
back (``latent_gather``), absorbed attention over the pages
(``latent_decode``), expanded attention (``latent_prefill``), and the layer
as they make it together."""
import numpy as np
import pytest

from oracle import latent as ol

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
HALF = 2.0 ** -8            # half a bf16 step, relative


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_linear_attention_gb300 import build
    build.build()
    _kda().device_error(reset=True)
    yield


def _kda():
    import kda_linear_attention_gb300 as kda
    return kda


def _rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def _bf(a):
    """fp64 numpy -> (bf16 device tensor, its exact values as fp64)."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def _i32(a):
    import torch
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


def _np(t):
    return t.detach().double().cpu().numpy()


def _clear(want=0):
    import torch
    torch.cuda.synchronize()
    assert _kda().device_error(reset=True) == want


def check(o, lse, r, what):
    """o and lse against the oracle's result, element by element.

    A score is an fp32 sum of at most 36 products of 16 terms each, exact
    before they are added; an addition is off by at most two units of 2^-23 of
    the row's largest sum |x||k| scale (r.mag), so a score by d = 80 2^-23 mag
    and a probability by the factor 1 +- (2 d + 2^-20) (its own score, the sum
    it is divided by, exponential and reciprocal).  Each probability is then
    rounded to bf16 for its product with the values: independent errors of at
    most HALF p |v|, whose sum exceeds 7 sqrt(sum (HALF p v)^2) with
    probability below 2 e^-24.5 (Hoeffding).  The sum is rounded to bf16
    once.  lse is not touched by the rounded probabilities."""
    o, lse = _np(o), _np(lse)
    d = 80 * 2.0 ** -23 * r.mag
    assert np.array_equal(np.isneginf(lse), np.isneginf(r.lse)), what + ": rows that see nothing"
    live = ~np.isneginf(r.lse)
    err = np.abs(lse[live] - r.lse[live])
    lim = d[live] + 2.0 ** -20 * (1 + np.abs(r.lse[live]))
    assert (err <= lim).all(), "%s: lse off by %.3g (allowed %.3g)" % (what, err.max(), lim[err.argmax()])
    err = np.abs(o - r.o)
    lim = (HALF * np.abs(r.o) + 7 * HALF * r.sqsum) * (1 + HALF) + (2 * d + 2.0 ** -20)[..., None] * r.absum
    bad = ~(err <= lim)
    assert not bad.any(), "%s: %d of %d outputs off, first at %s: %.6g for %.6g (allowed %.3g)" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], o[bad][0], r.o[bad][0], lim[bad][0])


class Paged:
    """A cache of random rows with NaN wherever no sequence has a row."""

    def __init__(self, seed, lens, page, nan=True):
        self.rng = _rng(seed)
        self.lens, self.page = list(lens), page
        self.table, self.P = ol.ragged_pages(self.rng, self.lens, page)
        rows = self.rng.normal(size=(self.P, page, ol.ROW))
        self.dev, self.ref = _bf(rows)
        if nan:
            held = np.zeros((self.P, page), dtype=bool)
            for b, n in enumerate(self.lens):
                p = np.arange(n)
                held[self.table[b, p // page], p % page] = True
            import torch
            self.dev[torch.from_numpy(~held).cuda()] = float("nan")
        self.table_dev = _i32(self.table)
        self.lens_dev = _i32(self.lens)

    def q(self, tokens, H, scale=1.0):
        return _bf(self.rng.normal(size=(tokens, H, ol.ROW)) * scale)


# ------------------------------------------------------------------ append, gather
LENS = [0, 1, 15, 16, 17, 64, 200, 129]


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("norm", [False, True])
def test_append_ragged(page, norm):
    import torch
    kda = _kda()
    c = Paged(11, LENS, page, nan=False)
    news = [0, 1, 15, 3, 0, 64, 130, 2]
    cu = np.cumsum([0] + news)
    x, xr = _bf(c.rng.normal(size=(cu[-1] + 2, ol.ROW)) * 3)      # two tokens behind the last sequence
    w = torch.from_numpy(c.rng.normal(size=512)).float().cuda() if norm else None
    want = ol.append(xr[:cu[-1]], c.ref, c.table, c.lens, cu, None if w is None else _np(w), 1e-6)
    got = kda.latent_append(x, c.dev, c.table_dev, c.lens_dev, _i32(cu), norm_w=w, eps=1e-6)
    assert got is c.dev
    _clear()
    got = _np(got)
    if not norm:
        assert np.array_equal(got, want)
        return
    assert np.array_equal(got[..., 512:], want[..., 512:])
    # one rounding to bf16 of a value computed in a few fp32 steps (2^-20)
    assert (np.abs(got - want) <= (HALF + 2.0 ** -20) * np.abs(want)).all()


def test_append_one_token_a_sequence_equals_the_packed_call():
    import torch
    kda = _kda()
    lens = [1, 16, 17, 100]
    c = Paged(12, lens, 16, nan=False)
    x, _ = _bf(c.rng.normal(size=(4, ol.ROW)))
    w = torch.ones(512, device="cuda")
    a = kda.latent_append(x, c.dev.clone(), c.table_dev, c.lens_dev, norm_w=w)
    b = kda.latent_append(x, c.dev.clone(), c.table_dev, c.lens_dev, _i32([0, 1, 2, 3, 4]), norm_w=w)
    _clear()
    assert torch.equal(a, b) and not torch.equal(a, c.dev)


def test_append_flags_bad_places_and_writes_none_of_them():
    import torch
    kda = _kda()
    c = Paged(13, [20, 20, 20, 20], 16, nan=False)
    x, _ = _bf(c.rng.normal(size=(4, ol.ROW)))
    table = c.table.copy()
    table[0, 1], table[1, 1] = -1, c.P                              # positions 19 of sequences 0 and 1
    before = c.dev.clone()
    kda.latent_append(x, c.dev, _i32(table), c.lens_dev)
    _clear(2)
    keep = torch.ones((c.P, 16), dtype=torch.bool)
    for b in (2, 3):
        row = int(table[b, 1])
        assert torch.equal(c.dev[row, 3].cpu(), x[b].cpu())
        keep[row, 3] = False
    assert torch.equal(c.dev[keep.cuda()], before[keep.cuda()])
    c.dev.copy_(before)                                             # lengths outside the table
    kda.latent_append(x, c.dev, c.table_dev, _i32([0, -5, 16 * c.table.shape[1] + 1, 2 ** 31 - 1]))
    _clear(1)
    assert torch.equal(c.dev, before)


@pytest.mark.parametrize("page", [16, 64])
def test_gather_ragged(page):
    import torch
    kda = _kda()
    c = Paged(14, LENS, page)
    cu = np.cumsum([0] + [n // 2 for n in LENS[:4]] + LENS[4:])
    out = torch.full((cu[-1] + 5, ol.ROW), 7.0, dtype=torch.bfloat16, device="cuda")
    kda.latent_gather(c.dev, c.table_dev, _i32(cu), out=out)
    _clear()
    want = np.concatenate([ol.sequence_rows(c.ref, c.table[b], 0, cu[b + 1] - cu[b]) for b in range(len(LENS))])
    assert np.array_equal(_np(out[:cu[-1]]), want)
    assert (out[cu[-1]:] == 7.0).all()                             # rows behind the last sequence
    again = kda.latent_gather(c.dev, c.table_dev, _i32(cu), total=int(cu[-1]))
    assert torch.equal(again, out[:cu[-1]])


@pytest.mark.parametrize("bad", [[0, 30, 20, 40], [-3, 10, 20, 40], [0, 10, 20, 41]])
def test_broken_offsets_are_flagged_and_touch_nothing_outside(bad):
    """Offsets that decrease or leave [0, T]: bit 0 from every call on them,
    and guard rows around the buffers keep their values."""
    import torch
    kda = _kda()
    c = Paged(16, [40, 40, 40], 16, nan=False)
    cu = _i32(bad)
    guard = torch.full((60, ol.ROW), 7.0, dtype=torch.bfloat16, device="cuda")
    kda.latent_gather(c.dev, c.table_dev, cu, out=guard[10:50])
    _clear(1)
    assert (guard[:10] == 7.0).all() and (guard[50:] == 7.0).all()
    kda.latent_append(guard[10:50], c.dev, c.table_dev, c.lens_dev, cu)
    _clear(1)
    q, _ = c.q(40, 4)
    o = torch.full((60, 4, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((60, 4), 7.0, device="cuda")
    kda.latent_decode(q, c.dev, c.table_dev, c.lens_dev, cu, o=o[10:50], lse=lse[12:52])
    _clear(1)
    assert (o[:10] == 7.0).all() and (o[50:] == 7.0).all() and (lse[:12] == 7.0).all() and (lse[52:] == 7.0).all()


def test_gather_reads_zeros_for_a_bad_page():
    import torch
    kda = _kda()
    c = Paged(15, [40], 16)
    table = c.table.copy()
    table[0, 1] = c.P + 3
    out = kda.latent_gather(c.dev, _i32(table), _i32([0, 40]), total=40)
    _clear(2)
    want = ol.sequence_rows(c.ref, c.table[0], 0, 40).copy()
    want[16:32] = 0
    assert np.array_equal(_np(out), want)


# ------------------------------------------------------------------ decode
def _decode(c, q, cu, **kw):
    return _kda().latent_decode(q, c.dev, c.table_dev, c.lens_dev, None if cu is None else _i32(cu), **kw)


@pytest.mark.parametrize("H", [1, 3, 16, 40, 96, 128])
@pytest.mark.parametrize("page", [16, 64])
def test_decode_one_token(H, page):
    lens = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 300, 1000]
    c = Paged(21, lens, page)
    q, qr = c.q(len(lens), H)
    o, lse = _decode(c, q, None)
    _clear()
    r = ol.decode(qr, c.ref, c.table, lens, np.arange(len(lens) + 1), SCALE)
    check(o, lse, r, "decode H=%d" % H)


@pytest.mark.parametrize("H", [130, 200, 530])
def test_decode_many_heads(H):
    """Three and four row tiles a token, taken side by side, and nine, which
    one CTA takes in turn."""
    lens = [1000, 3, 0, 129, 640]
    c = Paged(30, lens, 64)
    q, qr = c.q(len(lens), H)
    o, lse = _decode(c, q, None)
    _clear()
    check(o, lse, ol.decode(qr, c.ref, c.table, lens, np.arange(len(lens) + 1), SCALE), "decode H=%d" % H)


@pytest.mark.parametrize("H", [1, 5, 16, 96])
def test_decode_ragged_new_tokens(H):
    lens = [5, 130, 0, 64, 257, 3, 128, 140]
    news = [5, 3, 0, 1, 33, 0, 64, 7]
    c = Paged(22, lens, 32)
    cu = np.cumsum([0] + news)
    q, qr = c.q(cu[-1] + 1, H)                                      # one row behind the last sequence
    import torch
    o = torch.full((cu[-1] + 1, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((cu[-1] + 1, H), 7.0, device="cuda")
    _decode(c, q, cu, o=o, lse=lse)
    _clear()
    assert (o[-1] == 7.0).all() and (lse[-1] == 7.0).all()
    r = ol.decode(qr[:-1], c.ref, c.table, lens, cu, SCALE)
    check(o[:-1], lse[:-1], r, "ragged decode H=%d" % H)


def test_decode_more_new_tokens_than_positions():
    """A length shorter than the new tokens: the first ones see nothing."""
    c = Paged(23, [2, 70], 16)
    q, qr = c.q(5 + 3, 4)
    o, lse = _decode(c, q, [0, 5, 8])
    _clear()
    check(o, lse, ol.decode(qr, c.ref, c.table, c.lens, [0, 5, 8], SCALE), "short sequence")
    assert (o[:3] == 0).all() and np.isneginf(_np(lse)[:3]).all()


@pytest.mark.parametrize("lens,H,page", [([5000, 1, 2049], 16, 128), ([9001], 64, 16), ([300] * 200, 8, 64),
                                         ([(37 * i) % 150 for i in range(1000)], 1, 16)])
def test_decode_split_over_positions(lens, H, page):
    """Few long sequences (each split over the SMs) and many short ones."""
    c = Paged(24, lens, page)
    q, qr = c.q(len(lens), H)
    o, lse = _decode(c, q, None)
    _clear()
    check(o, lse, ol.decode(qr, c.ref, c.table, lens, np.arange(len(lens) + 1), SCALE), "split")


@pytest.mark.parametrize("lens,H", [([1300], 16), ([1300], 33), ([700] * 40, 64), ([5000, 4999, 1, 4000], 64),
                                    ([5000, 4999, 1, 4000], 16), ([10000, 9000], 16), ([20000], 5), ([20000], 70)])
def test_decode_joins_pieces(lens, H):
    """Row tiles in 2, 3, 4 to 8, 9 to 32 and more pieces, with few and many
    rows, into buffers that held other numbers before."""
    import torch
    kda = _kda()
    c = Paged(31, lens, 64)
    N = len(lens)
    q, qr = c.q(N, H)
    o = torch.full((N, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((N, H), 7.0, device="cuda")
    ws = torch.full((kda.latent_decode_workspace_bytes(N, N, H),), 0xFF, dtype=torch.uint8, device="cuda")
    _decode(c, q, None, o=o, lse=lse, workspace=ws)
    _clear()
    check(o, lse, ol.decode(qr, c.ref, c.table, lens, np.arange(N + 1), SCALE), "pieces H=%d" % H)


@pytest.mark.parametrize("kind", ["rising", "falling", "spike", "tiny", "flat"])
def test_decode_score_ranges(kind):
    """Scores that rise or fall by hundreds over the positions, one position
    that takes all, and none that stands out: the running maximum moves often,
    once, or never."""
    lens, H = [700, 129], 16
    c = Paged(25, lens, 64, nan=False)
    ref = c.ref.copy()
    u = np.zeros(ol.ROW)
    u[7] = 1.0
    for b, n in enumerate(lens):
        p = np.arange(n)
        ramp = {"rising": p * 2.0, "falling": -p * 2.0, "spike": (p == n // 2) * 3000.0, "tiny": p * 0.0,
                "flat": p * 0.0 + 500.0}[kind]
        ref[c.table[b, p // 64], p % 64, 7] = ramp
    c.dev, c.ref = _bf(ref)
    q, qr = c.q(2, H, scale=1e-3 if kind == "tiny" else 1.0)
    qr = qr.copy()
    qr[:, :, 7] = 13.0
    q, qr = _bf(qr)
    o, lse = _decode(c, q, None)
    _clear()
    check(o, lse, ol.decode(qr, c.ref, c.table, lens, np.arange(3), SCALE), kind)


def test_decode_is_reproducible_and_takes_a_workspace():
    import torch
    kda = _kda()
    c = Paged(26, [3000, 40, 777], 64)
    q, _ = c.q(3, 96)
    o, lse = _decode(c, q, None)
    n = kda.latent_decode_workspace_bytes(3, 3, 96)
    ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        o2, lse2 = _decode(c, q, None, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    _clear()


def test_decode_bad_pages_read_as_zeros():
    kda = _kda()
    c = Paged(27, [300, 100], 64)
    table = c.table.copy()
    table[0, 1], table[1, 0] = -7, 2 ** 31 - 1
    q, qr = c.q(2, 8)
    o, lse = kda.latent_decode(q, c.dev, _i32(table), c.lens_dev)
    _clear(2)
    ref = np.concatenate([c.ref, np.zeros((1, 64, ol.ROW))])        # a page of zeros in their place
    table[0, 1] = table[1, 0] = c.P
    check(o, lse, ol.decode(qr, ref, table, c.lens, np.arange(3), SCALE), "bad pages")


def test_decode_lengths_outside_the_table_are_flagged():
    kda = _kda()
    c = Paged(28, [64, 64], 64)
    q, qr = c.q(2, 4)
    o, lse = kda.latent_decode(q, c.dev, c.table_dev[:, :1].contiguous(), _i32([65, -1]))
    _clear(1)
    r = ol.decode(qr, c.ref, c.table, [64, 0], np.arange(3), SCALE)
    check(o, lse, r, "clamped lengths")


def test_decode_shared_pages():
    """Two sequences whose first pages are the same ones."""
    kda = _kda()
    c = Paged(29, [200, 90], 16, nan=False)
    table = c.table.copy()
    table[1, :4] = table[0, :4]
    q, qr = c.q(2, 16)
    o, lse = kda.latent_decode(q, c.dev, _i32(table), c.lens_dev)
    _clear()
    check(o, lse, ol.decode(qr, c.ref, table, c.lens, np.arange(3), SCALE), "shared pages")


# ------------------------------------------------------------------ prefill
def _prefill_inputs(seed, nq, nk, H, extra=0):
    rng = _rng(seed)
    cu, cuk = np.cumsum([0] + list(nq)), np.cumsum([0] + list(nk))
    q, qr = _bf(rng.normal(size=(cu[-1] + extra, H, 192)))
    kv, kvr = _bf(rng.normal(size=(cuk[-1] + extra, H, 256)))
    pe, per = _bf(rng.normal(size=(cuk[-1] + extra, 64)))
    return cu, cuk, (q, kv, pe), (qr, kvr, per)


@pytest.mark.parametrize("H", [1, 3])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_ragged(H, causal):
    kda = _kda()
    lens = [0, 1, 2, 17, 63, 64, 65, 127, 128, 129, 0, 200, 257, 300]
    cu, _, (q, kv, pe), (qr, kvr, per) = _prefill_inputs(31, lens, lens, H)
    o, lse = kda.latent_prefill(q, kv, pe, _i32(cu), causal=causal)
    _clear()
    check(o, lse, ol.prefill(qr, kvr, per, cu, cu, SCALE, causal), "prefill H=%d" % H)


@pytest.mark.parametrize("causal", [True, False])
def test_prefill_behind_a_context(causal):
    """New tokens behind contexts, more queries than keys, no keys at all; NaN
    behind the last sequence in every input, and output rows there untouched."""
    import torch
    kda = _kda()
    nq, nk, H = [3, 130, 1, 64, 5, 4, 300], [200, 131, 700, 64, 2, 0, 300], 2
    cu, cuk, (q, kv, pe), (qr, kvr, per) = _prefill_inputs(32, nq, nk, H, extra=3)
    for t, n in ((q, cu[-1]), (kv, cuk[-1]), (pe, cuk[-1])):
        t[int(n):] = float("nan")
    o = torch.full((q.shape[0], H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((q.shape[0], H), 7.0, device="cuda")
    kda.latent_prefill(q, kv, pe, _i32(cu), _i32(cuk), causal=causal, o=o, lse=lse)
    _clear()
    n = int(cu[-1])
    assert (o[n:] == 7.0).all() and (lse[n:] == 7.0).all()
    check(o[:n], lse[:n], ol.prefill(qr[:n], kvr, per, cu, cuk, SCALE, causal), "context")


def test_prefill_sequences_do_not_reach_into_each_other():
    """A neighbour of infinities and NaN changes nothing."""
    kda = _kda()
    lens = [70, 90, 140]
    cu, _, (q, kv, pe), (qr, kvr, per) = _prefill_inputs(33, lens, lens, 2)
    for t in (q, kv, pe):
        t[70:160] = float("nan")
        t[100:110] = float("inf")
    o, lse = kda.latent_prefill(q, kv, pe, _i32(cu))
    _clear()
    r = ol.prefill(qr, kvr, per, cu, cu, SCALE)
    for a, b in ((0, 70), (160, 300)):
        part = ol.Result((b - a, 2), 128)
        part.o, part.lse, part.absum, part.sqsum, part.mag = (getattr(r, n)[a:b] for n in
                                                              ("o", "lse", "absum", "sqsum", "mag"))
        check(o[a:b], lse[a:b], part, "rows %d.." % a)


@pytest.mark.parametrize("kind", ["rising", "falling", "spike"])
def test_prefill_score_ranges(kind):
    kda = _kda()
    n, H = 400, 2
    cu, _, (q, kv, pe), (qr, kvr, per) = _prefill_inputs(34, [n], [n], H)
    p = np.arange(n)
    qr, per = qr.copy(), per.copy()
    qr[:, :, 128] = 13.0
    per[:, 0] = {"rising": p * 2.0, "falling": -p * 2.0, "spike": (p == 37) * 3000.0}[kind]
    q, qr = _bf(qr)
    pe, per = _bf(per)
    o, lse = kda.latent_prefill(q, kv, pe, _i32(cu))
    _clear()
    check(o, lse, ol.prefill(qr, kvr, per, cu, cu, SCALE), kind)


def test_prefill_takes_strided_shared_keys():
    import torch
    kda = _kda()
    cu, _, (q, kv, pe), _ = _prefill_inputs(35, [150, 20], [150, 20], 2)
    rows = torch.full((170, ol.ROW), float("nan"), dtype=torch.bfloat16, device="cuda")
    rows[:, 512:] = pe
    a, la = kda.latent_prefill(q, kv, pe, _i32(cu))
    b, lb = kda.latent_prefill(q, kv, rows[:, 512:], _i32(cu))
    _clear()
    assert torch.equal(a, b) and torch.equal(la, lb)
    with pytest.raises(kda.KDAError):
        kda.latent_prefill(q, kv, torch.zeros((170, 68), dtype=torch.bfloat16, device="cuda")[:, :64], _i32(cu))


def test_prefill_many_sequences():
    """More sequences than a block has threads, lengths 0 to 12 and a few long
    ones among them."""
    kda = _kda()
    lens = [(7 * i) % 13 for i in range(1000)]
    lens[17], lens[640], lens[999] = 300, 513, 129
    cu, _, (q, kv, pe), (qr, kvr, per) = _prefill_inputs(37, lens, lens, 1)
    o, lse = kda.latent_prefill(q, kv, pe, _i32(cu))
    _clear()
    check(o, lse, ol.prefill(qr, kvr, per, cu, cu, SCALE), "many sequences")


def test_prefill_more_work_tiles_than_sms():
    """Work tiles taken over by running blocks: a batch whose tiles are several
    times the SMs', against the same heads in smaller calls."""
    import torch
    kda = _kda()
    lens, H = [1, 700, 260, 1300], 64
    cu, _, (q, kv, pe), _ = _prefill_inputs(38, lens, lens, H)
    cu = _i32(cu)
    o, lse = kda.latent_prefill(q, kv, pe, cu)
    for h in (0, 24, 48):
        oh, lh = kda.latent_prefill(q[:, h:h + 16].contiguous(), kv[:, h:h + 16].contiguous(), pe, cu)
        assert torch.equal(oh, o[:, h:h + 16]) and torch.equal(lh, lse[:, h:h + 16])
    for _ in range(3):
        o2, lse2 = kda.latent_prefill(q, kv, pe, cu)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    _clear()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,H", [([5], [9000], 1), ([1, 40, 0, 300], [700, 2500, 100, 300], 2),
                                     ([300], [1000], 3), ([128], [128 * 33 + 1], 4)])
def test_prefill_few_queries_over_many_keys(nq, nk, H, causal):
    """Keys cut into pieces and joined: rows that see none of a piece, pieces
    of sequences shorter than the pieces' number, rows behind the last
    sequence."""
    import torch
    kda = _kda()
    cu, cuk, (q, kv, pe), (qr, kvr, per) = _prefill_inputs(43, nq, nk, H, extra=2)
    n = int(cu[-1])
    assert kda.latent_prefill_workspace_bytes(len(nq), n + 2, int(cuk[-1]) + 2, H) > 0
    o = torch.full((n + 2, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n + 2, H), 7.0, device="cuda")
    kda.latent_prefill(q, kv, pe, _i32(cu), _i32(cuk), causal=causal, o=o, lse=lse)
    _clear()
    assert (o[n:] == 7.0).all() and (lse[n:] == 7.0).all()
    check(o[:n], lse[:n], ol.prefill(qr[:n], kvr, per, cu, cuk, SCALE, causal), "pieces")
    need = kda.latent_prefill_workspace_bytes(len(nq), n + 2, int(cuk[-1]) + 2, H)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    o2, lse2 = kda.latent_prefill(q, kv, pe, _i32(cu), _i32(cuk), causal=causal, workspace=ws)
    _clear()
    assert torch.equal(o2[:n], o[:n]) and torch.equal(lse2[:n], lse[:n])


def test_prefill_output_without_wide_alignment():
    """An output that starts on a 16-byte boundary but not on a 32-byte one."""
    import torch
    kda = _kda()
    cu, _, (q, kv, pe), _ = _prefill_inputs(39, [150], [150], 2)
    want, _ = kda.latent_prefill(q, kv, pe, _i32(cu))
    flat = torch.empty(150 * 2 * 128 + 8, dtype=torch.bfloat16, device="cuda")
    o = flat[8:].view(150, 2, 128)
    assert o.data_ptr() % 32 == 16
    kda.latent_prefill(q, kv, pe, _i32(cu), o=o)
    _clear()
    assert torch.equal(o, want)


def test_prefill_captured_and_replayed():
    import torch
    kda = _kda()
    cu, _, (q, kv, pe), _ = _prefill_inputs(40, [300, 77], [300, 77], 4)
    cu = _i32(cu)
    o, lse = kda.latent_prefill(q, kv, pe, cu)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.latent_prefill(q, kv, pe, cu, o=o, lse=lse)
    for seed in (1, 2):
        nq, nkv = _prefill_inputs(50 + seed, [300, 77], [300, 77], 4)[2][:2]
        q.copy_(nq)
        kv.copy_(nkv)
        g.replay()
        want = kda.latent_prefill(nq, nkv, pe, cu)
        _clear()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_prefill_flags_bad_offsets():
    kda = _kda()
    cu, _, (q, kv, pe), _ = _prefill_inputs(36, [40], [40], 1)
    for bad in ([0, 41], [-1, 40], [30, 20]):
        kda.latent_prefill(q, kv, pe, _i32([0, 40]), _i32(bad))
        _clear(1)


def test_prefill_broken_query_offsets_do_no_work_outside():
    """Offsets that go back and forth claim more queries than there are: the
    call is flagged and rows around the output keep their values."""
    import torch
    kda = _kda()
    T, H, N = 600, 2, 200
    rng = _rng(47)
    (q, _), (kv, _), (pe, _) = (_bf(rng.normal(size=n)) for n in ((T, H, 192), (T, H, 256), (T, 64)))
    cu = _i32([0, T] * (N // 2) + [0])
    o = torch.full((T + 20, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 40, H), 7.0, device="cuda")
    kda.latent_prefill(q, kv, pe, cu, o=o[10:10 + T], lse=lse[16:16 + T])
    _clear(1)
    assert (o[:10] == 7.0).all() and (o[10 + T:] == 7.0).all()
    assert (lse[:16] == 7.0).all() and (lse[16 + T:] == 7.0).all()


# ------------------------------------------------------------------ together
def _layer(seed, H):
    rng = _rng(seed)
    (wk, wkr), (wv, wvr) = (_bf(rng.normal(size=(H, 512, 128)) / 16) for _ in range(2))
    return rng, wk, wkr, wv, wvr


def test_layer_chunked_prefill_then_decode_both_forms():
    """A prompt in two chunks and three decode steps through the cache, each
    chunk attended to in the expanded form (rows gathered, expanded, prefill)
    and in the absorbed one (decode over the pages): the two agree to the
    roundings between them, and the cache holds what was written."""
    import torch
    kda = _kda()
    H, page, N = 4, 16, 3
    rng, wk, wkr, wv, wvr = _layer(41, H)
    total = [90, 33, 200]
    table, P = ol.ragged_pages(rng, [n + 3 for n in total], page)
    table_dev = _i32(table)
    cache = torch.full((P, page, ol.ROW), float("nan"), dtype=torch.bfloat16, device="cuda")
    norm_w = torch.from_numpy(1 + 0.1 * rng.normal(size=512)).float().cuda()
    have = [0, 0, 0]
    for news in ([60, 33, 128], [30, 0, 72], [1, 1, 1], [1, 1, 1], [1, 1, 1]):
        have = [a + b for a, b in zip(have, news)]
        cu, cuk = _i32(np.cumsum([0] + news)), _i32(np.cumsum([0] + have))
        lens = _i32(have)
        x, _ = _bf(rng.normal(size=(sum(news), ol.ROW)))
        q, _ = _bf(rng.normal(size=(sum(news), H, 192)))
        kda.latent_append(x, cache, table_dev, lens, cu, norm_w=norm_w)
        rows = kda.latent_gather(cache, table_dev, cuk, total=sum(have))
        kv = torch.cat([torch.einsum("nc,hcd->nhd", rows[:, :512].float(), w.float()) for w in (wk, wv)], 2)
        oe, le = kda.latent_prefill(q, kv.to(torch.bfloat16).contiguous(), rows[:, 512:], cu, cuk)
        qa = torch.cat([torch.einsum("thd,hcd->thc", q[..., :128].float(), wk.float()), q[..., 128:].float()], 2)
        oa, la = kda.latent_decode(qa.to(torch.bfloat16).contiguous(), cache, table_dev, lens, cu)
        oa = torch.einsum("thc,hcd->thd", oa.float(), wv.float())
        _clear()
        # the roundings to bf16 between the forms (q absorbed; keys and values expanded): errors of a
        # score of at most 2^-8 scale (|qa| . |row| + |q| . |k|), here below 2^-8 * 90, as random signs
        # (7 sqrt(n) instead of n of them): both sides' scores agree to 0.15
        assert (le - la).abs().max() < 0.15
        rel = ((oe.float() - oa).norm() / oa.norm()).item()
        assert rel < 0.03, rel
    assert torch.isnan(cache).any()                                 # what no token owns was never touched


def test_layer_captured_and_replayed():
    """A decode step (append, then attention) captured into a graph and
    replayed with new inputs in place."""
    import torch
    kda = _kda()
    lens = [130, 64, 1, 500]
    c = Paged(42, lens, 64)
    x, _ = _bf(c.rng.normal(size=(4, ol.ROW)))
    q, _ = c.q(4, 16)
    n = kda.latent_decode_workspace_bytes(4, 4, 16)
    ws = torch.empty((max(n, 1),), dtype=torch.uint8, device="cuda")
    o = torch.empty((4, 16, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((4, 16), device="cuda")

    def step():
        kda.latent_append(x, c.dev, c.table_dev, c.lens_dev)
        kda.latent_decode(q, c.dev, c.table_dev, c.lens_dev, o=o, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(3):
        nx, nq = _bf(c.rng.normal(size=(4, ol.ROW)))[0], c.q(4, 16)[0]
        x.copy_(nx)
        q.copy_(nq)
        c.lens_dev.copy_(_i32([m - k % 2 if m > 1 else m for m in lens]))
        g.replay()
        _clear()
        got = o.clone(), lse.clone()
        step()
        _clear()
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)


def test_calls_on_another_stream():
    import torch
    kda = _kda()
    c = Paged(43, [2000, 300], 64)
    q, _ = c.q(2, 16)
    want = _decode(c, q, None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [_decode(c, q, None, stream=s) for _ in range(4)]
    s.synchronize()
    _clear()
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_steps_follow_one_another_closely():
    """Kernels that begin under the end of the one before them see what it
    wrote: 100 decode steps (new rows and queries copied in, append,
    attention, expanded attention of the gathered rows) without a wait between
    them, against the same steps one at a time."""
    import torch
    kda = _kda()
    lens = [200, 64, 1000]
    c = Paged(49, lens, 64, nan=False)
    start = c.dev.clone()
    xs, qs = _bf(c.rng.normal(size=(100, 3, ol.ROW)))[0], _bf(c.rng.normal(size=(100, 3, 16, ol.ROW)))[0]
    pq = _bf(c.rng.normal(size=(3, 2, 192)))[0]
    cu, cuk = _i32([0, 1, 2, 3]), _i32(np.cumsum([0] + lens))
    x, q = torch.empty_like(xs[0]), torch.empty_like(qs[0])

    def steps(wait):
        c.dev.copy_(start)
        out = []
        for i in range(100):
            x.copy_(xs[i])
            q.copy_(qs[i])
            kda.latent_append(x, c.dev, c.table_dev, c.lens_dev)
            out += kda.latent_decode(q, c.dev, c.table_dev, c.lens_dev)
            rows = kda.latent_gather(c.dev, c.table_dev, cuk, total=sum(lens))
            kv = rows[:, :512].reshape(-1, 2, 256).contiguous()
            out += kda.latent_prefill(pq, kv, rows[:, 512:], cu, cuk)
            if wait:
                torch.cuda.synchronize()
        return out

    want = steps(True)
    for _ in range(3):
        for a, b in zip(steps(False), want):
            assert torch.equal(a, b)
    _clear()


def test_decode_captured_with_memory_of_its_own():
    """Two graphs that each take their workspace from the capture's memory."""
    import torch
    kda = _kda()
    c = Paged(50, [700, 90], 64)
    q, _ = c.q(2, 16)
    want = _decode(c, q, None)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _decode(c, q, None)
        graphs.append((g, out))
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    _clear()
    for _, (o, lse) in graphs:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_two_streams_at_once():
    """Decode and prefill calls of two streams in flight together, each with
    its own workspace, give what they give alone."""
    import torch
    kda = _kda()
    c = Paged(45, [3000, 300, 64], 64)
    q, _ = c.q(3, 48)
    want = _decode(c, q, None)
    cu, _, (pq, kv, pe), _ = _prefill_inputs(46, [900, 40], [900, 40], 16)
    cu = _i32(cu)
    pwant = kda.latent_prefill(pq, kv, pe, cu)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got, pgot = [], []
    for _ in range(5):
        for s in streams:
            got.append(_decode(c, q, None, stream=s))
            pgot.append(kda.latent_prefill(pq, kv, pe, cu, stream=s))
    _clear()
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    for o, lse in pgot:
        assert torch.equal(o, pwant[0]) and torch.equal(lse, pwant[1])


def test_c_entries_take_no_lse():
    import torch
    kda = _kda()
    c = Paged(47, [300, 5], 64)
    q, _ = c.q(2, 4)
    want, _ = _decode(c, q, None)
    o = torch.empty_like(want)
    n = kda.latent_decode_workspace_bytes(2, 2, 4)
    ws = torch.empty((n,), dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    assert kda.lib().kda_latent_decode(q.data_ptr(), c.dev.data_ptr(), c.table_dev.data_ptr(), c.lens_dev.data_ptr(),
                                       None, SCALE, o.data_ptr(), None, 2, 2, 4, c.P, 64, c.table.shape[1], 512, 64,
                                       ws.data_ptr(), n, st) == 0
    cu, _, (pq, kv, pe), _ = _prefill_inputs(48, [140], [140], 2)
    cu = _i32(cu)
    pwant, _ = kda.latent_prefill(pq, kv, pe, cu)
    po = torch.empty_like(pwant)
    assert kda.lib().kda_latent_prefill(pq.data_ptr(), kv.data_ptr(), pe.data_ptr(), 64, cu.data_ptr(), cu.data_ptr(),
                                        SCALE, 1, po.data_ptr(), None, 1, 140, 140, 2, 128, 64, 128, None, 0, st) == 0
    _clear()
    assert torch.equal(o, want) and torch.equal(po, pwant)


def test_calls_without_tokens_or_keys():
    import torch
    kda = _kda()
    c = Paged(51, [20, 5], 16, nan=False)
    before = c.dev.clone()
    none, bf = _i32([0, 0, 0]), torch.bfloat16
    kda.latent_append(torch.empty((0, ol.ROW), dtype=bf, device="cuda"), c.dev, c.table_dev, c.lens_dev, none)
    assert kda.latent_gather(c.dev, c.table_dev, none, total=0).shape == (0, ol.ROW)
    o, lse = kda.latent_decode(torch.empty((0, 4, ol.ROW), dtype=bf, device="cuda"), c.dev, c.table_dev, c.lens_dev, none)
    assert o.shape == (0, 4, 512) and lse.shape == (0, 4)
    _clear()
    assert torch.equal(c.dev, before)
    q, kv, pe = _prefill_inputs(52, [3, 4], [0, 0], 2)[2]
    o, lse = kda.latent_prefill(q, kv, pe, _i32([0, 3, 7]), none)       # queries without any key
    _clear()
    assert (o == 0).all() and torch.isneginf(lse).all()
    o, lse = kda.latent_prefill(q[:0], kv, pe, none, none)
    assert o.shape == (0, 2, 128)


def test_binding_refuses_wrong_tensors():
    import torch
    kda = _kda()
    c = Paged(44, [20], 16)
    q, _ = c.q(1, 4)
    two, _ = c.q(2, 4)
    with pytest.raises(TypeError):
        kda.latent_decode(q.float(), c.dev, c.table_dev, c.lens_dev)
    with pytest.raises(TypeError):
        kda.latent_decode(q, c.dev, c.table_dev.long(), c.lens_dev)
    with pytest.raises(ValueError):
        kda.latent_decode(q, c.dev[:, :, :512], c.table_dev, c.lens_dev)
    with pytest.raises(ValueError):
        kda.latent_decode(q, c.dev, c.table_dev, _i32([20, 20]))
    with pytest.raises(ValueError):
        kda.latent_decode(two.transpose(0, 1), c.dev, c.table_dev, c.lens_dev)
    with pytest.raises(ValueError):
        kda.latent_gather(c.dev, c.table_dev, _i32([0, 20]))
    with pytest.raises(kda.KDAError):
        kda.latent_decode(q, c.dev.view(-1, 8, 576), c.table_dev, c.lens_dev)
    with pytest.raises(kda.KDAError):
        kda.latent_decode(q, c.dev, c.table_dev, c.lens_dev, scale=-1.0)


# ------------------------------------------------------------------ queries that are not finite
KINDS = ["nan", "inf", "-inf", "both", "low", "high"]


def _poison(qr, rows, channel):
    """Copy of queries [T, H, d] whose rows (token, head) hold NaN or
    infinities.  Keys are negative in `channel`, so +inf there makes every
    score -inf ("low") and -inf every one +inf ("high")."""
    qr = qr.copy()
    for k, (t, h) in enumerate(rows):
        kind = KINDS[k % len(KINDS)]
        if kind == "nan":
            qr[t, h, 3] = np.nan
        elif kind == "both":
            qr[t, h, 3], qr[t, h, 100] = np.inf, -np.inf
        elif kind in ("inf", "-inf"):
            qr[t, h, 60] = float(kind)
        else:
            qr[t, h, channel] = np.inf if kind == "low" else -np.inf
    return qr


def _check_poisoned(o, lse, r, rows, low, sees, what):
    """Rows of finite queries as ever; the poisoned ones, where they see
    anything, NaN in every channel, with a NaN log-sum-exp unless all of their
    scores are -inf (ln 0); o = 0 and lse = -inf where they see nothing."""
    bad = np.zeros(r.lse.shape, dtype=bool)
    for t, h in rows:
        bad[t, h] = True
    part = ol.Result((1, 1), 1)
    part.o, part.lse, part.absum, part.sqsum, part.mag = (getattr(r, n)[~bad] for n in
                                                          ("o", "lse", "absum", "sqsum", "mag"))
    clean = (~bad).tolist()
    import torch
    clean = torch.tensor(clean, device=o.device)
    check(o[clean], lse[clean], part, what)
    o, lse = _np(o), _np(lse)
    for t, h in rows:
        at = "%s: row (%d, %d)" % (what, t, h)
        if sees[t] <= 0:
            assert (o[t, h] == 0).all() and np.isneginf(lse[t, h]), at + " sees nothing"
        else:
            assert np.isnan(o[t, h]).all(), at + ": o"
            assert np.isneginf(lse[t, h]) if (t, h) in low else np.isnan(lse[t, h]), at + ": lse"


def _spread_rows(rng, T, H, n):
    """n rows (token, head) in no order, the first and last token's among them."""
    n = min(n, T * H)
    flat = [0, T * H - 1] + [int(x) for x in rng.permutation(np.arange(1, T * H - 1))]
    return [(x // H, x % H) for x in flat[:n]]


@pytest.mark.parametrize("lens,news,H,page", [
    ([40, 129, 700, 2, 128, 1], [4, 3, 5, 5, 1, 1], 4, 16),       # tiles in one piece and in several
    ([300] * 200, [1] * 200, 5, 64), ([9001, 5000], [1, 1], 16, 64), ([20000], [2], 6, 128),
    ([700, 200, 150], [1, 230, 2], 2, 64)])                       # rows that see nothing, of a tile in pieces
def test_decode_of_queries_that_are_not_finite(lens, news, H, page):
    import torch
    c = Paged(61, lens, page)
    c.ref[:, :, 7] = -np.abs(c.ref[:, :, 7]) - 0.5
    c.ref = torch.from_numpy(c.ref).to(torch.bfloat16).double().numpy()
    c.dev[:, :, 7] = torch.where(torch.isnan(c.dev[:, :, 7]), c.dev[:, :, 7],
                                 torch.from_numpy(c.ref[:, :, 7]).to(torch.bfloat16).cuda())
    cu = np.cumsum([0] + news)
    _, qr = c.q(cu[-1], H)
    rows = _spread_rows(c.rng, int(cu[-1]), H, 12)
    rows += [(int(cu[b]), 0) for b in range(len(lens)) if news[b] > lens[b] and (int(cu[b]), 0) not in rows]
    q, qr = _bf(_poison(qr, rows, 7))
    o, lse = _decode(c, q, None if set(news) == {1} else cu)
    _clear()
    with np.errstate(all="ignore"):
        r = ol.decode(qr, c.ref, c.table, lens, cu, SCALE)
    sees = np.concatenate([m - n + 1 + np.arange(n) for m, n in zip(lens, news)])
    low = {rows[k] for k in range(len(rows)) if KINDS[k % len(KINDS)] == "low"}
    for t, h in rows:                                              # what a single score's sign leaves
        if sees[t] > 0 and not np.isnan(qr[t, h]).any():
            b = int(np.searchsorted(cu, t, side="right")) - 1
            with np.errstate(all="ignore"):
                s = ol.sequence_rows(c.ref, c.table[b], 0, int(sees[t])) @ qr[t, h]
            if np.isneginf(s).all():
                low.add((t, h))
    _check_poisoned(o, lse, r, rows, low, sees, "decode")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,H", [([40, 70, 300, 5, 1], [40, 200, 300, 2, 1], 3), ([5, 3], [9000, 1], 1),
                                     ([1, 40, 0, 300], [700, 2500, 100, 300], 2), ([600], [500], 2)])
def test_prefill_of_queries_that_are_not_finite(nq, nk, H, causal):
    kda = _kda()
    cu, cuk, _, (qr, kvr, per) = _prefill_inputs(62, nq, nk, H)
    per = per.copy()
    per[:, 2] = -np.abs(per[:, 2]) - 0.5
    rng = _rng(63)
    rows = _spread_rows(rng, int(cu[-1]), H, 12)
    (q, qr), (kv, kvr), (pe, per) = _bf(_poison(qr, rows, 130)), _bf(kvr), _bf(per)
    o, lse = kda.latent_prefill(q, kv, pe, _i32(cu), _i32(cuk), causal=causal)
    _clear()
    with np.errstate(all="ignore"):
        r = ol.prefill(qr, kvr, per, cu, cuk, SCALE, causal)
    sees = np.concatenate([m - n + 1 + np.arange(n) if causal else np.full(n, m) for m, n in zip(nk, nq)])
    low = {rows[k] for k in range(len(rows)) if KINDS[k % len(KINDS)] == "low"}
    for t, h in rows:
        if sees[t] > 0 and not np.isnan(qr[t, h]).any():
            b = int(np.searchsorted(cu, t, side="right")) - 1
            k0 = int(cuk[b])
            key = np.concatenate([kvr[k0:k0 + int(sees[t]), h, :128], per[k0:k0 + int(sees[t])]], 1)
            with np.errstate(all="ignore"):
                if np.isneginf(key @ qr[t, h]).all():
                    low.add((t, h))
    _check_poisoned(o, lse, r, rows, low, sees, "prefill")


# ------------------------------------------------------------------ rows of others beside a sequence's
def _others(q, at, seed):
    """Contents for the queries `at`: zeros, scores that run by hundreds, infinities, NaN."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    for scale in (0.0, 30.0, -30.0, float("inf"), float("nan")):
        wild = torch.randn(q[at].shape, generator=gen, device="cuda")
        yield (wild * scale if abs(scale) < 100 else torch.full_like(wild, scale)).to(q.dtype)


@pytest.mark.parametrize("H", [5, 20])
@pytest.mark.parametrize("lens,news", [([700] * 200, [1] * 200), ([900, 30] * 150, [2, 1] * 150), ([9000], [1])])
def test_decode_takes_nothing_from_other_rows(lens, news, H):
    """A tile's columns that another sequence or none holds: their contents
    leave a sequence's bits alone, however their scores run."""
    import torch
    c = Paged(64, lens, 64)
    cu = np.cumsum([0] + news)
    n = int(cu[-1])
    q, _ = c.q(n + 3, H)
    kept = [t for b in range(0, len(lens), 2) for t in range(cu[b], cu[b + 1])]
    others = [t for t in range(n + 3) if t not in set(kept)]
    for kept, others in ((kept, others), (list(range(n)), [n, n + 1, n + 2])):
        kept, others = torch.tensor(kept, device="cuda"), torch.tensor(others, device="cuda")
        want = None
        for k, x in enumerate(_others(q, others, 70)):
            q[others] = x
            o, lse = _decode(c, q, cu)
            _clear()
            if want is None:
                want = o[kept], lse[kept]
            assert torch.equal(o[kept], want[0]) and torch.equal(lse[kept], want[1]), k
        q[others] = torch.ones_like(q[others])


@pytest.mark.parametrize("nq,nk,H", [([40], [380], 2), ([7, 130, 1], [350, 300, 200], 3), ([3], [9000], 1)])
def test_prefill_takes_nothing_from_other_rows(nq, nk, H):
    import torch
    kda = _kda()
    cu, cuk, (q, kv, pe), _ = _prefill_inputs(65, nq, nk, H, extra=20)
    n = int(cu[-1])
    for b in range(len(nq)):                                       # each sequence among others, then padding
        kept = slice(int(cu[b]), int(cu[b + 1]))
        others = torch.tensor([t for t in range(n + 20) if not cu[b] <= t < cu[b + 1]], device="cuda")
        want = None
        for k, x in enumerate(_others(q, others, 71)):
            q[others] = x
            o, lse = kda.latent_prefill(q, kv, pe, _i32(cu), _i32(cuk))
            _clear()
            if want is None:
                want = o[kept].clone(), lse[kept].clone()
            assert torch.equal(o[kept], want[0]) and torch.equal(lse[kept], want[1]), (b, k)
        q[others] = torch.ones_like(q[others])


# ------------------------------------------------------------------ wide pages, uncut key loops
@pytest.mark.parametrize("page", [256, 512, 1024])
def test_pages_wider_than_a_tile_of_positions(page):
    """Append, gather and both forms of decode on pages that hold several
    tiles of positions, lengths around the tiles' and the pages' borders."""
    import torch
    kda = _kda()
    lens = [1, 127, 129, page - 1, page, page + 1, 2 * page + 130, 5 * page // 2, 0]
    news = [1, 3, 0, 2, 129, 2, 131, 1, 0]
    c = Paged(66, lens, page, nan=False)
    cu = np.cumsum([0] + news)
    n = int(cu[-1])
    x, xr = _bf(c.rng.normal(size=(n, ol.ROW)))
    c.ref = ol.append(xr, c.ref, c.table, lens, cu)
    kda.latent_append(x, c.dev, c.table_dev, c.lens_dev, _i32(cu))
    _clear()
    assert np.array_equal(_np(c.dev), c.ref)
    held = np.zeros((c.P, page), dtype=bool)
    for b, m in enumerate(lens):
        p = np.arange(m)
        held[c.table[b, p // page], p % page] = True
    c.dev[torch.from_numpy(~held).cuda()] = float("nan")
    cuk = np.cumsum([0] + lens)
    rows = kda.latent_gather(c.dev, c.table_dev, _i32(cuk), total=int(cuk[-1]))
    _clear()
    assert np.array_equal(_np(rows), np.concatenate([ol.sequence_rows(c.ref, c.table[b], 0, m)
                                                     for b, m in enumerate(lens)]))
    for H, offsets in ((5, cu), (16, None), (70, None)):
        at = np.arange(len(lens) + 1) if offsets is None else offsets
        q, qr = c.q(int(at[-1]), H)
        o, lse = _decode(c, q, offsets)
        _clear()
        check(o, lse, ol.decode(qr, c.ref, c.table, lens, at, SCALE), "page %d, H=%d" % (page, H))


@pytest.mark.parametrize("lens,ctx,H", [([4096], 0, 96), ([1024, 1000], 8192, 32), ([1, 700, 260, 1300], 0, 64),
                                        ([300, 257], 2500, 96)])
def test_prefill_uncut_against_the_oracle(lens, ctx, H):
    """Many work tiles of many key tiles, taken over by running blocks, heads
    in several groups: rows of first, middle and last tokens and heads."""
    import torch
    kda = _kda()
    gen = torch.Generator(device="cuda").manual_seed(67)
    cu, cuk = np.cumsum([0] + lens), np.cumsum([0] + [m + ctx for m in lens])

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)

    q, kv, pe = normal(cu[-1], H, 192), normal(cuk[-1], H, 256), normal(cuk[-1], 64)
    assert kda.latent_prefill_workspace_bytes(len(lens), int(cu[-1]), int(cuk[-1]), H) == 0
    o, lse = kda.latent_prefill(q, kv, pe, _i32(cu), _i32(cuk))
    _clear()
    per = _np(pe)
    for h in (0, 1, H // 2 - 1, H // 2, H - 2, H - 1):
        qh, kvh = _np(q[:, h]), _np(kv[:, h])
        for b, m in enumerate(lens):
            k0 = int(cuk[b])
            key = np.concatenate([kvh[k0:k0 + m + ctx, :128], per[k0:k0 + m + ctx]], 1)
            value = kvh[k0:k0 + m + ctx, 128:]
            toks = sorted({i for i in (0, 1, 127, 128, 255, 256, m // 2, m - 257, m - 2, m - 1) if 0 <= i < m})
            r = ol.Result((len(toks), 1), 128)
            for k, i in enumerate(toks):
                r.put(k, 0, qh[cu[b] + i], key[:ctx + i + 1], value[:ctx + i + 1], SCALE)
            at = torch.tensor([int(cu[b]) + i for i in toks], device="cuda")
            check(o[at, h:h + 1], lse[at, h:h + 1], r, "uncut, head %d, sequence %d" % (h, b))


def test_calls_without_torchs_inner_names(monkeypatch):
    """Workspaces as tensors and torch's public names: the same bits, on
    another stream and in a graph too."""
    import torch
    kda = _kda()
    c = Paged(68, [3000, 300], 64)
    q, _ = c.q(2, 16)
    cu, cuk, (pq, kv, pe), _ = _prefill_inputs(69, [5], [9000], 2)
    cu, cuk = _i32(cu), _i32(cuk)
    want = _decode(c, q, None) + kda.latent_prefill(pq, kv, pe, cu, cuk)
    monkeypatch.setattr(kda, "_raw_alloc", None)
    monkeypatch.setattr(kda, "_raw_free", None)
    monkeypatch.setattr(kda, "_current_device", torch.cuda.current_device)
    monkeypatch.setattr(kda, "_current_raw_stream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [_decode(c, q, None, stream=t) + kda.latent_prefill(pq, kv, pe, cu, cuk, stream=t)
           for t in (None, s, s, None)]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got.append(_decode(c, q, None) + kda.latent_prefill(pq, kv, pe, cu, cuk))
    g.replay()
    _clear()
    for some in got:
        for a, b in zip(some, want):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Caches, queries, outputs, keys and values of more than 4 GB, with the
    rows that are used at their ends."""
    import torch
    kda = _kda()
    rng, bf = _rng(72), torch.bfloat16
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    page, P, L = 64, 70_000, 300                                   # 5.2 GB
    cache = torch.empty((P, page, ol.ROW), dtype=bf, device="cuda")
    table = np.array([[P - 1 - 3 * i for i in range(5)], [P - 2 - 3 * i for i in range(5)]])
    x, xr = _bf(rng.normal(size=(2 * L, ol.ROW)))
    kda.latent_append(x, cache, _i32(table), _i32([L, L]), _i32([0, L, 2 * L]))
    assert torch.equal(kda.latent_gather(cache, _i32(table), _i32([0, L, 2 * L]), total=2 * L), x)
    T, H = 45_000, 96                                              # 5.0 GB of queries, 4.4 GB of outputs
    q = torch.empty((T, H, ol.ROW), dtype=bf, device="cuda")
    held, heldr = _bf(rng.normal(size=(3, H, ol.ROW)))
    q[-3:] = held
    o = torch.full((T, H, 512), 7.0, dtype=bf, device="cuda")
    o, lse = kda.latent_decode(q, cache, _i32(table), _i32([L, L]), _i32([T - 3, T - 2, T]), o=o)
    _clear()
    r = ol.Result((3, H), 512)
    for t, (b, n) in enumerate(((0, L), (1, L - 1), (1, L))):
        for h in range(H):
            r.put(t, h, heldr[t, h], xr[b * L:b * L + n], xr[b * L:b * L + n, :512], SCALE)
    check(o[-3:], lse[-3:], r, "decode")
    assert (o[:10] == 7.0).all() and (o[-13:-3] == 7.0).all()
    del q, o, cache
    Tq, Tk, nq, nk = 120_000, 100_000, 40, 400                     # 4.4 GB of queries, 4.9 GB of keys and values
    q = torch.empty((Tq, H, 192), dtype=bf, device="cuda")
    kv = torch.empty((Tk, H, 256), dtype=bf, device="cuda")
    pe = torch.empty((Tk, 64), dtype=bf, device="cuda")
    (hq, hqr), (hkv, hkvr), (hpe, hper) = (_bf(rng.normal(size=s)) for s in ((nq, H, 192), (nk, H, 256), (nk, 64)))
    q[-nq:], kv[-nk:], pe[-nk:] = hq, hkv, hpe
    o = torch.full((Tq, H, 128), 7.0, dtype=bf, device="cuda")
    o, lse = kda.latent_prefill(q, kv, pe, _i32([Tq - nq, Tq]), _i32([Tk - nk, Tk]), o=o)
    _clear()
    check(o[-nq:], lse[-nq:], ol.prefill(hqr, hkvr, hper, [0, nq], [0, nk], SCALE), "prefill")
    assert (o[:10] == 7.0).all() and (o[-nq - 10:-nq] == 7.0).all()


def test_decode_of_few_tokens_among_many_sequences():
    """Far more sequences than new tokens: tiles of 16 rows, several a token."""
    kda = _kda()
    N, H, lens = 400, 96, [(13 * i) % 90 for i in range(400)]
    lens[7], lens[399] = 700, 260
    news = [0] * N
    news[7], news[100], news[399] = 2, 1, 1
    c = Paged(73, lens, 16)
    cu = np.cumsum([0] + news)
    q, qr = c.q(int(cu[-1]), H)
    o, lse = _decode(c, q, cu)
    _clear()
    check(o, lse, ol.decode(qr, c.ref, c.table, lens, cu, SCALE), "few tokens")


@pytest.mark.parametrize("nq,Tk", [(5, 9000), (40, 200)])
def test_prefill_over_a_broken_range_of_keys_sees_nothing(nq, Tk):
    """In pieces and whole: a flagged key range counts as none."""
    kda = _kda()
    cu, _, (q, kv, pe), _ = _prefill_inputs(74, [nq], [Tk], 2)
    assert (kda.latent_prefill_workspace_bytes(1, nq, Tk, 2) > 0) == (Tk == 9000)
    for bad in ([0, Tk + 1], [-1, Tk], [Tk, 5]):
        o, lse = kda.latent_prefill(q, kv, pe, _i32(cu), _i32(bad))
        _clear(1)
        assert (o == 0).all() and np.isneginf(_np(lse)).all(), bad
