"""GPU parity of the rotary calls and of the 4-bit latent cache, through the
public calls, against the fp64 oracle: rows rotated (``latent_rotate``,
``latent_append_rotated``), quantised (``latent4_append``), read back
(``latent4_gather``) and attended to (``latent4_decode``), and a layer's steps
as they make it together."""
import numpy as np
import pytest

from oracle import latent as ol
from oracle import latent4 as o4

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
HALF = 2.0 ** -8            # half a bf16 step, relative
HALF16 = 2.0 ** -11         # half an fp16 step, relative


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


def _to(a, dtype):
    """fp64 numpy -> (device tensor, its exact values as fp64)."""
    t = _torch().from_numpy(np.ascontiguousarray(a)).to(dtype)
    return t.cuda(), t.double().numpy()


def _torch():
    import torch
    return torch


def _bf(a):
    return _to(a, _torch().bfloat16)


def _i32(a):
    return _torch().tensor(np.asarray(a), dtype=_torch().int32).cuda()


def _np(t):
    return t.detach().double().cpu().numpy()


def _clear(want=0):
    _torch().cuda.synchronize()
    assert _kda().device_error(reset=True) == want


def check(o, lse, r, what, seen=1 << 12):
    """o and lse against the oracle's result, element by element.

    A score is an fp32 sum of 36 products of 16 terms each, exact before they
    are added; an addition is off by at most two units of 2^-23 of the row's
    largest sum |x||k| scale (r.mag), so a score by d = 80 2^-23 mag and a
    probability by the factor 1 +- (2 d + 2^-20) (its own score, the sum it is
    divided by, exponential and reciprocal).  Each probability may then be
    rounded to fp16 for its product with the values: independent errors of at
    most HALF16 p |v|, whose sum exceeds 7 sqrt(sum (HALF16 p v)^2) with
    probability below 2 e^-24.5 (Hoeffding); those below fp16's normal numbers,
    with the row's largest at 2^7 or above, by 2^-32 of it at most, over `seen`
    positions of magnitudes up to vmax.  The sum is rounded to bf16 once.  lse
    is not touched by the rounded probabilities."""
    o, lse = _np(o), _np(lse)
    d = 80 * 2.0 ** -23 * r.mag
    assert np.array_equal(np.isneginf(lse), np.isneginf(r.lse)), what + ": rows that see nothing"
    live = ~np.isneginf(r.lse)
    err = np.abs(lse[live] - r.lse[live])
    lim = d[live] + 2.0 ** -20 * (1 + np.abs(r.lse[live]))
    assert (err <= lim).all(), "%s: lse off by %.3g (allowed %.3g)" % (what, err.max(), lim[err.argmax()])
    err = np.abs(o - r.o)
    vmax = r.absum.max() * 16 if r.absum.size else 0.0
    lim = ((HALF * np.abs(r.o) + 7 * HALF16 * r.sqsum) * (1 + HALF) + (2 * d + 2.0 ** -20)[..., None] * r.absum
           + 2.0 ** -32 * seen * vmax)
    bad = ~(err <= lim)
    assert not bad.any(), "%s: %d of %d outputs off, first at %s: %.6g for %.6g (allowed %.3g)" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], o[bad][0], r.o[bad][0], lim[bad][0])


# ------------------------------------------------------------------ rotary
BF16, F32 = "bfloat16", "float32"


def _rotation_limit(x, y, amplitude, half, interleaved):
    """An angle is off by 2^-22 at a position of 2^30 (two fp64 roundings of the
    table's frequency) and by 2^-23.4 for its part of a turn in fp32 (2^-25 of
    half a turn), sincospi by 2^-23, the three products and the amplitude by
    2^-24 each: below 2^-20 of |x_a| + |x_b| in all, and one rounding."""
    mag = np.abs(x)
    if interleaved:
        both = np.repeat(mag[..., 0::2] + mag[..., 1::2], 2, axis=-1)
    else:
        h = x.shape[-1] // 2
        both = np.concatenate([mag[..., :h] + mag[..., h:]] * 2, axis=-1)
    return (half * np.abs(y) + 2.0 ** -20 * abs(amplitude) * both) * (1 + half)


LENS = [5, 0, 70, 33, 1 << 30, 4000]
NEWS = [5, 0, 1, 20, 7, 34]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,H", [(64, 3), (16, 1), (64, 96), (256, 5), (48, 200)])
def test_rotate_ragged(d, H, dtype, interleaved, inverse):
    """In place on a part of the heads; the rest, and rows behind the last
    sequence, keep their bits."""
    torch, kda = _torch(), _kda()
    rng, cu = _rng(d + H), np.cumsum([0] + NEWS)
    T, at, W = int(cu[-1]), 8, d + 24
    x, xr = _to(rng.normal(size=(T + 2, H, W)), getattr(torch, dtype))
    before, amplitude = x.clone(), 1.25
    turns, _ = kda.rotary_turns(d, base=5e5)
    part = x[..., at:at + d]
    got = kda.latent_rotate(part, turns, _i32(LENS), _i32(cu), amplitude=amplitude, interleaved=interleaved,
                            inverse=inverse)
    _clear()
    assert got is part
    xr = xr[:T, :, at:at + d]
    want = o4.rotate(xr, o4.positions(LENS, cu), o4.frequencies(d, 5e5), amplitude, interleaved, inverse)
    half = HALF if dtype == BF16 else 2.0 ** -24
    assert (np.abs(_np(x[:T, :, at:at + d]) - want) <= _rotation_limit(xr, want, amplitude, half, interleaved)).all()
    x[:T, :, at:at + d] = before[:T, :, at:at + d]
    assert torch.equal(x, before)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotate_into_another_tensor(interleaved):
    """The expanded queries' last part into the absorbed queries' place: other
    strides; one new token a sequence without offsets."""
    torch, kda = _torch(), _kda()
    N, H, lens = 70, 6, [(17 * i) % 900 + 1 for i in range(70)]
    q, qr = _bf(_rng(3).normal(size=(N, H, 192)))
    out = torch.full((N, H, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    turns, _ = kda.rotary_turns()
    kept = q.clone()
    got = kda.latent_rotate(q[..., 128:], turns, _i32(lens), out=out[..., 512:], interleaved=interleaved)
    _clear()
    assert got.data_ptr() == out[..., 512:].data_ptr() and torch.equal(q, kept) and (out[..., :512] == 7.0).all()
    want = o4.rotate(qr[..., 128:], np.array(lens) - 1, o4.frequencies(64, 1e4), 1.0, interleaved)
    assert (np.abs(_np(got) - want) <= _rotation_limit(qr[..., 128:], want, 1.0, HALF, interleaved)).all()
    packed = kda.latent_rotate(q[..., 128:], turns, _i32(lens), _i32(np.arange(N + 1)), out=torch.empty_like(q)[..., 128:],
                               interleaved=interleaved)
    assert torch.equal(packed, got)
    # transposed memory: heads further apart than tokens
    swapped = q[..., 128:].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(kda.latent_rotate(swapped, turns, _i32(lens), interleaved=interleaved), got)


def test_rotate_one_token_and_none():
    torch, kda = _torch(), _kda()
    turns, _ = kda.rotary_turns(16)
    for H in (1, 2):
        x, xr = _to(_rng(H).normal(size=(1, H, 16)), torch.float32)
        kda.latent_rotate(x, turns, _i32([1]))                       # position 0
        assert np.array_equal(_np(x), xr)
    empty = torch.empty((0, 3, 16), device="cuda")
    assert kda.latent_rotate(empty, turns, _i32([4]), _i32([0, 0])) is empty
    _clear()


def test_rotate_a_row_for_all_heads():
    """A broadcast input into a dense output; in place it is refused."""
    torch, kda = _torch(), _kda()
    turns, _ = kda.rotary_turns()
    x, _ = _bf(_rng(9).normal(size=(5, 1, 64)))
    lens, cu = _i32([40]), _i32([0, 5])
    wide = x.expand(5, 7, 64)
    got = kda.latent_rotate(wide, turns, lens, cu, out=torch.empty((5, 7, 64), dtype=x.dtype, device="cuda"))
    _clear()
    assert torch.equal(got, kda.latent_rotate(x.clone(), turns, lens, cu).expand(5, 7, 64))
    before = x.clone()
    with pytest.raises(kda.KDAError):
        kda.latent_rotate(wide, turns, lens, cu)
    assert torch.equal(x, before)


def test_rotate_flags_bad_positions_and_offsets():
    torch, kda = _torch(), _kda()
    turns, _ = kda.rotary_turns()
    x, _ = _bf(_rng(4).normal(size=(6, 2, 64)))
    before = x.clone()
    kda.latent_rotate(x, turns, _i32([2, -1]), _i32([0, 4, 6]))      # tokens at -2, -1, 0, 1 and -3, -2
    _clear(1)
    assert torch.equal(x[[0, 1, 4, 5]], before[[0, 1, 4, 5]]) and torch.equal(x[2], before[2])
    assert not torch.equal(x[3], before[3])
    guard = torch.full((40, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    for bad in ([0, 30, 20], [-3, 10, 20], [0, 10, 21]):
        kda.latent_rotate(guard[10:30], turns, _i32([50, 50]), _i32(bad))
        _clear(1)
        assert (guard[:10] == 7.0).all() and (guard[30:] == 7.0).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_is_the_gradient(interleaved):
    """<rotate(x), g> = <x, inverse(g)>, and differences of the map along a
    coordinate are its gradient's entries (the map is linear)."""
    torch, kda = _torch(), _kda()
    rng, cu, lens = _rng(5), [0, 9, 13], [9, 5000]
    turns, amplitude = kda.rotary_turns(64, method="yarn", factor=8.0, trained_length=1024)
    (x, xr), (g, gr) = (_to(rng.normal(size=(13, 4, 64)), torch.float32) for _ in range(2))
    call = dict(amplitude=amplitude, interleaved=interleaved)
    y = _np(kda.latent_rotate(x, turns, _i32(lens), _i32(cu), out=torch.empty_like(x), **call))
    dx = _np(kda.latent_rotate(g, turns, _i32(lens), _i32(cu), out=torch.empty_like(g), inverse=True, **call))
    # a side's terms are off by 2^-20 amplitude (|x_a| + |x_b|) |g| at most
    lim = 2.0 ** -20 * amplitude * 4 * np.linalg.norm(xr) * np.linalg.norm(gr)
    assert abs((y * gr).sum() - (xr * dx).sum()) <= lim
    for t, h, c in ((0, 0, 3), (8, 1, 40), (11, 3, 63)):
        up, down = x.clone(), x.clone()
        up[t, h, c] += 1.0
        down[t, h, c] -= 1.0
        a, b = (_np(kda.latent_rotate(v, turns, _i32(lens), _i32(cu), **call)) for v in (up, down))
        diff = ((a - b) * gr)[t, h].sum() / 2
        assert abs(diff - dx[t, h, c]) <= 2.0 ** -17 * amplitude * np.abs(gr[t, h]).max() * (2 + np.abs(xr[t, h]).max())
    _clear()


# ------------------------------------------------------------------ append, gather
class Paged4:
    """A 4-bit cache with NaN scales and NaN shared parts wherever no sequence
    has a row."""

    def __init__(self, seed, lens, page, exponent=0, spread=1.0):
        self.rng = _rng(seed)
        self.lens, self.page, self.exponent = list(lens), page, exponent
        self.table, self.P = ol.ragged_pages(self.rng, self.lens, page)
        c = self.rng.normal(size=(self.P, page, 512)) * spread * 2.0 ** exponent
        pe = self.rng.normal(size=(self.P, page, 64)).astype(np.float32)
        codes, sc = o4.quantise(c, exponent)
        self.rows = o4.pack(codes, (pe.view(np.uint32) >> 16).astype(np.uint16), sc)
        self.ref = o4.unpack(self.rows, exponent)
        held = np.zeros((self.P, page), dtype=bool)
        for b, n in enumerate(self.lens):
            p = np.arange(n)
            held[self.table[b, p // page], p % page] = True
        self.held = held
        dirty = self.rows.copy()
        dirty[~held] = 0xFF
        self.dev = _torch().from_numpy(dirty).cuda()
        self.table_dev = _i32(self.table)
        self.lens_dev = _i32(self.lens)

    def q(self, tokens, H, scale=1.0):
        return _bf(self.rng.normal(size=(tokens, H, ol.ROW)) * scale)

    def decode(self, q, cu, **kw):
        if isinstance(cu, (list, np.ndarray)):
            cu = _i32(cu)
        return _kda().latent4_decode(q, self.dev, self.table_dev, self.lens_dev, cu,
                                     exponent=self.exponent, **kw)

    def want(self, qr, cu, scale=SCALE):
        cu = list(range(len(self.lens) + 1)) if cu is None else cu
        return ol.decode(qr, self.ref, self.table, self.lens, cu, scale)


RAGGED = [0, 1, 15, 16, 17, 64, 200, 129]
RAGGED_NEW = [0, 1, 15, 3, 0, 64, 130, 2]


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_append_rotated_ragged(page, norm, interleaved):
    """The latent part has latent_append's bits, the shared part is rotated."""
    torch, kda = _torch(), _kda()
    rng = _rng(page)
    table, P = ol.ragged_pages(rng, RAGGED, page)
    cu = np.cumsum([0] + RAGGED_NEW)
    x, xr = _bf(rng.normal(size=(cu[-1] + 2, ol.ROW)) * 3)
    w = torch.from_numpy(rng.normal(size=512)).float().cuda() if norm else None
    cache = torch.full((P, page, ol.ROW), 7.0, dtype=torch.bfloat16, device="cuda")
    turns, amplitude = kda.rotary_turns(64, method="yarn", factor=4.0, trained_length=64)
    args = (_i32(table), _i32(RAGGED))
    plain = kda.latent_append(x, cache.clone(), *args, _i32(cu), norm_w=w)
    got = kda.latent_append_rotated(x, cache, *args, turns, _i32(cu), norm_w=w, amplitude=amplitude,
                                    interleaved=interleaved)
    _clear()
    assert got is cache and torch.equal(got[..., :512], plain[..., :512])
    pos = o4.positions(RAGGED, cu)
    b = np.repeat(np.arange(len(RAGGED)), RAGGED_NEW)
    at = table[b, pos // page], pos % page
    freq = np.array([float(t) * 2.0 ** -64 * 2 * np.pi for t in turns.cpu().numpy().astype(np.uint64)])
    want = o4.rotate(xr[:cu[-1], 512:], pos, freq, amplitude, interleaved)
    err = np.abs(_np(got)[at][:, 512:] - want)
    assert (err <= _rotation_limit(xr[:cu[-1], 512:], want, amplitude, HALF, interleaved)).all()
    new = torch.zeros((P, page), dtype=torch.bool)
    new[at] = True
    assert (got[~new.cuda()] == 7.0).all()


def _quantised(rows, exponent=0):
    """bf16 rows (device, [..., 576]) as the oracle packs them."""
    bits = rows.view(_torch().int16).cpu().numpy().view(np.uint16)
    codes, sc = o4.quantise(_np(rows)[..., :512], exponent)
    return o4.pack(codes, bits[..., 512:], sc)


def _same_rows(got, want):
    """4-bit rows equal but for the codes of groups that are NaN."""
    got, want = got.copy(), want.copy()
    for g in range(32):
        nan = (want[..., 384 + g] & 0x7F) == 0x7F
        assert np.array_equal(nan, (got[..., 384 + g] & 0x7F) == 0x7F)
        for a in (got, want):
            a[nan, 8 * g:8 * g + 8] = 0
            a[nan, 384 + g] = 0x7F
    return np.array_equal(got, want)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("norm,turned,interleaved,exponent", [
    (False, False, False, 0), (True, False, False, 0), (True, True, False, 0), (False, True, True, 0),
    (True, True, True, -9), (False, False, False, 5)])
def test_append4_is_the_bf16_row_quantised(page, norm, turned, interleaved, exponent):
    """Bit by bit what the oracle makes of the rows that the bf16 calls store."""
    torch, kda = _torch(), _kda()
    rng = _rng(40 + page)
    table, P = ol.ragged_pages(rng, RAGGED, page)
    cu = np.cumsum([0] + RAGGED_NEW)
    x, _ = _bf(rng.normal(size=(cu[-1] + 2, ol.ROW)) * 3)
    w = torch.from_numpy(rng.normal(size=512) * 2.0 ** exponent).float().cuda() if norm else None
    turns, _ = kda.rotary_turns()
    args, rot = (_i32(table), _i32(RAGGED)), dict(amplitude=1.5, interleaved=interleaved)
    bf = torch.zeros((P, page, ol.ROW), dtype=torch.bfloat16, device="cuda")
    if turned:
        kda.latent_append_rotated(x, bf, *args, turns, _i32(cu), norm_w=w, **rot)
    else:
        kda.latent_append(x, bf, *args, _i32(cu), norm_w=w)
    got = torch.full((P, page, 416), 0xAB, dtype=torch.uint8, device="cuda")
    back = kda.latent4_append(x, got, *args, _i32(cu), norm_w=w, turns=turns if turned else None, exponent=exponent,
                              **(rot if turned else {}))
    _clear()
    assert back is got
    pos = o4.positions(RAGGED, cu)
    b = np.repeat(np.arange(len(RAGGED)), RAGGED_NEW)
    at = table[b, pos // page], pos % page
    new = np.zeros((P, page), dtype=bool)
    new[at] = True
    assert _same_rows(got.cpu().numpy()[new], _quantised(bf, exponent)[new])
    assert (got.cpu().numpy()[~new] == 0xAB).all()


def test_append4_of_every_magnitude():
    """Groups whose maxima run through all bf16 numbers, with their other
    channels at and beside the codes' borders; zeros, infinities, NaN."""
    torch, kda = _torch(), _kda()
    rng = _rng(50)
    mags = torch.arange(0, 0x7F81, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)      # 0 .. inf
    n = -(-len(mags) // 32)
    x = torch.zeros((n, 32, 16), dtype=torch.bfloat16)
    top = torch.zeros(n * 32, dtype=torch.bfloat16)
    top[:len(mags)] = mags
    x[:] = (top.view(n, 32, 1).double() * torch.from_numpy(rng.uniform(-1, 1, size=(n, 32, 16)))).bfloat16()
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.5, 0.2]) / 6
    x[..., 1:10] = (top.view(n, 32, 1).float() * border).bfloat16()
    x[..., 0] = top.view(n, 32) * torch.from_numpy(rng.choice([-1, 1], size=(n, 32))).bfloat16()
    x[3, 5, 7] = x[800, 0, 0] = float("nan")
    rows = torch.cat([x.view(n, 512), torch.zeros((n, 64), dtype=torch.bfloat16)], 1).cuda()
    cache = torch.zeros((1, 1024 if n <= 1024 else 0, 416), dtype=torch.uint8, device="cuda")
    kda.latent4_append(rows, cache, _i32([[0]]), _i32([n]), _i32([0, n]))
    _clear()
    with np.errstate(invalid="ignore"):
        assert _same_rows(cache.cpu().numpy()[0, :n], _quantised(rows))


@pytest.mark.parametrize("exponent", [-32, -20, -9, 9, 32])
def test_append4_of_every_magnitude_and_unit(exponent):
    """Magnitudes far above and below the cache's unit saturate and vanish with
    their signs."""
    torch, kda = _torch(), _kda()
    rng = _rng(52)
    mags = torch.arange(0, 0x7F81, 7, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    n = -(-len(mags) // 32)
    top = torch.zeros(n * 32, dtype=torch.bfloat16)
    top[:len(mags)] = mags
    share = torch.from_numpy(rng.choice([-1, 1], size=(n, 32, 16)) * rng.choice([0.0, 0.01, 0.3, 1.0], size=(n, 32, 16)))
    x = torch.where(share == 0, share, top.view(n, 32, 1).double() * share).bfloat16()
    rows = torch.cat([x.view(n, 512), torch.zeros((n, 64), dtype=torch.bfloat16)], 1).cuda()
    page = 1 << (n - 1).bit_length()
    cache = torch.zeros((1, page, 416), dtype=torch.uint8, device="cuda")
    kda.latent4_append(rows, cache, _i32([[0]]), _i32([n]), _i32([0, n]), exponent=exponent)
    _clear()
    with np.errstate(invalid="ignore"):
        assert _same_rows(cache.cpu().numpy()[0, :n], _quantised(rows, exponent))


def test_append4_keeps_the_bits_of_the_shared_part():
    """All 65,536 bit patterns, NaN's payloads among them."""
    torch, kda = _torch(), _kda()
    bits = torch.arange(-(1 << 15), 1 << 15, dtype=torch.int32).to(torch.int16).view(1024, 64)
    rows = torch.cat([torch.zeros((1024, 512), dtype=torch.int16), bits], 1).view(torch.bfloat16).cuda()
    cache = torch.zeros((16, 64, 416), dtype=torch.uint8, device="cuda")
    where = (_i32(np.arange(16)[None]), _i32([1024]), _i32([0, 1024]))
    kda.latent4_append(rows, cache, *where)
    back = kda.latent4_gather(cache, where[0], where[2], total=1024)
    _clear()
    assert np.array_equal(cache.cpu().numpy().reshape(1024, 416)[:, 256:384].copy().view(np.int16), bits.numpy())
    assert np.array_equal(back[:, 512:].contiguous().view(torch.int16).cpu().numpy(), bits.numpy())


def test_append4_one_token_a_sequence_and_bad_places():
    torch, kda = _torch(), _kda()
    lens = [1, 16, 17, 100]
    c = Paged4(51, lens, 16)
    x, _ = _bf(c.rng.normal(size=(4, ol.ROW)))
    a = kda.latent4_append(x, c.dev.clone(), c.table_dev, c.lens_dev)
    b = kda.latent4_append(x, c.dev.clone(), c.table_dev, c.lens_dev, _i32([0, 1, 2, 3, 4]))
    _clear()
    assert torch.equal(a, b) and not torch.equal(a, c.dev)
    table, before = c.table.copy(), c.dev.clone()
    table[2, 1], table[3, 6] = -1, c.P
    kda.latent4_append(x[2:], c.dev, _i32(table[2:]), _i32(lens[2:]))
    _clear(2)
    assert torch.equal(c.dev, before)
    kda.latent4_append(x, c.dev, c.table_dev, _i32([0, -5, 16 * c.table.shape[1] + 1, 2 ** 31 - 1]))
    _clear(1)
    assert torch.equal(c.dev, before)
    turns, _ = kda.rotary_turns()
    bf = torch.zeros((c.P, 16, ol.ROW), dtype=torch.bfloat16, device="cuda")
    kda.latent_append_rotated(x[2:], bf, _i32(table[2:]), _i32(lens[2:]), turns)
    _clear(2)
    kda.latent_append_rotated(x, bf, c.table_dev, _i32([0, -5, 16 * c.table.shape[1] + 1, 2 ** 31 - 1]), turns)
    _clear(1)
    assert (bf == 0).all()


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("exponent", [0, -7, 32, -32])
def test_gather4_ragged(page, exponent):
    torch, kda = _torch(), _kda()
    c = Paged4(52, RAGGED, page, exponent)
    cu = np.cumsum([0] + [n // 2 for n in RAGGED[:4]] + RAGGED[4:])
    out = torch.full((cu[-1] + 5, ol.ROW), 7.0, dtype=torch.bfloat16, device="cuda")
    kda.latent4_gather(c.dev, c.table_dev, _i32(cu), out=out, exponent=exponent)
    _clear()
    want = np.concatenate([ol.sequence_rows(c.ref, c.table[b], 0, cu[b + 1] - cu[b]) for b in range(len(RAGGED))])
    assert np.array_equal(_np(out[:cu[-1]]), want)
    assert (out[cu[-1]:] == 7.0).all()
    again = kda.latent4_gather(c.dev, c.table_dev, _i32(cu), total=int(cu[-1]), exponent=exponent)
    assert torch.equal(again, out[:cu[-1]])


def test_gather4_of_every_code_and_scale():
    """All pairs of codes under all 256 scale bytes."""
    torch, kda = _torch(), _kda()
    rows = np.zeros((256, 416), dtype=np.uint8)
    rows[:, :256] = np.arange(256)
    rows[:, 384:] = (np.arange(256)[:, None] + 8 * np.arange(32)) % 256
    cache = torch.from_numpy(rows).cuda().view(4, 64, 416)
    got = kda.latent4_gather(cache, _i32([[0, 1, 2, 3]]), _i32([0, 256]), total=256)
    _clear()
    assert np.array_equal(_np(got), o4.unpack(rows), equal_nan=True)


def test_gather4_bad_pages_and_offsets():
    torch, kda = _torch(), _kda()
    c = Paged4(53, [100, 100], 16)
    table = c.table.copy()
    table[0, 1], table[1, 0] = -1, c.P
    got = kda.latent4_gather(c.dev, _i32(table), _i32([0, 40, 80]), total=80)
    _clear(2)
    g = _np(got)
    assert (g[16:32] == 0).all() and (g[40:56] == 0).all()
    assert np.array_equal(g[:16], ol.sequence_rows(c.ref, c.table[0], 0, 16))
    guard = torch.full((100, ol.ROW), 7.0, dtype=torch.bfloat16, device="cuda")
    for bad in ([0, 60, 20], [-3, 10, 20], [0, 10, 81]):
        kda.latent4_gather(c.dev, c.table_dev, _i32(bad), out=guard[10:90])
        _clear(1)
        assert (guard[:10] == 7.0).all() and (guard[90:] == 7.0).all()


# ------------------------------------------------------------------ decode
@pytest.mark.parametrize("page", [16, 64, 128, 512])
@pytest.mark.parametrize("H", [1, 5, 16, 31, 48, 64, 96, 130])
def test_decode4_ragged(H, page):
    lens = [1, 15, 16, 17, 127, 128, 129, 255, 300, 0, 640]
    c = Paged4(60 + H, lens, page)
    q, qr = c.q(len(lens), H)
    o, lse = c.decode(q, None)
    _clear()
    check(o, lse, c.want(qr, None), "decode")


@pytest.mark.parametrize("H,news", [(16, [4, 3, 4, 1, 2, 0]), (4, [64, 1, 9, 33, 0, 2]), (64, [2, 5, 1, 0, 1, 3]),
                                    (96, [2, 1, 4, 2, 0, 1]), (1, [130, 1, 1, 7, 3, 1])])
def test_decode4_of_several_new_tokens(H, news):
    """Ragged new tokens; more of them than positions (the first see nothing)."""
    lens = [3, 129, 700, 33, 0, 256]
    c = Paged4(80 + H, lens, 32)
    cu = np.cumsum([0] + news)
    q, qr = c.q(int(cu[-1]) + 3, H)
    o = _torch().full((q.shape[0], H, 512), 7.0, dtype=_torch().bfloat16, device="cuda")
    o, lse = c.decode(q, cu, o=o)
    _clear()
    T = int(cu[-1])
    assert (o[T:] == 7.0).all()                                      # rows that no sequence holds
    check(o[:T], lse[:T], c.want(qr[:T], cu), "several tokens")
    for b, (n, m) in enumerate(zip(news, lens)):
        blind = max(0, n - m)
        assert (o[cu[b]:cu[b] + blind] == 0).all() and np.isneginf(_np(lse[cu[b]:cu[b] + blind])).all()


@pytest.mark.parametrize("H,lens", [(16, [5000]), (32, [9000, 3001]), (64, [4097, 1]), (128, [2500] * 3)])
def test_decode4_over_long_contexts(H, lens):
    """Contexts that are cut into pieces and joined."""
    c = Paged4(90 + H, lens, 64)
    q, qr = c.q(len(lens), H)
    o, lse = c.decode(q, None)
    _clear()
    check(o, lse, c.want(qr, None), "long", seen=max(lens))
    o2, lse2 = c.decode(q, list(range(len(lens) + 1)))
    check(o2, lse2, c.want(qr, None), "long, with offsets", seen=max(lens))


def test_decode4_many_sequences():
    lens = [(37 * i) % 200 for i in range(700)]
    c = Paged4(95, lens, 16)
    q, qr = c.q(len(lens), 2)
    o, lse = c.decode(q, None)
    _clear()
    check(o, lse, c.want(qr, None), "many")


@pytest.mark.parametrize("how", ["rising", "falling", "spike", "flat"])
def test_decode4_of_scores_that_move(how):
    """Scores over hundreds of powers of two, in orders that move the maximum at
    every tile, at one, or never."""
    lens, H = [700, 300], 8
    c = Paged4(97, lens, 64)
    q, qr = c.q(2, H, 0.0 if how == "flat" else 30.0)
    if how != "flat":
        # order the first sequence's rows by its first head's scores
        rows = ol.sequence_rows(c.rows, c.table[0], 0, 700)
        s = ol.sequence_rows(c.ref, c.table[0], 0, 700) @ qr[0, 0]
        order = np.argsort(s if how != "falling" else -s)
        if how == "spike":
            order = np.concatenate([order[:400], order[-1:], order[400:-1]])
        p = np.arange(700)
        c.rows[c.table[0, p // 64], p % 64] = rows[order]
        dirty = c.rows.copy()
        dirty[~c.held] = 0xFF
        c.dev, c.ref = _torch().from_numpy(dirty).cuda(), o4.unpack(c.rows)
    o, lse = c.decode(q, None)
    _clear()
    check(o, lse, c.want(qr, None), how)


@pytest.mark.parametrize("exponent", [-32, -10, 3, 32])
def test_decode4_exponents(exponent):
    """The cache's unit; queries whose latent part balances it."""
    c = Paged4(98, [300, 77], 32, exponent)
    q, qr = _bf(np.concatenate([c.rng.normal(size=(2, 20, 512)) * 2.0 ** -exponent, c.rng.normal(size=(2, 20, 64))], 2))
    o, lse = c.decode(q, None)
    _clear()
    check(o, lse, c.want(qr, None), "exponent")


@pytest.mark.parametrize("power", [-100, -40, 0, 30])
def test_decode4_of_queries_of_any_size(power):
    """Query rows from 2^-149 to 2^112, the scale taking it back; rows of one
    tile of very different sizes; a row of zeros."""
    c = Paged4(99, [200, 130, 64], 16)
    rows = c.rng.normal(size=(3, 24, ol.ROW))
    rows[1] *= 2.0 ** (8 * (np.arange(24) - 12))[:, None] / 64
    rows[2, 5] = 0
    q, qr = _bf(rows * 2.0 ** power)
    scale = SCALE * 2.0 ** -power
    o, lse = c.decode(q, None, scale=scale)
    _clear()
    r = c.want(qr, None, scale)
    keep = r.mag < 1e5                                               # beyond, a score's rounding decides who wins
    pick = lambda a: a[keep]  # noqa: E731
    s = ol.Result((int(keep.sum()), 1), 512)
    s.o, s.lse, s.absum, s.sqsum, s.mag = (pick(a)[:, None] for a in (r.o, r.lse, r.absum, r.sqsum, r.mag))
    t = _torch().from_numpy(keep).cuda()
    check(o[t][:, None], lse[t][:, None], s, "sizes")
    assert not _torch().isnan(o).any()


@pytest.mark.parametrize("H", [3, 40, 96])
def test_decode4_of_queries_that_are_not_finite(H):
    """NaN or infinities in a row of q: NaN where it sees anything, and the other
    rows' bits as without it."""
    torch = _torch()
    c = Paged4(101, [200, 0, 64], 16)
    q, _ = c.q(3, H)
    want, want_lse = c.decode(q, None)
    bad = q.clone()
    bad[0, 1, 7], bad[0, 2, 550], bad[1, 0, 0], bad[2, H - 1, 511] = float("nan"), float("nan"), float("nan"), float("inf")
    o, lse = c.decode(bad, None)
    _clear()
    hit = torch.zeros((3, H), dtype=torch.bool, device="cuda")
    hit[0, 1] = hit[0, 2] = hit[2, H - 1] = True
    assert torch.isnan(o[hit]).all()
    assert torch.equal(o[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()


def test_decode4_bad_pages_lengths_and_offsets():
    torch, kda = _torch(), _kda()
    lens = [100, 90, 40]
    c = Paged4(102, lens, 16)
    q, qr = c.q(3, 6)
    table = c.table.copy()
    table[0, 2], table[1, 0] = -1, c.P
    ref = np.concatenate([c.ref, np.zeros((1,) + c.ref.shape[1:])])  # a bad page reads as zeros
    t2 = np.where((table < 0) | (table >= c.P), c.P, table)
    o, lse = kda.latent4_decode(q, c.dev, _i32(table), c.lens_dev)
    _clear(2)
    check(o, lse, ol.decode(qr, ref, t2, lens, [0, 1, 2, 3], SCALE), "bad pages")
    width = 16 * c.table.shape[1]
    kda.latent4_decode(q, c.dev, c.table_dev, _i32([-3, width + 1, 40]))
    _clear(1 | 2)                                                    # flagged; what lies behind the table's pages is bad
    guard = torch.full((30, 6, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    q20, _ = c.q(20, 6)
    for bad in ([0, 30, 20, 20], [-3, 5, 9, 12], [0, 1, 2, 21]):
        kda.latent4_decode(q20, c.dev, c.table_dev, c.lens_dev, _i32(bad), o=guard[5:25])
        _clear(1)
        assert (guard[:5] == 7.0).all() and (guard[25:] == 7.0).all()


def test_decode4_is_reproducible_on_streams_and_in_graphs():
    torch = _torch()
    c = Paged4(103, [900, 1, 333, 64], 32)
    for H, cu in ((16, None), (96, None), (8, [0, 3, 4, 6, 7])):
        q, _ = c.q(7 if cu else 4, H)
        cu = cu and _i32(cu)
        want = c.decode(q, cu)
        torch.cuda.synchronize()
        s, t = torch.cuda.Stream(), torch.cuda.Stream()
        got = [c.decode(q, cu, stream=x) for x in (s, t, s, t, None)]
        graphs = []
        torch.cuda.synchronize()
        for _ in range(2):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                got.append(c.decode(q, cu))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graphs[0].replay()
        with torch.cuda.stream(t):
            graphs[1].replay()
        torch.cuda.synchronize()
        graphs[0].replay()
        _clear()
        for o, lse in got:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        # new inputs in a captured call's place
        q.copy_(c.q(q.shape[0], H)[0])
        fresh = c.decode(q, cu)
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(got[-1][0], fresh[0]) and not torch.equal(fresh[0], want[0])


def test_decode4_with_a_given_workspace():
    torch, kda = _torch(), _kda()
    c = Paged4(104, [700, 60], 16)
    q, _ = c.q(2, 20)
    want = c.decode(q, None)
    n = kda.latent4_decode_workspace_bytes(2, 2, 20)
    ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    got = c.decode(q, None, workspace=ws)
    _clear()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    if n:
        with pytest.raises(kda.KDAError):
            c.decode(q, None, workspace=ws[:n - 1])


def test_offsets_past_32_bits():
    """A 4-bit cache, rotated rows, queries and outputs of more than 4 GB, with
    the rows that are used at their ends."""
    torch, kda = _torch(), _kda()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    rng, bf = _rng(105), torch.bfloat16
    page, P, L = 64, 190_000, 300                                    # 5.1 GB
    cache = torch.empty((P, page, 416), dtype=torch.uint8, device="cuda")
    table = np.array([[P - 1 - 3 * i for i in range(5)], [P - 2 - 3 * i for i in range(5)]])
    x, _ = _bf(rng.normal(size=(2 * L, ol.ROW)))
    kda.latent4_append(x, cache, _i32(table), _i32([L, L]), _i32([0, L, 2 * L]))
    rows = o4.unpack(_quantised(x))
    assert np.array_equal(_np(kda.latent4_gather(cache, _i32(table), _i32([0, L, 2 * L]), total=2 * L)), rows)
    T, H = 45_000, 96                                                # 5.0 GB of queries, 4.4 GB of outputs
    q = torch.empty((T, H, ol.ROW), dtype=bf, device="cuda")
    held, heldr = _bf(rng.normal(size=(3, H, ol.ROW)))
    q[-3:] = held
    o = torch.full((T, H, 512), 7.0, dtype=bf, device="cuda")
    o, lse = kda.latent4_decode(q, cache, _i32(table), _i32([L, L]), _i32([T - 3, T - 2, T]), o=o)
    _clear()
    r = ol.Result((3, H), 512)
    for t, (b, n) in enumerate(((0, L), (1, L - 1), (1, L))):
        for h in range(H):
            r.put(t, h, heldr[t, h], rows[b * L:b * L + n], rows[b * L:b * L + n, :512], SCALE)
    check(o[-3:], lse[-3:], r, "decode")
    assert (o[:10] == 7.0).all() and (o[-13:-3] == 7.0).all()
    turns, _ = kda.rotary_turns()
    kda.latent_rotate(q[..., 512:], turns, _i32([L, L]), _i32([T - 3, T - 2, T]))
    _clear()
    want = o4.rotate(heldr[..., 512:], np.array([L - 1, L - 2, L - 1]), o4.frequencies(64, 1e4))
    assert (np.abs(_np(q[-3:, :, 512:]) - want) <= _rotation_limit(heldr[..., 512:], want, 1.0, HALF, False)).all()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("interleaved", [False, True])
def test_a_layer_in_chunks(interleaved):
    """Prompts, then a chunk, then single tokens: rows rotated and stored in 4
    bits, attended to absorbed over the pages and expanded after a gather, both
    against the oracle's rows."""
    torch, kda = _torch(), _kda()
    rng, H, page = _rng(106), 4, 16
    turns, amplitude = kda.rotary_turns(64, method="yarn", factor=4.0, trained_length=256)
    freq = np.array([float(t) * 2.0 ** -64 * 2 * np.pi for t in turns.cpu().numpy().astype(np.uint64)])
    rot = dict(amplitude=amplitude, interleaved=interleaved)
    wk, wv = rng.normal(size=(H, 512, 128)) / 16, rng.normal(size=(H, 512, 128)) / 16
    w = torch.from_numpy(1 + 0.1 * rng.normal(size=512)).float().cuda()
    steps = [[40, 130], [33, 7], [1, 1], [1, 1]]
    total = np.sum(steps, axis=0)
    table, P = ol.ragged_pages(rng, list(total), page)
    cache = torch.full((P, page, 416), 0xFF, dtype=torch.uint8, device="cuda")
    held = np.zeros(2, dtype=int)
    for news in steps:
        cu = np.cumsum([0] + news)
        held = held + news
        lens, T = _i32(held), int(cu[-1])
        q, qr = _bf(rng.normal(size=(T, H, 192)))
        x, xr = _bf(rng.normal(size=(T, ol.ROW)))
        pos = o4.positions(list(held), cu)
        kda.latent_rotate(q[..., 128:], turns, lens, _i32(cu), **rot)
        want = o4.rotate(qr[..., 128:], pos, freq, amplitude, interleaved)
        assert (np.abs(_np(q[..., 128:]) - want) <= _rotation_limit(qr[..., 128:], want, amplitude, HALF, interleaved)).all()
        kda.latent4_append(x, cache, _i32(table), lens, _i32(cu), norm_w=w, turns=turns, **rot)
        cu_k = np.cumsum([0] + list(held))
        rows = kda.latent4_gather(cache, _i32(table), _i32(cu_k), total=int(cu_k[-1]))
        # what was stored stands for the normalised rows to within the codes' steps
        for b in range(2):
            mine = _np(rows[cu_k[b + 1] - news[b]:cu_k[b + 1]])
            c = ol.normalised_row(xr[cu[b]:cu[b + 1]], _np(w), 1e-6)
            g = np.abs(c[:, :512]).reshape(-1, 32, 16).max(-1).repeat(16, -1)
            # half the widest step, 1/6 of the maximum, and a scale that is off by half an e4m3 step
            assert (np.abs(mine[:, :512] - c[:, :512]) <= g * (1 / 6 + 2.0 ** -4 + HALF)).all()
            far = o4.rotate(xr[cu[b]:cu[b + 1], 512:], pos[cu[b]:cu[b + 1]], freq, amplitude, interleaved)
            assert (np.abs(mine[:, 512:] - far)
                    <= _rotation_limit(xr[cu[b]:cu[b + 1], 512:], far, amplitude, HALF, interleaved)).all()
        qa, qar = _bf(ol.absorb(_np(q), wk))
        o, lse = kda.latent4_decode(qa, cache, _i32(table), lens, _i32(cu))
        ref = o4.unpack(cache.cpu().numpy())
        check(o, lse, ol.decode(qar, ref, table, list(held), cu, SCALE), "absorbed")
        kv, pe = ol.expand(_np(rows), wk, wv)
        kv, kvr = _bf(kv)
        po, plse = kda.latent_prefill(q, kv, rows[:, 512:], _i32(cu), _i32(cu_k))
        r = ol.prefill(_np(q), kvr, _np(rows[:, 512:]), cu, cu_k, SCALE)
        assert np.abs(_np(plse) - r.lse).max() <= 1e-4 * (1 + np.abs(r.lse).max())
        # the two forms: q' and the keys are rounded to bf16 before their products
        mag = SCALE * np.abs(_np(q)).max() * np.abs(kvr).max() * 192
        assert np.abs(_np(lse) - _np(plse)).max() <= 4 * HALF * mag
        _clear()


def test_append4_of_many_normalised_rows_is_the_bf16_row_quantised():
    """A sum of squares that is added in another order than the bf16 call's
    rounds differently in a row of ten and moves a code in a row of tens of
    thousands: half a million rows, plain and rotated, against the same rows
    stored in bf16 and quantised as they lie there."""
    torch, kda = _torch(), _kda()
    N, L, page = 8, 1 << 16, 64
    gen = torch.Generator(device="cuda").manual_seed(107)
    x = (torch.randn((N * L, ol.ROW), generator=gen, device="cuda") * 3).bfloat16()
    w = torch.randn(512, generator=gen, device="cuda")
    table = torch.arange(N * L // page, dtype=torch.int32, device="cuda").view(N, -1)
    where = (table, _i32([L] * N))
    cu = _i32(np.arange(N + 1) * L)
    turns, _ = kda.rotary_turns()
    rows = torch.empty((N * L // page, page, ol.ROW), dtype=torch.bfloat16, device="cuda")
    got, want = (torch.zeros((N * L // page, page, 416), dtype=torch.uint8, device="cuda") for _ in range(2))
    for rot in (None, dict(amplitude=1.25, interleaved=False), dict(amplitude=1.0, interleaved=True)):
        if rot is None:
            kda.latent_append(x, rows, *where, cu, norm_w=w)
        else:
            kda.latent_append_rotated(x, rows, *where, turns, cu, norm_w=w, **rot)
        kda.latent4_append(rows.view(-1, ol.ROW), want, *where, cu)
        kda.latent4_append(x, got, *where, cu, norm_w=w, turns=None if rot is None else turns, **(rot or {}))
        _clear()
        off = (got != want).any(2).sum().item()
        assert off == 0, "%d rows of %d differ" % (off, N * L)


@pytest.mark.parametrize("more", [0, 10])
@pytest.mark.parametrize("exponent", [-32, -28, -24, -20, 0, 20, 32])
def test_decode4_units_with_queries_of_one_size(exponent, more):
    """Latents and shared channels of the cache's unit, or the shared ones 2^10
    below it, under queries that balance them: both parts count alike in a
    score, whatever the unit."""
    c = Paged4(108, [300, 77], 32, exponent)
    pe = (c.rng.normal(size=(c.P, 32, 64)) * 2.0 ** (exponent - more)).astype(np.float32)
    c.rows[..., 256:384] = (pe.view(np.uint32) >> 16).astype(np.uint16).view(np.uint8)
    dirty = c.rows.copy()
    dirty[~c.held] = 0xFF
    c.dev, c.ref = _torch().from_numpy(dirty).cuda(), o4.unpack(c.rows, exponent)
    part = np.concatenate([np.ones(512), np.full(64, 2.0 ** more)])
    q, qr = _bf(c.rng.normal(size=(2, 20, ol.ROW)) * part * 2.0 ** -exponent)
    o, lse = c.decode(q, None)
    _clear()
    check(o, lse, c.want(qr, None), "exponent %d" % exponent)


def test_rotate_and_autograd():
    """A rotation raises the version of the tensor that it writes, and no other:
    a backward pass over a tensor that was rotated after it was saved is an error
    and not a wrong gradient.  Inside an autograd function it is differentiable."""
    torch, kda = _torch(), _kda()
    rng = _rng(112)
    turns, amplitude = kda.rotary_turns(64, method="yarn", factor=8.0, trained_length=1024)
    lens, cu = _i32([40]), _i32([0, 5])
    x, xr = _to(rng.normal(size=(5, 3, 192)), torch.float32)
    with pytest.raises(ValueError, match="gradient"):
        kda.latent_rotate(x.clone().requires_grad_()[..., 128:], turns, lens, cu)
    leaf = x.clone().requires_grad_()
    y = leaf * 2
    z = (y * y).sum()
    with torch.no_grad():
        kda.latent_rotate(y[..., 128:], turns, lens, cu)
    with pytest.raises(RuntimeError, match="inplace"):
        z.backward()
    out = torch.empty_like(x[..., 128:])
    before = x._version, out._version
    kda.latent_rotate(x[..., 128:], turns, lens, cu, out=out)
    assert x._version == before[0] and out._version > before[1]
    with torch.inference_mode():
        assert torch.equal(kda.latent_rotate(x[..., 128:].clone(), turns, lens, cu), out)

    class Rotate(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a):
            return kda.latent_rotate(a, turns, lens, cu, out=torch.empty_like(a), amplitude=amplitude)

        @staticmethod
        def backward(ctx, g):
            return kda.latent_rotate(g, turns, lens, cu, out=torch.empty_like(g), amplitude=amplitude, inverse=True)

    leaf = x.clone().requires_grad_()
    g, gr = _to(rng.normal(size=(5, 3, 64)), torch.float32)
    (Rotate.apply(leaf[..., 128:]) * g).sum().backward()
    _clear()
    freq = np.array([float(t) * 2.0 ** -64 * 2 * np.pi for t in turns.cpu().numpy().astype(np.uint64)])
    want = o4.rotate(gr, np.arange(35, 40), freq, amplitude, inverse=True)
    assert (np.abs(_np(leaf.grad[..., 128:]) - want) <= _rotation_limit(gr, want, amplitude, 2.0 ** -24, False)).all()
    assert (leaf.grad[..., :128] == 0).all()


def _forms_limits(qr, rows, wk, wv, o):
    """For one (token, head): how far lse and the value-expanded output of the
    absorbed form may be from the expanded form's, over the rows it sees.

    With q' = Wk q, k = c Wk and v = c Wv: the absorbed form rounds q' to bf16,
    the expanded one k and v, each by HALF of its size at most and independently.
    So a score is off by scale sum_j e_j q'_j c_pj there and by scale sum_j e_pj
    q_j k_pj here; 7 times the root of the summed squares (Hoeffding, as in
    check) bounds these sums, Da and De their largest over p, and also what they
    come to, to first order, in lse (weights p) and in an output (weights
    p (v - vm), vm = sum p v).  Second order: Da^2 / 2 in lse, 4 Da^2 e^2Da sum p
    |v - vm| in an output (the third cumulant of weights changed by e^2Da), and
    the same of De.  An output has the roundings of P (fp16 absorbed, bf16
    expanded), of v, of the absorbed o (each channel, through Wv) and of the
    expanded one besides, both the kernels' own fp32 as in check."""
    q, c, r = qr[:128], rows[:, :512], rows[:, 512:]
    k, v, qa = c @ wk, c @ wv, wk @ q
    s = SCALE * (k @ q + r @ qr[128:])
    p = np.exp(s - s.max())
    p /= p.sum()
    lse = s.max() + np.log(np.exp(s - s.max()).sum())
    a, e = 7 * HALF * SCALE * qa, 7 * HALF * SCALE * np.sqrt((q * q) @ (k * k).T)      # e: of each score
    da, de = np.sqrt((a * a) @ (c * c).T).max(), e.max()
    mag = SCALE * ((np.abs(c) @ np.abs(qa)).max() + (np.abs(k) @ np.abs(q)).max() + 2 * (np.abs(r) @ np.abs(qr[128:])).max())
    d = 80 * 2.0 ** -23 * mag                                       # of both kernels
    lim_lse = np.sqrt(((a * (p @ c)) ** 2).sum()) + np.sqrt(((p * e) ** 2).sum()) + (da * da + de * de) / 2
    lim_lse += d + 2 * 2.0 ** -20 * (1 + np.abs(lse))
    dev = v - p @ v
    first = np.sqrt((a * a) @ ((p[:, None] * c).T @ dev) ** 2) + np.sqrt((p * e) ** 2 @ dev ** 2)
    second = 4 * (da * da * np.exp(2 * da) + de * de * np.exp(2 * de)) * (p @ np.abs(dev))
    lim = first + second + 7 * (HALF16 + 2 * HALF) * np.sqrt((p * p) @ (v * v)) + (2 * d + 2 * 2.0 ** -20) * (p @ np.abs(v))
    lim += 7 * HALF * np.sqrt((o * o) @ (wv * wv)) + HALF * np.abs(p @ v) + 2.0 ** -20 * ((p @ np.abs(c)) @ np.abs(wv))
    return lim_lse, lim * (1 + 4 * HALF) + 2.0 ** -32 * len(rows) * 16 * np.abs(v).max()


@pytest.mark.parametrize("news", [[40, 130], [3, 20], [1, 1]])
def test_both_forms_over_the_same_rows(news):
    """The absorbed form over 4-bit pages and the expanded form over the gathered
    rows: each against the oracle, and the absorbed output, its values expanded,
    against the expanded output."""
    from test_gpu_latent import check as check_prefill
    torch, kda = _torch(), _kda()
    lens, H, page = [40, 163], 3, 16
    c = Paged4(109, lens, page)
    wk, wv = (c.rng.normal(size=(H, 512, 128)) / 16 for _ in range(2))
    cu, cu_k = np.cumsum([0] + news), np.cumsum([0] + lens)
    q, qr = _bf(c.rng.normal(size=(int(cu[-1]), H, 192)))
    rows = kda.latent4_gather(c.dev, c.table_dev, _i32(cu_k), total=int(cu_k[-1]))
    ref = [ol.sequence_rows(c.ref, c.table[b], 0, n) for b, n in enumerate(lens)]
    assert np.array_equal(_np(rows), np.concatenate(ref))
    qa, qar = _bf(ol.absorb(qr, wk))
    o, lse = c.decode(qa, cu)
    kv, kvr = _bf(ol.expand(_np(rows), wk, wv)[0])
    po, plse = kda.latent_prefill(q, kv, rows[:, 512:], _i32(cu), _i32(cu_k))
    _clear()
    check(o, lse, c.want(qar, cu), "absorbed")
    check_prefill(po, plse, ol.prefill(qr, kvr, _np(rows[:, 512:]), cu, cu_k, SCALE), "expanded")
    o, lse, po, plse = (_np(t) for t in (o, lse, po, plse))
    for b, (n, m) in enumerate(zip(news, lens)):
        for i in range(n):
            for h in range(H):
                t = cu[b] + i
                lim_lse, lim = _forms_limits(qr[t, h], ref[b][:m - n + i + 1], wk[h], wv[h], o[t, h])
                assert abs(lse[t, h] - plse[t, h]) <= lim_lse, (b, i, h)
                assert (np.abs(o[t, h] @ wv[h] - po[t, h]) <= lim).all(), (b, i, h)
