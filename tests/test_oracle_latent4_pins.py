"""Pins of the rotary and 4-bit oracle: hand values, closed forms and torch's
own e4m3 conversions."""
import numpy as np
import pytest

from oracle import latent4 as o4


def test_e4m3_values_are_torchs():
    torch = pytest.importorskip("torch")
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(o4.E4M3, want, equal_nan=True)
    assert o4.E4M3[126] == 448 and o4.E4M3[1] == 2.0 ** -9 and np.isnan(o4.E4M3[127])


def test_nearest_even_at_and_beside_borders():
    x = [0, 0.25, 0.2500001, 0.7499999, 0.75, 1.25, 1.75, 2.5, 2.500001, 3.5, 5, 5.000001, 6, 1e9]
    want = [0, 0, 0.5, 0.5, 1, 1, 2, 2, 3, 4, 4, 6, 6, 6]
    assert o4.E2M1[o4.nearest_even(np.array(x), o4.E2M1)].tolist() == want


def test_e4m3_rounding_is_torchs():
    torch = pytest.importorskip("torch")
    bf = torch.arange(0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).double()
    x = bf[bf <= 448]
    want = x.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(o4.nearest_even(x.numpy(), o4.E4M3[:127]), want)


def test_quantise_by_hand():
    c = np.zeros((1, 512))
    c[0, :4] = [6, -0.24, 5, -2.5]                 # group 0: scale 1
    c[0, 16:18] = [1.5, -0.75]                     # group 1: scale 1/4
    c[0, 32] = 1e6                                 # group 2: saturates at 6 * 448
    c[0, 48] = 6 * 2.0 ** -10                      # group 3: a border to the smallest scale, to even: 0
    c[0, 64], c[0, 65] = 6 * 2.0 ** -9, np.nan     # group 4: NaN
    codes, sc = o4.quantise(c)
    v = o4.values(codes, sc)[0]
    assert v[:4].tolist() == [6, 0, 4, -2] and np.signbit(v[1])
    assert v[16:18].tolist() == [1.5, -0.75] and o4.E4M3[sc[0, 1]] == 0.25
    assert v[32] == 2688 and v[48] == 0 and np.isnan(v[64:80]).all() and sc[0, 4] == 0x7F
    codes, sc = o4.quantise(c * 2.0 ** -7, exponent=-7)              # the same, in another unit
    assert np.array_equal(o4.values(codes, sc, -7)[0], v * 2.0 ** -7, equal_nan=True)


def test_pack_and_unpack():
    rng = np.random.Generator(np.random.PCG64(1))
    codes = rng.integers(0, 16, (3, 512)).astype(np.uint8)
    sc = rng.integers(0, 127, (3, 32)).astype(np.uint8)
    pe = rng.normal(size=(3, 64)).astype(np.float32)
    bits = (pe.view(np.uint32) >> 16).astype(np.uint16)
    rows = o4.pack(codes, bits, sc)
    assert rows.shape == (3, 416) and rows[0, 0] == codes[0, 0] | codes[0, 1] << 4 and rows[0, 415] == sc[0, 31]
    v = o4.unpack(rows)
    assert np.array_equal(v[:, :512], o4.values(codes, sc))
    assert np.array_equal(v[:, 512:].astype(np.float32).view(np.uint32), bits.astype(np.uint32) << 16)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation(interleaved):
    f = o4.frequencies(8, 1e4)
    assert np.allclose(f.astype(float), [1, 0.1, 0.01, 0.001], rtol=1e-15)
    rng = np.random.Generator(np.random.PCG64(2))
    x, k = rng.normal(size=(2, 5, 8))
    p = np.array([0, 1, 7, 100, 123456])
    y = o4.rotate(x, p, f, 1.0, interleaved)
    assert np.array_equal(y[0], x[0])                                # position 0
    a, b = (0, 1) if interleaved else (0, 4)                         # pair 0 at position 1: one radian
    assert np.isclose(y[1, a], x[1, a] * np.cos(1) - x[1, b] * np.sin(1))
    assert np.isclose(y[1, b], x[1, b] * np.cos(1) + x[1, a] * np.sin(1))
    assert np.allclose(o4.rotate(y, p, f, 1.0, interleaved, inverse=True), x)
    # products depend on the distance of the positions alone
    far = o4.rotate(x, p + 999, f, 1.0, interleaved), o4.rotate(k, p[::-1] + 999, f, 1.0, interleaved)
    assert np.allclose((y * o4.rotate(k, p[::-1], f, 1.0, interleaved)).sum(1), (far[0] * far[1]).sum(1), atol=1e-9)
    assert np.allclose(o4.rotate(x, p, f, 1.7, interleaved), 1.7 * y)


def test_positions():
    assert o4.positions([5, 3, 4], [0, 2, 2, 6]).tolist() == [3, 4, 0, 1, 2, 3]
