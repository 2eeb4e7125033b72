"""Pins of the latent-attention oracle (CPU): closed forms, the two forms of
the layer against each other, splits joined by their lse, and pages."""
import numpy as np
import pytest

from oracle import latent as ol


def _rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def test_one_key_gives_its_value():
    r = _rng(1)
    x, k, v = r.normal(size=8), r.normal(size=(1, 8)), r.normal(size=(1, 5))
    o, lse, p = ol.attend(x, k, v, 0.3)
    assert np.array_equal(o, v[0]) and p[0] == 1.0
    assert lse == pytest.approx(0.3 * float(k[0] @ x), rel=1e-14)


def test_equal_keys_give_the_mean():
    r = _rng(2)
    k = np.repeat(r.normal(size=(1, 8)), 7, axis=0)
    v = r.normal(size=(7, 5))
    x = r.normal(size=8)
    o, lse, _ = ol.attend(x, k, v, 0.5)
    assert np.allclose(o, v.mean(0), atol=1e-14)
    assert lse == pytest.approx(0.5 * float(k[0] @ x) + np.log(7), rel=1e-14)


def test_hand_worked_two_keys():
    # scores ln 3 and 0: weights 3/4 and 1/4, lse = ln 4
    o, lse, p = ol.attend(np.array([1.0]), np.array([[np.log(3.0)], [0.0]]), np.array([[4.0], [8.0]]), 1.0)
    assert p == pytest.approx([0.75, 0.25]) and o[0] == pytest.approx(5.0) and lse == pytest.approx(np.log(4.0))


def test_no_key_gives_zero():
    o, lse, _ = ol.attend(np.ones(4), np.zeros((0, 4)), np.zeros((0, 3)), 1.0)
    assert not o.any() and lse == -np.inf


def test_parts_join_by_their_lse():
    r = _rng(3)
    x, k, v = r.normal(size=8), r.normal(size=(11, 8)), r.normal(size=(11, 5))
    o, lse, _ = ol.attend(x, k, v, 0.7)
    (o1, l1, _), (o2, l2, _) = ol.attend(x, k[:4], v[:4], 0.7), ol.attend(x, k[4:], v[4:], 0.7)
    assert np.allclose(o, o1 * np.exp(l1 - lse) + o2 * np.exp(l2 - lse), atol=1e-14)
    assert lse == pytest.approx(np.logaddexp(l1, l2), rel=1e-14)


def test_absorbed_equals_expanded():
    """The same layer both ways: o_expanded = o_absorbed Wv, equal lse."""
    r = _rng(4)
    H, lens, news, page = 3, [5, 18], [2, 18], 16
    table, P = ol.ragged_pages(r, lens, page)
    cache = r.normal(size=(P, page, ol.ROW))
    wk, wv = r.normal(size=(2, H, 512, 128)) / 16
    cu = np.cumsum([0] + news)
    cu_k = np.cumsum([0] + lens)
    q = r.normal(size=(cu[-1], H, 192))
    scale = 192 ** -0.5
    a = ol.decode(ol.absorb(q, wk), cache, table, lens, cu, scale)
    rows = np.concatenate([ol.sequence_rows(cache, table[b], 0, n) for b, n in enumerate(lens)])
    kv, pe = ol.expand(rows, wk, wv)
    e = ol.prefill(q, kv, pe, cu, cu_k, scale)
    assert np.allclose(np.einsum("thc,hcd->thd", a.o, wv), e.o, atol=1e-11)
    assert np.allclose(a.lse, e.lse, atol=1e-11)


def test_new_tokens_one_at_a_time():
    """n new tokens in one call equal n calls of one token on shorter lengths."""
    r = _rng(5)
    page, L, n, H = 16, 21, 4, 2
    table, P = ol.ragged_pages(r, [L], page)
    cache = r.normal(size=(P, page, ol.ROW))
    q = r.normal(size=(n, H, ol.ROW))
    whole = ol.decode(q, cache, table, [L], [0, n], 0.1)
    for i in range(n):
        one = ol.decode(q[i:i + 1], cache, table, [L - n + i + 1], [0, 1], 0.1)
        assert np.allclose(one.o[0], whole.o[i], atol=1e-14) and np.allclose(one.lse[0], whole.lse[i])


def test_append_puts_rows_where_sequences_read_them():
    r = _rng(6)
    page, lens, news = 16, [17, 1, 40], [3, 1, 40]
    table, P = ol.ragged_pages(r, lens, page)
    cache = r.normal(size=(P, page, ol.ROW))
    cu = np.cumsum([0] + news)
    x = r.normal(size=(cu[-1], ol.ROW))
    out = ol.append(x, cache, table, lens, cu)
    for b, (n, k) in enumerate(zip(lens, news)):
        assert np.array_equal(ol.sequence_rows(out, table[b], n - k, n), x[cu[b]:cu[b + 1]])
        assert np.array_equal(ol.sequence_rows(out, table[b], 0, n - k), ol.sequence_rows(cache, table[b], 0, n - k))


def test_normalised_row():
    r = _rng(7)
    x, w = r.normal(size=(4, ol.ROW)) * 3, r.normal(size=512)
    y = ol.normalised_row(x, np.ones(512), 0.0)
    assert np.allclose((y[:, :512] ** 2).mean(1), 1.0) and np.array_equal(y[:, 512:], x[:, 512:])
    assert np.allclose(ol.normalised_row(5 * x, w, 0.0)[:, :512], ol.normalised_row(x, w, 0.0)[:, :512])
    assert np.array_equal(ol.normalised_row(x, None, 0.0), x)
    # mean square 3, eps 1: divided by 2
    assert np.allclose(ol.normalised_row(np.full(576, np.sqrt(3.0)), w, 1.0)[:512], np.sqrt(3.0) / 2 * w)


def test_causal_rows_see_up_to_their_own():
    r = _rng(8)
    q, kv, pe = r.normal(size=(3, 1, 192)), r.normal(size=(5, 1, 256)), r.normal(size=(5, 64))
    a = ol.prefill(q, kv, pe, [0, 3], [0, 5], 0.1)
    kv2, pe2 = kv.copy(), pe.copy()
    kv2[4], pe2[4] = 9.0, 9.0                           # the last key: only the last query sees it
    b = ol.prefill(q, kv2, pe2, [0, 3], [0, 5], 0.1)
    assert np.array_equal(a.o[:2], b.o[:2]) and not np.allclose(a.o[2], b.o[2])
    # more queries than keys: the first ones see nothing
    c = ol.prefill(q, kv[:1], pe[:1], [0, 3], [0, 1], 0.1)
    assert not c.o[:2].any() and np.all(c.lse[:2] == -np.inf) and np.allclose(c.o[2], kv[:1, 0, 128:])
