"""Latent attention over a paged cache, numpy fp64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``): it shares no code with
the CUDA path.

One row of 576 a token for all heads, [c (512) | r (64)].  A row x of a
(token, head) pair attends to the rows it may see,

    s_p = scale <x, key_p>,  o = sum_p softmax(s)_p value_p,  lse = ln sum_p e^{s_p},

with key = row and value = c (absorbed), or with key = [k | r] and value = v
multiplied out of c (expanded).  A row that sees nothing has o = 0 and
lse = -inf.
"""
from __future__ import annotations

from typing import List, Optional, Tuple

import numpy as np

LATENT, PE = 512, 64
ROW = LATENT + PE


def normalised_row(x: np.ndarray, norm_w: Optional[np.ndarray], eps: float) -> np.ndarray:
    """The cached row of raw x [..., 576]: the latent part RMS-normalised."""
    x = np.array(x, dtype=np.float64)
    if norm_w is not None:
        c = x[..., :LATENT]
        c /= np.sqrt(np.mean(c * c, axis=-1, keepdims=True) + eps)
        c *= np.asarray(norm_w, dtype=np.float64)
    return x


def sequence_rows(cache: np.ndarray, table_row: np.ndarray, start: int, stop: int) -> np.ndarray:
    """Rows of positions start .. stop - 1 of the sequence with this table row."""
    page = cache.shape[1]
    p = np.arange(start, stop)
    return cache[table_row[p // page], p % page]


def append(x, cache, table, seq_lens, cu, norm_w=None, eps=1e-6) -> np.ndarray:
    """The cache (fp64 copy) after the new tokens' rows were written."""
    out = np.array(cache, dtype=np.float64)
    page = out.shape[1]
    rows = normalised_row(x, norm_w, eps)
    for b in range(len(seq_lens)):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            p = seq_lens[b] - n + i
            out[table[b, p // page], p % page] = rows[cu[b] + i]
    return out


def attend(x: np.ndarray, key: np.ndarray, value: np.ndarray, scale: float
           ) -> Tuple[np.ndarray, float, np.ndarray]:
    """One row x over keys [n, d] and values [n, dv]: (o, lse, softmax)."""
    if len(key) == 0:
        return np.zeros(value.shape[1]), -np.inf, np.zeros(0)
    s = key @ x * scale
    m = s.max()
    p = np.exp(s - m)
    z = p.sum()
    return p @ value / z, float(m + np.log(z)), p / z


class Result:
    """o and lse of an attention call with what its rounding bounds need, all
    of o's shape or lse's: sum p |v|, sqrt(sum (p v)^2), and the largest
    scale * sum |x| |key| of a row."""

    def __init__(self, rows: Tuple[int, int], dv: int):
        self.o = np.zeros(rows + (dv,))
        self.lse = np.full(rows, -np.inf)
        self.absum = np.zeros(rows + (dv,))
        self.sqsum = np.zeros(rows + (dv,))
        self.mag = np.zeros(rows)

    def put(self, t, h, x, key, value, scale):
        self.o[t, h], self.lse[t, h], p = attend(x, key, value, scale)
        if len(key):
            self.absum[t, h] = p @ np.abs(value)
            self.sqsum[t, h] = np.sqrt((p * p) @ (value * value))
            self.mag[t, h] = scale * (np.abs(key) @ np.abs(x)).max()


def decode(q, cache, table, seq_lens, cu, scale) -> Result:
    """Absorbed attention of the new tokens cu[b] .. of every sequence."""
    q = np.asarray(q, dtype=np.float64)
    r = Result(q.shape[:2], LATENT)
    for b in range(len(seq_lens)):
        n = cu[b + 1] - cu[b]
        rows = np.asarray(sequence_rows(cache, table[b], 0, seq_lens[b]), dtype=np.float64).reshape(-1, ROW)
        for i in range(n):
            seen = rows[:max(0, seq_lens[b] - n + i + 1)]
            for h in range(q.shape[1]):
                r.put(cu[b] + i, h, q[cu[b] + i, h], seen, seen[:, :LATENT], scale)
    return r


def prefill(q, kv, k_pe, cu_q, cu_k, scale, causal=True) -> Result:
    """Expanded attention: kv [Tk, H, 256] = (key 128 | value 128)."""
    q, kv, k_pe = (np.asarray(a, dtype=np.float64) for a in (q, kv, k_pe))
    r = Result(q.shape[:2], 128)
    for b in range(len(cu_q) - 1):
        nq, nk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        pe = k_pe[cu_k[b]:cu_k[b + 1]]
        for h in range(q.shape[1]):
            key = np.concatenate([kv[cu_k[b]:cu_k[b + 1], h, :128], pe], axis=1)
            value = kv[cu_k[b]:cu_k[b + 1], h, 128:]
            for i in range(nq):
                seen = max(0, nk - nq + i + 1) if causal else nk
                r.put(cu_q[b] + i, h, q[cu_q[b] + i, h], key[:seen], value[:seen], scale)
    return r


def expand(rows: np.ndarray, wk: np.ndarray, wv: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """(kv [n, H, 256], k_pe [n, 64]) of cached rows [n, 576]; wk [H, 512, 128],
    wv [H, 512, 128]."""
    rows = np.asarray(rows, dtype=np.float64)
    c = rows[:, :LATENT]
    kv = np.concatenate([np.einsum("nc,hcd->nhd", c, wk), np.einsum("nc,hcd->nhd", c, wv)], axis=2)
    return kv, rows[:, LATENT:]


def absorb(q: np.ndarray, wk: np.ndarray) -> np.ndarray:
    """q [T, H, 192] -> [T, H, 576], the key expansion moved into it."""
    q = np.asarray(q, dtype=np.float64)
    return np.concatenate([np.einsum("thd,hcd->thc", q[..., :128], wk), q[..., 128:]], axis=2)


def ragged_pages(rng: np.random.Generator, lens: List[int], page: int, spare: int = 2
                 ) -> Tuple[np.ndarray, int]:
    """A block table [N, width] int32 that hands out pages in no order (-1
    where none is needed) and the number of pages."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + spare
    perm = rng.permutation(total).astype(np.int32)
    table = np.full((len(lens), max(need + [1]) + 1), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, total
