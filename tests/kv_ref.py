"""Plain 64-bit definitions of the key-value cache operators, on the CPU
(numpy), and the small batches the tests run them on.  Nothing here calls the
library; stored Q8_0 rows go through the oracle's quantizer."""
import numpy as np

import oracle as O

F32, BF16, F16, Q8 = "f32", "bf16", "f16", "q8_0"


def bf16_round(x):
    """fp32 values to the nearest bfloat16 (ties to even), as fp32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32)


def as_type(x, t):
    """fp32 values rounded to t (f32, bf16, f16), as fp32."""
    x = np.asarray(x, np.float32)
    return x if t == F32 else bf16_round(x) if t == BF16 else x.astype(np.float16).astype(np.float32)


def freqs64(n_rot, base=10000.0, scale=1.0, factors=None):
    f = scale * np.float64(base) ** (-2.0 * np.arange(n_rot // 2, dtype=np.float64) / n_rot)
    return f if factors is None else f / np.asarray(factors, np.float64)


def rotate64(x, pos, freqs, pairing, sections=None):
    """x (tokens, heads, D) fp32, pos (axes, tokens) -> float64 values."""
    y = np.asarray(x, np.float64).copy()
    half = len(freqs)
    axis = np.zeros(half, int) if sections is None else np.repeat(np.arange(len(sections)), sections)
    a = np.asarray(pos, np.float64)[axis].T * freqs  # tokens, pairs
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    if pairing == "pairs":
        i, j = np.arange(half) * 2, np.arange(half) * 2 + 1
    else:
        i, j = np.arange(half), np.arange(half) + half
    u, w = y[..., i].copy(), y[..., j].copy()
    y[..., i], y[..., j] = u * c - w * s, u * s + w * c
    return y


def stored_rows(x, cache):
    """fp32 rows (..., D) as the bytes of a cache row (..., row bytes)."""
    x = np.ascontiguousarray(x, np.float32)
    if not x.size:
        return np.zeros((*x.shape[:-1], x.shape[-1] // 32 * 34 if cache == Q8 else 2 * x.shape[-1]), np.uint8)
    if cache == Q8:
        flat = O.quantize(O.Q8_0, x.reshape(-1, x.shape[-1]))
        return np.asarray(flat).reshape(*x.shape[:-1], -1)
    if cache == F16:
        return x.astype(np.float16).view(np.uint8).reshape(*x.shape[:-1], -1)
    hi = (bf16_round(x).view(np.uint32) >> 16).astype(np.uint16)
    return hi.view(np.uint8).reshape(*x.shape[:-1], -1)


def row_values(rows, cache, dim):
    """Cache rows (..., row bytes) as float64 values (..., dim)."""
    rows = np.ascontiguousarray(rows)
    if not rows.size:
        return np.zeros((*rows.shape[:-1], dim))
    if cache == Q8:
        b = rows.reshape(*rows.shape[:-1], dim // 32, 34)
        d = np.ascontiguousarray(b[..., :2]).view(np.float16).astype(np.float64)
        q = np.ascontiguousarray(b[..., 2:]).view(np.int8).astype(np.float64)
        return (d * q).reshape(*rows.shape[:-1], dim)
    if cache == F16:
        return rows.view(np.float16).astype(np.float64)
    return (rows.view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


class Batch:
    """Sequences of (new, cached in all) tokens and their pages, shuffled
    through a pool with spare pages."""

    def __init__(self, g, seqs, page, spare=3, width_more=1):
        self.new = [n for n, _ in seqs]
        self.len = [m for _, m in seqs]
        self.page = page
        self.q_start = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.N = int(self.q_start[-1])
        need = [-(-m // page) for m in self.len]
        self.width = max(max(need), 1) + width_more
        self.n_pages = sum(need) + spare
        order = g.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((len(seqs), self.width), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n

    def tokens(self):
        """(row, sequence, index in the sequence) of every row."""
        for s, (n, m) in enumerate(zip(self.new, self.len)):
            for i in range(n):
                yield int(self.q_start[s]) + i, s, m - n + i


def attention64(q, batch, kv, vv, n_kv, scale, softcap=0.0, window=0, slopes=None, prefix=None):
    """q (N, n_q, D); kv, vv: lists of (len, n_kv, D) float64 per sequence.
    Returns (out, spread): spread bounds |terms|: sum of p |v|, and the
    largest sum of |q k| scale of a row, for tolerances."""
    N, n_q, D = q.shape
    out, T = np.zeros((N, n_q, D)), np.zeros((N, n_q, D))
    A = np.zeros((N, n_q, 1))
    G = n_q // n_kv
    for row, s, p in batch.tokens():
        L = kv[s].shape[0]
        j = np.arange(L)
        seen = (j <= p) & ((p - j < window) if window else True)
        if prefix is not None:
            seen = seen | (j < prefix[s])
        if not seen.any():
            continue
        jj = j[seen]
        for h in range(n_q):
            k, v = kv[s][jj, h // G], vv[s][jj, h // G]
            x = q[row, h].astype(np.float64)
            t = scale * (k @ x)
            A[row, h] = abs(scale) * (np.abs(k) @ np.abs(x)).max()
            if softcap:
                t = softcap * np.tanh(t / softcap)
            if slopes is not None:
                t = t - np.float64(slopes[h]) * np.abs(p - jj)
            w = np.exp(t - t.max())
            w /= w.sum()
            out[row, h], T[row, h] = w @ v, w @ np.abs(v)
    return out, T, A
