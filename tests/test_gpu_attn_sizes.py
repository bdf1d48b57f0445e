"""Attention over values of very different sizes side by side, and over the
largest ones: a result's error goes by what it is a sum of."""
import numpy as np
import pytest
import torch

import block_quantized_amd as Q
import kv_ref as R
import synth
from gpu_util import to_cpu, to_gpu
from test_gpu_attn import ALGOS, setup

pytestmark = pytest.mark.gpu


def rescaled(pool, b, kv, cache, factor):
    """Multiplies row j of sequence s by factor[s][j] (heads, 32-value blocks),
    in the pool and in kv, its values."""
    width = pool.shape[-1]
    host = pool.cpu().numpy()
    for s, L in enumerate(b.len):
        for j in range(L):
            row = host[b.table[s, j // b.page], :, j % b.page]
            f = np.asarray(factor[s][j], np.float64)
            if cache == R.Q8:
                d = row.reshape(row.shape[0], -1, 34)[..., :2].copy().view(np.float16)[..., 0]
                blocks = row.reshape(row.shape[0], -1, 34).copy()
                blocks[..., :2] = (d.astype(np.float64) * f).astype(np.float16)[..., None].view(np.uint8)
                row = blocks.reshape(row.shape)
            else:
                v = R.row_values(row, cache, width // 2).reshape(row.shape[0], -1, 32) * f[..., None]
                row = R.stored_rows(v.reshape(row.shape[0], -1).astype(np.float32), cache)
            host[b.table[s, j // b.page], :, j % b.page] = row
            kv[s][j] = R.row_values(row, cache, kv[s].shape[-1])
    pool.copy_(torch.from_numpy(host))


def block_errors(got, out):
    """The relative 2-norm of the error of each row's blocks of 32 values."""
    e = (np.asarray(got, np.float64) - out).reshape(*out.shape[:2], -1, 32)
    return np.linalg.norm(e, axis=-1) / np.linalg.norm(out.reshape(e.shape), axis=-1)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("cache", [R.Q8, R.F16, R.BF16])
@pytest.mark.parametrize("where", ["block", "unseen", "unweighted", "light", "mixed"])
@pytest.mark.parametrize("ratio", [1e4, 1e6])
@pytest.mark.parametrize("dim", [64, 256])
def test_values_of_different_sizes(algo, cache, where, ratio, dim):
    """One block of values, keys that only the last rows see, keys without
    weight, or with one of about 1 / ratio, `ratio` times larger than the rest:
    every block of 32 results keeps the bound of fp32 results, 2^-18 of its own
    norm.  (The smallest step of the 16-bit parts is 2^-39 of the largest
    weight and of the largest value, 2^-19 of values 2^20 times smaller.)"""
    g = synth.rng(73)
    n_kv, n_q = 1, 2
    b, c, kb, ks, vs = setup(g, [(1, 100), (40, 90)], 16, cache, n_kv, dim)
    small = {R.Q8: 100.0, R.F16: 20.0, R.BF16: 1.0}[cache] / ratio
    factor = [np.full((L, n_kv, dim // 32), small) for L in b.len]
    slopes = None
    for f, n in zip(factor, b.len):
        if where == "block":
            f[:, :, 1] *= ratio
        elif where == "unseen":
            f[n - 2:] *= ratio
        elif where == "mixed":
            f *= ratio ** g.random(f.shape)
        else:
            f[:3] *= ratio
    if where in ("unweighted", "light"):  # by distance: the first keys are 50 to 100 away
        slopes = np.full(n_q, 1.0 if where == "unweighted" else np.log(ratio) / 50, np.float32)
    rescaled(c.v, b, vs, cache, factor)
    q = R.as_type(synth.normal_f32(g, (b.N, n_q, dim)), R.F32)
    scale = np.float64(np.float32(dim ** -0.5))
    got = to_cpu(Q.attn(c, kb, to_gpu(q), scale=float(scale), slopes=None if slopes is None else to_gpu(slopes), algo=algo))
    out = R.attention64(q, b, ks, vs, n_kv, scale, slopes=slopes)[0]
    err = block_errors(got, out)
    bias = 0.0 if slopes is None else 100 * float(slopes[0])  # off by 4 u, as in test_gpu_attn.py
    assert err.max() <= 2.0 ** -18 + 4 * bias * 2.0 ** -24, (err.max(), np.unravel_index(err.argmax(), err.shape))


@pytest.mark.parametrize("algo", ALGOS)
def test_largest_bf16_values(algo):
    # values near bf16's largest: no weight above 2 meets them on the way
    g = synth.rng(89)
    b, c, kb, ks, vs = setup(g, [(1, 20), (20, 50)], 16, R.BF16, 1, 64)
    rescaled(c.v, b, vs, R.BF16, [np.full((L, 1, 2), 2.0 ** 120) for L in b.len])
    q = R.as_type(synth.normal_f32(g, (b.N, 2, 64)) * np.float32(3), R.F32)
    scale = np.float64(np.float32(64 ** -0.5))
    got = to_cpu(Q.attn(c, kb, to_gpu(q), algo=algo)).astype(np.float64)
    out = R.attention64(q, b, ks, vs, 1, scale)[0]
    assert np.isfinite(got).all()
    assert np.linalg.norm((got - out) * 2.0 ** -120) <= 2.0 ** -18 * np.linalg.norm(out * 2.0 ** -120)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("cache", [R.Q8, R.F16, R.BF16])
@pytest.mark.parametrize("what", ["queries", "keys"])
@pytest.mark.parametrize("ratio", [1e4, 1e6])
def test_queries_and_keys_of_different_sizes(algo, cache, what, ratio):
    """Query values that are `ratio` times larger than a head's others and meet
    keys of 0, or one key that is `ratio` times larger than its neighbours and
    far from every query.  Parts of fp16 step by 2^-24 where the largest value x
    is 2^13 or more, so each value is off by 2^-38 x at most, and a score by
    scale 2^-38 x |k| (2-norm) / sqrt(3) in the root mean square, x being the
    largest of the queries here, up to 4 ratio: a result by sqrt(2) of that (weights
    above and below the line), and by less than 4 times its 2-norm bound over all
    the rows looked at."""
    g = synth.rng(103)
    dim, n_q = 64, 2
    b, c, kb, ks, vs = setup(g, [(1, 100), (40, 90)], 16, cache, 1, dim)
    q = R.as_type(synth.normal_f32(g, (b.N, n_q, dim)), R.F32)
    host = c.k.cpu().numpy()
    for s, L in enumerate(b.len):
        for j in range(L):
            k = ks[s][j].astype(np.float32)
            if what == "queries":
                k[:, :32] = 0.0
            elif j == 30:
                k[:], k[:, 0] = 0.0, -ratio / 100
            else:
                k[:, :32] /= 100
            row = R.stored_rows(k, cache)
            host[b.table[s, j // 16], :, j % 16] = row
            ks[s][j] = R.row_values(row, cache, dim)
    c.k.copy_(torch.from_numpy(host))
    if what == "queries":
        q[..., :32] *= np.float32(ratio)
    else:
        q[..., 0] = 8.0  # the large key's score is -100 or less
    scale = np.float64(np.float32(dim ** -0.5))
    got = to_cpu(Q.attn(c, kb, to_gpu(q), scale=float(scale), algo=algo))
    out = R.attention64(q, b, ks, vs, 1, scale)[0]
    err = block_errors(got, out)
    step = 4 * np.sqrt(2 / 3) * scale * 2.0 ** -38 * np.abs(q).max() * max(np.linalg.norm(k[:, 0], axis=-1)[:30].max() for k in ks)
    assert err.max() <= 2.0 ** -18 + step, (err.max(), np.unravel_index(err.argmax(), err.shape))
