"""Appending rotated keys, values and queries on the GPU against the 64-bit
definition and the oracle's Q8_0 quantizer.

Tolerance.  The rotation is computed in 64 bits on both sides and rounded to
fp32 once.  The sides' angles and sines agree to about 1e-15 |pos|-independent
(both reduce the same fp64 angle), so fp32 values are equal but where the
64-bit value lies within ~1e-16 of a rounding border: bytes are compared for
equality.  Q8_0 codes follow from equal fp32 values by the oracle's rule."""
import numpy as np
import pytest
import torch

import block_quantized_amd as Q
import kv_ref as R
import synth
from gpu_util import assert_bytes_equal, to_cpu, to_gpu

pytestmark = pytest.mark.gpu

KIND = {R.Q8: Q.QMM_Q8_0, R.F16: Q.QMM_F16, R.BF16: Q.QMM_BF16}
DT = {R.F32: torch.float32, R.BF16: torch.bfloat16}
FILL = 0xA5


def make(g, cache, n_kv, dim, batch):
    row = Q.qmm_kv_bytes(KIND[cache], 1, dim, 16, 1) // 16
    k, v = (torch.full((batch.n_pages, n_kv, batch.page, row), FILL, dtype=torch.uint8, device="cuda") for _ in range(2))
    return Q.KVCache(k, v, KIND[cache], n_kv, dim, batch.page)


def kv_batch(b, table=None, kv_len=None, n_tokens=None):
    return Q.KVBatch(to_gpu(b.q_start), to_gpu(np.array(b.len if kv_len is None else kv_len, np.int32)),
                     to_gpu(b.table if table is None else table), b.N if n_tokens is None else n_tokens)


def expect(b, rows, cache, n_kv, page_bytes_shape, table=None, kv_len=None):
    """The pool of bytes after rows (N, n_kv, row bytes) are stored."""
    want = np.full(page_bytes_shape, FILL, np.uint8)
    table = b.table if table is None else table
    kv_len = b.len if kv_len is None else kv_len
    for row, s, _ in b.tokens():
        p = kv_len[s] - b.new[s] + (row - b.q_start[s])
        if p < 0 or p // b.page >= table.shape[1]:
            continue
        pg = table[s, p // b.page]
        if 0 <= pg < want.shape[0]:
            want[pg, :, p % b.page] = rows[row]
    return want


SEQS = ([(1, 1)], [(1, 77), (0, 30), (5, 5), (1, 16), (3, 35)], [(70, 81), (1, 17)])


@pytest.mark.parametrize("cache", [R.Q8, R.F16, R.BF16])
@pytest.mark.parametrize("xt", [R.F32, R.BF16])
@pytest.mark.parametrize("dim,n_rot,pairing", [(128, 128, "pairs"), (128, 64, "halves"), (64, 64, "halves"),
                                               (96, 96, "halves"), (96, 26, "pairs"), (192, 130, "halves"),
                                               (256, 256, "halves"), (64, 2, "pairs")])
@pytest.mark.parametrize("which", range(3))
def test_append(cache, xt, dim, n_rot, pairing, which):
    g = synth.rng(which)
    n_kv, n_q, page = (2, 6, 16) if which != 1 else (3, 3, 48)
    b = R.Batch(g, SEQS[which], page)
    k, v, q = (R.as_type(synth.normal_f32(g, (b.N, h, dim)), xt) for h in (n_kv, n_kv, n_q))
    freqs = R.freqs64(n_rot)
    c = make(g, cache, n_kv, dim, b)
    t = lambda x: to_gpu(x).to(DT[xt])  # noqa: E731
    rope = Q.Rope(to_gpu(freqs), Q.QMM_ROPE_PAIRS if pairing == "pairs" else Q.QMM_ROPE_HALVES)
    got = Q.kv_append(c, kv_batch(b), t(k), t(v), q=t(q), rope=rope)
    pos = np.array([p for _, _, p in b.tokens()])[None]
    rk, rq = (R.rotate64(x, pos, freqs, pairing).astype(np.float32) for x in (k, q))
    shape = tuple(c.k.shape)
    assert_bytes_equal(to_cpu(c.k), expect(b, R.stored_rows(rk, cache), cache, n_kv, shape), "keys")
    assert_bytes_equal(to_cpu(c.v), expect(b, R.stored_rows(v, cache), cache, n_kv, shape), "values")
    assert np.array_equal(to_cpu(got.float()), R.as_type(rq, xt)), "queries"


def test_far_positions_axes_and_strides():
    # three axes with far and negative positions, rows apart, q rotated in place
    g = synth.rng(5)
    dim, n_kv, n_q = 128, 2, 4
    b = R.Batch(g, [(9, 20), (4, 4)], 16)
    wide = torch.from_numpy(synth.normal_f32(g, (b.N, (n_q + 2 * n_kv) * dim + 8))).cuda()  # q|k|v of one product
    q, k, v = (wide[:, a * dim:e * dim].unflatten(1, (-1, dim)) for a, e in ((0, 4), (4, 6), (6, 8)))
    sections = [16, 24, 24]
    pos = g.integers(-5, 2 ** 31 - 1, (3, b.N)).astype(np.int32)
    freqs = R.freqs64(128, base=1e6, factors=np.linspace(1, 8, 64).astype(np.float32))
    got_f = Q.rope_freqs(128, 1e6, factors=to_gpu(np.linspace(1, 8, 64).astype(np.float32)))
    assert np.allclose(to_cpu(got_f), freqs, rtol=1e-14, atol=0)
    rope = Q.Rope(to_gpu(freqs), Q.QMM_ROPE_HALVES, pos=to_gpu(pos), sections=sections)
    c = make(g, R.F16, n_kv, dim, b)
    ref = {n: x.cpu().numpy() for n, x in (("q", q), ("k", k), ("v", v))}
    got = Q.kv_append(c, kv_batch(b), k, v, q=q, rope=rope)
    turn = lambda x: R.rotate64(x, pos, freqs, "halves", sections).astype(np.float32)  # noqa: E731
    assert np.array_equal(to_cpu(got), turn(ref["q"]))
    assert_bytes_equal(to_cpu(c.k), expect(b, R.stored_rows(turn(ref["k"]), R.F16), R.F16, n_kv, tuple(c.k.shape)), "keys")
    assert_bytes_equal(to_cpu(c.v), expect(b, R.stored_rows(ref["v"], R.F16), R.F16, n_kv, tuple(c.v.shape)), "values")
    own = q.contiguous()
    assert Q.kv_append(c, kv_batch(b), k, v, q=own, rope=rope, q_out=own) is own
    assert torch.equal(own, got)


def test_without_rotation_is_the_quantizer():
    g = synth.rng(6)
    b = R.Batch(g, [(33, 33)], 16)
    x = synth.normal_f32(g, (b.N, 4, 64))
    c = make(g, R.Q8, 4, 64, b)
    assert Q.kv_append(c, kv_batch(b), to_gpu(x), to_gpu(-x)) is None
    assert_bytes_equal(to_cpu(c.k), expect(b, R.stored_rows(x, R.Q8), R.Q8, 4, tuple(c.k.shape)))
    assert_bytes_equal(to_cpu(c.v), expect(b, R.stored_rows(-x, R.Q8), R.Q8, 4, tuple(c.v.shape)))
    # the whole array is rows that the library dequantizes
    rows = c.k.numel() // c.k.shape[-1]
    assert Q.dequantize(Q.QMM_Q8_0, c.k, rows, 64).shape == (rows, 64)


def test_what_must_not_be_stored():
    # missing and out-of-range pages, lengths below the new tokens and beyond
    # the table, rows behind the last sequence: nothing else is touched
    g = synth.rng(7)
    b = R.Batch(g, [(3, 40), (4, 4), (2, 50), (5, 21)], 16, width_more=0)
    table = b.table.copy()
    table[0, 2] = b.n_pages      # the page of sequence 0's new tokens is outside the pool
    table[3, 1] = -2 ** 31
    kv_len = [40, 2, 2000, 21]   # 1: two tokens before the start; 2: beyond the table
    N = b.N + 3
    x = synth.normal_f32(g, (N, 1, 64))
    q = torch.full((N, 1, 64), 7.0, device="cuda")
    c = make(g, R.F16, 1, 64, b)
    out = torch.full_like(q, -3.0)
    rope = Q.Rope(to_gpu(R.freqs64(64)), Q.QMM_ROPE_PAIRS)
    Q.kv_append(c, kv_batch(b, table, kv_len, N), to_gpu(x), to_gpu(x), q=q, rope=rope, q_out=out)
    want = expect(b, R.stored_rows(x[:b.N], R.F16), R.F16, 1, tuple(c.v.shape), table, kv_len)
    assert_bytes_equal(to_cpu(c.v), want)
    assert (want != FILL).any()
    o = to_cpu(out)
    assert np.all(o[b.N:] == -3.0) and not np.any(o[:b.N] == -3.0)


def test_garbage_metadata_stays_in_bounds():
    # contents that no program means: every access stays inside the buffers
    g = synth.rng(8)
    b = R.Batch(g, [(4, 9), (4, 9)], 16)
    c = make(g, R.Q8, 2, 64, b)
    guard = c.k.clone()
    x = to_gpu(synth.normal_f32(g, (b.N, 2, 64)))
    for q_start, kv_len in (([5, -7, 2 ** 31 - 1], [2 ** 31 - 1, -2 ** 31]), ([0, 3, 1], [-1, 0]), ([8, 8, 8], [9, 9])):
        kb = Q.KVBatch(to_gpu(np.array(q_start, np.int32)), to_gpu(np.array(kv_len, np.int32)),
                       to_gpu(np.full_like(b.table, 10 ** 9)), b.N)
        Q.kv_append(c, kb, x, x, q=x, rope=Q.Rope(to_gpu(R.freqs64(64)), 0))
        torch.cuda.synchronize()
    assert torch.equal(c.k, guard)


def test_rows_of_any_contents_are_the_quantizers():
    # infinities, NaN, zeros of both signs, subnormals, blocks whose scale
    # overflows or vanishes: byte for byte what the activation quantizer stores
    g = synth.rng(9)
    b = R.Batch(g, [(64, 64)], 64)
    x = synth.normal_f32(g, (64, 2, 64)) * np.float32(10.0) ** g.integers(-44, 38, (64, 2, 1)).astype(np.float32)
    odd = np.array([np.inf, -np.inf, np.nan, 0.0, -0.0, 1e-45, 3e38, -3e38], np.float32)
    x[:8, 0, 5] = odd
    x[8:16, 1, :32] = 0.0
    x[8:16, 1, 40] = odd
    c = make(g, R.Q8, 2, 64, b)
    Q.kv_append(c, kv_batch(b), to_gpu(x), to_gpu(x))
    want = to_cpu(Q.quantize_act(Q.QMM_Q8_0, to_gpu(x.reshape(64, 128)))).reshape(64, 2, 68)
    for pool in (c.k, c.v):
        assert_bytes_equal(to_cpu(pool), expect(b, want, R.Q8, 2, tuple(pool.shape)))
