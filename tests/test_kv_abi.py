"""The key-value cache's C ABI: sizes, the choice of kernels, and refusals.
None of these calls reaches the GPU: validation returns first."""
import ctypes

import pytest

import block_quantized_amd as Q

A, S = 0x7F0000000000, 0  # a fake, never dereferenced device address; the null stream


def cache(**k):
    c = dict(k=A, v=A, type=Q.QMM_Q8_0, n_kv=2, head_dim=128, page_size=16, n_pages=4)
    c.update(k)
    return Q.qmm_kv_cache(*(c[n] for n, _ in Q.qmm_kv_cache._fields_))


def batch(**k):
    b = dict(q_start=A, kv_len=A, table=A, n_seqs=2, table_width=2, n_tokens=3, max_kv=0)
    b.update(k)
    return Q.qmm_kv_batch(*(b[n] for n, _ in Q.qmm_kv_batch._fields_))


def rope(sections=(0, 0, 0, 0), **k):
    r = dict(freqs=A, pos=A, n_rot=128, pairing=0, n_axes=1)
    r.update(k)
    return Q.qmm_rope(r["freqs"], r["pos"], r["n_rot"], r["pairing"], r["n_axes"], (ctypes.c_int32 * 4)(*sections))


def opts(**k):
    o = dict(scale=0.1, softcap=0.0, window=0, algo=0, slopes=None, prefix=None)
    o.update(k)
    return Q.qmm_attn_opts(*(o[n] for n, _ in Q.qmm_attn_opts._fields_))


def append(c=cache(), b=batch(), r=None, xtype=Q.QMM_F32, k=A, ldk=256, v=A, ldv=256, q=A, ldq=512, n_q=4, q_out=A + 16):
    return Q.qmm_kv_append(c, b, r, xtype, k, ldk, v, ldv, q, ldq, n_q, q_out, S)


def attn(c=cache(), b=batch(), o=opts(), xtype=Q.QMM_F32, q=A, ldq=512, n_q=4, out=A, work=A, work_bytes=1 << 40):
    return Q.qmm_attn(c, b, o, xtype, q, ldq, n_q, out, work, work_bytes, S)


def test_bytes():
    assert Q.qmm_kv_bytes(Q.QMM_Q8_0, 8, 128, 16, 3) == 3 * 8 * 16 * 136
    assert Q.qmm_kv_bytes(Q.QMM_F16, 8, 96, 48, 3) == 3 * 8 * 48 * 192
    assert Q.qmm_kv_bytes(Q.QMM_BF16, 1, 64, 16, 1) == 16 * 128
    for bad in ((Q.QMM_Q4_0, 8, 128, 16, 3), (Q.QMM_F32, 8, 128, 16, 3), (99, 8, 128, 16, 3), (Q.QMM_F16, 0, 128, 16, 3),
                (Q.QMM_F16, 8, 80, 16, 3), (Q.QMM_F16, 8, 128, 8, 3), (Q.QMM_F16, 8, 128, 24, 3),
                (Q.QMM_F16, 8, 128, 16, 0), (Q.QMM_F16, 8, 128, 16, 2 ** 60)):
        assert Q.qmm_kv_bytes(*bad) == 0, bad


GEOMETRY = [
    (dict(c=None), Q.QMM_ERR_NULL), (dict(b=None), Q.QMM_ERR_NULL),
    (dict(c=cache(type=99)), Q.QMM_ERR_TYPE), (dict(c=cache(type=Q.QMM_Q4_K)), Q.QMM_ERR_UNSUPPORTED),
    (dict(c=cache(type=Q.QMM_F32)), Q.QMM_ERR_UNSUPPORTED),
    (dict(xtype=99), Q.QMM_ERR_TYPE), (dict(xtype=Q.QMM_F16), Q.QMM_ERR_UNSUPPORTED),
    (dict(xtype=Q.QMM_Q8_0), Q.QMM_ERR_UNSUPPORTED),
    (dict(c=cache(n_kv=0)), Q.QMM_ERR_SHAPE), (dict(c=cache(head_dim=0)), Q.QMM_ERR_SHAPE),
    (dict(c=cache(head_dim=80)), Q.QMM_ERR_UNSUPPORTED), (dict(c=cache(page_size=8)), Q.QMM_ERR_SHAPE),
    (dict(c=cache(page_size=40)), Q.QMM_ERR_SHAPE), (dict(c=cache(n_pages=0)), Q.QMM_ERR_SHAPE),
    (dict(c=cache(n_pages=2 ** 60)), Q.QMM_ERR_SHAPE),
    (dict(c=cache(k=None)), Q.QMM_ERR_NULL), (dict(c=cache(v=A + 8)), Q.QMM_ERR_ALIGN),
    (dict(b=batch(n_seqs=0)), Q.QMM_ERR_SHAPE), (dict(b=batch(n_tokens=0)), Q.QMM_ERR_SHAPE),
    (dict(b=batch(table_width=0)), Q.QMM_ERR_SHAPE), (dict(b=batch(table_width=2 ** 30)), Q.QMM_ERR_SHAPE),
    (dict(b=batch(max_kv=-1)), Q.QMM_ERR_SHAPE), (dict(b=batch(n_tokens=2 ** 31)), Q.QMM_ERR_SHAPE),
    (dict(b=batch(n_seqs=2 ** 30)), Q.QMM_ERR_SHAPE), (dict(b=batch(n_seqs=2 ** 16 + 1)), Q.QMM_ERR_SHAPE),
    (dict(b=batch(n_tokens=2 ** 23)), Q.QMM_ERR_SHAPE),
    (dict(b=batch(q_start=None)), Q.QMM_ERR_NULL), (dict(b=batch(kv_len=A + 2)), Q.QMM_ERR_ALIGN),
    (dict(b=batch(table=None)), Q.QMM_ERR_NULL),
    (dict(q=A + 4), Q.QMM_ERR_ALIGN), (dict(ldq=508), Q.QMM_ERR_SHAPE), (dict(ldq=504), Q.QMM_ERR_SHAPE),
    (dict(ldq=2 ** 62), Q.QMM_ERR_SHAPE), (dict(n_q=-4), Q.QMM_ERR_SHAPE), (dict(n_q=10 ** 6), Q.QMM_ERR_SHAPE),
]


@pytest.mark.parametrize("call", [append, attn])
@pytest.mark.parametrize("k,want", GEOMETRY)
def test_refusals_of_both(call, k, want):
    assert call(**k) == want


@pytest.mark.parametrize("k,want", [
    (dict(k=None), Q.QMM_ERR_NULL), (dict(v=None), Q.QMM_ERR_NULL), (dict(v=A + 2), Q.QMM_ERR_ALIGN),
    (dict(ldk=248), Q.QMM_ERR_SHAPE), (dict(ldv=260), Q.QMM_ERR_SHAPE),
    (dict(q=None), Q.QMM_ERR_NULL), (dict(q_out=None), Q.QMM_ERR_NULL), (dict(q=None, q_out=None), Q.QMM_ERR_NULL),
    (dict(q_out=A + 4), Q.QMM_ERR_ALIGN), (dict(q_out=A, ldq=520), Q.QMM_ERR_SHAPE), (dict(n_q=0), Q.QMM_ERR_SHAPE),
    (dict(r=rope(freqs=None)), Q.QMM_ERR_NULL), (dict(r=rope(freqs=A + 4)), Q.QMM_ERR_ALIGN),
    (dict(r=rope(pos=A + 2)), Q.QMM_ERR_ALIGN), (dict(r=rope(n_rot=0)), Q.QMM_ERR_SHAPE),
    (dict(r=rope(n_rot=63)), Q.QMM_ERR_SHAPE), (dict(r=rope(n_rot=130)), Q.QMM_ERR_SHAPE),
    (dict(r=rope(pairing=2)), Q.QMM_ERR_UNSUPPORTED), (dict(r=rope(n_axes=0)), Q.QMM_ERR_SHAPE),
    (dict(r=rope(n_axes=5)), Q.QMM_ERR_SHAPE), (dict(r=rope(n_axes=3, sections=(16, 24, 25, 0))), Q.QMM_ERR_SHAPE),
    (dict(r=rope(n_axes=2, sections=(-1, 65, 0, 0))), Q.QMM_ERR_SHAPE),
])
def test_append_refusals(k, want):
    assert append(**k) == want


@pytest.mark.parametrize("k,want", [
    (dict(q=None), Q.QMM_ERR_NULL), (dict(out=None), Q.QMM_ERR_NULL), (dict(out=A + 8), Q.QMM_ERR_ALIGN),
    (dict(n_q=3, ldq=512), Q.QMM_ERR_SHAPE), (dict(n_q=0), Q.QMM_ERR_SHAPE), (dict(o=None), Q.QMM_ERR_NULL),
    (dict(o=opts(scale=float("nan"))), Q.QMM_ERR_UNSUPPORTED), (dict(o=opts(scale=float("inf"))), Q.QMM_ERR_UNSUPPORTED),
    (dict(o=opts(softcap=-1.0)), Q.QMM_ERR_UNSUPPORTED), (dict(o=opts(window=-1)), Q.QMM_ERR_UNSUPPORTED),
    (dict(o=opts(algo=3)), Q.QMM_ERR_UNSUPPORTED), (dict(o=opts(algo=-1)), Q.QMM_ERR_UNSUPPORTED),
    (dict(o=opts(slopes=A + 2)), Q.QMM_ERR_ALIGN), (dict(o=opts(prefix=A + 1)), Q.QMM_ERR_ALIGN),
])
def test_attn_refusals(k, want):
    assert attn(**k) == want


def test_workspace_refusals():
    b = batch(n_seqs=1, n_tokens=1, table_width=512)  # one token over 8192 keys: the length is split
    need = Q.qmm_attn_work(cache(), b, opts(), Q.QMM_F32, 4)
    assert need > 0 and need % 16 == 0
    assert attn(b=b, work=None, work_bytes=need) == Q.QMM_ERR_NULL
    assert attn(b=b, work=A + 8, work_bytes=need) == Q.QMM_ERR_ALIGN
    assert attn(b=b, work_bytes=need - 1) == Q.QMM_ERR_SHAPE
    # a known bound on the lengths, or a window, lowers the number of splits
    assert Q.qmm_attn_work(cache(), batch(n_seqs=1, n_tokens=1, table_width=512, max_kv=100), opts(), Q.QMM_F32, 4) == 0
    assert Q.qmm_attn_work(cache(), b, opts(window=1000), Q.QMM_F32, 4) < need
    # rejected arguments need none
    assert Q.qmm_attn_work(cache(head_dim=80), b, opts(), Q.QMM_F32, 4) == 0
    assert Q.qmm_attn_work(cache(), b, opts(algo=7), Q.QMM_F32, 4) == 0
    assert Q.qmm_attn_work(None, b, opts(), Q.QMM_F32, 4) == 0 and Q.qmm_attn_work(cache(), None, opts(), Q.QMM_F32, 4) == 0


def test_choice():
    assert Q.qmm_attn_choice(cache(), batch(), Q.QMM_F32, 4) == 1
    assert Q.qmm_attn_choice(cache(), batch(), Q.QMM_F32, 3) == 0
    assert Q.qmm_attn_choice(cache(), batch(), Q.QMM_F16, 4) == 0
    assert Q.qmm_attn_choice(cache(page_size=15), batch(), Q.QMM_F32, 4) == 0
    # single tokens and short questions take the split kernels, prompts the tile kernels
    c = cache(n_kv=8, page_size=64)
    for n_seqs, n_tokens, width, want in ((64, 64, 256, 1), (1, 61, 32, 1), (1, 2048, 32, 2), (4, 8000, 35, 2)):
        assert Q.qmm_attn_choice(c, batch(n_seqs=n_seqs, n_tokens=n_tokens, table_width=width), Q.QMM_F32, 32) == want


def test_grids_of_too_many_workgroups():
    # 2^23 - 1 single rows of 512 heads, in row tiles of 16 (split) or 128 (tile kernels)
    c, b = cache(n_kv=512), batch(n_tokens=2 ** 23 - 1, n_seqs=1, table_width=4)
    for algo in (0, 1, 2):
        o = opts(algo=algo)
        assert Q.qmm_attn_work(c, b, o, Q.QMM_F32, 512) == 0
        assert attn(c=c, b=b, o=o, n_q=512, ldq=512 * 128) == Q.QMM_ERR_SHAPE
    assert Q.qmm_attn_choice(c, b, Q.QMM_F32, 512) == 0
    # the largest sizes of all leave no product past 64 bits behind
    c = cache(n_kv=4096, page_size=2 ** 20, n_pages=1)
    assert Q.qmm_attn_work(c, batch(n_tokens=2 ** 23 - 1, n_seqs=2 ** 16, table_width=2 ** 10), opts(algo=1), Q.QMM_F32,
                           4096) == 0


def test_rope_freqs_refusals():
    f = Q.qmm_rope_freqs
    assert f(None, 64, 1e4, 1.0, None, S) == Q.QMM_ERR_NULL
    assert f(A + 4, 64, 1e4, 1.0, None, S) == Q.QMM_ERR_ALIGN
    assert f(A, 64, 1e4, 1.0, A + 1, S) == Q.QMM_ERR_ALIGN
    assert f(A, 0, 1e4, 1.0, None, S) == Q.QMM_ERR_SHAPE and f(A, 63, 1e4, 1.0, None, S) == Q.QMM_ERR_SHAPE
    for base, scale in ((0.0, 1.0), (-2.0, 1.0), (float("nan"), 1.0), (1e4, 0.0), (1e4, float("inf"))):
        assert f(A, 64, base, scale, None, S) == Q.QMM_ERR_UNSUPPORTED


def test_holders_refuse_cpu_tensors_and_shapes():
    import torch
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    for make, code in ((lambda: Q.KVBatch(i(3), i(2), i(2, 2), 2), Q.QMM_ERR_UNSUPPORTED),
                       (lambda: Q.KVBatch(i(2), i(2), i(2, 2), 2), Q.QMM_ERR_SHAPE),
                       (lambda: Q.KVBatch(i(3).long(), i(2), i(2, 2), 2), Q.QMM_ERR_SHAPE),
                       (lambda: Q.KVBatch(i(3), i(2), i(2, 4)[:, ::2], 2), Q.QMM_ERR_SHAPE),
                       (lambda: Q.KVBatch(i(3), i(2), i(4), 2), Q.QMM_ERR_SHAPE),
                       (lambda: Q.KVCache(torch.zeros(2176), torch.zeros(2176), Q.QMM_Q8_0, 1, 80, 16), Q.QMM_ERR_UNSUPPORTED),
                       (lambda: Q.KVCache(torch.zeros(9), torch.zeros(9), Q.QMM_F16, 1, 64, 16), Q.QMM_ERR_SHAPE),
                       (lambda: Q.Rope(torch.zeros(4), 0), Q.QMM_ERR_SHAPE),
                       (lambda: Q.Rope(torch.zeros(4, dtype=torch.float64), 0, sections=[1] * 5), Q.QMM_ERR_SHAPE),
                       (lambda: Q.Rope(torch.zeros(4, dtype=torch.float64), 0, pos=i(2, 3)), Q.QMM_ERR_SHAPE),
                       (lambda: Q.Rope(torch.zeros(4, dtype=torch.float64), 0, pos=i(1)[0]), Q.QMM_ERR_SHAPE),
                       (lambda: Q.Rope(torch.zeros(4, dtype=torch.float64), 0, pos=i(1, 1, 3)), Q.QMM_ERR_SHAPE),
                       (lambda: Q.KVBatch(i(3), i(2), i(2, 2), 0), Q.QMM_ERR_SHAPE),
                       (lambda: Q.KVBatch(i(3), i(2), i(2, 2), 2 ** 23), Q.QMM_ERR_SHAPE),
                       (lambda: Q.KVBatch(i(3), i(2), i(2, 2), 2, max_kv=-1), Q.QMM_ERR_SHAPE),
                       (lambda: Q.KVCache(torch.zeros(1088), torch.zeros(1088), Q.QMM_Q8_0, 1, 64, 2 ** 32 + 16),
                        Q.QMM_ERR_UNSUPPORTED)):
        with pytest.raises(Q.QmmError) as e:
            make()
        assert e.value.code == code
