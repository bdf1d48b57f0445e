"""Offsets past 32 bits: caches of more than 4 GiB and logits of more than 2^32
bytes, and the largest counts."""
import numpy as np
import pytest
import torch

import block_quantized_amd as Q
import draft_ref as D
import kv_ref as R
import synth
from gpu_util import to_cpu, to_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,cache", [(Q.QMM_F16, R.F16), (Q.QMM_Q8_0, R.Q8)])
def test_a_cache_past_four_gigabytes(kind, cache):
    # 8 heads of 128, pages of 256 tokens: the pages in use are the last ones of 5 GiB
    n_kv, dim, page = 8, 128, 256
    row = Q.qmm_kv_bytes(kind, 1, dim, 16, 1) // 16
    n_pages = 5 * 2 ** 30 // (n_kv * page * row) + 1
    assert (n_pages - 4) * n_kv * page * row > 2 ** 32
    pools = [torch.zeros((n_pages, n_kv, page, row), dtype=torch.uint8, device="cuda") for _ in range(2)]
    c = Q.KVCache(*pools, kind, n_kv, dim, page)
    g = synth.rng(51)
    L, new = 600, 5
    pages = [n_pages - 1, n_pages - 3, n_pages - 2]
    table = to_gpu(np.array([pages], np.int32))
    vals = []
    for p in pools:
        rows = R.stored_rows(synth.normal_f32(g, (L, n_kv, dim)), cache)
        t = to_gpu(rows)
        for j0 in range(0, L, page):
            p[pages[j0 // page], :, :min(page, L - j0)] = t[j0:j0 + page].transpose(0, 1)
        vals.append(R.row_values(rows, cache, dim))
    kb = Q.KVBatch(to_gpu(np.array([0, new], np.int32)), to_gpu(np.array([L], np.int32)), table, new)
    parents = [-1, 0, 0, 1, 2]
    q = synth.normal_f32(g, (new, 2 * n_kv, dim))

    class B:
        tokens = staticmethod(lambda: [(i, 0, L - new + i) for i in range(new)])
        len, new = [L], [5]

    out, T, A = D.attention_tree64(q, B, [parents], [vals[0]], [vals[1]], n_kv, dim ** -0.5)
    for algo in (1, 2):
        got = to_cpu(Q.attn(c, kb, to_gpu(q), algo=algo, tree=Q.KVTree(kb, to_gpu(np.array(parents, np.int32)))))
        assert np.linalg.norm(got - out) <= 2.0 ** -18 * np.linalg.norm(out)
    # a copy from the last page to the first, and back past 4 GiB; rows that move within the last pages
    l = Q.KVLayers([c])
    last = pools[0][pages[0]].clone()
    Q.kv_copy(l, to_gpu(np.array([pages[0]], np.int32)), to_gpu(np.array([0], np.int32)))
    assert torch.equal(pools[0][0], last)
    Q.kv_copy(l, to_gpu(np.array([0], np.int32)), to_gpu(np.array([n_pages - 4], np.int32)), rows=to_gpu(np.array([7], np.int32)))
    assert torch.equal(pools[0][n_pages - 4, :, :7], last[:, :7]) and not pools[0][n_pages - 4, :, 7:].any()
    keep = np.array([[597, 599]], np.int32)
    want = [pools[1][pages[2], :, j - 512].clone() for j in (597, 599)]
    Q.kv_compact(l, table, to_gpu(np.array([595], np.int32)), to_gpu(keep), to_gpu(np.array([2], np.int32)))
    assert all(torch.equal(pools[1][pages[2], :, 595 + i - 512], w) for i, w in enumerate(want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_far_apart(dtype):
    g = synth.rng(52)
    vocab, ld = 30001, 2 ** 31 // 2 + 12345  # values: the third row begins past 2^32 bytes
    whole = torch.empty(2 * ld + vocab, dtype=dtype, device="cuda")
    x = synth.normal_f32(g, (3, vocab), 3.0)
    t = whole.as_strided((3, vocab), (ld, 1))
    t.copy_(to_gpu(x))
    got = Q.logprobs(t, top=7)
    near = Q.logprobs(t.contiguous(), top=7)
    # (rows that begin elsewhere among 16 bytes are summed in another order: both within 2 (V / 256 + 274) 2^-24)
    tol = 4 * (vocab / 256 + 274) * 2.0 ** -24
    assert torch.equal(got.top_ids, near.top_ids)
    assert (got.top - near.top).abs().max() <= tol * 2 and ((got.entropy - near.entropy).abs() <= tol * (1 + near.entropy)).all()


def test_most_rows_and_longest_vocabulary():
    n = 2 ** 20 + 3
    x = torch.zeros(n, 3, device="cuda")
    x[:, 1] = 1.0
    got = Q.logprobs(x, top=1)
    assert (got.top_ids == 1).all()
    want = float(torch.log_softmax(torch.tensor([0.0, 1.0, 0.0], dtype=torch.float64), 0)[1])
    assert (got.top - want).abs().max() < 1e-6
    v = 2 ** 28
    y = torch.full((1, v), -3.0, dtype=torch.bfloat16, device="cuda")
    y[0, v - 1] = 2.0
    got = Q.logprobs(y, tokens=to_gpu(np.array([[0, v - 1]], np.int32)), top=2)
    rest = (v - 1) * np.exp(-5.0)
    assert got.top_ids.tolist() == [[v - 1, 0]]
    # parts of 2^20 values: sums of 2^20 / 256 terms a lane in 32s, so 2^-24 (V / (256 parts 256) + 66 + ..) as in the header of the sizes' test
    assert abs(float(got.tokens[0, 1]) + np.log1p(rest)) < 4 * 2.0 ** -24 * (2 ** 28 / 2 ** 16 + 300)


def test_most_sequences():
    # 65536 sequences of one new token each, and 4096 heads
    n = 65536
    kb = Q.KVBatch(torch.arange(n + 1, dtype=torch.int32, device="cuda"), torch.ones(n, dtype=torch.int32, device="cuda"),
                   torch.zeros(n, 1, dtype=torch.int32, device="cuda"), n)
    tree = Q.KVTree(kb, torch.full((n,), -1, dtype=torch.int32, device="cuda"), max_new=1)
    assert (tree.seen == 1).all() and (tree.depth == 0).all() and (tree.pos == 0).all()
    c = Q.KVCache.allocate(Q.QMM_F16, 1, 64, 16, 1)
    c.k.fill_(0.5), c.v.fill_(0.25)
    q = torch.ones(8, 4096, 64, device="cuda")
    kb = Q.KVBatch(to_gpu(np.array([0, 8], np.int32)), to_gpu(np.array([8], np.int32)), to_gpu(np.array([[0]], np.int32)), 8)
    tree = Q.KVTree(kb, to_gpu(np.array([-1, 0, 0, 1, 1, 2, 2, 3], np.int32)))
    for algo in (0, 1, 2):
        assert (Q.attn(c, kb, q, tree=tree, algo=algo) - 0.25).abs().max() < 1e-6
