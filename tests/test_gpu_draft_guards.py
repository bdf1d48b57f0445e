"""Contents that no program means: whatever the device arrays of a call hold,
nothing outside its buffers is written.  Every written buffer lies between
guard bytes."""
import numpy as np
import pytest
import torch

import block_quantized_amd as Q
import synth
from gpu_util import to_gpu
from test_gpu_kv_guards import KV_LENS, PAGE, PAGES, Q_STARTS, ROWS, Guarded, table

pytestmark = pytest.mark.gpu
BAD = [2 ** 31 - 1, -2 ** 31, 0, -1, 7, 10 ** 9]


def junk(g, *shape):
    return to_gpu(g.choice(np.array(BAD, np.int64), shape).astype(np.int32))


@pytest.mark.parametrize("words", [1, 16])
def test_tree_build(words):
    g = synth.rng(1)
    for q_start in Q_STARTS:
        for kv_len in KV_LENS:
            kb = Q.KVBatch(to_gpu(np.array(q_start, np.int32)), to_gpu(np.array(kv_len, np.int32)), table(g), ROWS)
            seen, depth, pos = Guarded(8 * ROWS * words), Guarded(4 * ROWS), Guarded(4 * ROWS)
            t = Q.qmm_kv_tree()
            t.seen, t.depth, t.words = seen.view(torch.int64, ROWS * words).data_ptr(), depth.view(torch.int32, ROWS).data_ptr(), words
            assert Q.qmm_kv_tree_build(kb.c, junk(g, ROWS), t, pos.view(torch.int32, ROWS)) == Q.QMM_OK
            torch.cuda.synchronize()
            assert seen.kept() and depth.kept() and pos.kept(), (q_start, kv_len)


@pytest.mark.parametrize("kind,row", [(Q.QMM_Q8_0, 68), (Q.QMM_F16, 128), (Q.QMM_BF16, 128)])
@pytest.mark.parametrize("algo", [1, 2])
@pytest.mark.parametrize("width", [4, 64])
def test_attention(kind, row, algo, width):
    g = synth.rng(2)
    k, v = (torch.zeros(PAGES, 2, PAGE, row, dtype=torch.uint8, device="cuda") for _ in range(2))
    c = Q.KVCache(k, v, kind, 2, 64, PAGE)
    q = to_gpu(synth.normal_f32(g, (ROWS, 4, 64)))
    prefix, slopes = to_gpu(np.array([2 ** 31 - 1, -9, 40, 64, 0], np.int32)), torch.ones(4, device="cuda")
    t = table(g) if width == 4 else to_gpu(g.integers(-2, PAGES + 2, (5, width)).astype(np.int32))
    for words in (1, 5):
        tree, depth = to_gpu(g.integers(-2 ** 63, 2 ** 63 - 1, (ROWS, words))), junk(g, ROWS)
        ct = Q.qmm_kv_tree()
        ct.seen, ct.depth, ct.words = tree.data_ptr(), depth.data_ptr(), words
        for q_start in Q_STARTS:
            for kv_len in KV_LENS + ([1024, 1000, 1024, 7, 513],):
                kb = Q.KVBatch(to_gpu(np.array(q_start, np.int32)), to_gpu(np.array(kv_len, np.int32)), t, ROWS)
                for window, sl, pre in ((0, None, None), (5, slopes, prefix)):
                    o = Q.qmm_attn_opts(0.125, 0.0, window, algo, None if sl is None else sl.data_ptr(), None if pre is None else pre.data_ptr())
                    need = Q.qmm_attn_tree_work(c.c, kb.c, o, Q.QMM_F32, 4)
                    out, work = Guarded(ROWS * 4 * 64 * 4), Guarded(need, 0xFF)
                    rc = Q.qmm_attn_tree(c.c, kb.c, ct, o, Q.QMM_F32, q, 256, 4, out.view(torch.float32, ROWS, 4, 64),
                                         work.view(torch.uint8, need), need)
                    torch.cuda.synchronize()
                    assert rc == Q.QMM_OK and out.kept() and work.kept(), (q_start, kv_len, window)


@pytest.mark.parametrize("kind,row", [(Q.QMM_Q8_0, 68), (Q.QMM_Q8_0, 102), (Q.QMM_BF16, 128)])
def test_moves(kind, row):
    g = synth.rng(3)
    dim = 96 if row == 102 else 64
    n = PAGES * 2 * PAGE * row
    for round_ in range(20):
        pools = [Guarded(n), Guarded(n), Guarded(n), Guarded(n)]
        v = [p.view(torch.uint8, PAGES, 2, PAGE, row) for p in pools]
        l = Q.KVLayers([Q.KVCache(v[0], v[1], kind, 2, dim, PAGE), Q.KVCache(v[2], v[3], kind, 2, dim, PAGE)])
        m = int(g.integers(1, 12))
        pages = g.integers(-2, PAGES + 2, (2, m)).astype(np.int32)
        Q.kv_copy(l, to_gpu(pages[0]), to_gpu(pages[1]), rows=None if round_ % 2 else junk(g, m))
        keep = g.integers(-3, 70, (5, 30)).astype(np.int32) if round_ % 3 else g.choice(np.array(BAD), (5, 30)).astype(np.int32)
        lens = Guarded(20)
        Q.kv_compact(l, table(g), to_gpu(g.choice(np.array([0, 1, -5, 60, 2 ** 31 - 1, -2 ** 31]), 5).astype(np.int32)), to_gpu(keep),
                     to_gpu(g.choice(np.array([30, 0, -1, 2 ** 31 - 1, 12]), 5).astype(np.int32)), kv_len=lens.view(torch.int32, 5))
        torch.cuda.synchronize()
        assert lens.kept() and all(p.kept() for p in pools)


@pytest.mark.parametrize("xt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 9), (2, 8191), (5, 20011), (1100, 33)])
def test_logprobs(xt, rows, vocab):
    g = synth.rng(4)
    x = to_gpu(g.standard_normal((rows, vocab), dtype=np.float32)).to(xt)
    x.view(torch.int16 if xt == torch.bfloat16 else torch.int32)[0, ::3] = -1  # NaNs
    top, given = min(vocab, 64), 3
    code = Q.QMM_BF16 if xt == torch.bfloat16 else Q.QMM_F32
    need = Q.qmm_logprobs_work(code, rows, vocab, top)
    logp, ent, ids, best, work = (Guarded(4 * rows * given), Guarded(4 * rows), Guarded(4 * rows * top), Guarded(4 * rows * top), Guarded(need, 0xFF))
    assert Q.qmm_logprobs(code, x, vocab, rows, vocab, 1.0, 0.0, junk(g, rows, given), given, logp.view(torch.float32, rows, given),
                          ent.view(torch.float32, rows), top, ids.view(torch.int32, rows, top), best.view(torch.float32, rows, top),
                          work.view(torch.uint8, need), need) == Q.QMM_OK
    torch.cuda.synchronize()
    assert all(b.kept() for b in (logp, ent, ids, best, work))
    i = ids.view(torch.int32, rows, top)
    assert ((i >= 0) & (i < vocab)).all()
    s = i.sort(1).values
    assert top == 1 or (s[:, 1:] != s[:, :-1]).all()  # each once
