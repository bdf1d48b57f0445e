"""Batches that no program means, over pages that exist: whatever q_start,
kv_len, table, pos and prefix hold, nothing outside the buffers is written.
Every buffer that a call writes lies between guard bytes."""
import numpy as np
import pytest
import torch

import block_quantized_amd as Q
import synth
from gpu_util import to_gpu

pytestmark = pytest.mark.gpu

GUARD, FILL = 4096, 0x5A
ROWS, PAGES, WIDTH, PAGE = 8, 6, 4, 16
Q_STARTS = ([0, 8, 0, 8, 2, 8], [0, 3, 3, 1, 7, 8], [5, -7, 2 ** 31 - 1, 0, 8, 4], [-2 ** 31, 8, -1, 8, 8, 2 ** 31 - 1],
            [0, 1, 2, 3, 4, 5])
KV_LENS = ([64, 64, 64, 64, 64], [2 ** 31 - 1, -2 ** 31, 1, 0, 63], [5, 9, 2, 300, 17])


class Guarded:
    """A device buffer of n bytes with guards on both sides."""

    def __init__(self, n, fill=FILL):
        self.n = n
        self.whole = torch.full((n + 2 * GUARD,), fill, dtype=torch.uint8, device="cuda")
        self.whole[:GUARD] = FILL
        self.whole[GUARD + n:] = FILL

    def view(self, dtype, *shape):
        return self.whole[GUARD:GUARD + self.n].view(dtype).view(*shape)

    def kept(self):
        return bool((self.whole[:GUARD] == FILL).all() and (self.whole[GUARD + self.n:] == FILL).all())


def table(g):
    """Valid, negative and too large page numbers, valid ones several times."""
    t = g.integers(0, PAGES, (5, WIDTH)).astype(np.int32)
    t[1, 0], t[2, 1], t[3, 2], t[4, 3], t[0, 2] = -1, PAGES, 2 ** 31 - 1, -2 ** 31, 10 ** 9
    return to_gpu(t)


@pytest.mark.parametrize("kind,row", [(Q.QMM_Q8_0, 68), (Q.QMM_F16, 128), (Q.QMM_BF16, 128)])
@pytest.mark.parametrize("algo", [1, 2])
def test_attention(kind, row, algo):
    g = synth.rng(97)
    k, v = (torch.zeros(PAGES, 2, PAGE, row, dtype=torch.uint8, device="cuda") for _ in range(2))
    c = Q.KVCache(k, v, kind, 2, 64, PAGE)
    q = to_gpu(synth.normal_f32(g, (ROWS, 4, 64)))
    t, prefix = table(g), to_gpu(np.array([2 ** 31 - 1, -9, 40, 64, 0], np.int32))
    for q_start in Q_STARTS:
        for kv_len in KV_LENS:
            # max_kv too large: the keys are split although there are few
            kb = Q.KVBatch(to_gpu(np.array(q_start, np.int32)), to_gpu(np.array(kv_len, np.int32)), t, ROWS)
            for window, pre in ((0, None), (5, prefix)):
                o = Q.qmm_attn_opts(0.125, 0.0, window, algo, None, None if pre is None else pre.data_ptr())
                need = Q.qmm_attn_work(c.c, kb.c, o, Q.QMM_F32, 4)
                out, work = Guarded(ROWS * 4 * 64 * 4), Guarded(need, 0xFF)
                rc = Q.qmm_attn(c.c, kb.c, o, Q.QMM_F32, q, 256, 4, out.view(torch.float32, ROWS, 4, 64),
                                work.view(torch.uint8, need), need)
                torch.cuda.synchronize()
                assert rc == Q.QMM_OK and out.kept() and work.kept(), (q_start, kv_len, window)


@pytest.mark.parametrize("kind,row", [(Q.QMM_Q8_0, 68), (Q.QMM_F16, 128), (Q.QMM_BF16, 128)])
@pytest.mark.parametrize("algo", [1, 2])
def test_attention_in_parts(kind, row, algo):
    # the same over a table long enough that rows are split and joined
    g = synth.rng(98)
    width = 64
    k, v = (torch.zeros(PAGES, 2, PAGE, row, dtype=torch.uint8, device="cuda") for _ in range(2))
    c = Q.KVCache(k, v, kind, 2, 64, PAGE)
    q = to_gpu(synth.normal_f32(g, (ROWS, 4, 64)))
    t = to_gpu(g.integers(-2, PAGES + 2, (5, width)).astype(np.int32))
    for q_start in Q_STARTS:
        for kv_len in ([1024, 1000, 1024, 7, 513], [2 ** 31 - 1, -2 ** 31, 1, 0, 1023]):
            kb = Q.KVBatch(to_gpu(np.array(q_start, np.int32)), to_gpu(np.array(kv_len, np.int32)), t, ROWS)
            o = Q.qmm_attn_opts(0.125, 0.0, 0, algo, None, None)
            need = Q.qmm_attn_work(c.c, kb.c, o, Q.QMM_F32, 4)
            assert need > 0
            out, work = Guarded(ROWS * 4 * 64 * 4), Guarded(need, 0xFF)
            rc = Q.qmm_attn(c.c, kb.c, o, Q.QMM_F32, q, 256, 4, out.view(torch.float32, ROWS, 4, 64),
                            work.view(torch.uint8, need), need)
            torch.cuda.synchronize()
            assert rc == Q.QMM_OK and out.kept() and work.kept(), (q_start, kv_len)


@pytest.mark.parametrize("kind,row", [(Q.QMM_Q8_0, 68), (Q.QMM_F16, 128), (Q.QMM_BF16, 128)])
def test_append(kind, row):
    g = synth.rng(99)
    n = PAGES * 2 * PAGE * row
    x = to_gpu(synth.normal_f32(g, (ROWS, 2, 64)))
    freqs = to_gpu(10.0 ** -np.arange(32, dtype=np.float64))
    pos = to_gpu(g.integers(-2 ** 31, 2 ** 31 - 1, (1, ROWS)).astype(np.int32))
    t = table(g)
    for q_start in Q_STARTS:
        for kv_len in KV_LENS:
            pools = [Guarded(n), Guarded(n)]
            c = Q.KVCache(*(p.view(torch.uint8, PAGES, 2, PAGE, row) for p in pools), kind, 2, 64, PAGE)
            kb = Q.KVBatch(to_gpu(np.array(q_start, np.int32)), to_gpu(np.array(kv_len, np.int32)), t, ROWS)
            for p in (None, pos):
                q_out = Guarded(ROWS * 2 * 64 * 4)
                Q.kv_append(c, kb, x, x, q=x, rope=Q.Rope(freqs, Q.QMM_ROPE_HALVES, pos=p),
                            q_out=q_out.view(torch.float32, ROWS, 2, 64))
                torch.cuda.synchronize()
                assert q_out.kept() and all(p.kept() for p in pools), (q_start, kv_len)
