"""Trees of new tokens over the forms that the kernels take: tiles of 32 and of
64 rows, half filled and full ones, several to a sequence, divided and whole
keys; masks of a caller's own; unseen rows of any contents.  Tolerances as in
test_gpu_attn.py."""
import numpy as np
import pytest
import torch

import block_quantized_amd as Q
import draft_ref as D
import kv_ref as R
import synth
from gpu_util import to_cpu, to_gpu
from test_gpu_attn import DT, KIND, check, setup
from test_gpu_attn_tree import run, trees

pytestmark = pytest.mark.gpu


# tokens of a sequence, query heads of a key-value head: 1 .. 32 rows, 33 .. 64, more
@pytest.mark.parametrize("algo", (1, 2))
@pytest.mark.parametrize("cache", [R.Q8, R.F16, R.BF16])
@pytest.mark.parametrize("xt", [R.F32, R.BF16])
@pytest.mark.parametrize("dim,new,group", [(d, *f) for d in (64, 128, 256) for f in (((7, 8, 6), 4), ((30, 32, 31), 1), ((16, 15, 13), 4), ((3, 2, 3), 20))]
                         + [(d, *f) for d in (96, 192) for f in (((1, 2, 3), 5), ((21, 40, 33), 3))])
def test_forms(algo, cache, xt, dim, new, group):
    g = synth.rng(dim + group)
    case = setup(g, [(n, n + m) for n, m in zip(new, (700, 31, 1))], 16, cache, 1, dim)
    q = R.as_type(synth.normal_f32(g, (case[0].N, group, dim)), xt)
    run(case, trees(g, case[0].new, 4), q, xt, 1, dim, algo)


@pytest.mark.parametrize("algo", (1, 2))
@pytest.mark.parametrize("cache", [R.Q8, R.F16])
@pytest.mark.parametrize("words", [1, 3])
def test_masks_of_ones_own(algo, cache, words):
    # any set of new tokens, later ones and not oneself among them; any depth
    g = synth.rng(words)
    n_kv, G, dim = 2, 3, 64
    b, c, kb, ks, vs = setup(g, [(20, 75), (60 * words, 60 * words), (5, 800)], 16, cache, n_kv, dim)
    N = b.N
    bits = g.random((N, 64 * words)) < 0.3
    depth = g.integers(0, 9, N).astype(np.int32)
    held = np.minimum(depth, np.repeat(b.new, b.new) - 1)  # no tree is deeper than it has tokens
    seen = np.zeros((N, words), np.uint64)
    for j in range(64 * words):
        seen[:, j // 64] |= bits[:, j].astype(np.uint64) << np.uint64(j % 64)
    t = Q.qmm_kv_tree()
    ts, td = to_gpu(seen.view(np.int64)), to_gpu(depth)
    t.seen, t.depth, t.words = ts.data_ptr(), td.data_ptr(), words
    q = synth.normal_f32(g, (N, n_kv * G, dim))
    slopes = np.array([0.5, 0.1, 0.02, 1.0, 0.0, 0.3], np.float32)
    for window, sl in ((0, None), (6, None), (0, slopes), (40, slopes)):
        tsl = None if sl is None else to_gpu(sl)
        o = Q.qmm_attn_opts(0.125, 0.0, window, algo, None if sl is None else tsl.data_ptr(), None)
        need = Q.qmm_attn_tree_work(c.c, kb.c, o, Q.QMM_F32, n_kv * G)
        work, out = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda"), torch.empty(N, n_kv * G, dim, device="cuda")
        tq = to_gpu(q)
        assert Q.qmm_attn_tree(c.c, kb.c, t, o, Q.QMM_F32, tq, n_kv * G * dim, n_kv * G, out, work, need) == Q.QMM_OK
        want, T, A = np.zeros(q.shape), np.zeros(q.shape), np.zeros((N, n_kv * G, 1))
        for row, s, _ in b.tokens():
            L, base, r0 = b.len[s], b.len[s] - b.new[s], int(b.q_start[s])
            place = np.concatenate([np.arange(base), base + held[r0:r0 + b.new[s]]])
            p = base + held[row]
            vis = np.concatenate([np.ones(base, bool), bits[row, :b.new[s]]])
            vis &= (p - place < window) if window else True
            if not vis.any():
                continue
            for h in range(n_kv * G):
                k, v, x = ks[s][vis, h // G], vs[s][vis, h // G], q[row, h].astype(np.float64)
                sc = 0.125 * (k @ x)
                A[row, h] = 0.125 * (np.abs(k) @ np.abs(x)).max()
                if sl is not None:
                    sc = sc - np.float64(sl[h]) * np.abs(p - place[vis])
                w = np.exp(sc - sc.max())
                w /= w.sum()
                want[row, h], T[row, h] = w @ v, w @ np.abs(v)
        kind = {v: k for k, v in KIND.items()}[c.type]
        check(to_cpu(out), (want, T, A), R.F32, dim, max(b.len), 0.0 if sl is None else float(max(b.len)), kind, algo)


@pytest.mark.parametrize("algo", (1, 2))
@pytest.mark.parametrize("cache", [R.Q8, R.F16, R.BF16])
def test_what_nobody_sees_may_be_anything(algo, cache):
    # pages' rows behind the lengths and below every window are NaN (setup fills pools with NaN bytes); keys below the window, too
    g = synth.rng(21)
    b, c, kb, ks, vs = setup(g, [(6, 300), (9, 200)], 16, cache, 1, 128)
    window = 50
    row_bytes = c.k.shape[-1]
    for pool in (c.k, c.v):
        flat = pool.view(torch.uint8).view(b.n_pages, 1, 16, -1)
        for s in range(2):
            for j in range(b.len[s] - b.new[s] - window - 1):  # below position base - window + 1
                flat[int(b.table[s, j // 16]), :, j % 16] = 0xFF
    q = R.as_type(synth.normal_f32(g, (b.N, 4, 128)), R.F32)
    run((b, c, kb, ks, vs), trees(g, b.new, 3), q, R.F32, 1, 128, algo, window=window)
    run((b, c, kb, ks, vs), trees(g, b.new, 3), q, R.F32, 1, 128, algo, window=window, softcap=20.0)
    assert row_bytes


@pytest.mark.parametrize("cache", [R.Q8, R.F16])
@pytest.mark.parametrize("algo", (1, 2))
def test_values_of_very_different_sizes(cache, algo):
    # blocks and keys 2^20 apart keep their bits: Q8_0 scales and rows from 2^-14 to 2^6, by blocks of 32 and by keys
    g = synth.rng(22)
    b = R.Batch(g, [(8, 150), (5, 37)], 16)
    dim, n_kv = 128, 1
    row = Q.qmm_kv_bytes(KIND[cache], 1, dim, 16, 1) // 16
    k, v = (np.zeros((b.n_pages, n_kv, 16, row), np.uint8) for _ in range(2))
    ks, vs = [], []
    for s, L in enumerate(b.len):
        pair = []
        for pool, by in ((k, 0), (v, 1)):
            x = synth.normal_f32(g, (L, n_kv, dim))
            if by:  # values: each block of 32 another size; a few keys of another too
                x *= (2.0 ** np.repeat([0, -14, 6, -7], 32)).astype(np.float32)
                x[::7] *= np.float32(2.0 ** -6)
            rows = R.stored_rows(x, cache)
            for j in range(L):
                pool[b.table[s, j // 16], :, j % 16] = rows[j]
            pair.append(R.row_values(rows, cache, dim))
        ks.append(pair[0]), vs.append(pair[1])
    c = Q.KVCache(to_gpu(k), to_gpu(v), KIND[cache], n_kv, dim, 16)
    kb = Q.KVBatch(to_gpu(b.q_start), to_gpu(np.array(b.len, np.int32)), to_gpu(b.table), b.N)
    parents = trees(g, b.new, 3)
    q = synth.normal_f32(g, (b.N, 4, dim))
    got = to_cpu(Q.attn(c, kb, to_gpu(q), algo=algo, tree=Q.KVTree(kb, to_gpu(np.array(sum(parents, []), np.int32)))))
    out, T, A = D.attention_tree64(q, b, parents, ks, vs, n_kv, dim ** -0.5)
    for blk in range(4):  # each block of 32 values by itself, in the 2-norm
        e = slice(32 * blk, 32 * blk + 32)
        assert np.linalg.norm(got[..., e] - out[..., e]) <= 2.0 ** -18 * np.linalg.norm(out[..., e])


def test_bf16_results_are_the_fp32_ones_rounded():
    g = synth.rng(23)
    for cache in (R.Q8, R.F16, R.BF16):
        b, c, kb, ks, vs = setup(g, [(16, 900), (12, 40)], 16, cache, 2, 64)
        par = to_gpu(np.array(sum(trees(g, b.new, 4), []), np.int32))
        q = to_gpu(R.as_type(synth.normal_f32(g, (b.N, 8, 64)), R.BF16))
        tree = Q.KVTree(kb, par)
        for algo in (1, 2):
            f32, bf = Q.attn(c, kb, q, algo=algo, tree=tree), Q.attn(c, kb, q.to(torch.bfloat16), algo=algo, tree=tree)
            diff = (f32.to(torch.bfloat16) != bf).float().mean().item()
            # both round nearly the same fp32 value: a border lies between them where they differ by 2^-16 or less of a value (weights of
            # 16 bits over bf16 rows), that is for 2^-16 / 2^-8 of the values at most, and as many again for the spread of terms
            assert diff < 2 * 2.0 ** -8, (cache, algo, diff)
            # step between neighbours: one bf16 step, 2^-7 of the value
            assert ((f32 - bf.float()).abs() <= 2.0 ** -7 * f32.abs() + 2.0 ** -16 * f32.abs().max()).all()


@pytest.mark.parametrize("cache,n_tokens", [(R.F16, 1000), (R.Q8, 1000)])
def test_many_sequences(cache, n_tokens):
    # more sequences than a wavefront looks through at once, most with one new token, one with many
    g = synth.rng(24)
    seqs = [(1, int(g.integers(1, 40))) for _ in range(150)] + [(37, 90)] + [(0, 10), (2, 2)]
    case = setup(g, seqs, 16, cache, 1, 64)
    q = R.as_type(synth.normal_f32(g, (case[0].N, 2, 64)), R.F32)
    parents = trees(g, case[0].new, 6)
    for algo in (0, 1, 2):
        run(case, parents, q, R.F32, 1, 64, algo)


@pytest.mark.parametrize("cache,dim", [(R.Q8, 64), (R.Q8, 128), (R.F16, 128), (R.BF16, 256)])
@pytest.mark.parametrize("n_kv,lens,new", [
    (32, (1900, 700, 1300), (9, 5, 12)),                                    # 16 (8) places, parts to grow until they fit
    (8, (2100, 600, 900, 1500, 1, 0, 700, 40), (16, 8, 0, 9, 1, 0, 3, 20)),  # sequences without tokens and without old keys among them
    (1, tuple(520 + 13 * (7 * i % 37) for i in range(70)), (1, 2) * 35),     # more sequences than a wavefront looks through at once
    (2, tuple(600 + 9 * (5 * i % 61) for i in range(64)), (3,) * 64)])       # as many as that
def test_divisions(cache, dim, n_kv, lens, new):
    g = synth.rng(n_kv + dim)
    case = setup(g, [(n, n + m) for n, m in zip(new, lens)], 64, cache, n_kv, dim)
    q = R.as_type(synth.normal_f32(g, (case[0].N, n_kv * 2, dim)), R.F32)
    run(case, trees(g, case[0].new, 5), q, R.F32, n_kv, dim, 2)
