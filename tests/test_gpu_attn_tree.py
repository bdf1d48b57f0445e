"""Attention for trees of new tokens on the GPU against the 64-bit definition.

The kernels are the ones of test_gpu_attn.py with another mask, and the
tolerances are that file's: what a key's visibility and distance are does not
change how its score and weight are rounded."""
import numpy as np
import pytest
import torch

import block_quantized_amd as Q
import draft_ref as D
import kv_ref as R
import synth
from gpu_util import to_cpu, to_gpu
from test_gpu_attn import DT, KIND, check, setup

pytestmark = pytest.mark.gpu
ALGOS = (1, 2)


def trees(g, new, branch):
    """Parents of each sequence's tokens: one of the `branch` places before each, or none."""
    return [[max(-1, i - 1 - int(g.integers(branch))) for i in range(n)] for n in new]


def run(case, parents, q, xt, n_kv, dim, algo, max_new=None, **o):
    b, c, kb, ks, vs = case
    tree = Q.KVTree(kb, to_gpu(np.array(sum(parents, []), np.int32)), max_new=max_new)
    slopes, prefix = o.get("slopes"), o.get("prefix")
    got = Q.attn(c, kb, to_gpu(q).to(DT[xt]), softcap=o.get("softcap", 0.0), window=o.get("window", 0), algo=algo, tree=tree,
                 slopes=None if slopes is None else to_gpu(slopes),
                 prefix=None if prefix is None else to_gpu(np.array(prefix, np.int32)))
    ref = D.attention_tree64(q, b, parents, ks, vs, n_kv, np.float64(np.float32(dim ** -0.5)), **o)
    bias = 0.0 if slopes is None else float(np.abs(slopes).max() * max(b.len))
    kind = {v: k for k, v in KIND.items()}[c.type]
    check(to_cpu(got.float()), ref, xt, dim, max(b.len), bias, kind, algo)
    return got


@pytest.mark.parametrize("words,new", [(1, [1, 5, 0, 64, 2]), (2, [65, 128, 3]), (3, [300, 1, 192]), (16, [1024, 700])])
def test_build(words, new):
    g = synth.rng(words)
    parents = trees(g, new, 4)
    for p in parents:  # what is no parent: too large, itself, far below
        for i, bad in zip(range(1, len(p), 7), (2 ** 31 - 1, -2 ** 31, 10 ** 6, -2)):
            p[i] = bad
        if len(p) > 2:
            p[2] = 2
    kv = [n + 10 * s for s, n in enumerate(new)]
    q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    N = int(q_start[-1]) + 3  # three rows of no sequence
    kb = Q.KVBatch(to_gpu(q_start), to_gpu(np.array(kv, np.int32)), to_gpu(np.zeros((len(new), 1), np.int32)), N)
    par = to_gpu(np.array(sum(parents, []) + [0, 0, 0], np.int32))
    c = Q.qmm_kv_tree()
    seen = torch.full((N, words), 0x5A5A5A5A5A5A5A5A, dtype=torch.int64, device="cuda")
    depth, pos = (torch.full((N,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    c.seen, c.depth, c.words = seen.data_ptr(), depth.data_ptr(), words
    assert Q.qmm_kv_tree_build(kb.c, par, c, pos) == Q.QMM_OK
    want_seen, want_depth = D.tree_arrays(parents, words)
    assert np.array_equal(to_cpu(seen)[:N - 3].view(np.uint64), want_seen)
    assert np.array_equal(to_cpu(depth)[:N - 3], want_depth)
    base = np.repeat(np.array(kv) - np.array(new), new)
    assert np.array_equal(to_cpu(pos)[:N - 3], base + want_depth)
    assert (to_cpu(seen)[N - 3:] == 0x5A5A5A5A5A5A5A5A).all() and (to_cpu(depth)[N - 3:] == 77).all() and (to_cpu(pos)[N - 3:] == 77).all()
    assert Q.qmm_kv_tree_build(kb.c, par, c, None) == Q.QMM_OK
    if max(new) <= 64 * words:
        t = Q.KVTree(kb, par, max_new=max(new))
        assert np.array_equal(to_cpu(t.seen)[:N - 3].view(np.uint64), want_seen) and t.pos.shape == (1, N)


# drafts behind caches whose lengths put the first new token before, at and
# behind borders of tiles and pages; single tokens, none at all, all tokens new
BATCH = [(9, 41), (1, 33), (64, 96), (17, 17), (0, 20), (33, 160), (5, 69)]


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("cache", [R.Q8, R.F16, R.BF16])
@pytest.mark.parametrize("xt", [R.F32, R.BF16])
@pytest.mark.parametrize("dim,n_kv,n_q", [(64, 2, 14), (96, 1, 3), (128, 2, 8), (192, 1, 1), (256, 1, 20)])
def test_trees(algo, cache, xt, dim, n_kv, n_q):
    g = synth.rng(dim)
    case = setup(g, BATCH, 16 if dim % 64 else 48, cache, n_kv, dim)
    q = R.as_type(synth.normal_f32(g, (case[0].N, n_q, dim)), xt)
    run(case, trees(g, case[0].new, 5), q, xt, n_kv, dim, algo)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("cache", [R.Q8, R.F16, R.BF16])
@pytest.mark.parametrize("options", [dict(softcap=3.0), dict(window=1), dict(window=7), dict(window=45), dict(slopes=True),
                                     dict(prefix=[0, 50, 500, 9, 3]), dict(window=20, prefix=[40, 95, 33, 0, -4]),
                                     dict(softcap=50.0, window=40, slopes=True, prefix=[10, 80, 0, 1, 9])])
def test_masks_and_scores(algo, cache, options):
    g = synth.rng(5)
    n_kv, n_q, dim = 2, 6, 64
    case = setup(g, [(1, 90), (37, 101), (3, 7), (70, 70), (25, 52)], 16, cache, n_kv, dim)
    q = R.as_type(synth.normal_f32(g, (case[0].N, n_q, dim)), R.F32)
    o = dict(options)
    if o.pop("slopes", False):
        o["slopes"] = (2.0 ** -np.arange(1, n_q + 1)).astype(np.float32)
    run(case, trees(g, case[0].new, 9), q, R.F32, n_kv, dim, algo, **o)


@pytest.mark.parametrize("algo", ALGOS)
def test_a_chain_is_a_prompt(algo):
    # parents one before another: as without a tree.  (Its rows go through all new tokens' tiles, which may divide the
    # keys in another way: both are within 2^-18 of the exact results in the 2-norm.)
    g = synth.rng(6)
    b, c, kb, ks, vs = setup(g, [(40, 130), (1, 77), (64, 64)], 32, R.F16, 2, 128)
    q = to_gpu(synth.normal_f32(g, (b.N, 8, 128)))
    par = to_gpu(np.concatenate([np.arange(n) - 1 for n in b.new]).astype(np.int32))
    tree = Q.KVTree(kb, par)
    for o in (dict(), dict(window=19), dict(slopes=to_gpu(np.full(8, 0.25, np.float32)))):
        got, want = Q.attn(c, kb, q, algo=algo, tree=tree, **o), Q.attn(c, kb, q, **o)
        assert float((got - want).norm() / want.norm()) <= 2 * 2.0 ** -18, o


@pytest.mark.parametrize("algo", (0, 1, 2))
@pytest.mark.parametrize("cache", [R.Q8, R.BF16])
def test_split_length(algo, cache):
    # few drafts behind long caches: the keys are split, and the parts joined
    g = synth.rng(8)
    case = setup(g, [(11, 5003), (3, 40), (30, 2100)], 128, cache, 1, 128)
    q = R.as_type(synth.normal_f32(g, (case[0].N, 4, 128)), R.F32)
    for o in (dict(), dict(window=900, prefix=[70, 1, 0])):
        run(case, trees(g, case[0].new, 4), q, R.F32, 1, 128, algo, **o)


@pytest.mark.parametrize("algo", ALGOS)
def test_large_tree(algo):
    # more than one word of new tokens, keys of all of them in several tiles
    g = synth.rng(9)
    case = setup(g, [(300, 331), (129, 500)], 16, R.F16, 1, 64)
    q = R.as_type(synth.normal_f32(g, (case[0].N, 2, 64)), R.F32)
    for branch in (1, 40):
        run(case, trees(g, case[0].new, branch), q, R.F32, 1, 64, algo, window=70, slopes=np.array([0.5, 0.01], np.float32))


@pytest.mark.parametrize("algo", ALGOS)
def test_more_new_tokens_than_cached_and_missing_pages(algo):
    # kv_len below the number of new tokens: the first of them have no place; a page that is none hides its keys
    g = synth.rng(10)
    b, c, kb, ks, vs = setup(g, [(20, 90), (40, 60)], 16, R.F16, 1, 64)
    parents = trees(g, b.new, 3)
    q = synth.normal_f32(g, (b.N, 2, 64))
    table = b.table.copy()
    table[0, 1] = -1
    kv_len = np.array([90, 25], np.int32)
    kb = Q.KVBatch(to_gpu(b.q_start), to_gpu(kv_len), to_gpu(table), b.N)
    got = to_cpu(Q.attn(c, kb, to_gpu(q), algo=algo, tree=Q.KVTree(kb, to_gpu(np.array(sum(parents, []), np.int32)))))
    out = np.zeros((b.N, 2, 64))
    for row, s, _ in b.tokens():
        i = row - b.q_start[s]
        base = int(kv_len[s]) - b.new[s]
        keys = [j for j in range(max(base, 0))] + [base + j for j in D.chains(parents[s])[0][i] if base + j >= 0]
        keys = [j for j in keys if table[s, j // 16] >= 0]
        if not keys:
            continue
        for h in range(2):
            t = ks[s][keys, 0] @ q[row, h].astype(np.float64) / 8
            w = np.exp(t - t.max())
            out[row, h] = w @ vs[s][keys, 0] / w.sum()
    assert np.abs(got - out).max() < 1e-4
    assert (out[b.q_start[1]] == 0).all() and (got[b.q_start[1]] == 0).all()
