"""One long sequence among short ones, each with drafts: its keys are cut into
parts that are no longer than twice the even share of what runs at once, which
the workspace shows, and the results are right.  Tolerances as in
test_gpu_attn.py."""
import numpy as np
import pytest
import torch

import block_quantized_amd as Q
import draft_ref as D
import kv_ref as R
import synth
from gpu_util import to_cpu, to_gpu
from test_gpu_attn import DT, check, setup
from test_gpu_attn_tree import trees

pytestmark = pytest.mark.gpu

LONG = 9000
TILE = 8  # tokens of a row tile: as many as a sequence has on average, one head a key-value head
BATCHES = {
    "row tiles fill the places": [8] * 64,
    "real row tiles pass them": [4] * 25 + [12] * 25,
    "places for few parts": [8] * 60,
    "more sequences than a wavefront looks through at once": [8] * 70,
    "idle sequences": [16, 0] * 32,
}


@pytest.mark.parametrize("cache,xt,dim", [(R.Q8, R.F32, 128), (R.Q8, R.BF16, 64), (R.F16, R.BF16, 128), (R.F16, R.F32, 64), (R.BF16, R.F32, 128)])
@pytest.mark.parametrize("name", BATCHES)
def test_one_long_sequence(cache, xt, dim, name):
    g = synth.rng(dim + len(name))
    new, n_kv = BATCHES[name], 8
    lens = [60 + 7 * (s % 11) for s in range(len(new))]
    lens[len(new) // 2 - len(new) // 2 % 2] = LONG
    b, c, kb, ks, vs = setup(g, [(n, m) for n, m in zip(new, lens)], 64, cache, n_kv, dim)
    parents = trees(g, new, 4)
    tree = Q.KVTree(kb, to_gpu(np.array(sum(parents, []), np.int32)), max_new=max(new))
    q = R.as_type(synth.normal_f32(g, (b.N, n_kv, dim)), xt)
    o = Q.qmm_attn_opts(dim ** -0.5, 0.0, 0, 2, None, None)
    x = Q.QMM_F32 if xt == R.F32 else Q.QMM_BF16
    need = Q.qmm_attn_tree_work(c.c, kb.c, o, x, n_kv)
    assert need > 0
    work = torch.zeros(need, dtype=torch.uint8, device="cuda")
    tq = to_gpu(q).to(DT[xt])
    out = torch.empty_like(tq)
    assert Q.qmm_attn_tree(c.c, kb.c, tree.c, o, x, tq, n_kv * dim, n_kv, out, work, need) == Q.QMM_OK
    # the workspace ends with, for each row and head, where its parts are: the first, how many (0: one), their step, and the slot
    parts = to_cpu(work[need - b.N * n_kv * 16:].view(torch.int32)).reshape(b.N, n_kv, 4)[..., 1]
    s, places = lens.index(LONG), 512 // n_kv
    blocks = [-(-n // 32) for n in lens]
    share = sum(-(-n // TILE) * k for n, k in zip(new, blocks)) / places
    cut = parts[b.q_start[s]:b.q_start[s + 1]]
    assert (cut == cut[0, 0]).all() and cut[0, 0] > 1
    # (a part has whole blocks, four at least)
    assert -(-blocks[s] // int(cut[0, 0])) <= max(2 * (share + 1), 8), (int(cut[0, 0]), share)
    extra = sum(-(-n // TILE) * (max(int(parts[a, 0]), 1) - 1) for n, a in zip(new, b.q_start) if n)
    assert extra <= places
    ref = D.attention_tree64(q, b, parents, ks, vs, n_kv, np.float64(np.float32(dim ** -0.5)))
    check(to_cpu(out.float()), ref, xt, dim, LONG, 0.0, cache, 2)
    check(to_cpu(Q.attn(c, kb, tq, tree=tree).float()), ref, xt, dim, LONG, 0.0, cache, 2)
