"""A run of the calls together, as a program that drafts uses them: drafts of
several sequences are appended as trees, attended to, scored by the head's
logits, the accepted paths kept; a conversation forks.  It has to give what the
same tokens give one at a time.

Also: other streams, captured graphs and their replays, gradients."""
import numpy as np
import pytest
import torch

import block_quantized_amd as Q
import kv_ref as R
import oracle as O
import synth
from gpu_util import to_gpu

pytestmark = pytest.mark.gpu

N_Q, N_KV, DIM, PAGE, LAYERS, VOCAB = 4, 2, 64, 16, 3, 512
WIDE = N_Q * DIM


class Model:
    """A few attention layers with a residual stream, quantized products and a Q6_K head."""

    def __init__(self, seed, kind):
        g = synth.rng(seed)
        self.kind = kind
        q4 = lambda m, k: to_gpu(O.quantize(O.Q4_0, synth.normal_f32(g, (m, k), 0.08)))  # noqa: E731
        self.qkv = [[q4(WIDE, WIDE), q4(N_KV * DIM, WIDE), q4(N_KV * DIM, WIDE)] for _ in range(LAYERS)]
        self.out = [q4(WIDE, WIDE) for _ in range(LAYERS)]
        self.head = to_gpu(synth.q6_k_random(g, VOCAB, WIDE))
        self.embed = to_gpu(synth.normal_f32(g, (VOCAB, WIDE)))
        self.freqs = Q.rope_freqs(DIM, 10000.0)
        self.layers = Q.KVLayers([Q.KVCache.allocate(kind, N_KV, DIM, PAGE, 64) for _ in range(LAYERS)])

    def __call__(self, tokens, batch, tree=None):
        x = self.embed[tokens]
        n = x.shape[0]
        rope = Q.Rope(self.freqs, Q.QMM_ROPE_HALVES, pos=None if tree is None else tree.pos)
        for cache, w, o in zip(self.layers.caches, self.qkv, self.out):
            xq = Q.quantize_act(Q.QMM_Q8_0, x / x.norm(dim=1, keepdim=True) * 16)
            q, k, v = (Q.mul_mat(Q.QMM_Q4_0, m, xq, m.shape[0], n, WIDE, algo=1) for m in w)
            q = Q.kv_append(cache, batch, k.view(n, N_KV, DIM), v.view(n, N_KV, DIM), q=q.view(n, N_Q, DIM), rope=rope)
            y = Q.attn(cache, batch, q, tree=tree).view(n, WIDE)
            x = x + Q.mul_mat(Q.QMM_Q4_0, o, Q.quantize_act(Q.QMM_Q8_0, y), WIDE, n, WIDE, algo=1)
        xq = Q.quantize_act(Q.QMM_Q8_K, x / x.norm(dim=1, keepdim=True) * 16)
        return Q.mul_mat(Q.QMM_Q6_K, self.head, xq, VOCAB, n, WIDE, algo=1)


def ints(*x):
    return torch.tensor(*x, dtype=torch.int32, device="cuda")


def batch_of(new, lens, table):
    starts = np.concatenate([[0], np.cumsum(new)])
    return Q.KVBatch(ints(starts.tolist()), ints(list(lens)), table, int(starts[-1]))


@pytest.mark.parametrize("kind", [Q.QMM_F16, Q.QMM_Q8_0, Q.QMM_BF16])
def test_drafts_give_what_single_tokens_give(kind):
    g = synth.rng(31)
    table = ints(g.permutation(64)[:40].reshape(4, 10).tolist())  # the fourth sequence is for the fork
    spare = table[3].clone()
    prompts = [g.integers(0, VOCAB, n).tolist() for n in (21, 5, 40)]
    parents = [[-1, 0, 0, 1, 1, 2, 3, 6, 5], [-1, -1, 0, 2, 3], [-1, 0, 1, 2, 3, 3]]
    paths = [[0, 2, 5, 8], [1], [0, 1, 2, 3, 5]]  # what is accepted
    drafts = [g.integers(0, VOCAB, len(p)).tolist() for p in parents]
    # ---- one token at a time, along the accepted paths, then one more token each
    plain = Model(7, kind)
    lens = [len(p) for p in prompts]
    plain(torch.tensor(sum(prompts, []), device="cuda"), batch_of(lens, lens, table[:3]))
    want = [[] for _ in range(3)]
    for s in range(3):
        for i in paths[s]:
            lens[s] += 1
            want[s].append(plain(torch.tensor([drafts[s][i]], device="cuda"), batch_of([1], [lens[s]], table[s:s + 1]))[0])
    last = [17, 400, 3]
    after = plain(torch.tensor(last, device="cuda"), batch_of([1] * 3, [n + 1 for n in lens], table[:3]))
    # ---- as trees
    m = Model(7, kind)
    lens = [len(p) for p in prompts]
    m(torch.tensor(sum(prompts, []), device="cuda"), batch_of(lens, lens, table[:3]))
    new = [len(p) for p in parents]
    batch = batch_of(new, [a + b for a, b in zip(lens, new)], table[:3])
    tree = Q.KVTree(batch, ints(sum(parents, [])), max_new=max(new))
    logits = m(torch.tensor(sum(drafts, []), device="cuda"), batch, tree)
    start = np.concatenate([[0], np.cumsum(new)])
    # the layers' products are quantized: a difference in a last bit may move a code by one, 1/254 of a block's largest value
    tol = 0.03
    for s in range(3):
        for got_row, w in zip([int(start[s]) + i for i in paths[s]], want[s]):
            assert float((logits[got_row] - w).norm() / w.norm()) < tol
    lp = Q.logprobs(logits, tokens=ints([[1, 2]] * len(logits)), top=3)
    ref = torch.log_softmax(logits.double(), 1)
    assert torch.allclose(lp.tokens.double(), ref[:, 1:3], atol=1e-4)
    assert torch.equal(lp.top_ids.long(), torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :3])
    # ---- the accepted rows move together; all without a copy to the host
    width = max(len(p) for p in paths)
    keep = ints([[a + i for i in p] + [0] * (width - len(p)) for a, p in zip(lens, paths)])
    kv_len = batch.kv_len
    Q.kv_compact(m.layers, table[:3].contiguous(), ints(lens), keep, ints([len(p) for p in paths]), kv_len=kv_len)
    assert kv_len.tolist() == [a + len(p) for a, p in zip(lens, paths)]
    # ---- sequence 0 forks: whole pages are shared, its last one is copied
    n0 = int(kv_len[0])
    full, part = n0 // PAGE, n0 % PAGE
    fork = table[0].clone()
    fork[full] = spare[0]
    Q.kv_copy(m.layers, table[0, full:full + 1].contiguous(), spare[:1].contiguous(), rows=ints([part]))
    tables = torch.cat([table[:3], fork[None]]).contiguous()
    got = m(torch.tensor(last + [250], device="cuda"), batch_of([1] * 4, [n + 1 for n in kv_len.tolist()] + [n0 + 1], tables))
    for a, b in zip(got[:3], after):
        assert float((a - b).norm() / b.norm()) < tol
    # the fork's own token differs from its sibling's, and what it saw was the same
    again = m(torch.tensor([last[0]], device="cuda"), batch_of([1], [n0 + 1], fork[None].contiguous()))
    assert float((again[0] - got[0]).norm() / got[0].norm()) < tol
    assert float((got[3] - got[0]).norm()) > 0.1 * float(got[0].norm())


def small_case(g, n_pages=6):
    c = Q.KVLayers([Q.KVCache.allocate(Q.QMM_F16, 1, 64, 16, n_pages) for _ in range(2)])
    for l in c.caches:
        l.k.copy_(to_gpu(synth.normal_f32(g, tuple(l.k.shape)))), l.v.copy_(to_gpu(synth.normal_f32(g, tuple(l.v.shape))))
    return c


def step(layers, q_start, kv_len, table, parents, q, logits, tokens, src, dst, first, keep, n_keep, new_len):
    """Everything that a checking step does, on the current stream."""
    batch = Q.KVBatch(q_start, kv_len, table, q.shape[0])
    tree = Q.KVTree(batch, parents, max_new=8)
    y = Q.attn(layers.caches[0], batch, q, tree=tree)
    lp = Q.logprobs(logits, tokens=tokens, top=4)
    Q.kv_copy(layers, src, dst)
    Q.kv_compact(layers, table, first, keep, n_keep, kv_len=new_len)
    return [y, *lp, tree.pos, new_len, *[t for l in layers.caches for t in (l.k, l.v)]]


def arguments(g):
    N = 9
    return dict(q_start=ints([0, 4, 9]), kv_len=ints([30, 20]), table=ints([[0, 1], [2, 3]]), parents=ints([-1, 0, 0, 1, -1, 0, 1, 2, 2]),
                q=to_gpu(synth.normal_f32(g, (N, 2, 64))), logits=to_gpu(synth.normal_f32(g, (N, 9000))), tokens=ints([[5]] * N),
                src=ints([4]), dst=ints([5]), first=ints([26, 15]), keep=ints([[26, 28, 29], [16, 18, 0]]), n_keep=ints([3, 2]), new_len=ints([0, 0]))


def test_on_a_stream_of_ones_own():
    g = synth.rng(41)
    layers, a = small_case(g), arguments(g)
    saved = [t.clone() for l in layers.caches for t in (l.k, l.v)]
    want = [t.clone() for t in step(layers, **a)]
    for t, s in zip([t for l in layers.caches for t in (l.k, l.v)], saved):
        t.copy_(s)
    a["new_len"].zero_()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step(layers, **a)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    # the same by the calls' own argument
    for t, sv in zip([t for l in layers.caches for t in (l.k, l.v)], saved):
        t.copy_(sv)
    torch.cuda.synchronize()
    batch = Q.KVBatch(a["q_start"], a["kv_len"], a["table"], 9)
    tree = Q.KVTree(batch, a["parents"], max_new=8, stream=s)
    y = Q.attn(layers.caches[0], batch, a["q"], tree=tree, stream=s)
    lp = Q.logprobs(a["logits"], tokens=a["tokens"], top=4, stream=s)
    Q.kv_copy(layers, a["src"], a["dst"], stream=s)
    Q.kv_compact(layers, a["table"], a["first"], a["keep"], a["n_keep"], kv_len=a["new_len"], stream=s.cuda_stream)
    s.synchronize()
    got = [y, *lp, tree.pos, a["new_len"], *[t for l in layers.caches for t in (l.k, l.v)]]
    assert all(torch.equal(x, z) for x, z in zip(got, want))


def test_captured_and_replayed_with_other_contents():
    g = synth.rng(42)
    layers, a = small_case(g), arguments(g)
    pools = [t for l in layers.caches for t in (l.k, l.v)]
    saved = [t.clone() for t in pools]

    def restore():
        for t, s in zip(pools, saved):
            t.copy_(s)

    step(layers, **a)  # (loads the library)
    restore()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(layers, **a)
    for parents, kv, keep in (([-1, 0, 0, 1, -1, 0, 1, 2, 2], [30, 20], [[26, 28, 29], [16, 18, 0]]),
                              ([-1, 0, 1, 2, -1, -1, 0, 1, 0], [32, 9], [[27, 28, 31], [15, 17, 1]]),
                              ([-1, -1, -1, 2, -1, 0, 1, 2, 3], [5, 32], [[26, 27, 28], [15, 16, 17]])):
        for name, x in (("parents", parents), ("kv_len", kv), ("keep", keep)):
            a[name].copy_(ints(x))
        a["q"].copy_(torch.randn_like(a["q"]))
        a["logits"].copy_(torch.randn_like(a["logits"]))
        restore()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        restore()
        want = step(layers, **a)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_two_graphs_in_turn_keep_their_workspaces():
    # divided rows and joins in both; replayed in turn and at the same time on two streams
    g = synth.rng(43)
    x = [to_gpu(synth.normal_f32(g, (2, 100000))) for _ in range(2)]
    ref = [Q.logprobs(t, top=5) for t in x]
    graphs, outs = [], []
    for t in x:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(Q.logprobs(t, top=5))
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in x]
    torch.cuda.synchronize()
    for _ in range(5):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for o, r in zip(outs, ref):
        assert torch.equal(o.entropy, r.entropy) and torch.equal(o.top_ids, r.top_ids) and torch.equal(o.top, r.top)


def test_gradients_are_refused_not_dropped():
    layers, a = small_case(synth.rng(44)), arguments(synth.rng(44))
    batch = Q.KVBatch(a["q_start"], a["kv_len"], a["table"], 9)
    tree = Q.KVTree(batch, a["parents"])
    q, x = a["q"].clone().requires_grad_(), a["logits"].clone().requires_grad_()
    for call in (lambda: Q.attn(layers.caches[0], batch, q, tree=tree), lambda: Q.logprobs(x)):
        with pytest.raises(Q.QmmError, match="gradients") as e:
            call()
        assert e.value.code == Q.QMM_ERR_UNSUPPORTED
    with torch.no_grad():
        assert Q.attn(layers.caches[0], batch, q, tree=tree).shape == q.shape and Q.logprobs(x).entropy.shape == (9,)


def test_refusals_of_the_helpers():
    layers, a = small_case(synth.rng(45)), arguments(synth.rng(45))
    batch = Q.KVBatch(a["q_start"], a["kv_len"], a["table"], 9)
    tree = Q.KVTree(batch, a["parents"])
    other = Q.KVBatch(a["q_start"], a["kv_len"], a["table"], 8)
    one = Q.KVCache.allocate(Q.QMM_F16, 1, 64, 16, 7)
    cpu = lambda t: t.cpu()  # noqa: E731
    for call, code in ((lambda: Q.KVTree(batch, a["parents"][:5]), Q.QMM_ERR_SHAPE), (lambda: Q.KVTree(batch, a["parents"].long()), Q.QMM_ERR_SHAPE),
                       (lambda: Q.KVTree(batch, a["parents"], max_new=0), Q.QMM_ERR_SHAPE), (lambda: Q.KVTree(batch, a["parents"], max_new=1025), Q.QMM_ERR_SHAPE),
                       (lambda: Q.KVTree(batch, cpu(a["parents"])), Q.QMM_ERR_UNSUPPORTED), (lambda: Q.attn(layers.caches[0], other, a["q"][:8], tree=tree), Q.QMM_ERR_SHAPE),
                       (lambda: Q.attn(layers.caches[0], batch, a["q"], tree=tree, algo=3), Q.QMM_ERR_UNSUPPORTED),
                       (lambda: Q.KVLayers([*layers.caches, one]), Q.QMM_ERR_SHAPE), (lambda: Q.kv_copy(layers, a["src"], ints([1, 2])), Q.QMM_ERR_SHAPE),
                       (lambda: Q.kv_copy(layers, cpu(a["src"]), a["dst"]), Q.QMM_ERR_UNSUPPORTED), (lambda: Q.kv_copy(layers, a["src"], a["dst"], rows=ints([1, 2])), Q.QMM_ERR_SHAPE),
                       (lambda: Q.kv_compact(layers, a["table"], a["first"], a["keep"][0], a["n_keep"]), Q.QMM_ERR_SHAPE),
                       (lambda: Q.kv_compact(layers, a["table"], a["first"], a["keep"], a["n_keep"], kv_len=a["first"]), Q.QMM_ERR_UNSUPPORTED),
                       (lambda: Q.kv_compact(layers, a["table"], a["first"][:1], a["keep"], a["n_keep"]), Q.QMM_ERR_SHAPE),
                       (lambda: Q.kv_compact(layers, a["table"], a["first"], cpu(a["keep"]), a["n_keep"]), Q.QMM_ERR_UNSUPPORTED),
                       (lambda: Q.logprobs(a["logits"], scale=0.0), Q.QMM_ERR_UNSUPPORTED), (lambda: Q.logprobs(a["logits"][:, :3], top=4), Q.QMM_ERR_SHAPE),
                       (lambda: Q.logprobs(a["logits"][:0]), Q.QMM_ERR_SHAPE), (lambda: Q.logprobs(a["logits"], tokens=cpu(a["tokens"])), Q.QMM_ERR_UNSUPPORTED)):
        with pytest.raises(Q.QmmError) as e:
            call()
        assert e.value.code == code
    Q.kv_copy(layers, a["src"][:0], a["dst"][:0])  # nothing to do
    kv_len = ints([9, 9])
    Q.kv_compact(layers, a["table"], a["first"], a["keep"][:, :0].contiguous(), a["n_keep"], kv_len=kv_len)  # nothing is kept
    assert kv_len.tolist() == a["first"].tolist()
