"""Attention over a paged cache on the GPU against the 64-bit definition.

Tolerance, fp32 outputs.  With u = 2^-24: a score is a sum of D products of
exact parts (at most three a product) in fp32, off by at most (3 D + 8) u S
with S = scale sum |q k| (the 8: scale, log2 e, cap, bias, the parts' last
bits; 2 u |s| more where a score passes the cap or a bias, both below S + the
bias).  exp2 turns an absolute error e of its argument into a relative e, twice
(numerator and denominator), and adds a few u itself; a sum over L keys adds
at most (L + 32) u.  So |o - o64| <= T (2 (3 D + 8) u S + 4 (bias) u + (2 L +
64) u), T = sum p |v|: worst case.  Roundings are independent, so the 2-norm
over an output is held to 2^-18 of the result's, some ten times the
square-root law's value at these sizes.

bf16 outputs add half a step, 2^-8 of the value.  The tile kernels also round
what a bf16 result need not keep: P to 16 bits (e = 2^-11 for the fp16
products, 2^-8 for a bf16 cache), which is off by at most e T, and the values
of Q8_0 rows to fp16: V adds 2^-11 T, and K moves a score by 2^-11 S, so 2 x
2^-11 S T.  In the 2-norm the roundings of the output and of P are independent
and uniform, 1/sqrt(3) of their bounds each."""
import numpy as np
import pytest
import torch

import block_quantized_amd as Q
import kv_ref as R
import synth
from gpu_util import to_cpu, to_gpu

pytestmark = pytest.mark.gpu

KIND = {R.Q8: Q.QMM_Q8_0, R.F16: Q.QMM_F16, R.BF16: Q.QMM_BF16}
DT = {R.F32: torch.float32, R.BF16: torch.bfloat16}
NAN_BYTE = 0xFF  # every 16-bit pattern of it is a NaN, and so is a Q8_0 scale
ALGOS = (1, 2)


def setup(g, seqs, page, cache, n_kv, dim, spread=1.0, width_more=1):
    b = R.Batch(g, seqs, page, width_more=width_more)
    row = Q.qmm_kv_bytes(KIND[cache], 1, dim, 16, 1) // 16
    k, v = (np.full((b.n_pages, n_kv, page, row), NAN_BYTE, np.uint8) for _ in range(2))  # stale: NaN
    ks, vs = [], []
    for s, L in enumerate(b.len):
        pair = []
        for pool in (k, v):
            rows = R.stored_rows(synth.normal_f32(g, (L, n_kv, dim), spread), cache)
            for j in range(L):
                pool[b.table[s, j // page], :, j % page] = rows[j]
            pair.append(R.row_values(rows, cache, dim) if L else np.zeros((0, n_kv, dim)))
        ks.append(pair[0]), vs.append(pair[1])
    c = Q.KVCache(to_gpu(k), to_gpu(v), KIND[cache], n_kv, dim, page)
    kb = Q.KVBatch(to_gpu(b.q_start), to_gpu(np.array(b.len, np.int32)), to_gpu(b.table), b.N)
    return b, c, kb, ks, vs


def check(got, ref, xt, dim, L, bias=0.0, cache=None, algo=1):
    """algo: 1 where only the split kernels can have run."""
    out, T, A = ref
    u = 2.0 ** -24
    got = np.asarray(got, np.float64)
    tol = T * (2 * (3 * dim + 8) * u * A + 4 * bias * u + (2 * L + 64) * u) + 1e-30
    half = 2.0 ** -8 if xt == R.BF16 else 0.0
    part = 0.0
    if xt == R.BF16 and algo != 1:
        part = 2.0 ** -8 if cache == R.BF16 else 2.0 ** -11
        tol = tol + part * T + (2.0 ** -11 * (1 + 2 * A) * T if cache == R.Q8 else 0.0)
    err = np.abs(got - out)
    bad = err > tol * (1 + half) + half * np.abs(out)
    assert not bad.any(), (np.argwhere(bad)[:4].tolist(), got[bad][:4], out[bad][:4], tol[np.broadcast_to(bad, tol.shape)][:4])
    norm = np.linalg.norm(out)
    if norm:
        rel = np.linalg.norm(err) / norm
        assert rel <= 2.0 ** -18 + np.hypot(half, 4 * part if cache == R.Q8 else part) / np.sqrt(3), rel


def run(b, c, kb, ks, vs, q, xt, n_kv, dim, algo, scale=None, softcap=0.0, window=0, slopes=None, prefix=None):
    scale = dim ** -0.5 if scale is None else scale
    got = Q.attn(c, kb, to_gpu(q).to(DT[xt]), scale=scale, softcap=softcap, window=window,
                 slopes=None if slopes is None else to_gpu(slopes), algo=algo,
                 prefix=None if prefix is None else to_gpu(np.array(prefix, np.int32)))
    assert got.dtype == DT[xt]
    ref = R.attention64(q, b, ks, vs, n_kv, np.float64(np.float32(scale)), softcap, window, slopes, prefix)
    bias = 0.0 if slopes is None else float(np.abs(slopes).max() * max(b.len))
    kind = {v: k for k, v in KIND.items()}[c.type]
    check(to_cpu(got.float()), ref, xt, dim, max(b.len), bias, kind, algo)
    return got


# one token each: lengths around the tile (32 keys), the page, and the splits;
# an empty sequence, and one with no new token
DECODE = [(1, 1), (1, 2), (1, 15), (1, 16), (1, 17), (0, 40), (1, 31), (1, 32), (1, 33), (1, 64), (1, 127), (1, 130)]


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("cache", [R.Q8, R.F16, R.BF16])
@pytest.mark.parametrize("xt", [R.F32, R.BF16])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_single_tokens(algo, cache, xt, dim):
    g = synth.rng(dim)
    n_kv, n_q, page = {64: (2, 14, 16), 96: (3, 3, 32), 128: (2, 8, 48), 192: (1, 5, 16), 256: (1, 20, 64)}[dim]
    case = setup(g, DECODE, page, cache, n_kv, dim)
    q = R.as_type(synth.normal_f32(g, (case[0].N, n_q, dim)), xt)
    run(*case, q, xt, n_kv, dim, algo)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("cache", [R.Q8, R.F16, R.BF16])
@pytest.mark.parametrize("options", [dict(softcap=3.0), dict(window=1), dict(window=45), dict(slopes=True),
                                     dict(prefix=[0, 50, 500, 9, 3]), dict(window=20, prefix=[40, 3, 33, 0, -4]),
                                     dict(softcap=50.0, window=40, slopes=True, prefix=[10, 80, 0, 1, 9]), dict(scale=0.0),
                                     dict(scale=-0.3)])
def test_masks_and_scores(algo, cache, options):
    # a mixed batch: single tokens, prompts, a prompt behind a cache
    g = synth.rng(3)
    n_kv, n_q, dim = 2, 6, 64
    case = setup(g, [(1, 90), (37, 101), (1, 7), (70, 70), (5, 32)], 16, cache, n_kv, dim)
    q = R.as_type(synth.normal_f32(g, (case[0].N, n_q, dim)), R.F32)
    o = dict(options)
    if o.pop("slopes", False):
        o["slopes"] = (2.0 ** -np.arange(1, n_q + 1)).astype(np.float32)
    run(*case, q, R.F32, n_kv, dim, algo, **o)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("cache", [R.Q8, R.F16, R.BF16])
@pytest.mark.parametrize("xt", [R.F32, R.BF16])
@pytest.mark.parametrize("dim,n_kv,n_q", [(64, 1, 1), (96, 2, 10), (128, 2, 8), (192, 1, 3), (256, 1, 2)])
def test_prompts(algo, cache, xt, dim, n_kv, n_q):
    g = synth.rng(dim + n_q)
    case = setup(g, [(2, 2), (33, 33), (130, 150), (65, 200)], 32, cache, n_kv, dim)
    q = R.as_type(synth.normal_f32(g, (case[0].N, n_q, dim)), xt)
    run(*case, q, xt, n_kv, dim, algo)


@pytest.mark.parametrize("cache", [R.Q8, R.F16, R.BF16])
def test_split_length(cache):
    # one long conversation: many splits, joined; bounds on the length change
    # the splits and not the result
    g = synth.rng(11)
    b, c, kb, ks, vs = setup(g, [(1, 5003)], 128, cache, 1, 128)
    q = R.as_type(synth.normal_f32(g, (1, 4, 128)), R.F32)
    opts = Q.qmm_attn_opts(0.1, 0.0, 0, 0, None, None)
    assert Q.qmm_attn_work(kb.c, kb.c, opts, Q.QMM_F32, 4) == 0  # (not a cache: refused)
    assert Q.qmm_attn_work(c.c, kb.c, opts, Q.QMM_F32, 4) > 0
    for max_kv in (0, 5003, 64, 700, 10 ** 12):
        kb = Q.KVBatch(kb.q_start, kb.kv_len, kb.table, b.N, max_kv=max_kv)
        run(b, c, kb, ks, vs, q, R.F32, 1, 128, 0)
        run(b, c, kb, ks, vs, q, R.F32, 1, 128, 0, window=3000, prefix=[900])


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("cache", [R.Q8, R.F16, R.BF16])
@pytest.mark.parametrize("spread", [1e-4, 30.0, 3000.0])
def test_ranges(algo, cache, spread):
    # small and large cached values, queries scaled against them so that the
    # softmax is neither flat nor a single key
    g = synth.rng(13)
    case = setup(g, [(1, 100), (40, 90)], 16, cache, 1, 128, spread=spread)
    q = R.as_type(synth.normal_f32(g, (case[0].N, 2, 128)) * np.float32(2.0 / spread), R.F32)
    run(*case, q, R.F32, 1, 128, algo)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("cache", [R.Q8, R.F16, R.BF16])
def test_rows_that_see_nothing_and_missing_pages(algo, cache):
    # a window over keys whose page is missing leaves nothing: zeros; other
    # rows ignore the missing keys; kv_len below the new tokens
    g = synth.rng(17)
    n_kv, n_q, dim, page = 1, 2, 64, 16
    b, c, kb, ks, vs = setup(g, [(1, 64), (8, 64), (4, 20)], page, cache, n_kv, dim)
    table = b.table.copy()
    table[0, 3] = -1            # the last 16 keys of sequence 0
    table[1, 1] = c.n_pages     # keys 16..31 of sequence 1
    kb = Q.KVBatch(kb.q_start, to_gpu(np.array([64, 64, 2], np.int32)), to_gpu(table), b.N)
    q = synth.normal_f32(g, (b.N, n_q, dim))
    got = to_cpu(Q.attn(c, kb, to_gpu(q), window=16, algo=algo))
    assert np.all(got[0] == 0)
    assert np.all(got[9:11] == 0)  # sequence 2: two tokens stand before its start
    full = to_cpu(Q.attn(c, kb, to_gpu(q), algo=algo))
    keep = np.r_[0:16, 32:64]
    for row, s, p in [(0, 0, 63)] + [(1 + i, 1, 56 + i) for i in range(8)] + [(11, 2, 0), (12, 2, 1)]:
        j = np.arange(48) if s == 0 else keep[keep <= p] if s == 1 else np.arange(p + 1)
        for h in range(n_q):
            w = ks[s][j, 0] @ q[row, h].astype(np.float64) * dim ** -0.5
            w = np.exp(w - w.max())
            want = (w / w.sum()) @ vs[s][j, 0]
            assert np.linalg.norm(full[row, h] - want) <= 2.0 ** -18 * np.linalg.norm(want), (row, h)
    assert np.isfinite(full).all()


@pytest.mark.parametrize("algo", ALGOS)
def test_rows_behind_the_last_and_strided_queries(algo):
    g = synth.rng(19)
    b, c, kb, ks, vs = setup(g, [(3, 30), (1, 9)], 16, R.Q8, 2, 64)
    N = b.N + 2
    kb = Q.KVBatch(kb.q_start, kb.kv_len, kb.table, N)
    wide = torch.from_numpy(synth.normal_f32(g, (N, 4 * 64 + 40))).cuda()
    q = wide[:, 8:8 + 256].unflatten(1, (4, 64))
    out = torch.full((N, 4, 64), 5.0, device="cuda")
    assert Q.attn(c, kb, q, out=out, algo=algo) is out
    o = to_cpu(out)
    assert np.all(o[b.N:] == 5.0)
    ref = R.attention64(q.cpu().numpy()[:b.N], b, ks, vs, 2, np.float64(np.float32(64 ** -0.5)))
    check(o[:b.N], ref, R.F32, 64, 30)


@pytest.mark.parametrize("algo", ALGOS)
def test_garbage_metadata_stays_in_bounds(algo):
    g = synth.rng(23)
    b, c, kb, ks, vs = setup(g, [(4, 9), (4, 9)], 16, R.Q8, 2, 64)
    q = to_gpu(synth.normal_f32(g, (b.N, 4, 64)))
    for q_start, kv_len in (([5, -7, 2 ** 31 - 1], [2 ** 31 - 1, -2 ** 31]), ([0, 3, 1], [-1, 0]), ([8, 8, 8], [9, 9])):
        kb = Q.KVBatch(to_gpu(np.array(q_start, np.int32)), to_gpu(np.array(kv_len, np.int32)),
                       to_gpu(np.full_like(b.table, 10 ** 9)), b.N)
        Q.attn(c, kb, q, window=5, prefix=to_gpu(np.array([2 ** 31 - 1, -9], np.int32)), algo=algo)
        torch.cuda.synchronize()


@pytest.mark.parametrize("cache", [R.Q8, R.F16, R.BF16])
@pytest.mark.parametrize("xt", [R.F32, R.BF16])
def test_append_then_attend(cache, xt):
    """A run as a layer makes it: a prompt, then single tokens, each appended
    and attended to, against the definition on the values stored so far."""
    g = synth.rng(29)
    n_kv, n_q, dim, page = 2, 8, 128, 16
    freqs = R.freqs64(dim, base=500000.0)
    rope = Q.Rope(Q.rope_freqs(dim, 500000.0), Q.QMM_ROPE_HALVES)
    c = Q.KVCache.allocate(KIND[cache], n_kv, dim, page, 24)
    c.k.fill_(float("nan") if cache != R.Q8 else NAN_BYTE), c.v.fill_(float("nan") if cache != R.Q8 else NAN_BYTE)
    table = g.permutation(24).astype(np.int32).reshape(2, 12)
    ks, vs = [np.zeros((0, n_kv, dim))] * 2, [np.zeros((0, n_kv, dim))] * 2
    length = np.zeros(2, int)
    for new in ((50, 3), (1, 1), (1, 0), (1, 1), (20, 1)):
        length = length + new
        q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        N = int(q_start[-1])
        x = [R.as_type(synth.normal_f32(g, (N, h, dim)), xt) for h in (n_q, n_kv, n_kv)]
        kb = Q.KVBatch(to_gpu(q_start), to_gpu(length.astype(np.int32)), to_gpu(table), N)
        q, k, v = (to_gpu(y).to(DT[xt]) for y in x)
        rq = Q.kv_append(c, kb, k, v, q=q, rope=rope)
        got = Q.attn(c, kb, rq)
        b = R.Batch.__new__(R.Batch)
        b.new, b.len, b.q_start, b.N = list(new), [int(i) for i in length], q_start, N
        pos = np.array([p for _, _, p in b.tokens()])[None]
        rot = lambda y: R.rotate64(y, pos, freqs, "halves").astype(np.float32)  # noqa: E731
        for s in range(2):
            a, e = q_start[s], q_start[s + 1]
            for store, val in ((ks, rot(x[1])), (vs, x[2])):
                store[s] = np.concatenate([store[s], R.row_values(R.stored_rows(val[a:e], cache), cache, dim)])
        ref = R.attention64(R.as_type(rot(x[0]), xt), b, ks, vs, n_kv, np.float64(np.float32(dim ** -0.5)))
        check(to_cpu(got.float()), ref, xt, dim, int(length.max()), 0.0, cache, 0)


def test_streams_and_graph():
    """On a side stream, and captured: the graph is replayed on new inputs and
    a grown cache, with eager work between the replays, two graphs in turn."""
    g = synth.rng(31)
    b, c, kb, ks, vs = setup(g, [(1, 700), (1, 90)], 16, R.Q8, 2, 64)
    qs = [to_gpu(synth.normal_f32(g, (2, 4, 64))) for _ in range(4)]
    xs = [to_gpu(synth.normal_f32(g, (2, 2, 64))) for _ in range(4)]
    rope = Q.Rope(Q.rope_freqs(64, 1e4), Q.QMM_ROPE_HALVES)

    def step(q, x, stream=None):
        return Q.attn(c, kb, Q.kv_append(c, kb, x, x, q=q, rope=rope, stream=stream), stream=stream)

    want = [step(q, x).clone() for q, x in zip(qs, xs)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(qs[1], xs[1], stream=side)
    side.synchronize()
    assert torch.equal(got, want[1])
    got = step(qs[2], xs[2], stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want[2])
    q0, x0 = qs[0].clone(), xs[0].clone()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(q0, x0)
        graphs.append((graph, out))
    for i in (1, 0, 3, 2, 1):
        q0.copy_(qs[i]), x0.copy_(xs[i])
        graph, out = graphs[i % 2]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]), i
        step(qs[(i + 1) % 4], xs[(i + 1) % 4])  # eager work between
        torch.cuda.synchronize()


def test_python_refusals():
    g = synth.rng(37)
    b, c, kb, ks, vs = setup(g, [(2, 9)], 16, R.Q8, 2, 64)
    q = torch.zeros(2, 4, 64, device="cuda")
    for call, code in ((lambda: Q.attn(c, kb, q.half()), Q.QMM_ERR_UNSUPPORTED),
                       (lambda: Q.attn(c, kb, q[:1]), Q.QMM_ERR_SHAPE),
                       (lambda: Q.attn(c, kb, q[:, :3]), Q.QMM_ERR_SHAPE),
                       (lambda: Q.attn(c, kb, q.transpose(0, 1).contiguous().transpose(0, 1)), Q.QMM_ERR_UNSUPPORTED),
                       (lambda: Q.attn(c, kb, q.cpu()), Q.QMM_ERR_UNSUPPORTED),
                       (lambda: Q.attn(c, kb, q, out=q[:, :2]), Q.QMM_ERR_SHAPE),
                       (lambda: Q.attn(c, kb, q, slopes=torch.zeros(3, device="cuda")), Q.QMM_ERR_SHAPE),
                       (lambda: Q.attn(c, kb, q, prefix=torch.zeros(1, device="cuda")), Q.QMM_ERR_SHAPE),
                       (lambda: Q.attn(c, kb, q, softcap=-1.0), Q.QMM_ERR_UNSUPPORTED),
                       (lambda: Q.kv_append(c, kb, q[:, :2], q[:, :2].bfloat16()), Q.QMM_ERR_UNSUPPORTED),
                       (lambda: Q.kv_append(c, kb, q[:, :1], q[:, :2]), Q.QMM_ERR_SHAPE),
                       (lambda: Q.kv_append(c, kb, q[:, :2], q[:, :2], q_out=q), Q.QMM_ERR_NULL),
                       (lambda: Q.kv_append(c, kb, q[:, :2], q[:, :2], q=q, rope=Q.Rope(
                           torch.ones(32, device="cuda", dtype=torch.float64), 0,
                           pos=torch.zeros(1, 3, device="cuda", dtype=torch.int32))), Q.QMM_ERR_SHAPE)):
        with pytest.raises(Q.QmmError) as e:
            call()
        assert e.value.code == code


@pytest.mark.parametrize("algo", (0, 1, 2))
@pytest.mark.parametrize("cache", [R.Q8, R.BF16])
def test_many_uneven_sequences(algo, cache):
    # more sequences than a wavefront looks at together, short ones and none
    # among them, one long: the keys are divided over all
    g = synth.rng(41)
    seqs = [(int(n), int(n) + int(m)) for n, m in zip(g.integers(0, 3, 150), g.integers(0, 40, 150))]
    seqs[97], seqs[20] = (1, 2500), (9, 700)
    case = setup(g, seqs, 16, cache, 2, 64)
    q = R.as_type(synth.normal_f32(g, (case[0].N, 4, 64)), R.F32)
    run(*case, q, R.F32, 2, 64, algo)
    b, c, kb, ks, vs = case
    kb = Q.KVBatch(kb.q_start, kb.kv_len, kb.table, b.N, max_kv=2500)
    run(b, c, kb, ks, vs, q, R.F32, 2, 64, algo, window=300)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("n_q", [40, 200])
def test_many_query_heads_of_one(algo, n_q):
    # more query heads of a key-value head than a row tile holds
    g = synth.rng(43)
    case = setup(g, [(1, 50), (5, 300)], 16, R.F16, 1, 64)
    q = R.as_type(synth.normal_f32(g, (case[0].N, n_q, 64)), R.BF16)
    run(*case, q, R.BF16, 1, 64, algo, window=170)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("spreads", [(300.0, 1e-3), (1e-3, 300.0)])
def test_keys_and_values_of_other_sizes(algo, spreads):
    # Q8_0 scales of keys and values five orders apart, in either direction
    g = synth.rng(47)
    b, c, kb, ks, vs = setup(g, [(1, 100), (40, 90)], 16, R.Q8, 1, 64)
    other = setup(synth.rng(47), [(1, 100), (40, 90)], 16, R.Q8, 1, 64)  # the same pages again
    for pool, rows, s in ((c.k, ks, spreads[0]), (c.v, vs, spreads[1])):
        blocks = pool.view(torch.int16).view(*pool.shape[:3], -1, 17)[..., 0].view(torch.float16)
        blocks.mul_(s)
        d = blocks.cpu().numpy()
        for i, L in enumerate(b.len):
            for j in range(L):
                row = pool[b.table[i, j // 16], :, j % 16].cpu().numpy()
                rows[i][j] = R.row_values(row, R.Q8, 64)
        assert np.isfinite(d).any()
    q = R.as_type(synth.normal_f32(g, (b.N, 2, 64)) * np.float32(2.0 / spreads[0]), R.F32)
    run(b, c, kb, ks, vs, q, R.F32, 1, 64, algo)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("cache", [R.Q8, R.F16])
def test_offsets_past_32_bits(algo, cache):
    # the same pages at the start and at the end of a pool of over 4 GiB each
    g = synth.rng(53)
    n_kv, dim, page = 8, 256, 256
    per = Q.qmm_kv_bytes(KIND[cache], n_kv, dim, page, 1)
    n_pages = (1 << 32) // per + 40
    if torch.cuda.mem_get_info()[0] < 3 * n_pages * per:
        pytest.skip("not enough free memory")
    c = Q.KVCache.allocate(KIND[cache], n_kv, dim, page, n_pages)
    assert c.k.numel() * c.k.element_size() > 1 << 32
    x = [to_gpu(synth.normal_f32(g, (600, n_kv, dim))) for _ in range(2)]
    q = to_gpu(synth.normal_f32(g, (600, n_kv, dim)))
    outs = []
    for first in (0, n_pages - 3):
        kb = Q.KVBatch(to_gpu(np.array([0, 600], np.int32)), to_gpu(np.array([600], np.int32)),
                       to_gpu(np.arange(first, first + 3, dtype=np.int32)[None]), 600)
        Q.kv_append(c, kb, *x)
        outs.append(Q.attn(c, kb, q, algo=algo).clone())
    assert torch.equal(*outs)
    assert torch.isfinite(outs[0]).all() and outs[0].abs().max() > 0
    del c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("algo", ALGOS)
def test_lengths_past_the_table(algo):
    # kv_len beyond the table's pages: the keys behind them do not exist, the
    # positions count on
    g = synth.rng(59)
    b, c, kb, ks, vs = setup(g, [(2, 64)], 16, R.F16, 1, 64, width_more=0)
    kb = Q.KVBatch(kb.q_start, to_gpu(np.array([80], np.int32)), kb.table, b.N)
    q = synth.normal_f32(g, (b.N, 1, 64))
    got = to_cpu(Q.attn(c, kb, to_gpu(q), window=30, algo=algo))
    for i, p in enumerate((78, 79)):
        j = np.arange(p - 29, 64)
        w = np.exp(ks[0][j, 0] @ q[i, 0].astype(np.float64) / 8)
        want = (w / w.sum()) @ vs[0][j, 0]
        assert np.linalg.norm(got[i, 0] - want) <= 2.0 ** -18 * np.linalg.norm(want)


@pytest.mark.parametrize("algo", ALGOS)
def test_capped_scores_beside_stale_pages(algo):
    # large scores under a cap in a tile whose rest holds NaNs: the masked
    # scores must not decide how the others are computed
    g = synth.rng(61)
    for cache in (R.Q8, R.F16, R.BF16):
        case = setup(g, [(1, 5), (3, 21), (1, 70)], 16, cache, 1, 64, spread=6.0)
        q = R.as_type(synth.normal_f32(g, (case[0].N, 2, 64)), R.F32)
        run(*case, q, R.F32, 1, 64, algo, softcap=2.0)


def test_two_streams_at_once_and_a_captured_prompt():
    g = synth.rng(67)
    cases = [setup(g, [(1, 900), (1, 333)], 16, R.Q8, 2, 128), setup(g, [(90, 400)], 32, R.F16, 2, 128)]
    qs = [to_gpu(synth.normal_f32(g, (c[0].N, 8, 128))) for c in cases]
    want = [Q.attn(c[1], c[2], q, window=200).clone() for c, q in zip(cases, qs)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i, (c, q) in enumerate(zip(cases, qs)):
            got[i].append(Q.attn(c[1], c[2], q, window=200, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])
    graph = torch.cuda.CUDAGraph()
    q = qs[1].clone()
    with torch.cuda.graph(graph):
        out = Q.attn(cases[1][1], cases[1][2], q, window=200)
    for k in (1.0, 0.5, 1.0):
        q.copy_(qs[1] * k)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, Q.attn(cases[1][1], cases[1][2], q, window=200))
        torch.cuda.synchronize()
    assert torch.equal(out, want[1])


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("cache", [R.Q8, R.F16])
def test_largest_window_and_tokens_before_the_first(algo, cache):
    # an index below 0 less a window of 2^31 - 1 passes 32 bits
    g = synth.rng(30)
    b, c, kb, ks, vs = setup(g, [(40, 25), (3, 2), (70, 69)], 16, cache, 1, 64)
    q = synth.normal_f32(g, (b.N, 2, 64))
    run(b, c, kb, ks, vs, q, R.F32, 1, 64, algo, window=2 ** 31 - 1)


def test_python_refuses_what_ctypes_would_cut():
    g = synth.rng(31)
    b, c, kb, ks, vs = setup(g, [(2, 9)], 16, R.F16, 2, 64)
    q = torch.zeros(2, 4, 64, device="cuda")
    for options in (dict(window=2 ** 31), dict(window=2 ** 32 + 5), dict(window=-1), dict(algo=3), dict(algo=2 ** 32 + 1)):
        with pytest.raises(Q.QmmError) as e:
            Q.attn(c, kb, q, **options)
        assert e.value.code == Q.QMM_ERR_UNSUPPORTED
    with pytest.raises(Q.QmmError):
        Q.rope_freqs(2 ** 32 + 64, 1e4)


@pytest.mark.parametrize("cache", [R.Q8, R.F16, R.BF16])
@pytest.mark.parametrize("xt", [R.F32, R.BF16])
def test_long_walks_of_the_tile_kernels(cache, xt):
    # more than 64 tiles of 64 keys in one part: page numbers are looked up for
    # 64 tiles together; a bound on the length that is too low keeps the part whole
    g = synth.rng(32)
    b, c, kb, ks, vs = setup(g, [(3, 8300), (2, 4200)], 64, cache, 1, 64)
    q = R.as_type(synth.normal_f32(g, (b.N, 2, 64)), xt)
    for max_kv in (64, 0):
        kb = Q.KVBatch(kb.q_start, kb.kv_len, kb.table, b.N, max_kv=max_kv)
        run(b, c, kb, ks, vs, q, xt, 1, 64, 2)
        run(b, c, kb, ks, vs, q, xt, 1, 64, 2, window=100, prefix=[5000, 4200])


@pytest.mark.parametrize("xt", [R.F32, R.BF16])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_joins_of_many_rows(xt, dim):
    # from 2048 rows and heads on the join gives each wavefront rows of its own
    g = synth.rng(33)
    seqs = [(1, 1100)] + [(1, 1 + (37 * i) % 50) for i in range(64)] + [(0, 9), (3, 600)]
    b, c, kb, ks, vs = setup(g, seqs, 16, R.F16, 1, dim)
    q = R.as_type(synth.normal_f32(g, (b.N, 32, dim)), xt)
    assert b.N * 32 >= 2048 and Q.qmm_attn_work(c.c, kb.c, Q.qmm_attn_opts(0.1, 0.0, 0, 1, None, None), Q.QMM_F32, 32) > 0
    run(b, c, kb, ks, vs, q, xt, 1, dim, 1)
    run(b, c, kb, ks, vs, q, xt, 1, dim, 1, window=300)
