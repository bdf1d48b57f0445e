"""Log probabilities, entropy and top tokens against the 64-bit definition.

Tolerance, u = 2^-24: x - m is rounded once and scaled once, so off by at most
2 u |x - m| scale; exp2 turns that into a relative error of its term and adds 2 u;
a sum of V terms of one sign, 32 a lane at a time and then in pairs, adds at most
(V / 256 + 64) u relative to it; so log1p(R) is off by at most R / (1 + R) times
that, at most (2 D scale + V / 256 + 66) u with D the largest |x - m| scale whose
weight counts (below 104 = -log of the smallest fp32, else the term is 0 in
both).  A cap adds 2^-21 of the larger of |x| and 0.35 cap to every x, scaled.
So log p within u (4 |log p| + V / 256 + 66 + 2 * 104) + cap's, the entropy (with
its terms m - x, once more) within twice that times (1 + entropy): worst case; at
V = 300000 that is 9e-5, and the square-root law's value a hundredth of it.
Where nearly all is on one token, R itself has that relative error: the log
probability of that token is held to it relative to itself."""
import numpy as np
import pytest
import torch

import block_quantized_amd as Q
import draft_ref as D
import kv_ref as R
import synth
from gpu_util import to_cpu, to_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def check(x, xt, tokens=None, top=0, scale=1.0, softcap=0.0, logits=None):
    t = to_gpu(x) if logits is None else logits
    if xt == R.BF16:
        t = t.to(torch.bfloat16) if logits is None else t
    got = Q.logprobs(t, tokens=None if tokens is None else to_gpu(tokens), top=top, scale=scale, softcap=softcap)
    lp, h, order = D.logprobs64(x, np.float64(np.float32(scale)), np.float64(np.float32(softcap)))
    V = x.shape[1]
    extra = 2.0 ** -21 * scale * np.maximum(np.minimum(np.abs(x[np.isfinite(x)]).max(initial=0), softcap), 0.35 * softcap)
    base = U * (V / 256 + 66 + 208) + 2 * extra

    def close(a, b, tol):
        a = np.asarray(a, np.float64)
        assert np.array_equal(np.isneginf(a), np.isneginf(b))
        ok = np.isneginf(b) | (np.abs(a - np.where(np.isneginf(b), 0, b)) <= tol)
        assert ok.all(), (a[~ok][:4], b[~ok][:4])

    close(to_cpu(got.entropy), h, 2 * base * (1 + h))
    if tokens is not None:
        r = np.arange(len(x))[:, None]
        inside = (tokens >= 0) & (tokens < V)
        want = np.where(inside, lp[r, np.where(inside, tokens, 0)], -np.inf)
        close(to_cpu(got.tokens), want, base + 4 * U * np.abs(np.where(np.isneginf(want), 0, want)))
    else:
        assert got.tokens is None
    if top:
        ids = to_cpu(got.top_ids)
        assert np.array_equal(ids, order[:, :top])
        want = np.take_along_axis(lp, order[:, :top], 1)
        close(to_cpu(got.top), want, base + 4 * U * np.abs(np.where(np.isneginf(want), 0, want)))
    else:
        assert got.top_ids is None and got.top is None
    return got


def rows(g, n, v, xt, spread=3.0):
    return R.as_type(synth.normal_f32(g, (n, v), spread), xt)


@pytest.mark.parametrize("xt", [R.F32, R.BF16])
@pytest.mark.parametrize("v", [1, 2, 3, 63, 64, 65, 100, 2047, 2048, 2049, 8191, 8192, 8200, 32003, 128256])
def test_sizes(xt, v):
    g = synth.rng(v)
    for n in (1, 3):
        x = rows(g, n, v, xt)
        for top in sorted({0, 1, min(v, 5), min(v, 20), min(v, 64)}):
            tokens = g.integers(0, v, (n, 4)).astype(np.int32)
            tokens[0, 1], tokens[-1, 2] = -1, v
            check(x, xt, tokens, top)


@pytest.mark.parametrize("xt", [R.F32, R.BF16])
@pytest.mark.parametrize("n,v", [(1500, 3001), (1024, 20000), (300, 50257), (5, 260000)])
def test_many_rows(xt, n, v):
    g = synth.rng(n)
    check(rows(g, n, v, xt), xt, g.integers(0, v, (n, 2)).astype(np.int32), 10)


@pytest.mark.parametrize("xt", [R.F32, R.BF16])
@pytest.mark.parametrize("scale,softcap", [(0.25, 0.0), (7.0, 0.0), (1.0, 30.0), (1.6, 5.0), (1e-3, 1e4)])
def test_scale_and_cap(xt, scale, softcap):
    g = synth.rng(2)
    check(rows(g, 4, 30011, xt, 8.0), xt, g.integers(0, 30011, (4, 3)).astype(np.int32), 12, scale, softcap)


@pytest.mark.parametrize("xt", [R.F32, R.BF16])
@pytest.mark.parametrize("kind", ["rising", "falling", "equal", "zeros of both signs", "two values", "blocks", "huge"])
@pytest.mark.parametrize("top", [1, 20, 64])
def test_orders(xt, kind, top):
    # orders that a running selection meets worst, and ties, which go by the lowest index
    g = synth.rng(3)
    v = 20011
    x = {"rising": np.arange(v), "falling": -np.arange(v), "equal": np.full(v, 1.5),
         "zeros of both signs": np.where(g.random(v) < 0.5, 0.0, -0.0), "two values": (g.random(v) < 0.01) * 4.0,
         "blocks": np.repeat(g.standard_normal(v // 100 + 1) * 5, 100)[:v],
         "huge": g.standard_normal(v) * 1e36}[kind]
    x = R.as_type(np.stack([x, x[::-1], np.roll(x, 777)]).astype(np.float32), xt)
    scale = 1e-3 if kind in ("rising", "falling") else 1e-36 if kind == "huge" else 1.0
    check(x, xt, np.array([[0], [v - 1], [5]], np.int32), top, scale)


@pytest.mark.parametrize("n", [1, 2000])
def test_masked_and_empty_rows(n):
    g = synth.rng(4)
    x = rows(g, n, 9001, R.F32)
    x[:, g.random(9001) < 0.5] = -np.inf
    x[0] = -np.inf  # nothing can be drawn
    if n > 1:
        x[1], x[1, 4000] = -np.inf, 2.0  # one token can
        x[2], x[2, [7, 8999]] = -np.finfo(np.float32).max, [1.0, 1.0]
    check(x, R.F32, np.full((n, 1), 4000, np.int32), 30, softcap=20.0)
    got = check(x, R.F32, np.full((n, 1), 4000, np.int32), 30)
    assert to_cpu(got.entropy)[0] == 0 and (to_cpu(got.top_ids)[0] == np.arange(30)).all()
    if n > 1:
        assert to_cpu(got.tokens)[1, 0] == 0 and to_cpu(got.entropy)[1] == 0
        assert abs(to_cpu(got.entropy)[2] - np.log(2)) < 1e-6


def test_nearly_certain():
    # all but one part in 10^7 on one token: what is left keeps its bits
    g = synth.rng(5)
    x = rows(g, 3, 40000, R.F32, 1.0)
    x[:, 123] = 27.0
    got = Q.logprobs(to_gpu(x), tokens=to_gpu(np.full((3, 1), 123, np.int32)), top=1)
    lp, h, _ = D.logprobs64(x)
    x64 = x.astype(np.float64)
    rest = np.exp(np.delete(x64, 123, 1) - 27.0).sum(1)
    rel = U * (40000 / 256 + 66 + 60)
    assert np.abs(to_cpu(got.tokens)[:, 0] / -np.log1p(rest) - 1).max() < rel
    assert (to_cpu(got.tokens) == to_cpu(got.top)).all() and (to_cpu(got.top_ids) == 123).all()
    e = (np.exp(np.delete(x64, 123, 1) - 27.0) * (27.0 - np.delete(x64, 123, 1))).sum(1)
    assert np.abs(to_cpu(got.entropy) / (np.log1p(rest) + e / (1 + rest)) - 1).max() < 2 * rel


@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("n", [1, 1100])
def test_rows_of_nan_and_infinity(bad, n):
    g = synth.rng(6)
    x = rows(g, n, 30000, R.F32)
    clean = x.copy()
    x[0, 17000] = bad
    got = Q.logprobs(to_gpu(x), tokens=to_gpu(np.full((n, 1), 3, np.int32)), top=8)
    assert np.isnan(to_cpu(got.entropy)[0]) and np.isnan(to_cpu(got.tokens)[0, 0]) and np.isnan(to_cpu(got.top)[0]).all()
    ids = to_cpu(got.top_ids)
    want = np.argsort(-np.where(np.isnan(x[0]), -np.inf, x[0]), kind="stable")[:8]
    assert np.array_equal(ids[0], want)
    if n > 1:
        ref = Q.logprobs(to_gpu(clean), tokens=to_gpu(np.full((n, 1), 3, np.int32)), top=8)
        assert all(torch.equal(a[1:], b[1:]) for a, b in zip(got, ref))


@pytest.mark.parametrize("xt", [R.F32, R.BF16])
def test_rows_apart_and_anywhere(xt):
    # a slice of wider rows, beginning at any value; what lies around is NaN
    g = synth.rng(7)
    for v, off, wide in ((5000, 1, 5003), (4099, 3, 5001), (8192, 5, 8200), (9, 2, 31)):
        x = rows(g, 6, v, xt)
        whole = torch.full((6, wide), float("nan"), device="cuda", dtype=torch.bfloat16 if xt == R.BF16 else torch.float32)
        part = whole[:, off:off + v]
        part.copy_(to_gpu(x))
        check(x, xt, g.integers(0, v, (6, 2)).astype(np.int32), min(9, v), logits=part)
        check(x[3:4], xt, g.integers(0, v, (1, 2)).astype(np.int32), min(9, v), logits=part[3:4])


def test_what_is_not_asked_for():
    g = synth.rng(8)
    x = rows(g, 2, 777, R.F32)
    check(x, R.F32)
    t = to_gpu(x)
    e = torch.zeros(2, device="cuda")
    assert Q.qmm_logprobs(Q.QMM_F32, t, 777, 2, 777, 1.0, 0.0, None, 0, None, e, 0, None, None, None, 0) == Q.QMM_OK
    assert np.allclose(to_cpu(e), D.logprobs64(x)[1], rtol=1e-5)
    ids, lp = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.zeros(2, 3, device="cuda")
    assert Q.qmm_logprobs(Q.QMM_F32, t, 777, 2, 777, 1.0, 0.0, None, 0, None, None, 3, ids, lp, None, 0) == Q.QMM_OK
    assert np.array_equal(to_cpu(ids), D.logprobs64(x)[2][:, :3])
