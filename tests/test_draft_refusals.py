"""What the calls for drafted tokens and logits refuse, before a GPU is needed:
every check comes before anything is enqueued."""
import ctypes

import pytest
import torch

import block_quantized_amd as Q

A, S = 1 << 20, 0  # an aligned address that is never read; the null stream
F32, BF16 = Q.QMM_F32, Q.QMM_BF16


def cache(**k):
    c = dict(k=A, v=A, type=Q.QMM_F16, n_kv=2, head_dim=64, page_size=16, n_pages=8)
    c.update(k)
    return Q.qmm_kv_cache(*c.values())


def batch(**k):
    b = dict(q_start=A, kv_len=A, table=A, n_seqs=2, table_width=4, n_tokens=6, max_kv=0)
    b.update(k)
    return Q.qmm_kv_batch(*b.values())


def tree(**k):
    t = dict(seen=A, depth=A, words=1)
    t.update(k)
    return Q.qmm_kv_tree(*t.values())


@pytest.mark.parametrize("change,code", [
    (dict(batch=None), Q.QMM_ERR_NULL), (dict(batch=batch(q_start=0)), Q.QMM_ERR_NULL), (dict(batch=batch(kv_len=0)), Q.QMM_ERR_NULL),
    (dict(parents=0), Q.QMM_ERR_NULL), (dict(tree=None), Q.QMM_ERR_NULL), (dict(tree=tree(seen=0)), Q.QMM_ERR_NULL),
    (dict(tree=tree(depth=0)), Q.QMM_ERR_NULL), (dict(tree=tree(seen=A + 8)), Q.QMM_ERR_ALIGN), (dict(tree=tree(depth=A + 2)), Q.QMM_ERR_ALIGN),
    (dict(parents=A + 1), Q.QMM_ERR_ALIGN), (dict(pos=A + 2), Q.QMM_ERR_ALIGN), (dict(batch=batch(q_start=A + 2)), Q.QMM_ERR_ALIGN),
    (dict(tree=tree(words=0)), Q.QMM_ERR_SHAPE), (dict(tree=tree(words=17)), Q.QMM_ERR_SHAPE), (dict(tree=tree(words=-1)), Q.QMM_ERR_SHAPE),
    (dict(batch=batch(n_seqs=0)), Q.QMM_ERR_SHAPE), (dict(batch=batch(n_seqs=65537)), Q.QMM_ERR_SHAPE),
    (dict(batch=batch(n_tokens=0)), Q.QMM_ERR_SHAPE), (dict(batch=batch(n_tokens=1 << 23)), Q.QMM_ERR_SHAPE)])
def test_tree_build(change, code):
    a = dict(batch=batch(), parents=A, tree=tree(), pos=0)
    a.update(change)
    assert Q.qmm_kv_tree_build(a["batch"], a["parents"], a["tree"], a["pos"], S) == code


@pytest.mark.parametrize("change,code", [
    (dict(tree=None), Q.QMM_ERR_NULL), (dict(tree=tree(words=40)), Q.QMM_ERR_SHAPE), (dict(tree=tree(seen=A + 4)), Q.QMM_ERR_ALIGN),
    (dict(cache=None), Q.QMM_ERR_NULL), (dict(opts=None), Q.QMM_ERR_NULL), (dict(xtype=Q.QMM_F16), Q.QMM_ERR_UNSUPPORTED),
    (dict(xtype=77), Q.QMM_ERR_TYPE), (dict(q=0), Q.QMM_ERR_NULL), (dict(out=0), Q.QMM_ERR_NULL), (dict(q=A + 4), Q.QMM_ERR_ALIGN),
    (dict(n_q=3), Q.QMM_ERR_SHAPE), (dict(ldq=255), Q.QMM_ERR_SHAPE), (dict(batch=batch(n_tokens=0)), Q.QMM_ERR_SHAPE),
    (dict(opts=Q.qmm_attn_opts(float("nan"), 0, 0, 0, None, None)), Q.QMM_ERR_UNSUPPORTED),
    (dict(opts=Q.qmm_attn_opts(1, 0, -1, 0, None, None)), Q.QMM_ERR_UNSUPPORTED),
    (dict(opts=Q.qmm_attn_opts(1, 0, 0, 3, None, None)), Q.QMM_ERR_UNSUPPORTED),
    (dict(batch=batch(table_width=4096), work=0), Q.QMM_ERR_NULL), (dict(batch=batch(table_width=4096), work_bytes=64), Q.QMM_ERR_SHAPE),
    (dict(batch=batch(table_width=4096), work=A + 8), Q.QMM_ERR_ALIGN)])
def test_attn_tree(change, code):
    a = dict(cache=cache(), batch=batch(), tree=tree(), opts=Q.qmm_attn_opts(1, 0, 0, 0, None, None), xtype=F32, q=A, ldq=256, n_q=4, out=A,
             work=A, work_bytes=1 << 40)
    a.update(change)
    assert Q.qmm_attn_tree(*a.values(), S) == code


@pytest.mark.parametrize("type,dim", [(Q.QMM_Q8_0, 64), (Q.QMM_Q8_0, 96), (Q.QMM_Q8_0, 256), (Q.QMM_F16, 128), (Q.QMM_BF16, 192)])
def test_attn_tree_work(type, dim):
    o = Q.qmm_attn_opts(1, 0, 0, 0, None, None)
    c = cache(type=type, head_dim=dim)
    assert Q.qmm_attn_tree_work(c, batch(table_width=4), o, F32, 4) == 0  # 64 keys: never divided
    small = Q.qmm_attn_tree_work(c, batch(table_width=4096), o, F32, 4)
    assert small > 0 and small % 16 == 0
    assert Q.qmm_attn_tree_work(c, batch(table_width=4096), o, F32, 3) == 0
    assert Q.qmm_attn_tree_work(c, batch(table_width=4096), None, F32, 4) == 0
    for tokens in (1, 64, 1000, 2 ** 23 - 1):  # no size overflows
        assert 0 <= Q.qmm_attn_tree_work(c, batch(table_width=4096, n_tokens=tokens, n_seqs=min(tokens, 65536)), o, F32, 4096) < 1 << 62


def layers(*changes):
    return (Q.qmm_kv_cache * max(1, len(changes)))(*[cache(**c) for c in changes])


@pytest.mark.parametrize("change,code", [
    (dict(caches=None), Q.QMM_ERR_NULL), (dict(count=0), Q.QMM_ERR_SHAPE), (dict(count=4097), Q.QMM_ERR_SHAPE), (dict(count=-1), Q.QMM_ERR_SHAPE),
    (dict(caches=layers({}, dict(n_pages=9)), count=2), Q.QMM_ERR_SHAPE), (dict(caches=layers({}, dict(page_size=32)), count=2), Q.QMM_ERR_SHAPE),
    (dict(caches=layers({}, dict(type=Q.QMM_BF16)), count=2), Q.QMM_ERR_SHAPE), (dict(caches=layers({}, dict(n_kv=1)), count=2), Q.QMM_ERR_SHAPE),
    (dict(caches=layers({}, dict(head_dim=128)), count=2), Q.QMM_ERR_SHAPE), (dict(caches=layers({}, dict(v=0)), count=2), Q.QMM_ERR_NULL),
    (dict(caches=layers(dict(k=A + 8))), Q.QMM_ERR_ALIGN), (dict(caches=layers(dict(type=Q.QMM_Q4_K))), Q.QMM_ERR_UNSUPPORTED),
    (dict(src=0), Q.QMM_ERR_NULL), (dict(dst=0), Q.QMM_ERR_NULL), (dict(src=A + 2), Q.QMM_ERR_ALIGN), (dict(rows=A + 1), Q.QMM_ERR_ALIGN),
    (dict(n=0), Q.QMM_ERR_SHAPE), (dict(n=-1), Q.QMM_ERR_SHAPE), (dict(n=1 << 24), Q.QMM_ERR_SHAPE), (dict(n=1 << 40), Q.QMM_ERR_SHAPE)])
def test_copy(change, code):
    a = dict(caches=layers({}), count=1, src=A, dst=A, rows=0, n=2)
    a.update(change)
    assert Q.qmm_kv_copy(*a.values(), S) == code


@pytest.mark.parametrize("change,code", [
    (dict(caches=None), Q.QMM_ERR_NULL), (dict(count=0), Q.QMM_ERR_SHAPE), (dict(caches=layers({}, dict(n_pages=9)), count=2), Q.QMM_ERR_SHAPE),
    (dict(table=0), Q.QMM_ERR_NULL), (dict(first=0), Q.QMM_ERR_NULL), (dict(keep=0), Q.QMM_ERR_NULL), (dict(n_keep=0), Q.QMM_ERR_NULL),
    (dict(table=A + 1), Q.QMM_ERR_ALIGN), (dict(kv_len=A + 2), Q.QMM_ERR_ALIGN), (dict(n_seqs=0), Q.QMM_ERR_SHAPE),
    (dict(n_seqs=65537), Q.QMM_ERR_SHAPE), (dict(table_width=0), Q.QMM_ERR_SHAPE), (dict(table_width=1 << 27), Q.QMM_ERR_SHAPE),
    (dict(width=-1), Q.QMM_ERR_SHAPE), (dict(width=(1 << 30) + 1), Q.QMM_ERR_SHAPE),
    (dict(kv_len=A), Q.QMM_ERR_UNSUPPORTED), (dict(kv_len=A + 16), Q.QMM_ERR_UNSUPPORTED),
    (dict(caches=layers(dict(n_kv=4096)), n_seqs=65536), Q.QMM_ERR_SHAPE)])
def test_compact(change, code):
    a = dict(caches=layers({}), count=1, table=A + 64, n_seqs=2, table_width=4, first=A, keep=A + 64, n_keep=A + 16, width=3, kv_len=0)
    a.update(change)
    assert Q.qmm_kv_compact(*a.values(), S) == code


@pytest.mark.parametrize("change,code", [
    (dict(xtype=Q.QMM_F16), Q.QMM_ERR_UNSUPPORTED), (dict(xtype=Q.QMM_Q8_0), Q.QMM_ERR_UNSUPPORTED), (dict(xtype=5000), Q.QMM_ERR_TYPE),
    (dict(logits=0), Q.QMM_ERR_NULL), (dict(logits=A + 2), Q.QMM_ERR_ALIGN), (dict(xtype=BF16, logits=A + 1), Q.QMM_ERR_ALIGN),
    (dict(ld=99), Q.QMM_ERR_SHAPE), (dict(rows=0), Q.QMM_ERR_SHAPE), (dict(rows=1 << 23), Q.QMM_ERR_SHAPE), (dict(ld=1 << 62), Q.QMM_ERR_SHAPE),
    (dict(vocab=0), Q.QMM_ERR_SHAPE), (dict(vocab=(1 << 28) + 1, ld=1 << 29), Q.QMM_ERR_SHAPE), (dict(n_top=-1), Q.QMM_ERR_SHAPE),
    (dict(n_top=65), Q.QMM_ERR_SHAPE), (dict(vocab=4, n_top=5), Q.QMM_ERR_SHAPE), (dict(scale=0.0), Q.QMM_ERR_UNSUPPORTED),
    (dict(scale=-1.0), Q.QMM_ERR_UNSUPPORTED), (dict(scale=float("inf")), Q.QMM_ERR_UNSUPPORTED), (dict(scale=float("nan")), Q.QMM_ERR_UNSUPPORTED),
    (dict(softcap=-1.0), Q.QMM_ERR_UNSUPPORTED), (dict(softcap=float("inf")), Q.QMM_ERR_UNSUPPORTED), (dict(n_tokens=-1), Q.QMM_ERR_SHAPE),
    (dict(n_tokens=65537), Q.QMM_ERR_SHAPE), (dict(tokens=0), Q.QMM_ERR_NULL), (dict(logp=0), Q.QMM_ERR_NULL), (dict(tokens=A + 1), Q.QMM_ERR_ALIGN),
    (dict(top_ids=0), Q.QMM_ERR_NULL), (dict(top_logp=A + 2), Q.QMM_ERR_ALIGN), (dict(entropy=A + 2), Q.QMM_ERR_ALIGN),
    (dict(n_tokens=0, n_top=0, entropy=0), Q.QMM_ERR_NULL), (dict(vocab=100000, ld=100000, work=0), Q.QMM_ERR_NULL),
    (dict(vocab=100000, ld=100000, work_bytes=16), Q.QMM_ERR_SHAPE), (dict(vocab=100000, ld=100000, work=A + 4), Q.QMM_ERR_ALIGN)])
def test_logprobs(change, code):
    a = dict(xtype=F32, logits=A, ld=100, rows=3, vocab=100, scale=1.0, softcap=0.0, tokens=A, n_tokens=2, logp=A, entropy=A, n_top=5, top_ids=A,
             top_logp=A, work=A, work_bytes=1 << 40)
    a.update(change)
    assert Q.qmm_logprobs(*a.values(), S) == code


@pytest.mark.parametrize("scale,softcap", [(3e38, 0.0), (1e-39, 0.0), (1e30, 1e30), (1e-30, 1e-30), (1.0, 1e-39), (1.0, 1e-45)])
def test_logprobs_numbers_that_fp32_does_not_hold(scale, softcap):
    # scale log2 e, that times the cap, or 1 / cap would be infinite or no normal number
    assert Q.qmm_logprobs(F32, A, 100, 3, 100, scale, softcap, A, 2, A, A, 5, A, A, A, 1 << 40, S) == Q.QMM_ERR_UNSUPPORTED


def test_logprobs_work():
    assert Q.qmm_logprobs_work(F32, 1, 8185, 5) == 0  # one turn of a workgroup
    one = Q.qmm_logprobs_work(F32, 1, 128256, 20)
    assert one == (16 * (4 + 2 * 20) * 4 + 15) // 16 * 16
    assert Q.qmm_logprobs_work(F32, 1024, 128256, 20) == 0  # enough rows
    assert Q.qmm_logprobs_work(Q.QMM_F16, 1, 128256, 20) == 0 and Q.qmm_logprobs_work(F32, 1, 3, 20) == 0
    for rows in (1, 2, 1023, 2 ** 23 - 1):
        for vocab in (1, 2 ** 28):
            assert 0 <= Q.qmm_logprobs_work(BF16, rows, vocab, 0) < 1 << 40


def test_python_helpers_without_a_gpu():
    i = lambda *x: torch.zeros(*x, dtype=torch.int32)  # noqa: E731
    x = torch.zeros(2, 10)
    for call, code, text in (
            (lambda: Q.logprobs(x[0]), Q.QMM_ERR_SHAPE, "rows x vocab"), (lambda: Q.logprobs(x.half()), Q.QMM_ERR_UNSUPPORTED, "float32 or bfloat16"),
            (lambda: Q.logprobs(x, top=65), Q.QMM_ERR_SHAPE, "0 to 64"), (lambda: Q.logprobs(x.T.contiguous().T), Q.QMM_ERR_UNSUPPORTED, "one after another"),
            (lambda: Q.logprobs(x, tokens=i(2)), Q.QMM_ERR_SHAPE, "rows x any"), (lambda: Q.logprobs(x, tokens=i(3, 1)), Q.QMM_ERR_SHAPE, "int32"),
            (lambda: Q.logprobs(x, tokens=i(2, 1).long()), Q.QMM_ERR_SHAPE, "int32"), (lambda: Q.logprobs(x), Q.QMM_ERR_UNSUPPORTED, "one GPU"),
            (lambda: Q.KVLayers([]), Q.QMM_ERR_SHAPE, "1 to 4096")):
        with pytest.raises(Q.QmmError, match=text) as e:
            call()
        assert e.value.code == code


def test_structures_match_the_header():
    assert ctypes.sizeof(Q.qmm_kv_tree) == 24 and Q.qmm_kv_tree.words.offset == 16
