"""Lengths that compaction would write over what it reads are refused, wherever
they lie in it; beside it they are not.  (So many sequences of so many heads
that the next check refuses those: nothing is launched.)"""
import pytest

import block_quantized_amd as Q

N, S = 2048, 0
AT = dict(first=1 << 20, n_keep=2 << 20, keep=3 << 20, table=4 << 20)  # aligned addresses that are never read
BYTES = dict(first=4 * N, n_keep=4 * N, keep=5 * 4 * N, table=3 * 4 * N)


def compact(kv_len, width=5):
    c = (Q.qmm_kv_cache * 1)(Q.qmm_kv_cache(1 << 30, 2 << 30, Q.QMM_F16, 4096, 64, 16, 8))
    return Q.qmm_kv_compact(c, 1, AT["table"], N, 3, AT["first"], AT["keep"], AT["n_keep"], width, kv_len, S)


@pytest.mark.parametrize("name", AT)
def test_overlaps(name):
    at, end = AT[name], AT[name] + BYTES[name]
    for kv_len in (at - 4 * N + 4, at - 4, at, at + 4, end - 4):
        assert compact(kv_len) == Q.QMM_ERR_UNSUPPORTED, (name, kv_len - at)
    for kv_len in (0, at - 4 * N, end):
        assert compact(kv_len) == Q.QMM_ERR_SHAPE, (name, kv_len - at)


def test_a_list_that_is_not_read_does_not_count():
    assert compact(AT["keep"], width=0) == Q.QMM_ERR_SHAPE
