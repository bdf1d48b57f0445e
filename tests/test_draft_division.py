"""Batches of drafts whose row tiles fill the chip keep places to cut a long
sequence among them (host logic only: what the workspace is sized for)."""
import pytest

import block_quantized_amd as Q


@pytest.mark.parametrize("type", [Q.QMM_Q8_0, Q.QMM_F16, Q.QMM_BF16])
@pytest.mark.parametrize("xtype", [Q.QMM_F32, Q.QMM_BF16])
@pytest.mark.parametrize("seqs,new", [(64, 8), (32, 16), (70, 8), (64, 16), (300, 2)])
def test_long_caches_can_be_cut(type, xtype, seqs, new):
    c = Q.qmm_kv_cache(None, None, type, 8, 128, 64, 1 << 20)
    for algo in (0, 1, 2):
        o = Q.qmm_attn_opts(0.1, 0.0, 0, algo, None, None)
        for n_q in (8, 32):
            # as the header says, max_kv is the longest sequence, as far as known, or the table's width counts
            for width, most in ((2049, 131072), (2049, 0)):
                b = Q.qmm_kv_batch(None, None, None, seqs, width, seqs * new, most)
                assert Q.qmm_attn_tree_work(c, b, o, xtype, n_q) > 0
        b = Q.qmm_kv_batch(None, None, None, seqs, 2, seqs * new, 128)
        assert Q.qmm_attn_tree_work(c, b, o, xtype, 32) == 0


@pytest.mark.parametrize("type", [Q.QMM_Q8_0, Q.QMM_F16, Q.QMM_BF16])
def test_the_workspace_stays_small(type):
    # every row has room in it, so batches of very many rows keep none for a long sequence
    c = Q.qmm_kv_cache(None, None, type, 8, 128, 64, 1 << 24)
    o = Q.qmm_attn_opts(0.1, 0.0, 0, 2, None, None)
    for seqs in (64, 256, 1024, 4096, 65536):
        b = Q.qmm_kv_batch(None, None, None, seqs, 2049, 8 * seqs, 131072)
        assert Q.qmm_attn_tree_work(c, b, o, Q.QMM_BF16, 32) <= 300 << 20
