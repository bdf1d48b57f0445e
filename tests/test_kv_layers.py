"""Layers whose rows are moved together are each there once (host logic: the
caches stand for tensors on a GPU)."""
import types

import pytest
import torch

import block_quantized_amd as Q

PAGE = Q.qmm_kv_bytes(Q.QMM_F16, 2, 64, 16, 1)


def cache(k, v, dev=0):
    t = torch.empty(3, 2, 16, 64, dtype=torch.float16)  # 3 pages
    return types.SimpleNamespace(k=t, v=t, type=Q.QMM_F16, n_kv=2, head_dim=64, page_size=16, n_pages=3, dev=dev,
                                 c=Q.qmm_kv_cache(k, v, Q.QMM_F16, 2, 64, 16, 3))


@pytest.mark.parametrize("change", ["the same cache", "the same keys", "keys and values", "a page of the next", "the values before"])
def test_overlapping_layers_are_refused(change):
    size = 3 * PAGE
    base = 1 << 20
    a, b = cache(base, base + size), cache(base + 2 * size, base + 3 * size)
    other = {"the same cache": a, "the same keys": cache(base, base + 8 * size), "keys and values": cache(base + 8 * size, base + 8 * size),
             "a page of the next": cache(base + 8 * size, base + 4 * size - PAGE), "the values before": cache(base - PAGE, base + 8 * size)}[change]
    layers = Q.KVLayers([b, a])  # side by side, in any order
    assert layers.n == 2 and layers.c[1].k == base
    with pytest.raises(Q.QmmError, match="overlap") as e:
        Q.KVLayers([a, b, other])
    assert e.value.code == Q.QMM_ERR_UNSUPPORTED
