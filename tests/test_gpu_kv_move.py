"""Copied pages and compacted rows against plain moves of bytes, bit for bit."""
import numpy as np
import pytest
import torch

import block_quantized_amd as Q
import synth
from gpu_util import to_cpu, to_gpu

pytestmark = pytest.mark.gpu

KINDS = [(Q.QMM_Q8_0, 34 / 32), (Q.QMM_F16, 2), (Q.QMM_BF16, 2)]


def pools(g, layers, n_pages, n_kv, page, row):
    return [g.integers(0, 256, (2, n_pages, n_kv, page, row), dtype=np.uint8) for _ in range(layers)]


def on_gpu(data, kind, n_kv, dim, page):
    t = [(to_gpu(p[0]), to_gpu(p[1])) for p in data]
    return t, Q.KVLayers([Q.KVCache(k, v, kind, n_kv, dim, page) for k, v in t])


def same(t, want):
    return all(np.array_equal(to_cpu(x), y) for pair, w in zip(t, want) for x, y in zip(pair, w))


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kind,size", KINDS)
@pytest.mark.parametrize("n_kv,page,layers", [(1, 16, 1), (3, 48, 3), (8, 128, 2)])
def test_copy(kind, size, dim, n_kv, page, layers):
    g = synth.rng(dim + page)
    row, n_pages = int(dim * size), 11
    data = pools(g, layers, n_pages, n_kv, page, row)
    for n, part in ((1, True), (1, False), (4, True), (5, False)):
        t, l = on_gpu(data, kind, n_kv, dim, page)
        order = g.permutation(n_pages).astype(np.int32)
        src, dst = order[:n].copy(), order[n:2 * n].copy()
        rows = None
        if part:
            rows = g.integers(1, page, n).astype(np.int32)
            rows[0] = [0, page + 5, -3, 1, page - 1][n % 5]
        if n == 4:  # pairs that are left out
            src[1], dst[2] = n_pages, -1
        Q.kv_copy(l, to_gpu(src), to_gpu(dst), rows=None if rows is None else to_gpu(rows))
        want = [d.copy() for d in data]
        for i in range(n):
            if 0 <= src[i] < n_pages and 0 <= dst[i] < n_pages:
                r = page if rows is None else min(max(int(rows[i]), 0), page)
                for w in want:
                    w[:, dst[i], :, :r] = w[:, src[i], :, :r]
        assert same(t, want), (n, part)


def compacted(data, table, first, keep, n_keep, page):
    want = [d.copy() for d in data]
    for s in range(len(first)):
        for i in range(min(max(int(n_keep[s]), 0), keep.shape[1])):
            a, b = int(keep[s, i]), int(first[s]) + i
            if not (0 <= a < table.shape[1] * page and 0 <= b < table.shape[1] * page):
                continue
            pa, pb = table[s, a // page], table[s, b // page]
            if pa < 0 or pb < 0 or max(pa, pb) >= data[0].shape[1]:
                continue
            for d, w in zip(data, want):  # every row as it was before
                w[:, pb, :, b % page] = d[:, pa, :, a % page]
    return want


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kind,size", KINDS)
def test_compact(kind, size, dim):
    # overlapping moves over chunks and pages; rows already in place; nothing kept; whole sequences
    g = synth.rng(dim)
    row, n_kv, page, layers, width = int(dim * size), 2, 16, 2, 30
    order = g.permutation(5 * width).astype(np.int32)
    table = order.reshape(5, width)
    room = width * page
    lists = [(0, np.sort(g.choice(room, 300, replace=False))), (37, np.sort(37 + g.choice(room - 37, 41, replace=False))),
             (5, np.zeros(0, int)), (0, np.arange(1, room)), (64, np.arange(64, 64 + 50))]
    most = max(len(k) for _, k in lists)
    first = np.array([f for f, _ in lists], np.int32)
    keep = np.full((5, most), -7, np.int32)
    for s, (_, k) in enumerate(lists):
        keep[s, :len(k)] = k
    n_keep = np.array([len(k) for _, k in lists], np.int32)
    n_keep[2] = -4  # none
    data = pools(g, layers, 5 * width, n_kv, page, row)
    t, l = on_gpu(data, kind, n_kv, dim, page)
    kv_len = to_gpu(np.full(5, 999, np.int32))
    Q.kv_compact(l, to_gpu(table), to_gpu(first), to_gpu(keep), to_gpu(n_keep), kv_len=kv_len)
    assert same(t, compacted(data, table, first, keep, n_keep, page))
    assert np.array_equal(to_cpu(kv_len), first + np.maximum(n_keep, 0))


def test_compact_without_pages_and_lengths():
    g = synth.rng(4)
    page, n_kv, row = 32, 1, 128
    table = np.array([[3, -1, 2, 9], [0, 1, 4, 10 ** 9]], np.int32)
    first, n_keep = np.array([0, 20], np.int32), np.array([60, 500], np.int32)  # more than the width: held to it
    keep = np.stack([np.sort(g.choice(128, 60, replace=False)), 20 + np.sort(g.choice(140, 60, replace=False))]).astype(np.int32)
    data = pools(g, 1, 5, n_kv, page, row)
    t, l = on_gpu(data, Q.QMM_F16, n_kv, 64, page)
    Q.kv_compact(l, to_gpu(table), to_gpu(first), to_gpu(keep), to_gpu(n_keep))
    assert same(t, compacted(data, table, first, keep, n_keep, page))


def test_many_layers():
    # more than one launch takes
    g = synth.rng(5)
    data = pools(g, 70, 3, 1, 16, 128)
    t, l = on_gpu(data, Q.QMM_BF16, 1, 64, 16)
    Q.kv_copy(l, to_gpu(np.array([0], np.int32)), to_gpu(np.array([2], np.int32)))
    for d in data:
        d[:, 2] = d[:, 0]
    assert same(t, data)
    table, keep = np.array([[1, 2]], np.int32), np.array([[3, 9, 30]], np.int32)
    first, n_keep, kv_len = (np.array([x], np.int32) for x in (1, 3, 0))
    kl = to_gpu(kv_len)
    Q.kv_compact(l, to_gpu(table), to_gpu(first), to_gpu(keep), to_gpu(n_keep), kv_len=kl)
    assert same(t, compacted(data, table, first, keep, n_keep, 16)) and to_cpu(kl)[0] == 4
