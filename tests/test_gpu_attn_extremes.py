"""Scales and caps at the ends of the ranges that attention accepts."""
import numpy as np
import pytest
import torch

import block_quantized_amd as Q
import kv_ref as R
import synth
from test_gpu_attn import ALGOS, run, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-38, -1e-44])
@pytest.mark.parametrize("xt", [R.F32, R.BF16])
def test_no_scale_over_the_smallest_keys(algo, scale, xt):
    # Q8_0 keys whose scales are fp16's smallest numbers: a factor of the scores
    # that rounds to 0 must not meet the -inf of masked keys
    g = synth.rng(79)
    b, c, kb, ks, vs = setup(g, [(1, 100), (40, 90), (3, 5)], 16, R.Q8, 1, 64)
    blocks = c.k.view(torch.int16).view(*c.k.shape[:3], -1, 17)[..., 0]
    blocks[blocks != -1] = 1  # 2^-24
    for i, L in enumerate(b.len):
        for j in range(L):
            ks[i][j] = R.row_values(c.k[b.table[i, j // 16], :, j % 16].cpu().numpy(), R.Q8, 64)
    q = R.as_type(synth.normal_f32(g, (b.N, 2, 64)), xt)
    run(b, c, kb, ks, vs, q, xt, 1, 64, algo, scale=scale)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("cache", [R.Q8, R.F16, R.BF16])
def test_smallest_cap(algo, cache):
    # a cap whose inverse passes fp32, over keys of zeros and of all sizes: no
    # score counts, so the values' mean
    g = synth.rng(83)
    b, c, kb, ks, vs = setup(g, [(1, 40), (20, 50)], 16, cache, 1, 64)
    for s in range(2):
        page = int(b.table[s, 1])
        c.k[page] = 0
        ks[s][16:32] = 0.0
    q = R.as_type(synth.normal_f32(g, (b.N, 2, 64)), R.F32)
    for cap in (1e-44, 1e-38, 1e-30):
        run(b, c, kb, ks, vs, q, R.F32, 1, 64, algo, softcap=cap)
