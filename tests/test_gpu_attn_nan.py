"""NaN in a query: its row's results are NaN, and no other row's are touched by it."""
import numpy as np
import pytest
import torch

import block_quantized_amd as Q
import kv_ref as R
import synth
from gpu_util import to_gpu
from test_gpu_attn import ALGOS, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("cache", [R.Q8, R.F16, R.BF16])
@pytest.mark.parametrize("softcap", [0.0, 5.0])
@pytest.mark.parametrize("seqs", [[(3, 40), (20, 33)], [(5, 900), (1, 300)]])  # whole, and in parts that are joined
def test_a_query_of_nan_stays_alone(algo, cache, softcap, seqs):
    g = synth.rng(101)
    b, c, kb, ks, vs = setup(g, seqs, 16, cache, 1, 64)
    q = to_gpu(synth.normal_f32(g, (b.N, 2, 64)))
    want = Q.attn(c, kb, q, softcap=softcap, algo=algo)
    assert torch.isfinite(want).all()
    bad = q.clone()
    bad[2, 1, 7] = float("nan")
    bad[b.N - 1, 0] = float("nan")
    got = Q.attn(c, kb, bad, softcap=softcap, algo=algo)
    hit = torch.zeros(b.N, 2, dtype=torch.bool, device="cuda")
    hit[2, 1] = hit[b.N - 1, 0] = True
    assert torch.isnan(got[hit]).all()
    # the rows of a wavefront raise their maxima together, so a row that raises none moves when its neighbours do:
    # by the roundings of fp32 results, each side's within 2^-18 of the norm of the exact ones
    err = (got[~hit].double() - want[~hit].double()).norm(dim=-1)
    assert (err <= 2.0 ** -17 * want[~hit].double().norm(dim=-1)).all()
