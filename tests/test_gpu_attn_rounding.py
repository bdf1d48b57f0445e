"""bf16 results of attention are the fp32 ones rounded once, whichever kernels run."""
import numpy as np
import pytest
import torch

import block_quantized_amd as Q
import kv_ref as R
import synth
from gpu_util import to_cpu, to_gpu
from test_gpu_attn import ALGOS, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("cache", [R.Q8, R.F16, R.BF16])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_bf16_results_are_rounded_once(algo, cache, dim, softcap):
    """A result differs from the 64-bit one rounded to bf16 only where a border
    between two bf16 values lies within its error: borders are 2^-8 to 2^-7 of
    the value apart, so an error of rms rho against values of rms 1 and a
    normal law moves a share of about 2^8 rho sqrt(2/pi) ln(1 / (2^8 rho)).
    Weights in two bf16 parts are off by at most 2^-18 of themselves (fp16
    parts by less), and the scores' fp32 sums by some 2^-19: rho below 2^-17.4,
    so 1%.  2% are allowed.  (One fp16 part, off by 2^-12, would move 10%, and
    one bf16 part almost half.)"""
    g = synth.rng(71 + dim)
    n_kv, n_q = 2, 6
    b, c, kb, ks, vs = setup(g, [(61, 61), (33, 250), (1, 77)], 32, cache, n_kv, dim)
    q = R.as_type(synth.normal_f32(g, (b.N, n_q, dim)), R.BF16)
    scale = np.float64(np.float32(dim ** -0.5))
    got = to_cpu(Q.attn(c, kb, to_gpu(q).to(torch.bfloat16), scale=float(scale), softcap=softcap, algo=algo).float())
    want = R.bf16_round(R.attention64(q, b, ks, vs, n_kv, scale, softcap)[0].astype(np.float32))
    assert np.mean(got != want) <= 0.02
