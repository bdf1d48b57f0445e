"""Trees of new tokens whose prefix reaches into them: tiles of keys that every
row sees still hold new tokens, whose distances go by their positions.
Tolerances as in test_gpu_attn.py."""
import numpy as np
import pytest

import kv_ref as R
import synth
from test_gpu_attn import setup
from test_gpu_attn_tree import run, trees

pytestmark = pytest.mark.gpu

# (new, all) tokens with the prefix of each: whole tiles of 32 and of 64 keys that hold new tokens alone, tiles that begin
# before them and end among them, all tokens new, and a prefix that ends in a tile, or before the new tokens
BATCH = [((70, 134), 128), ((64, 64), 64), ((100, 131), 96), ((100, 150), 150), ((40, 200), 70), ((200, 300), 290)]


@pytest.mark.parametrize("algo", (1, 2))
@pytest.mark.parametrize("cache", [R.Q8, R.F16, R.BF16])
@pytest.mark.parametrize("xt", [R.F32, R.BF16])
@pytest.mark.parametrize("dim,n_kv,n_q", [(64, 2, 6), (128, 1, 4), (256, 1, 2)])
def test_slopes_and_a_prefix_of_new_tokens(algo, cache, xt, dim, n_kv, n_q):
    g = synth.rng(dim + n_q)
    case = setup(g, [s for s, _ in BATCH], 16, cache, n_kv, dim)
    q = R.as_type(synth.normal_f32(g, (case[0].N, n_q, dim)), xt)
    parents = trees(g, case[0].new, 9)
    slopes, prefix = (2.0 ** -np.arange(2, n_q + 2)).astype(np.float32), [p for _, p in BATCH]
    for o in (dict(), dict(window=11), dict(softcap=20.0)):
        run(case, parents, q, xt, n_kv, dim, algo, slopes=slopes, prefix=prefix, **o)
