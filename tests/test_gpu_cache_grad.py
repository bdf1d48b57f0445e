"""Caches of keys and values that require a gradient (a learned prefix) are
refused where torch records: none reaches them, and none is dropped."""
import pytest
import torch

import block_quantized_amd as Q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", ["k", "v"])
def test_caches_that_require_gradients(which):
    pools = {n: torch.ones(2, 2, 16, 64, device="cuda", dtype=torch.float16, requires_grad=n == which) for n in ("k", "v")}
    c = Q.KVCache(pools["k"], pools["v"], Q.QMM_F16, 2, 64, 16)
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    b = Q.KVBatch(i(0, 2), i(2), i(0)[None], 2)
    tree = Q.KVTree(b, i(-1, 0))
    x = lambda h: torch.ones(2, h, 64, device="cuda")  # noqa: E731
    for call in (lambda: Q.attn(c, b, x(4)), lambda: Q.attn(c, b, x(4), tree=tree), lambda: Q.kv_append(c, b, x(2), x(2))):
        with pytest.raises(Q.QmmError, match="gradients") as e:
            call()
        assert e.value.code == Q.QMM_ERR_UNSUPPORTED
        with torch.no_grad():
            call()
    with torch.no_grad():
        assert torch.equal(Q.attn(c, b, x(4), tree=tree), x(4))
