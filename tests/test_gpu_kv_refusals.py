"""Inputs that require gradients are refused where torch would record them."""
import pytest
import torch

import block_quantized_amd as Q

pytestmark = pytest.mark.gpu


def test_gradients_are_refused_not_dropped():
    c = Q.KVCache.allocate(Q.QMM_F16, 2, 64, 16, 2)
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    b = Q.KVBatch(i(0, 2), i(2), i(0)[None], 2)
    x = lambda h, grad=False: torch.ones(2, h, 64, device="cuda", requires_grad=grad)  # noqa: E731
    slopes = torch.ones(4, device="cuda", requires_grad=True)
    for call in (lambda: Q.kv_append(c, b, x(2, True), x(2)), lambda: Q.kv_append(c, b, x(2), x(2, True)),
                 lambda: Q.kv_append(c, b, x(2), x(2), q=x(4, True)), lambda: Q.kv_append(c, b, x(2), x(2), q=x(4), q_out=x(4, True)),
                 lambda: Q.attn(c, b, x(4, True)), lambda: Q.attn(c, b, x(4), slopes=slopes),
                 lambda: Q.attn(c, b, x(4), out=x(4, True))):
        with pytest.raises(Q.QmmError, match="gradients") as e:
            call()
        assert e.value.code == Q.QMM_ERR_UNSUPPORTED
    # where nothing is recorded the same tensors do
    with torch.no_grad():
        assert Q.kv_append(c, b, x(2, True), x(2, True), q=x(4, True)).shape == (2, 4, 64)
        assert Q.attn(c, b, x(4, True), slopes=slopes).shape == (2, 4, 64)
    with torch.inference_mode():
        assert Q.attn(c, b, x(4)).shape == (2, 4, 64)
    Q.kv_append(c, b, x(2), x(2))
    assert torch.equal(Q.attn(c, b, x(4, True).detach()), torch.ones(2, 4, 64, device="cuda"))
