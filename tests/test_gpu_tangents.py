"""Inputs that carry a tangent of forward-mode differentiation are refused, as
those that require a gradient are: none is computed, and none is dropped."""
import pytest
import torch
import torch.autograd.forward_ad as F

import block_quantized_amd as Q


def test_the_check_itself():
    Q._need_torch()
    x = torch.ones(2, 3)
    Q._no_grad("call", x, None)
    with F.dual_level():
        dual = F.make_dual(x, torch.ones(2, 3))
        Q._no_grad("call", x, None, torch.ones(2, dtype=torch.int32), dual.detach())
        for where in (torch.enable_grad, torch.no_grad):
            with where(), pytest.raises(Q.QmmError, match="gradients") as e:
                Q._no_grad("call", x, dual)
            assert e.value.code == Q.QMM_ERR_UNSUPPORTED
    Q._no_grad("call", x)


@pytest.mark.gpu
def test_tangents_are_refused_not_dropped():
    c = Q.KVCache.allocate(Q.QMM_F16, 2, 64, 16, 2)
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    b = Q.KVBatch(i(0, 2), i(2), i(0)[None], 2)
    tree = Q.KVTree(b, i(-1, 0))
    x = lambda h: torch.ones(2, h, 64, device="cuda")  # noqa: E731
    logits, slopes = torch.ones(2, 9, device="cuda"), torch.ones(4, device="cuda")
    with F.dual_level():
        dual = lambda t: F.make_dual(t, torch.ones_like(t))  # noqa: E731
        for call in (lambda: Q.logprobs(dual(logits)), lambda: Q.attn(c, b, dual(x(4)), tree=tree), lambda: Q.attn(c, b, dual(x(4))),
                     lambda: Q.attn(c, b, x(4), slopes=dual(slopes), tree=tree), lambda: Q.kv_append(c, b, dual(x(2)), x(2)),
                     lambda: Q.kv_append(c, b, x(2), dual(x(2))), lambda: Q.kv_append(c, b, x(2), x(2), q=dual(x(4)))):
            with pytest.raises(Q.QmmError, match="gradients") as e:
                call()
            assert e.value.code == Q.QMM_ERR_UNSUPPORTED
        # others within a dual level, and detached ones, do
        Q.kv_append(c, b, dual(x(2)).detach(), x(2))
        assert torch.equal(Q.attn(c, b, dual(x(4)).detach(), tree=tree), torch.ones(2, 4, 64, device="cuda"))
        assert Q.logprobs(logits).entropy.shape == (2,)
