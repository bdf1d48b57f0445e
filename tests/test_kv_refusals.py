"""What the key-value cache's Python holders refuse before a GPU is needed."""
import pytest
import torch

import block_quantized_amd as Q


@pytest.mark.parametrize("type,dtype", [(Q.QMM_F16, torch.bfloat16), (Q.QMM_BF16, torch.float16), (Q.QMM_F16, torch.float32),
                                        (Q.QMM_BF16, torch.int16), (Q.QMM_Q8_0, torch.float16), (Q.QMM_Q8_0, torch.int8)])
def test_pools_of_another_type(type, dtype):
    n = Q.qmm_kv_bytes(type, 1, 64, 16, 1) // torch.empty(0, dtype=dtype).element_size()
    right = torch.zeros(Q.qmm_kv_bytes(type, 1, 64, 16, 1), dtype=torch.uint8)
    for k, v in ((torch.zeros(n, dtype=dtype), right), (right, torch.zeros(n, dtype=dtype))):
        with pytest.raises(Q.QmmError, match="have to hold") as e:
            Q.KVCache(k, v, type, 1, 64, 16)
        assert e.value.code == Q.QMM_ERR_UNSUPPORTED
    with pytest.raises(Q.QmmError, match="one GPU"):  # bytes are taken; what is wrong with them is where they lie
        Q.KVCache(right, right, type, 1, 64, 16)


def test_rotations_that_ctypes_would_cut():
    f = torch.zeros(4, dtype=torch.float64)
    for pairing in (2, -1, 2 ** 32, 2 ** 32 + 1):
        with pytest.raises(Q.QmmError, match="pairing") as e:
            Q.Rope(f, pairing)
        assert e.value.code == Q.QMM_ERR_UNSUPPORTED
    for sections in ([2 ** 32 + 2, 2], [-1, 5], [5, 0]):
        with pytest.raises(Q.QmmError, match="axes") as e:
            Q.Rope(f, 0, sections=sections)
        assert e.value.code == Q.QMM_ERR_SHAPE
