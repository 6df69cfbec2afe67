"""Torch-facing MX4 calls refuse storage that is an operand of another K, on
the host (the check comes before the one for GPU tensors), and take padded storage."""

import pytest
import torch

import dense_gemm_tuning_amd as dgt


def operand(rows, K):
    return dgt.mx4_empty(rows, K, device="cpu")


@pytest.mark.parametrize("K,other", [(64, 128), (4096, 8192), (330, 400), (512, 544), (33, 512), (0, 32)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_weight_of_another_k_is_refused(K, other, dtype):
    B, SB = operand(8, other)
    with pytest.raises(ValueError, match="operand of"):
        dgt.gemm_quantized(torch.zeros(4, K, dtype=dtype), None, B, SB, torch.zeros(4, 8))


@pytest.mark.parametrize("K,other", [(64, 128), (330, 400), (4096, 8192)])
def test_quantising_into_an_operand_of_another_k_is_refused(K, other):
    """Its rows would keep what was there past K."""
    Q, S = operand(4, other)
    with pytest.raises(ValueError, match="operand of"):
        dgt.quantize_mx4(torch.zeros(4, K), Q, S)
    with pytest.raises(ValueError, match="operand of"):
        dgt.quantize_mx4(torch.zeros(K, 4), Q, S, trans=True)
    with pytest.raises(ValueError, match="operand of"):
        dgt.dequantize_mx4(Q, S, torch.zeros(4, K))


def test_views_of_padded_storage_and_equal_block_counts_pass():
    """Each of these gets as far as the check for GPU tensors."""
    A, C = torch.zeros(4, 330, dtype=torch.bfloat16), torch.zeros(4, 8)
    wide, scales = torch.zeros(8, 224, dtype=torch.uint8), torch.zeros(8, 48, dtype=torch.uint8)
    B, SB = operand(8, 352)  # eleven blocks, as 330 elements take
    for b, s in ((wide[:, :176], scales[:, :16]), (wide, scales), (wide[:, :176], scales), (B, SB)):
        with pytest.raises(ValueError, match="GPU tensor"):
            dgt.gemm_quantized(A, None, b, s, C)


def test_more_workgroups_than_a_launch_holds_are_refused():
    """2^32 threads are one launch's limit; the counts are not cut on the way."""
    A, SA, B, SB, C = (i << 50 for i in range(1, 6))
    top = 2 ** 31 - 1

    def mx4(M, N, K=32):
        return dgt.gemm_mx4(M, N, K, 1.0, A, 16, SA, 16, B, 16, SB, 16, 0.0, C, N)

    def a16(M, N, dtype=dgt.DTYPE_BF16, lda=32):
        return dgt.gemm_mx4_a16(dtype, M, N, 32, 1.0, A, lda, B, 16, SB, 16, 0.0, C, N)

    assert mx4(top, 1) == mx4(1, top) == mx4(2 ** 22, 2 ** 22) == dgt.GEMM_ERR_DIM
    assert a16(top, 1) == a16(1, top) == a16(2 ** 26, 64) == dgt.GEMM_ERR_DIM
    assert a16(top, 1, dgt.DTYPE_F16, 33) == a16(top, 1, dgt.DTYPE_F16) == dgt.GEMM_ERR_DIM
    assert dgt.gemm_mx4_quantize(dgt.DTYPE_BF16, 1, top, 32, A, top, B, 16, SB, 16) == dgt.GEMM_ERR_DIM
