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
