"""gemm_orthogonalize's refusals on the host: sizes that its kernels' 32-bit
offsets and FP16 ranges do not hold.  Nothing here reaches a launch."""

import os

import pytest
import torch

import dense_gemm_tuning_amd as dgt

G_, O_, W_ = (i << 44 for i in (1, 2, 3))


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(dgt.LIB_PATH):
        from dense_gemm_tuning_amd import build
        build.build()


def call(M, N, dtype=1, batch=1, nbytes=0):
    """With a workspace that is too small, so that an accepted size ends there."""
    return dgt.gemm_orthogonalize(dtype, M, N, G_, N, M * N, O_, N, M * N, batch, 5, 3.0, -4.0, 2.0,
                                  1e-7, W_, nbytes)


@pytest.mark.parametrize("M,N", [(32, 70_000_000), (64, 70_000_000), (1, 2 ** 24 + 1), (8, 2 ** 28),
                                 (1, 2 ** 31 - 1), (2 ** 26 + 1, 1), (2 ** 31 - 1, 1), (2 ** 31 - 1, 64)])
def test_sizes_past_the_limits_are_refused(M, N):
    """Longer rows pass 2^32 bytes within a tile's rows; more rows hold X times 2^14
    and more, which leaves FP16's range."""
    assert dgt.gemm_orthogonalize_workspace_size(M, N, 1) == dgt.GEMM_ERR_DIM
    assert call(M, N) == dgt.GEMM_ERR_DIM
    assert dgt.gemm_orthogonalize_workspace_size(M, N, 0) == dgt.GEMM_ERR_DIM


@pytest.mark.parametrize("M,N", [(1, 2 ** 24), (64, 2 ** 24), (2 ** 26, 1), (2 ** 26, 16), (70001, 2)])
def test_sizes_at_the_limits_are_taken(M, N):
    need = dgt.gemm_orthogonalize_workspace_size(M, N, 1)
    assert need >= 8 * M * N  # X in two halves, twice
    assert call(M, N) == call(M, N, nbytes=need - 1) == dgt.GEMM_ERR_WORKSPACE


def test_counts_past_an_int_are_refused():
    """The C entry points take them as int, which would cut them: a batch of
    2^32 + 1 to 1, as many steps plus four to five."""
    far = torch.empty(2 ** 32 + 1, 1, 1, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="2\\^31"):
        dgt.orthogonalize(far, far)
    one = torch.zeros(1, 1, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="2\\^31"):
        dgt.orthogonalize(one, one, steps=2 ** 32 + 5)
    with pytest.raises(ValueError, match="2\\^31"):
        dgt.mx4_empty(2, 2 ** 32 + 64, device="meta")
