"""Gated and 4-bit calls of more workgroups than a launch holds are refused on the host, before any launch."""

import dense_gemm_tuning_amd as dgt

A, B, C, D, E, F, G = (i << 50 for i in range(1, 8))
BF, TOP = dgt.DTYPE_BF16, dgt.GATED_MAX_DIM


def test_gated():
    def f(M, N, K, ldx):
        return dgt.gemm_gated(BF, 0, M, N, K, A, ldx, B, ldx, C, ldx, 0, 0, D, N)

    # whole 16-byte rows, rows off them, and no k
    assert f(2 ** 22, 2 ** 22, 8, 8) == f(2 ** 22, 2 ** 22, 9, 9) == f(TOP, 2 ** 14, 0, 1) == dgt.GEMM_ERR_DIM
    assert f(64, TOP + 1, 8, 8) == dgt.GEMM_ERR_DIM


def test_gradient():
    def f(M, N, K):
        return dgt.gemm_gated_grad(BF, 0, M, N, K, A, K, B, N, C, N, D, N, E, N, F, N)

    assert f(2 ** 22, 2 ** 22, 8) == f(2 ** 22, 2 ** 22 + 1, 9) == dgt.GEMM_ERR_DIM


def test_w4():
    def product(M, N, ld=32):
        return dgt.gemm_w4_a16(BF, 32, BF, M, N, 32, 1.0, A, ld, B, 16, C, 1, 0, 0, 0.0, D, N)

    def gated(M, N, ld=32):
        return dgt.gemm_w4_gated(BF, 0, 32, BF, M, N, 32, A, ld, B, 16, C, 1, 0, 0, 0, 0, D, N)

    # strips are counted eight at a time: 2^20 blocks of 32 rows are too many for a single output
    assert product(2 ** 26, 1) == product(2 ** 26, 1, 33) == product(2 ** 20, 2 ** 20) == dgt.GEMM_ERR_DIM
    assert gated(2 ** 26, 1) == gated(2 ** 26, 1, 33) == gated(2 ** 20, 2 ** 20) == dgt.GEMM_ERR_DIM
