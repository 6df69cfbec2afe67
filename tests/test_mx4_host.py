"""MX4 and orthogonalisation entry points on the host: argument checks and
refusals, none of which reaches a kernel launch, and the plain format model's
own pins."""

import numpy as np
import pytest
import torch

import dense_gemm_tuning_amd as dgt
import mx4_plain as mp

Q_, S_, X_, Y_, C_, W_ = (0x1000000 * i for i in range(1, 7))


@pytest.fixture(scope="module", autouse=True)
def built():
    import os
    if not os.path.exists(dgt.LIB_PATH):
        from dense_gemm_tuning_amd import build
        build.build()


def test_pitches():
    for K in (1, 31, 32, 33, 511, 512, 513, 8192, 28672):
        assert dgt.gemm_mx4_code_pitch(K) == mp.code_pitch(K)
        assert dgt.gemm_mx4_scale_pitch(K) == mp.scale_pitch(K)
    assert dgt.gemm_mx4_code_pitch(0) == 0 and dgt.gemm_mx4_scale_pitch(-5) == 0


def test_quantize_argument_checks():
    def q(dtype=1, trans=0, M=4, K=64, X=X_, ldx=64, Q=Q_, ldq=32, S=S_, lds=16):
        return dgt.gemm_mx4_quantize(dtype, trans, M, K, X, ldx, Q, ldq, S, lds)

    assert q(dtype=3) == q(dtype=-1) == q(trans=2) == dgt.GEMM_ERR_ARG
    assert q(M=-1) == q(K=-1) == dgt.GEMM_ERR_DIM
    assert q(ldx=63) == q(ldq=16) == q(lds=0) == dgt.GEMM_ERR_LD
    assert q(trans=1, ldx=3) == dgt.GEMM_ERR_LD
    assert q(ldq=dgt.MX4_MAX_PITCH + 16) == q(lds=dgt.MX4_MAX_PITCH + 16) == dgt.GEMM_ERR_LD
    assert q(M=0) == dgt.GEMM_OK and q(K=0, X=0) == dgt.GEMM_OK
    assert q(X=0) == q(Q=0) == q(S=0) == dgt.GEMM_ERR_NULL
    assert q(Q=Q_ + 8) == q(S=S_ + 4) == q(ldq=40) == q(lds=24) == dgt.GEMM_ERR_ALIGN
    assert q(X=Q_ + 16) == q(S=Q_ + 96) == q(S=X_) == dgt.GEMM_ERR_OVERLAP


def test_dequantize_argument_checks():
    def d(dtype=0, M=4, K=64, Q=Q_, ldq=32, S=S_, lds=16, Y=Y_, ldy=64):
        return dgt.gemm_mx4_dequantize(dtype, M, K, Q, ldq, S, lds, Y, ldy)

    assert d(dtype=7) == dgt.GEMM_ERR_ARG
    assert d(M=-1) == dgt.GEMM_ERR_DIM
    assert d(ldy=63) == d(ldq=31) == d(lds=8) == dgt.GEMM_ERR_LD
    assert d(M=0) == d(K=0) == dgt.GEMM_OK
    assert d(Y=0) == d(Q=0) == d(S=0) == dgt.GEMM_ERR_NULL
    assert d(Q=Q_ + 1) == d(S=S_ + 15) == dgt.GEMM_ERR_ALIGN
    assert d(Y=Q_) == d(Y=S_ - 16) == dgt.GEMM_ERR_OVERLAP


def test_product_argument_checks():
    def g(M=4, N=8, K=64, alpha=1.0, A=X_, lda=32, SA=Y_, ldsa=16, B=Q_, ldb=32, SB=S_, ldsb=16,
          C=C_, ldc=8, bias=0):
        return dgt.gemm_mx4(M, N, K, alpha, A, lda, SA, ldsa, B, ldb, SB, ldsb, 0.0, C, ldc, bias)

    assert g(M=-1) == g(N=-1) == g(K=-1) == dgt.GEMM_ERR_DIM
    assert g(lda=16) == g(ldsa=0) == g(ldb=16) == g(ldsb=0) == g(ldc=7) == dgt.GEMM_ERR_LD
    assert g(ldb=dgt.MX4_MAX_PITCH + 16) == dgt.GEMM_ERR_LD
    assert g(M=0) == g(N=0) == dgt.GEMM_OK
    assert g(A=0) == g(SA=0) == g(B=0) == g(SB=0) == g(C=0) == dgt.GEMM_ERR_NULL
    assert g(A=X_ + 4) == g(SA=Y_ + 2) == g(B=Q_ + 8) == g(SB=S_ + 1) == dgt.GEMM_ERR_ALIGN
    assert g(lda=40) == g(ldb=36) == dgt.GEMM_ERR_ALIGN
    assert g(C=X_) == g(C=Y_) == g(C=Q_) == g(C=S_) == g(bias=C_) == dgt.GEMM_ERR_OVERLAP


def test_product16_argument_checks():
    def g(dtype=1, M=4, N=8, K=64, A=X_, lda=64, B=Q_, ldb=32, SB=S_, ldsb=16, C=C_, ldc=8):
        return dgt.gemm_mx4_a16(dtype, M, N, K, 1.0, A, lda, B, ldb, SB, ldsb, 0.0, C, ldc)

    assert g(dtype=0) == g(dtype=3) == dgt.GEMM_ERR_ARG
    assert g(K=-2) == dgt.GEMM_ERR_DIM
    assert g(lda=63) == g(ldb=16) == g(ldsb=0) == dgt.GEMM_ERR_LD
    assert g(N=0) == dgt.GEMM_OK
    assert g(A=0) == g(SB=0) == dgt.GEMM_ERR_NULL
    assert g(SB=S_ + 8) == dgt.GEMM_ERR_ALIGN
    assert g(C=X_) == g(C=Q_) == dgt.GEMM_ERR_OVERLAP


def test_orthogonalize_argument_checks():
    need = dgt.gemm_orthogonalize_workspace_size(32, 48, 2)
    assert need > 0
    assert dgt.gemm_orthogonalize_workspace_size(0, 48, 2) == 0
    assert dgt.gemm_orthogonalize_workspace_size(-1, 48, 2) == dgt.GEMM_ERR_DIM
    assert dgt.gemm_orthogonalize_workspace_size(4, 48, -2) == dgt.GEMM_ERR_ARG
    assert dgt.gemm_orthogonalize_workspace_size(2 ** 30, 2 ** 30, 8) == dgt.GEMM_ERR_DIM

    def o(dtype=0, M=32, N=48, G=X_, ldg=48, sg=32 * 48, O=Y_, ldo=48, so=32 * 48, batch=2, steps=5,
          a=3.0, b=-4.0, c=2.0, eps=1e-7, ws=W_, nbytes=None):
        return dgt.gemm_orthogonalize(dtype, M, N, G, ldg, sg, O, ldo, so, batch, steps, a, b, c,
                                      eps, ws, need if nbytes is None else nbytes)

    assert o(dtype=5) == o(batch=-1) == o(batch=65536) == o(steps=0) == o(steps=65) == dgt.GEMM_ERR_ARG
    assert o(a=float("nan")) == o(c=float("inf")) == o(eps=-1.0) == o(nbytes=-1) == dgt.GEMM_ERR_ARG
    assert o(sg=-1) == o(so=2 ** 48) == dgt.GEMM_ERR_ARG
    assert o(M=-1) == o(N=-1) == dgt.GEMM_ERR_DIM
    assert o(ldg=47) == o(ldo=47) == dgt.GEMM_ERR_LD
    assert o(M=0) == o(N=0) == o(batch=0) == dgt.GEMM_OK
    assert o(G=0) == o(O=0) == dgt.GEMM_ERR_NULL
    assert o(ws=0) == o(nbytes=need - 1) == dgt.GEMM_ERR_WORKSPACE
    assert o(ws=W_ + 8) == dgt.GEMM_ERR_ALIGN
    assert o(so=32 * 48 - 1) == o(G=W_ + 64) == o(O=W_) == dgt.GEMM_ERR_OVERLAP


def _u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def test_torch_calls_refuse_host_tensors_and_wrong_shapes():
    X = torch.zeros(4, 64)
    Q, S = _u8(4, 32), _u8(4, 16)
    with pytest.raises(ValueError, match="GPU tensor"):
        dgt.quantize_mx4(X, Q, S)
    with pytest.raises(ValueError, match="rows"):
        dgt.quantize_mx4(X, Q, S, trans=True)
    with pytest.raises(ValueError, match="code"):
        dgt.quantize_mx4(X, _u8(4, 16), S)
    with pytest.raises(TypeError):
        dgt.quantize_mx4(X.double(), Q, S)
    with pytest.raises(TypeError):
        dgt.quantize_mx4(X, Q.int(), S)
    with pytest.raises(ValueError, match="row-major"):
        dgt.quantize_mx4(torch.zeros(64, 4).t(), Q, S)
    with pytest.raises(ValueError, match="GPU tensor"):
        dgt.dequantize_mx4(Q, S, X)
    with pytest.raises(ValueError, match="scale"):
        dgt.dequantize_mx4(Q, _u8(4, 8), X)
    C = torch.zeros(4, 8)
    B, SB = _u8(8, 32), _u8(8, 16)
    with pytest.raises(ValueError, match="GPU tensor"):
        dgt.gemm_quantized(Q, S, B, SB, C)
    with pytest.raises(ValueError, match="one length"):
        dgt.gemm_quantized(Q, S, _u8(8, 48), SB, C)
    with pytest.raises(TypeError):
        dgt.gemm_quantized(X, None, B, SB, C)
    with pytest.raises(ValueError, match="shape mismatch"):
        dgt.gemm_quantized(torch.zeros(5, 64, dtype=torch.bfloat16), None, B, SB, C)
    with pytest.raises(ValueError, match="bias"):
        dgt.gemm_quantized(Q, S, B, SB, C, bias=torch.zeros(4))
    with pytest.raises(TypeError):
        dgt.gemm_quantized(Q, S, B, SB, C.bfloat16())
    O = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        dgt.orthogonalize(X, O)
    with pytest.raises(TypeError):
        dgt.orthogonalize(X, O.float())
    with pytest.raises(ValueError, match="shape mismatch"):
        dgt.orthogonalize(X, O[:, :32])
    with pytest.raises(ValueError, match="contiguous"):
        dgt.orthogonalize(X, O, workspace=_u8(8, 8).t())


def test_torch_calls_refuse_pitches_past_an_int():
    """A pitch that the C entry points' int would cut is refused; a single
    row's, which is never used, is not looked at."""
    far = torch.empty_strided((2, 64), (2 ** 32 + 64, 1), dtype=torch.bfloat16, device="meta")
    q, s = _u8(2, 32), _u8(2, 16)
    c = torch.empty(2, 2)
    for call in (lambda: dgt.quantize_mx4(far, q, s), lambda: dgt.dequantize_mx4(q, s, far),
                 lambda: dgt.gemm_quantized(far, None, q, s, c)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
    assert dgt._matrix(far[:1], "X") == (1, 64, 64)


def test_plain_format_pins():
    """The plain model itself: every code stands for its value and quantises
    back to itself; ties go to the even code; saturation; zero and NaN blocks."""
    codes = np.arange(16, dtype=np.uint8).repeat(2).reshape(1, 32)
    packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
    v = mp.values(packed, np.array([[129]], np.uint8), 32)
    assert list(v[0, 0:16:2]) == [0, 2, 4, 6, 8, 12, 16, 24]  # times 2^2
    q, s = mp.quantize(v)
    assert s[0, 0] == 129 and np.array_equal(q, packed)
    x = np.array([[6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.0, 7.9] + [0.0] * 22])
    q, s = mp.quantize(x)
    y = mp.values(q, s, 32)[0]
    assert s[0, 0] == 127 and list(y[:8]) == [6, 0, 1, 1, 2, 2, 4, 4] and y[9] == 6
    q, s = mp.quantize(np.zeros((1, 40)))
    assert not q.any() and list(s[0]) == [0, 0]
    bad = np.ones((1, 40))
    bad[0, 33] = np.inf
    q, s = mp.quantize(bad)
    assert list(s[0]) == [125, 255] and np.isnan(mp.values(q, s, 40)[0, 32:]).all()
