"""Gated projections and W4 entry points on the host: argument checks and
refusals, none of which reaches a kernel launch, and pins of the plain forms."""

import math

import numpy as np
import pytest
import torch

import dense_gemm_tuning_amd as dgt
import gated_plain as gp

X_, A_, B_, H_, G_, U_, D_, E_, W_ = (0x1000000 * i for i in range(1, 10))


@pytest.fixture(scope="module", autouse=True)
def built():
    import os
    if not os.path.exists(dgt.LIB_PATH):
        from dense_gemm_tuning_amd import build
        build.build()


def test_gated_argument_checks():
    def f(dtype=1, act=0, M=4, N=8, K=16, X=X_, ldx=16, Wg=A_, ldwg=16, Wu=B_, ldwu=16, bg=0, bu=0,
          H=H_, ldh=8, G=0, ldg=0, U=0, ldu=0):
        return dgt.gemm_gated(dtype, act, M, N, K, X, ldx, Wg, ldwg, Wu, ldwu, bg, bu, H, ldh, G, ldg, U, ldu)

    assert f(dtype=0) == f(dtype=3) == f(act=-1) == f(act=6) == dgt.GEMM_ERR_ARG
    assert f(M=-1) == f(N=-1) == f(K=-1) == f(M=dgt.GATED_MAX_DIM + 1) == dgt.GEMM_ERR_DIM
    assert f(ldx=15) == f(ldwg=15) == f(ldwu=15) == f(ldh=7) == dgt.GEMM_ERR_LD
    assert f(G=G_, ldg=7) == f(U=U_, ldu=7) == dgt.GEMM_ERR_LD
    assert f(M=0) == f(N=0) == f(M=0, X=0, H=0) == dgt.GEMM_OK
    assert f(X=0) == f(Wg=0) == f(Wu=0) == f(H=0) == f(H=0, K=0) == dgt.GEMM_ERR_NULL
    assert f(H=X_) == f(H=A_ + 32) == f(H=B_) == f(bg=H_) == f(bu=H_ + 60) == dgt.GEMM_ERR_OVERLAP
    assert f(G=H_, ldg=8) == f(U=H_, ldu=8) == f(G=G_, ldg=8, U=G_ + 14, ldu=8) == dgt.GEMM_ERR_OVERLAP
    # column ranges that share a column, or of unlike pitches
    assert f(G=G_, ldg=16, U=G_ + 14, ldu=16) == f(G=G_, ldg=16, U=G_ + 16, ldu=17) == dgt.GEMM_ERR_OVERLAP
    assert f(G=G_ + 14, ldg=16, U=G_, ldu=16) == f(H=G_ + 16, ldh=16, G=G_, ldg=15) == dgt.GEMM_ERR_OVERLAP


def test_grad_argument_checks():
    need = dgt.gemm_gated_grad_workspace_size(4, 8)
    assert need >= 64
    assert dgt.gemm_gated_grad_workspace_size(0, 8) == dgt.gemm_gated_grad_workspace_size(4, 0) == 0
    assert dgt.gemm_gated_grad_workspace_size(-1, 8) == dgt.GEMM_ERR_DIM

    def f(dtype=2, act=0, M=4, N=8, K=16, dY=X_, lddy=16, Wd=A_, ldw=8, G=G_, ldg=8, U=U_, ldu=8, dG=D_,
          lddg=8, dU=E_, lddu=8, H=0, ldh=0, sg=0, su=0, ws=0, nbytes=0):
        return dgt.gemm_gated_grad(dtype, act, M, N, K, dY, lddy, Wd, ldw, G, ldg, U, ldu, dG, lddg, dU, lddu, H,
                                   ldh, sg, su, ws, nbytes)

    assert f(dtype=0) == f(act=9) == f(nbytes=-1) == dgt.GEMM_ERR_ARG
    assert f(M=-1) == f(N=-1) == f(K=dgt.GATED_MAX_DIM + 1) == dgt.GEMM_ERR_DIM
    assert f(lddy=15) == f(ldw=7) == f(ldg=7) == f(ldu=7) == f(lddg=7) == f(lddu=7) == dgt.GEMM_ERR_LD
    assert f(H=H_, ldh=7) == dgt.GEMM_ERR_LD
    assert f(N=0, sg=B_) == f(M=0) == dgt.GEMM_OK
    assert f(dY=0) == f(Wd=0) == f(G=0) == f(U=0) == f(dG=0) == f(dU=0) == dgt.GEMM_ERR_NULL
    assert f(sg=B_) == f(su=B_, ws=W_, nbytes=need - 1) == dgt.GEMM_ERR_WORKSPACE
    assert f(sg=B_, ws=W_ + 8, nbytes=need) == dgt.GEMM_ERR_ALIGN
    assert f(sg=B_, su=B_ + 4, ws=W_, nbytes=need) == f(sg=W_, ws=W_, nbytes=need) == dgt.GEMM_ERR_OVERLAP
    assert f(sg=B_, ws=G_, nbytes=need) == f(sg=G_, ws=W_, nbytes=need) == dgt.GEMM_ERR_OVERLAP
    assert f(dG=X_) == f(dG=A_) == f(dG=U_) == f(dU=G_) == f(dG=E_) == f(H=D_, ldh=8) == dgt.GEMM_ERR_OVERLAP
    assert f(dG=G_ + 2) == f(dG=G_, lddg=9) == f(H=G_, ldh=8) == dgt.GEMM_ERR_OVERLAP


def test_grad_outputs_over_the_products_operands():
    need = dgt.gemm_gated_grad_workspace_size(1, 8)

    def f(M=1, N=8, K=8, dY=X_, Wd=A_, H=0, sg=0, su=0):
        return dgt.gemm_gated_grad(2, 0, M, N, K, dY, K, Wd, N, G_, N, U_, N, D_, N, E_, N, H, N, sg, su,
                                   W_ if sg or su else 0, need if sg or su else 0)

    # only dG over G and dU over U may share memory: each output stands against every input
    assert f(H=X_) == f(M=4, H=X_) == f(H=A_) == f(H=U_) == dgt.GEMM_ERR_OVERLAP
    for k in (1, 8):
        assert f(K=k, sg=A_) == f(K=k, sg=X_) == f(K=k, sg=G_) == f(K=k, su=A_) == dgt.GEMM_ERR_OVERLAP


def _w(group=64, K=100):
    return dict(ldq=64, lds=gp.groups(K, group), ldz=gp.groups(K, group))


def test_w4_quantize_argument_checks():
    def f(dtype=0, group=64, st=2, M=4, K=100, X=X_, ldx=100, Q=A_, ldq=64, S=B_, lds=2, Z=G_, ldz=2):
        return dgt.gemm_w4_quantize(dtype, group, st, M, K, X, ldx, Q, ldq, S, lds, Z, ldz)

    assert f(dtype=3) == f(group=16) == f(group=256) == f(group=0) == f(st=0) == f(st=3) == dgt.GEMM_ERR_ARG
    assert f(M=-1) == f(K=-1) == f(M=dgt.GATED_MAX_DIM + 1) == dgt.GEMM_ERR_DIM
    assert f(ldx=99) == f(ldq=48) == f(lds=1) == f(ldz=1) == f(ldq=dgt.MX4_MAX_PITCH + 16) == dgt.GEMM_ERR_LD
    assert f(M=0) == f(K=0, X=0) == dgt.GEMM_OK
    assert f(X=0) == f(Q=0) == f(S=0) == dgt.GEMM_ERR_NULL
    assert f(Q=A_ + 8) == f(ldq=72) == f(S=B_ + 1) == dgt.GEMM_ERR_ALIGN
    assert f(X=A_) == f(S=A_) == f(Z=A_ + 5) == f(Z=B_) == f(Z=X_ + 1) == dgt.GEMM_ERR_OVERLAP
    assert f(Z=0, ldz=0, X=A_) == dgt.GEMM_ERR_OVERLAP


def test_w4_dequantize_argument_checks():
    def f(dtype=1, group=32, st=1, M=4, K=100, Q=A_, ldq=64, S=B_, lds=4, Z=G_, ldz=4, Y=H_, ldy=100):
        return dgt.gemm_w4_dequantize(dtype, group, st, M, K, Q, ldq, S, lds, Z, ldz, Y, ldy)

    assert f(dtype=-1) == f(group=48) == f(st=0) == dgt.GEMM_ERR_ARG
    assert f(M=-1) == f(K=-1) == dgt.GEMM_ERR_DIM
    assert f(ldy=99) == f(ldq=32) == f(lds=3) == f(ldz=3) == dgt.GEMM_ERR_LD
    assert f(M=0) == f(K=0) == dgt.GEMM_OK
    assert f(Q=0) == f(S=0) == f(Y=0) == dgt.GEMM_ERR_NULL
    assert f(Q=A_ + 4) == dgt.GEMM_ERR_ALIGN
    assert f(Y=A_) == f(Y=B_) == f(Y=G_) == dgt.GEMM_ERR_OVERLAP


def test_w4_product_argument_checks():
    def f(dtype=1, group=128, st=2, M=4, N=8, K=100, alpha=1.0, A=X_, lda=100, Q=A_, ldq=64, S=B_, lds=1, Z=G_,
          ldz=1, beta=0.0, C=H_, ldc=8, bias=0):
        return dgt.gemm_w4_a16(dtype, group, st, M, N, K, alpha, A, lda, Q, ldq, S, lds, Z, ldz, beta, C, ldc, bias)

    assert f(dtype=0) == f(group=1) == f(st=0) == dgt.GEMM_ERR_ARG
    assert f(M=-1) == f(N=-1) == f(K=-1) == dgt.GEMM_ERR_DIM
    assert f(lda=99) == f(ldq=48) == f(lds=0) == f(ldz=0) == f(ldc=7) == dgt.GEMM_ERR_LD
    assert f(M=0) == f(N=0) == dgt.GEMM_OK
    assert f(A=0) == f(Q=0) == f(S=0) == f(C=0) == f(C=0, alpha=0.0) == dgt.GEMM_ERR_NULL
    assert f(Q=A_ + 1) == f(ldq=65) == dgt.GEMM_ERR_ALIGN
    assert f(C=X_) == f(C=A_) == f(C=B_) == f(C=G_) == f(bias=H_) == dgt.GEMM_ERR_OVERLAP
    assert f(bias=H_, alpha=0.0) == dgt.GEMM_ERR_OVERLAP


def test_w4_gated_argument_checks():
    def f(dtype=1, act=0, group=128, st=2, M=4, N=8, K=100, X=X_, ldx=100, Q=A_, ldq=64, S=B_, lds=1, Z=G_,
          ldz=1, bg=0, bu=0, H=H_, ldh=8):
        return dgt.gemm_w4_gated(dtype, act, group, st, M, N, K, X, ldx, Q, ldq, S, lds, Z, ldz, bg, bu, H, ldh)

    assert f(dtype=0) == f(act=6) == f(group=129) == f(st=5) == dgt.GEMM_ERR_ARG
    assert f(M=-1) == f(N=-1) == f(K=-1) == f(N=dgt.GATED_MAX_DIM // 2 + 1) == dgt.GEMM_ERR_DIM
    assert f(ldx=99) == f(ldq=48) == f(lds=0) == f(ldz=0) == f(ldh=7) == dgt.GEMM_ERR_LD
    assert f(M=0) == f(N=0) == dgt.GEMM_OK
    assert f(X=0) == f(Q=0) == f(S=0) == f(H=0) == dgt.GEMM_ERR_NULL
    assert f(Q=A_ + 2) == dgt.GEMM_ERR_ALIGN
    # the second half of the weight's rows counts too
    assert f(H=X_) == f(H=A_ + 64 * 15) == f(H=B_ + 30) == f(H=G_ + 15) == f(bg=H_) == dgt.GEMM_ERR_OVERLAP


def test_torch_calls_refuse_host_tensors_and_wrong_shapes():
    h = torch.float16
    X, W, H = torch.zeros(4, 64, dtype=h), torch.zeros(8, 64, dtype=h), torch.zeros(4, 8, dtype=h)
    with pytest.raises(ValueError, match="GPU tensor"):
        dgt.gated(X, W, W, H)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        dgt.gated(X.float(), W.float(), W.float(), H.float())
    with pytest.raises(TypeError, match="Wu must be"):
        dgt.gated(X, W, W.bfloat16(), H)
    with pytest.raises(ValueError, match="shape mismatch: Wu"):
        dgt.gated(X, W, W[:7], H)
    with pytest.raises(ValueError, match="shape mismatch: H"):
        dgt.gated(X, W, W, H[:3])
    with pytest.raises(ValueError, match="row-major"):
        dgt.gated(X, W, W, torch.zeros(8, 4, dtype=h).t())
    with pytest.raises(ValueError, match="bias_u"):
        dgt.gated(X, W, W, H, bias_u=torch.zeros(9))
    with pytest.raises(ValueError, match="act must be"):
        dgt.gated(X[:0], W[:0], W[:0], H[:0, :0], act="tanh")
    with pytest.raises(ValueError, match="GPU tensor"):
        dgt.gated_grad(X, W.t().contiguous(), H, H, H, H)
    with pytest.raises(ValueError, match="shape mismatch: Wd"):
        dgt.gated_grad(X, W, H, H, H, H)
    with pytest.raises(ValueError, match="shape mismatch: dU"):
        dgt.gated_grad(X, W.t().contiguous(), H, H, H, H[:, :4])
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        dgt.gated_grad(X, W.t().contiguous(), H, H, H, H, workspace=torch.zeros(4, 4).t()[1:])
    assert dgt.gated(X[:0], W[:0], W[:0], H[:0, :0]) == dgt.GEMM_OK


def test_torch_w4_calls_refuse_host_tensors_and_wrong_shapes():
    X, C, H = torch.zeros(4, 100), torch.zeros(4, 8), torch.zeros(4, 4, dtype=torch.float16)
    A = X.half()
    Q, S, Z = dgt.w4_empty(8, 100, group=64, device="cpu")
    assert Q.shape == (8, 64) and S.shape == Z.shape == (8, 2) and S.dtype is torch.float16
    assert dgt.w4_empty(8, 100, scale_dtype=torch.bfloat16, zeros=False, device="cpu")[1:] is not None
    with pytest.raises(ValueError, match="group must be"):
        dgt.w4_empty(8, 100, group=96, device="cpu")
    with pytest.raises(ValueError, match="GPU tensor"):
        dgt.gemm_w4(A, Q, S, Z, C, group=64)
    with pytest.raises(ValueError, match="in groups of 128"):
        dgt.gemm_w4(A, Q, S, Z, C)
    with pytest.raises(ValueError, match="in groups of 64"):  # of another K
        dgt.gemm_w4(torch.zeros(4, 64, dtype=torch.float16), Q, S, Z, C, group=64)
    with pytest.raises(ValueError, match="code bytes"):
        dgt.gemm_w4(A, Q[:, :48], S, Z, C, group=64)
    with pytest.raises(TypeError, match="Z"):
        dgt.gemm_w4(A, Q, S, Z.int(), C, group=64)
    with pytest.raises(TypeError, match="S"):
        dgt.gemm_w4(A, Q, S.float(), Z, C, group=64)
    with pytest.raises(TypeError, match="A must be"):
        dgt.gemm_w4(X, Q, S, Z, C, group=64)
    with pytest.raises(TypeError, match="C must be"):
        dgt.gemm_w4(A, Q, S, Z, C.half(), group=64)
    with pytest.raises(ValueError, match="GPU tensor"):
        dgt.gated_w4(A, Q, S, Z, H, group=64)
    with pytest.raises(ValueError, match="must have 16 rows"):
        dgt.gated_w4(A, Q, S, Z, torch.zeros(4, 8, dtype=torch.float16), group=64)
    with pytest.raises(ValueError, match="GPU tensor"):
        dgt.quantize_w4(torch.zeros(8, 100), Q, S, Z, group=64)
    with pytest.raises(ValueError, match="GPU tensor"):
        dgt.dequantize_w4(Q, S, None, torch.zeros(8, 100), group=64)
    with pytest.raises(ValueError, match="rows"):
        dgt.quantize_w4(X, Q, S, Z, group=64)


# ---- the plain forms' own pins

@pytest.mark.parametrize("name", gp.ACTS)
def test_plain_slope_is_the_activations_derivative(name):
    x = torch.linspace(-9, 9, 361, dtype=torch.float64) + 0.0123
    h = 1e-6
    diff = (gp.act(x + h, name) - gp.act(x - h, name)) / (2 * h)
    assert (diff - gp.slope(x, name)).abs().max() < 1e-8
    want = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "relu": torch.relu,
            "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh"), "sigmoid": torch.sigmoid,
            "identity": lambda t: t}[name](x)
    assert (want - gp.act(x, name)).abs().max() < 1e-14


def test_plain_quantizer_by_hand():
    x = np.array([[0.0, 1.5, -0.5, 3.25]])
    q, s, z = gp.quantize(x, 32, torch.float16, True)  # s = 3.75/15, z = 2
    assert s.item() == 0.25 and z.item() == 2 and q.tolist() == [[2, 8, 0, 15]]
    assert gp.values(q, s, z, 32).tolist() == x.tolist()
    x = np.array([[7.0, -8.0, 2.5, 3.5, -0.5]])  # ties to the even side
    q, s, z = gp.quantize(x, 32, torch.bfloat16, False)
    assert s.item() == 1.0 and q.tolist() == [[15, 0, 10, 12, 8]]
    q, s, z = gp.quantize(np.zeros((1, 3)), 32, torch.bfloat16, True)
    assert s.item() == 0 and z.item() == 0 and not q.any()
    q, s, z = gp.quantize(np.array([[1.0, math.inf]]), 32, torch.bfloat16, True)
    assert math.isnan(s.item()) and not q.any()
    assert gp.pack(np.array([[1, 2, 3]], np.uint8)).tolist() == [[0x21, 0x03] + [0] * 14]
