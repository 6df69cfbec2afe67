"""The gated projections and their gradient on rows that start on 16-byte boundaries and whose K, or N, ends inside
a 16-byte piece, NaN behind it: what the DMA tiles copy past the end must not reach a sum.  Whole numbers make the
results exact."""

import pytest
import torch

import dense_gemm_tuning_amd as dgt
import gated_plain as gp
from gpu_util import say
from test_gated_gpu import gen_for, ints, out_like, stored

pytestmark = pytest.mark.gpu

DT = gp.DT

KS = [1, 7, 31, 65, 130, 1001]
# few rows, tiles of 128 that end inside, and sizes that take tiles of 256
MN = [(1, 17), (8, 130), (33, 64), (64, 200), (65, 65), (129, 301), (300, 127), (2900, 3333)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("K", KS)
@pytest.mark.parametrize("M,N", MN)
def test_forward(M, N, K, dtype):
    say("gated, K tail", M, N, K, dtype)
    gen = gen_for(M, N, K, 71)
    X = stored(ints(gen, M, K, top=1), dtype, -K % 8)
    Wg, Wu = (stored(ints(gen, N, K, top=1), dtype, -K % 8 + extra) for extra in (0, 8))
    b = ints(gen, 2, N).cuda()
    H, h_ok = out_like(M, N, dtype, 1)
    G, g_ok = out_like(M, N, dtype, 0, 1)
    U, u_ok = out_like(M, N, dtype, 3)
    dgt.check(dgt.gated(X, Wg, Wu, H, act="relu", bias_g=b[0], bias_u=b[1], G=G, U=U))
    g, u = X.float() @ Wg.float().T + b[0], X.float() @ Wu.float().T + b[1]
    assert torch.equal(G, g.to(DT[dtype])) and torch.equal(U, u.to(DT[dtype]))
    assert torch.equal(H, (g.clamp(min=0) * u).to(DT[dtype]))
    assert h_ok() and g_ok() and u_ok()


@pytest.mark.parametrize("M,K", [(1, 7), (1, 1001), (1, 65)])
def test_a_single_row_at_any_pitch(M, K):
    """Through the C call, which takes a single row's pitch as it is given."""
    gen = gen_for(M, K, 79)
    N = 100
    X, Wg, Wu = (stored(ints(gen, r, K, top=1), "bf16", -K % 8) for r in (M, N, N))
    want = (X.float() @ Wg.float().T) * (X.float() @ Wu.float().T)
    for ldx in (K, K - K % 8 + 8, K - K % 8 + 16):
        say("gated, one row", K, ldx)
        H, h_ok = out_like(M, N, "bf16", 1)
        dgt.check(dgt.gemm_gated(dgt.DTYPE_BF16, dgt.ACT_IDENTITY, M, N, K, X.data_ptr(), ldx, Wg.data_ptr(), Wg.stride(0),
                                 Wu.data_ptr(), Wu.stride(0), 0, 0, H.data_ptr(), N + 1,
                                 stream=torch.cuda.current_stream().cuda_stream))
        assert torch.equal(H, want.bfloat16()) and h_ok()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("K", KS)
@pytest.mark.parametrize("M,N", MN)
def test_gradient(M, N, K, dtype):
    say("gated_grad, K tail", M, N, K, dtype)
    gen = gen_for(M, N, K, 73)
    t = DT[dtype]
    dY, Wd = stored(ints(gen, M, K, top=1), dtype, -K % 8), stored(ints(gen, K, N, top=1), dtype, -N % 8)
    G, U = stored(ints(gen, M, N), dtype, -N % 8), stored(ints(gen, M, N), dtype, 1)
    dG, g_ok = out_like(M, N, dtype, 1)
    dU, u_ok = out_like(M, N, dtype, -N % 8)
    H, h_ok = out_like(M, N, dtype, 2)
    sums = torch.full((2, N), 5.0, device="cuda")
    dgt.check(dgt.gated_grad(dY, Wd, G, U, dG, dU, act="relu", H=H, dbias_g=sums[0], dbias_u=sums[1]))
    dh, g, u = dY.float() @ Wd.float(), G.float(), U.float()
    dg, du = dh * u * (g > 0), dh * g.clamp(min=0)
    assert torch.equal(dG, dg.to(t)) and torch.equal(dU, du.to(t)) and torch.equal(H, (g.clamp(min=0) * u).to(t))
    want = torch.stack([dg.double().sum(0), du.double().sum(0)])
    assert want.abs().max() < 2 ** 23
    assert torch.equal(sums.double(), want)
    assert g_ok() and u_ok() and h_ok()
