"""gemm_orthogonalize at its size limits: rows that span more than 2^31 bytes
within a tile, and as many of them as FP16's range allows."""

import pytest
import torch

import dense_gemm_tuning_amd as dgt
import orth_model as om
from gpu_util import say

pytestmark = pytest.mark.gpu

# Five steps, normwise: half a bf16 step of the result, and half an FP16 step for
# each of S, B and X in the last step and as much again for the steps before.
NORMWISE = 2.0 ** -8 + 6 * 2.0 ** -11


def plain(G, steps=5, eps=1e-7):
    """The iteration in 64 bits as polynomials of one Gram matrix: every X is P X0
    with P of the smaller dimension.  The Gram matrix of a long X0 is summed in 256
    pieces of k (a whole one would run on one compute unit)."""
    a, b, c = om.COEF
    tall = G.shape[0] > G.shape[1]
    X = (G.t() if tall else G).double()
    X = X / (torch.linalg.vector_norm(X) + eps)
    n, k = X.shape
    Z = torch.nn.functional.pad(X, (0, -k % 256)).view(n, 256, -1).transpose(0, 1).contiguous()
    S0 = torch.bmm(Z, Z.transpose(1, 2).contiguous()).sum(0)
    P = torch.eye(n, dtype=X.dtype, device=X.device)
    for _ in range(steps):
        S = P.mm(S0).mm(P.t().contiguous())
        P = a * P + (b * S + c * S.mm(S)).mm(P)
    X = P.mm(X)
    return X.t() if tall else X


@pytest.mark.parametrize("M,N,kind", [(64, 2 ** 24, "normal"), (33, 2 ** 24 - 5, "rank8"), (2 ** 26, 8, "normal"),
                                      (2 ** 26, 1, "normal"), (1, 2 ** 24, "normal")])
def test_longest_matrices(M, N, kind):
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    G = om.matrix(gen, M, N, kind).to(torch.bfloat16)
    O = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dgt.check(dgt.orthogonalize(G, O))
    rel = om.normwise(O, plain(G))
    say("orth", M, N, kind, "normwise", rel)
    assert rel <= NORMWISE


def test_one_large_element_in_a_long_matrix():
    """A singular direction along one column, where X's elements are near 1 and
    held times 2^13."""
    M, N = 2 ** 26, 2
    G = torch.zeros(M, N, device="cuda")
    G[12345, 0] = 3.0
    G[M - 1, 1] = -2.0
    O = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dgt.check(dgt.orthogonalize(G, O))
    # Every sum has one term, so the documented roundings give these values
    # whatever the scale; then half a bf16 step, and as much as one FP16 operand
    # may differ where a term's fp32 rounding crosses one of its borders.
    want = om.rounded(G[[12345, M - 1]])
    got = O[[12345, M - 1]].double()
    assert ((got - want).abs() <= (2.0 ** -8 + 2.0 ** -10) * want.abs()).all()
    O[[12345, M - 1]] = 0.0
    assert not O.any()
