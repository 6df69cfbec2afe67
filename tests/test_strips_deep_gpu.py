"""The kernels that stream weights past a few rows, over their whole steady state: strips of every width with
wavefronts of several steps (rings that wrap, second runs of scales), each against plain results that whole numbers
make exact."""

import pytest
import torch

import dense_gemm_tuning_amd as dgt
import gated_plain as gp
from gpu_util import say
from test_gated_gpu import out_like

pytestmark = pytest.mark.gpu

DT = gp.DT


def whole(gen, *shape, top=1):
    return torch.randint(-top, top + 1, shape, generator=gen, device="cuda").float()


def packed(gen, rows, K, group, st, zeros, room):
    """A weight (codes in the stored layout, scales, zero points or None) and its values in fp32, whole multiples of
    1/2.  `room`: how far zero points lie from the middle."""
    n = gp.groups(K, group)
    q = torch.randint(0, 16, (rows, -(-K // 32) * 32), generator=gen, device="cuda", dtype=torch.uint8)
    s = torch.tensor([0.5, 1.0, -1.0], device="cuda")[torch.randint(0, 3, (rows, n), generator=gen, device="cuda")]
    z = torch.randint(8 - room, 9 + room, (rows, n), generator=gen, device="cuda", dtype=torch.uint8)
    if not zeros:
        z.fill_(8)
    w = torch.empty(rows, K, device="cuda")
    for r in range(0, rows, 4096):  # some rows at a time: the wide ones take gigabytes
        at = slice(r, r + 4096)
        sw, zw = (t[at].float().repeat_interleave(group, 1)[:, :K] for t in (s, z))
        w[at] = sw * (q[at, :K].float() - zw)
    return (q[:, 0::2] | (q[:, 1::2] << 4), s.to(DT[st]), z if zeros else None), w


# outputs where strips have 1, 2, 4 and 8 blocks of 16 stored rows (gated: 2, 4 and 8), cut off inside a block;
# K where wavefronts have a second step, more than a ring, and a second run of scales of every group size
W4_N = [130, 4101, 8203, 16410]
W4_K = [2100, 4616, 9000]


@pytest.mark.parametrize("M,dtype", [(1, "bf16"), (16, "f16")])
@pytest.mark.parametrize("K", W4_K)
@pytest.mark.parametrize("N", W4_N)
def test_w4_strips_are_exact(N, K, M, dtype):
    gen = torch.Generator(device="cuda").manual_seed(N + K + M)
    for group, st, zeros in ((128, "f16", True), (64, "bf16", True), (32, "f16", False), (128, "bf16", False)):
        say("w4 strips", M, N, K, dtype, group, st, zeros)
        W, w = packed(gen, N, K, group, st, zeros, 8)
        X = whole(gen, M, K)
        want = X @ w.t()
        assert X.abs().sum(1).max() * 16 < 2 ** 22  # every partial sum is exact
        b = whole(gen, N, top=8)
        C = torch.full((M, N + 1), 4.0, device="cuda")
        dgt.check(dgt.gemm_w4(X.to(DT[dtype]), *W, C[:, :N], group=group, beta=0.5, bias=b))
        assert torch.equal(C[:, :N], want + 2.0 + b) and (C[:, N] == 4.0).all()


@pytest.mark.parametrize("M,dtype", [(1, "f16"), (16, "bf16")])
@pytest.mark.parametrize("K", W4_K)
@pytest.mark.parametrize("N", [130, 4101, 8203])
def test_w4_gated_strips_are_exact(N, K, M, dtype):
    gen = torch.Generator(device="cuda").manual_seed(N + K + M + 1)
    for group, st, zeros in ((128, "f16", True), (64, "bf16", False), (32, "f16", True)):
        say("w4 gated strips", M, N, K, dtype, group, st, zeros)
        W, w = packed(gen, 2 * N, K, group, st, zeros, 1)
        X = whole(gen, M, K) * (torch.rand(M, K, generator=gen, device="cuda") < 64 / K)
        b = whole(gen, 2, N, top=8)
        g, u = (X @ w.t()).split(N, dim=1)
        want = (g + b[0]).clamp(min=0) * (u + b[1])
        assert want.abs().max() < 2 ** 22  # a multiple of 1/4: exact in fp32
        H = torch.full((M, N + 1), 77.0, dtype=DT[dtype], device="cuda")
        dgt.check(dgt.gated_w4(X.to(DT[dtype]), *W, H[:, :N], act="relu", group=group, bias_g=b[0], bias_u=b[1]))
        assert torch.equal(H[:, :N], want.to(DT[dtype])) and (H[:, N] == 77.0).all()


# two chunks of rows of one strip
@pytest.mark.parametrize("M,N,K", [(17, 4101, 4616), (32, 2050, 9000), (30, 8190, 2100)])
def test_w4_strips_of_two_row_chunks(M, N, K):
    gen = torch.Generator(device="cuda").manual_seed(N + K + M + 2)
    for group in (32, 64, 128):
        say("w4 strips, two chunks", M, N, K, group)
        W, w = packed(gen, N, K, group, "f16", True, 8)
        X = whole(gen, M, K)
        C = torch.empty(M, N, device="cuda")
        dgt.check(dgt.gemm_w4(X.half(), *W, C, group=group))
        assert torch.equal(C, X @ w.t())


# 16-bit weights: 2, 4 and 8 blocks of 16 stored rows; up to 16 rows, 32, 64; wavefronts of 2, 5 and 9 steps (up to 32
# rows), 3 to 17 above
@pytest.mark.parametrize("K", [1032, 4104, 8200])
@pytest.mark.parametrize("N", [34, 4100, 8200])
@pytest.mark.parametrize("M,dtype", [(1, "f16"), (15, "bf16"), (16, "f16"), (27, "bf16"), (32, "f16"), (50, "f16"), (64, "bf16")])
def test_gated_strips_are_exact(M, dtype, N, K):
    say("gated strips", M, N, K, dtype)
    gen = torch.Generator(device="cuda").manual_seed(N + K + M + 3)
    X, W, b = whole(gen, M, K), whole(gen, 2 * N, K), whole(gen, 2, N, top=8)
    H, h_ok = out_like(M, N, dtype, 1)
    G, g_ok = out_like(M, N, dtype, 0, 1)
    U, u_ok = out_like(M, N, dtype, 3)
    Wt = W.to(DT[dtype])
    dgt.check(dgt.gated(X.to(DT[dtype]), Wt[:N], Wt[N:], H, act="relu", bias_g=b[0], bias_u=b[1], G=G, U=U))
    g, u = (X @ W.t()).split(N, dim=1)
    g, u = g + b[0], u + b[1]
    want = g.clamp(min=0) * u
    assert want.abs().max() < 2 ** 24
    assert torch.equal(G, g.to(DT[dtype])) and torch.equal(U, u.to(DT[dtype]))
    assert torch.equal(H, want.to(DT[dtype]))
    assert h_ok() and g_ok() and u_ok()
