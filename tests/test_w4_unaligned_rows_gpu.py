"""4-bit products of many rows whose activations start off 16-byte boundaries, which pass through registers on
their way to LDS: rows of fewer than 8 elements, steps that end everywhere, stages that are refilled, and workgroups that
start at every run of the scales.  Against plain results that whole numbers make exact."""

import pytest
import torch

import dense_gemm_tuning_amd as dgt
import gated_plain as gp
from gpu_util import say
from test_gated_gpu import stored as stored16
from test_strips_deep_gpu import packed, whole

pytestmark = pytest.mark.gpu

DT = gp.DT

# (rows, outputs): up to one block of 32 rows over 8192 outputs, blocks that end inside, several blocks
SIZES = [(33, 130), (17, 8300), (65, 700), (130, 257)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 6, 7, 8, 9, 31, 255, 257, 769, 1025, 2055, 4109, 8191])
def test_rows_anywhere_are_exact(K, dtype):
    gen = torch.Generator(device="cuda").manual_seed(K + len(dtype))
    for M, N in SIZES:
        for group, zeros, pad, offset in ((128, True, 1, 1), (64, False, 2, 3), (32, True, 0, 5)):
            if (K + pad) % 8 == 0 and offset % 8 == 0:
                continue
            say("w4 rows anywhere", M, N, K, dtype, group, zeros, pad, offset)
            W, w = packed(gen, N, K, group, "f16", zeros, 8)
            X, b = whole(gen, M, K), whole(gen, N, top=8)
            want = X @ w.t()
            assert X.abs().sum(1).max() * 16 < 2 ** 22
            C = torch.full((M, N + 1), 4.0, device="cuda")
            dgt.check(dgt.gemm_w4(stored16(X, dtype, pad, offset), *W, C[:, :N], group=group, alpha=2.0, beta=0.5, bias=b))
            assert torch.equal(C[:, :N], 2 * want + 2.0 + b) and (C[:, N] == 4.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(33, 65, 3), (65, 700, 769), (40, 300, 1025), (17, 4150, 2055), (100, 520, 8191)])
def test_gated_rows_anywhere(M, N, K, dtype):
    gen = torch.Generator(device="cuda").manual_seed(M + N + K + len(dtype))
    for group, zeros, pad, offset in ((128, True, 1, 1), (64, False, 2, 3), (32, True, 0, 5)):
        say("w4 gated rows anywhere", M, N, K, dtype, group, zeros)
        W, w = packed(gen, 2 * N, K, group, "bf16", zeros, 1)
        X = whole(gen, M, K) * (torch.rand(M, K, generator=gen, device="cuda") < 64 / K)
        b = whole(gen, 2, N, top=8)
        g, u = (X @ w.t()).split(N, dim=1)
        want = (g + b[0]).clamp(min=0) * (u + b[1])
        assert want.abs().max() < 2 ** 22
        H = torch.full((M, N + 1), 77.0, dtype=DT[dtype], device="cuda")
        dgt.check(dgt.gated_w4(stored16(X, dtype, pad, offset), *W, H[:, :N], act="relu", group=group, bias_g=b[0],
                               bias_u=b[1]))
        assert torch.equal(H[:, :N], want.to(DT[dtype])) and (H[:, N] == 77.0).all()


@pytest.mark.parametrize("M,N,K", [(300, 3600, 2055), (65, 16400, 1025)])
def test_sizes_whose_aligned_form_takes_larger_tiles(M, N, K):
    gen = torch.Generator(device="cuda").manual_seed(M)
    for group in (32, 128):
        say("w4 rows anywhere", M, N, K, group)
        W, w = packed(gen, N, K, group, "bf16", True, 8)
        X = whole(gen, M, K)
        C = torch.empty(M, N, device="cuda")
        dgt.check(dgt.gemm_w4(stored16(X, "bf16", 1, 1), *W, C, group=group))
        assert torch.equal(C, X @ w.t())
