"""4-bit products at the ends of the activations' range: infinities and NaN, and the largest sums that are
still exact."""

import numpy as np
import pytest
import torch

import dense_gemm_tuning_amd as dgt
import gated_plain as gp
from gpu_util import say
from test_gated_gpu import stored as stored16
from test_w4_gpu import on_gpu, rng_for, whole_weight

pytestmark = pytest.mark.gpu

DT = gp.DT
# few rows, and the kernel that shares the activations: on 16-byte rows and off them
FORMS = [(3, 0), (40, 0), (40, 1)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,pad", FORMS)
def test_a_bad_activation_makes_its_row_nan(M, pad, dtype, group):
    rng = rng_for(M, pad, len(dtype), group)
    N, K = 70, 520
    for zeros in (True, False):
        say("w4 bad activations", M, pad, dtype, group, zeros)
        q, s, z = whole_weight(rng, 2 * N, K, group, "f16", zeros)
        s[7], z[9] = 0.0, 0  # neither a scale of 0 nor a zero point of 0 hides it
        W = on_gpu(q, s, z, zeros, 0)
        X = torch.from_numpy(rng.integers(-1, 2, (M, K)).astype(np.float32))
        bad = X.clone()
        bad[0, K - 1], bad[1, 0], bad[2, 300] = float("inf"), float("-inf"), float("nan")
        got = []
        for x in (X, bad):
            C = torch.empty(M, 2 * N, device="cuda")
            H = torch.empty(M, N, dtype=DT[dtype], device="cuda")
            dgt.check(dgt.gemm_w4(stored16(x, dtype, pad), *W, C, group=group))
            dgt.check(dgt.gated_w4(stored16(x, dtype, pad), *W, H, act="relu", group=group))
            got.append((C, H))
        for clean, poor in zip(*got):
            assert torch.isnan(poor[:3]).all() and torch.equal(poor[3:], clean[3:])
            assert not torch.isnan(clean).any()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,pad", FORMS)
def test_sums_below_2_to_119_are_exact(M, pad, group):
    """Whole numbers times 2^108, at most 2 of them: a group's |x| add up to 2^116 at most.  x q and z x are below 2^125,
    scales of 2^-100 bring the results back, all powers of two times whole numbers below 2^24."""
    rng = rng_for(M, pad, group, 5)
    N, K = 70, 520
    q, s, z = whole_weight(rng, N, K, group, "bf16", True)
    z[5] = 255
    s = s.abs().clamp(max=1).double()
    X = torch.from_numpy(rng.integers(-2, 3, (M, K)).astype(np.float64))
    want = X @ torch.from_numpy(gp.values(q, s, z, group).T.copy())
    assert want.abs().max() < 2 ** 22
    C = torch.empty(M, N, device="cuda")
    W = on_gpu(q, (s * 2.0 ** -100).bfloat16(), z, True, 0)
    dgt.check(dgt.gemm_w4(stored16(X * 2.0 ** 108, "bf16", pad), *W, C, group=group))
    assert torch.equal(C.cpu().double(), want * 256)
