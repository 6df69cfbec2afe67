"""gemm_orthogonalize on matrices whose weak directions show every rounding of
X: exactly low rank, and singular values that fall as a power.  Each step
multiplies what rounding X adds in the weak directions by 3.4, so an iterate
kept in one FP16 half only is 0.15 off on a matrix of rank one, and one whose low
half is lost before the last two steps 3e-3; the documented scheme is 1.7e-3."""

import math

import pytest
import torch

import dense_gemm_tuning_amd as dgt
import orth_model as om
from gpu_util import say

pytestmark = pytest.mark.gpu

# small matrices (direct tiles) and large ones (DMA tiles; Gram parts), wide and tall
SIZES = [(256, 256), (200, 520), (520, 200), (1030, 1030), (400, 2100), (2100, 400), (1152, 1280), (1280, 1152)]


@pytest.mark.parametrize("kind", ["rank1", "rank8", "power1", "power2", "normal", "lowrank"])
@pytest.mark.parametrize("M,N", SIZES)
def test_five_steps_by_spectrum(M, N, kind):
    gen = torch.Generator(device="cuda").manual_seed(1000 * M + N)
    G = (0.01 * om.matrix(gen, M, N, kind)).float()
    O = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dgt.check(dgt.orthogonalize(G, O))
    want = om.plain(G)
    rel, gate = om.normwise(O, want), om.gate(G, want)
    say("orth", M, N, kind, "normwise", rel, "gate", gate)
    assert rel <= gate


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 7])
@pytest.mark.parametrize("M,N", [(256, 256), (1030, 1030), (400, 2100), (2100, 400)])
def test_other_step_counts(M, N, steps):
    """Each number of steps ends with another copy of X and its low half."""
    gen = torch.Generator(device="cuda").manual_seed(steps)
    G = om.matrix(gen, M, N, "rank8").float()
    O = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dgt.check(dgt.orthogonalize(G, O, steps=steps))
    want = om.plain(G, steps)
    rel, gate = om.normwise(O, want), om.gate(G, want, steps)
    say("orth", M, N, steps, "steps, normwise", rel, "gate", gate)
    assert rel <= gate


@pytest.mark.parametrize("M,N", [(1, 5000), (8, 300), (300, 8), (48, 48), (48, 2600), (2600, 48), (100, 700)])
def test_few_rows(M, N):
    """With few rows each rounding of the Gram matrix and of the polynomial
    weighs more: a diagonal rounded to FP16 makes one row 2.4 times as far off
    as its own rounding to bf16, normal values of 48 x 2600 1.9 times.  Over
    eight matrices, within 1.3 times the error of the documented roundings."""
    gen = torch.Generator(device="cuda").manual_seed(10 * M + N)
    G = torch.stack([om.matrix(gen, M, N, "normal").float() for _ in range(8)])
    O = torch.full(G.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    dgt.check(dgt.orthogonalize(G, O))
    want = [om.plain(g) for g in G]

    def rms(errors):
        return math.sqrt(sum(e * e for e in errors) / len(G))

    rel = rms(om.normwise(o, w) for o, w in zip(O, want))
    own = rms(om.normwise(w.to(torch.bfloat16), w) for w in want)
    before = rms(om.normwise(om.rounded(g), w) for g, w in zip(G, want))
    say("orth", M, N, "rms", rel, "own rounding", own, "documented roundings before it", before)
    assert rel <= math.sqrt((1.02 * own) ** 2 + (1.3 * before) ** 2)
