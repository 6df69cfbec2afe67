"""gemm_orthogonalize at sizes that reach every form of the tile kernels:
256 x 256 and 128 x 128 tiles, with and without edges and a K tail, the Gram
matrix whole and in parts, wide and tall."""

import pytest
import torch

import dense_gemm_tuning_amd as dgt
import mx4_plain as mp
import orth_model as om
from gpu_util import say

pytestmark = pytest.mark.gpu

# More than 512 tiles of 128 take tiles of 256: the batches of 16, and the single ones.
# n a multiple of 256, of 128 only, and of neither; k likewise.
FORMS = [
    (16, 1024, 1024), (16, 1152, 1280), (16, 1280, 1152), (16, 1000, 1100), (16, 1100, 1000),
    (16, 1024, 1100), (16, 1100, 1024), (16, 1000, 1024), (16, 1024, 1000),
    # 128 x 128, the Gram matrix whole
    (8, 1024, 1024), (8, 1152, 1280), (8, 1280, 1152), (8, 1000, 1024), (8, 1024, 1000), (8, 1024, 1100),
    (8, 1100, 1024), (8, 1000, 1100), (8, 1100, 1000),
    # the Gram matrix in parts, whole and cut
    (1, 1152, 1280), (1, 1280, 1152), (1, 1024, 4096), (1, 4096, 1024), (1, 640, 2000), (1, 2000, 640),
    # one weight of ordinary size
    (1, 4096, 4096), (1, 2048, 8192), (1, 8192, 2048), (1, 4000, 4100), (1, 4100, 4000),
]


def inputs(batch, M, N, dtype):
    gen = torch.Generator(device="cuda").manual_seed(batch * 100003 + M * 1009 + N)
    G = torch.stack([om.matrix(gen, M, N, ("lowrank", "normal", "rank8")[z % 3]).float() for z in range(batch)])
    return (0.01 * G).to(dtype)


@pytest.mark.parametrize("batch,M,N", FORMS)
def test_five_steps(batch, M, N):
    """Every problem within the gate of the documented roundings, a workspace
    that starts as NaN, and the same bits again."""
    G = inputs(batch, M, N, torch.float32 if (M + N) % 3 else torch.bfloat16)
    need = dgt.gemm_orthogonalize_workspace_size(M, N, batch)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    O = torch.full((batch, M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dgt.check(dgt.orthogonalize(G, O, workspace=ws))
    worst = 0.0
    for z in range(batch):
        want = om.plain(G[z])
        rel, gate = om.normwise(O[z], want), om.gate(G[z], want)
        assert rel <= gate, (z, rel, gate)
        worst = max(worst, rel)
    say("orth form", batch, M, N, "normwise", worst)
    again = torch.empty_like(O)
    ws.fill_(0x3C)
    dgt.check(dgt.orthogonalize(G, again, workspace=ws))
    assert torch.equal(again, O)


@pytest.mark.parametrize("batch,M,N", [f for f in FORMS if max(f[1:]) <= 4096])
def test_one_step_within_its_rounding_bound(batch, M, N):
    """Every element of the first and the last problem within the bound
    derived from the documented roundings, rows off 16 bytes."""
    G = inputs(batch, M, N, torch.bfloat16 if M % 3 else torch.float16)
    flat = torch.full((batch * M * (N + 3) + 1,), float("nan"), dtype=G.dtype, device="cuda")
    Gs = flat[1:].as_strided(G.shape, (M * (N + 3), N + 3, 1))
    Gs.copy_(G)
    out = torch.full((batch * M * (N + 5) + 1,), -7.0, dtype=torch.bfloat16, device="cuda")
    O = out[1:].as_strided(G.shape, (M * (N + 5), N + 5, 1))
    dgt.check(dgt.orthogonalize(Gs, O, steps=1, coefficients=om.COEF))
    for z in {0, batch - 1}:
        g = G[z].double()
        err = (O[z].double() - om.plain(g, 1)).abs().cpu().numpy()
        assert (err <= mp.newton_schulz_step_bound(g.cpu().numpy(), *om.COEF, 1e-7)).all(), z
    O.fill_(-7.0)
    assert (out == -7.0).all()  # and nothing beside O was written
