"""gemm_orthogonalize on the GPU against the plain 64-bit iteration."""

import numpy as np
import pytest
import torch

import dense_gemm_tuning_amd as dgt
import mx4_plain as mp
from gpu_util import say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
COEF = (3.4445, -4.7750, 2.0315)


def matrix(rng, M, N, dtype, kind="lowrank"):
    if kind == "normal":
        g = rng.standard_normal((M, N))
    else:
        r = max(1, min(M, N) // 8)
        g = (rng.standard_normal((M, r)) @ rng.standard_normal((r, N)) / np.sqrt(r)
             + 0.3 * rng.standard_normal((M, N)))
    return torch.from_numpy(g * 0.01).to(DT[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N", [(1, 1), (1, 7), (9, 1), (2, 2), (33, 64), (64, 33), (128, 128), (100, 257),
                                 (257, 100), (130, 520), (384, 129)])
def test_one_step_within_its_rounding_bound(M, N, dtype):
    """Every element within the bound derived from the documented roundings."""
    say("orth step", M, N, dtype)
    rng = np.random.default_rng([M, N])
    G = matrix(rng, M, N, dtype)
    O = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dgt.check(dgt.orthogonalize(G.cuda(), O, steps=1, coefficients=COEF))
    g = G.double().numpy()
    want = mp.newton_schulz(g, 1, *COEF, 1e-7)
    err = np.abs(O.double().cpu().numpy() - want)
    bound = mp.newton_schulz_step_bound(g, *COEF, 1e-7)
    assert (err <= bound).all(), (err / bound).max()


# Five steps, normwise.  The result's own rounding is at most 2^-8 of each
# element; rounding the products' operands (half an FP16 step, 2^-11, for each
# of S, B and X) is what the steps add: three of them in the last step, whose
# singular values are near 1, and less than as much again from the steps
# before, whose errors later steps move by factors below 1 along the strong
# directions while the halves of X keep the weak ones: 2^-8 + 6 * 2^-11.
NORMWISE = 2.0 ** -8 + 6 * 2.0 ** -11


@pytest.mark.parametrize("kind", ["normal", "lowrank"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(48, 48), (64, 200), (256, 256), (300, 129), (256, 1000), (1025, 320), (777, 777)])
def test_five_steps(M, N, dtype, kind):
    rng = np.random.default_rng([M, N, 1])
    G = matrix(rng, M, N, dtype, kind)
    O = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dgt.check(dgt.orthogonalize(G.cuda(), O))
    want = mp.newton_schulz(G.double().numpy(), 5, *COEF, 1e-7)
    rel = np.linalg.norm(O.double().cpu().numpy() - want) / np.linalg.norm(want)
    say("orth", M, N, dtype, kind, "normwise", rel)
    assert rel <= NORMWISE


@pytest.mark.parametrize("M,N", [(96, 160), (200, 72), (256, 256)])
def test_batch_strides_and_guards(M, N):
    """A batch with padded rows and problem strides equals its problems one by
    one, bit for bit, and nothing else is written."""
    nb = 3
    rng = np.random.default_rng([M, N, 2])
    gp, op = N + 3, N + 5
    gs, os_ = M * gp + 11, M * op + 9
    Gf = torch.full((nb * gs,), float("nan"), device="cuda")
    Of = torch.full((nb * os_ + 1,), -7.0, dtype=torch.bfloat16, device="cuda")
    G = Gf.as_strided((nb, M, N), (gs, gp, 1))
    O = Of[1:].as_strided((nb, M, N), (os_, op, 1))
    for z in range(nb):
        G[z] = matrix(rng, M, N, "f32").cuda()
    dgt.check(dgt.orthogonalize(G, O))
    for z in range(nb):
        one = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        dgt.check(dgt.orthogonalize(G[z].contiguous(), one))
        assert torch.equal(one, O[z])
    guard = torch.ones(nb * os_ + 1, dtype=torch.bool)
    guard[1:].as_strided((nb, M, N), (os_, op, 1)).fill_(False)
    assert (Of.cpu()[guard] == -7.0).all()


def test_in_place_and_workspace_guard():
    G = matrix(np.random.default_rng(5), 130, 260, "bf16").cuda()
    want = torch.empty_like(G)
    dgt.check(dgt.orthogonalize(G, want))
    need = dgt.gemm_orthogonalize_workspace_size(130, 260, 1)
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    O = G.clone()
    dgt.check(dgt.orthogonalize(O, O, workspace=ws[:need]))
    assert torch.equal(O, want)
    assert (ws[need:] == 0x5A).all()
    assert dgt.orthogonalize(G, O, workspace=ws[:need - 1]) == dgt.GEMM_ERR_WORKSPACE


def test_special_inputs():
    """Zero stays zero; the result does not depend on the input's size; an
    infinity or NaN gives NaN; the norm of values whose squares pass fp32's range."""
    O = torch.full((40, 70), float("nan"), dtype=torch.bfloat16, device="cuda")
    dgt.check(dgt.orthogonalize(torch.zeros(40, 70, device="cuda"), O))
    assert not O.any()
    G = matrix(np.random.default_rng(6), 40, 70, "f32").cuda()
    dgt.check(dgt.orthogonalize(G, O, eps=0.0))
    base = O.clone()
    for f in (2.0 ** 90, 2.0 ** -90):
        dgt.check(dgt.orthogonalize(G * f, O, eps=0.0))
        assert torch.equal(O, base)
    for bad in (float("nan"), float("inf")):
        H = G.clone()
        H[3, 4] = bad
        dgt.check(dgt.orthogonalize(H, O))
        assert torch.isnan(O).all()
    dgt.check(dgt.orthogonalize(torch.zeros(40, 70, device="cuda"), O, eps=0.0))
    assert torch.isnan(O).all()


def test_other_coefficients_and_step_counts():
    """The cubic iteration (1.5, -0.5, 0), many steps: orthonormal rows."""
    rng = np.random.default_rng(8)
    g = rng.standard_normal((32, 512))
    G = torch.from_numpy(g).float()
    O = torch.empty(32, 512, dtype=torch.bfloat16, device="cuda")
    dgt.check(dgt.orthogonalize(G.cuda(), O, steps=20, coefficients=(1.5, -0.5, 0.0)))
    want = mp.newton_schulz(G.double().numpy(), 20, 1.5, -0.5, 0.0, 1e-7)
    o = O.double().cpu().numpy()
    assert np.linalg.norm(o - want) <= NORMWISE * np.linalg.norm(want)
    assert np.abs(o @ o.T - np.eye(32)).max() < 0.02


def test_graph_capture_and_streams():
    """Captured and replayed on new inputs; two calls on two streams at once,
    each with its own workspace."""
    rng = np.random.default_rng(9)
    G = torch.empty(192, 320, device="cuda")
    O = torch.empty(192, 320, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(dgt.gemm_orthogonalize_workspace_size(192, 320, 1), dtype=torch.uint8, device="cuda")
    G.copy_(matrix(rng, 192, 320, "f32"))
    dgt.check(dgt.orthogonalize(G, O, workspace=ws))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dgt.check(dgt.orthogonalize(G, O, workspace=ws))
    for _ in range(4):
        G.copy_(matrix(rng, 192, 320, "f32"))
        graph.replay()
        torch.cuda.synchronize()
        got = O.clone()
        dgt.check(dgt.orthogonalize(G, O, workspace=ws))
        torch.cuda.synchronize()
        assert torch.equal(got, O)
    H = matrix(rng, 192, 320, "f32").cuda()
    P = torch.empty_like(O)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dgt.check(dgt.orthogonalize(H, P, stream=side))
    dgt.check(dgt.orthogonalize(G, O))
    torch.cuda.synchronize()
    assert torch.equal(got, O)
    dgt.check(dgt.orthogonalize(H, O))
    torch.cuda.synchronize()
    assert torch.equal(P, O)


def test_update_then_serve():
    """The operators in a row: weight gradient, its orthogonalised update, the
    new weight packed into 4 bits, and a decode batch against it."""
    T, I, OUT = 256, 320, 192
    rng = np.random.default_rng(10)
    X, Gy = (torch.from_numpy(rng.standard_normal(s)).to(torch.bfloat16).cuda() for s in ((T, I), (T, OUT)))
    W = torch.from_numpy(0.05 * rng.standard_normal((OUT, I))).float().cuda()
    dW = torch.empty(OUT, I, device="cuda")
    dgt.check(dgt.gemm(Gy, X, dW, trans_a=True))
    U = torch.empty(OUT, I, dtype=torch.bfloat16, device="cuda")
    dgt.check(dgt.orthogonalize(dW, U))
    W.add_(U.float(), alpha=-0.02)
    Q, S = dgt.mx4_empty(OUT, I)
    dgt.check(dgt.quantize_mx4(W, Q, S))
    D = torch.from_numpy(rng.standard_normal((4, I))).to(torch.bfloat16).cuda()
    Y = torch.empty(4, OUT, device="cuda")
    dgt.check(dgt.gemm_quantized(D, None, Q, S, Y))
    dw = Gy.double().cpu().numpy().T @ X.double().cpu().numpy()
    u = mp.newton_schulz(dw, 5, *COEF, 1e-7)
    assert np.linalg.norm(U.double().cpu().numpy() - u) <= NORMWISE * np.linalg.norm(u)
    w = mp.values(*mp.quantize(W.double().cpu().numpy()), I)
    d = D.double().cpu().numpy()
    assert (np.abs(Y.double().cpu().numpy() - d @ w.T) <= (I + 4) * 2.0 ** -23 * (np.abs(d) @ np.abs(w).T)).all()


# The tests above run matrices small enough for 32 x 32 tiles; these sizes
# take the large tiles: edges in both dimensions, K tails, a long k summed in
# parts, and a few rows or columns only.
LARGE = [(1100, 900), (900, 2100), (2100, 260), (260, 2100), (1030, 1030), (1, 2300), (2305, 3), (2304, 130)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N", LARGE)
def test_large_one_step_within_its_rounding_bound(M, N, dtype):
    say("orth large step", M, N, dtype)
    G = matrix(np.random.default_rng([M, N, 3]), M, N, dtype)
    O = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dgt.check(dgt.orthogonalize(G.cuda(), O, steps=1, coefficients=COEF))
    g = G.double().numpy()
    err = np.abs(O.double().cpu().numpy() - mp.newton_schulz(g, 1, *COEF, 1e-7))
    bound = mp.newton_schulz_step_bound(g, *COEF, 1e-7)
    assert (err <= bound).all(), (err / bound).max()


@pytest.mark.parametrize("kind", ["normal", "lowrank"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", LARGE)
def test_large_five_steps(M, N, dtype, kind):
    G = matrix(np.random.default_rng([M, N, 4]), M, N, dtype, kind)
    O = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dgt.check(dgt.orthogonalize(G.cuda(), O))
    want = mp.newton_schulz(G.double().numpy(), 5, *COEF, 1e-7)
    rel = np.linalg.norm(O.double().cpu().numpy() - want) / np.linalg.norm(want)
    say("orth large", M, N, dtype, kind, "normwise", rel)
    assert rel <= NORMWISE


@pytest.mark.parametrize("M,N", [(950, 1000), (1000, 940), (260, 2100), (2100, 130)])
def test_large_batch_strides_and_guards(M, N):
    """Padded rows and problem strides, results off 16-byte rows, a workspace
    that starts as NaN: every problem right, nothing else written, and a NaN
    in one problem stays there."""
    nb = 3
    rng = np.random.default_rng([M, N, 5])
    gp, op = N + 3, N + 5
    gs, os_ = M * gp + 11, M * op + 9
    Gf = torch.full((nb * gs,), float("nan"), device="cuda")
    Of = torch.full((nb * os_ + 1,), -7.0, dtype=torch.bfloat16, device="cuda")
    G = Gf.as_strided((nb, M, N), (gs, gp, 1))
    O = Of[1:].as_strided((nb, M, N), (os_, op, 1))
    for z in range(nb):
        G[z] = matrix(rng, M, N, "f32").cuda()
    need = dgt.gemm_orthogonalize_workspace_size(M, N, nb)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    dgt.check(dgt.orthogonalize(G, O, workspace=ws[:need]))
    for z in range(nb):
        want = mp.newton_schulz(G[z].double().cpu().numpy(), 5, *COEF, 1e-7)
        rel = np.linalg.norm(O[z].double().cpu().numpy() - want) / np.linalg.norm(want)
        assert rel <= NORMWISE
    guard = torch.ones(nb * os_ + 1, dtype=torch.bool)
    guard[1:].as_strided((nb, M, N), (os_, op, 1)).fill_(False)
    assert (Of.cpu()[guard] == -7.0).all()
    assert (ws[need:] == 0xFF).all()
    base = O.clone()
    G[1, M // 2, N // 2] = float("nan")
    dgt.check(dgt.orthogonalize(G, O, workspace=ws[:need]))
    assert torch.isnan(O[1]).all()
    assert torch.equal(O[0], base[0]) and torch.equal(O[2], base[2])


@pytest.mark.parametrize("M,N", [(2200, 300), (1000, 1100)])
def test_large_in_place_and_replayed(M, N):
    """The result over its input; captured and replayed on new inputs."""
    rng = np.random.default_rng([M, N, 6])
    G = matrix(rng, M, N, "bf16").cuda()
    O = torch.empty_like(G)
    ws = torch.empty(dgt.gemm_orthogonalize_workspace_size(M, N, 1), dtype=torch.uint8, device="cuda")
    dgt.check(dgt.orthogonalize(G, O, workspace=ws))
    H = G.clone()
    dgt.check(dgt.orthogonalize(H, H, workspace=ws))
    assert torch.equal(H, O)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dgt.check(dgt.orthogonalize(G, O, workspace=ws))
    for _ in range(3):
        G.copy_(matrix(rng, M, N, "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        got = O.clone()
        O.zero_()
        dgt.check(dgt.orthogonalize(G, O, workspace=ws))
        torch.cuda.synchronize()
        assert torch.equal(got, O)
    dgt.check(dgt.orthogonalize(torch.zeros_like(G), O, workspace=ws))
    assert not O.any()


def test_many_tiny_matrices():
    """A batch large enough for the large tiles, of matrices far smaller than one."""
    rng = np.random.default_rng(11)
    G = torch.stack([matrix(rng, 24, 40, "f32") for _ in range(400)])
    O = torch.full((400, 24, 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    dgt.check(dgt.orthogonalize(G.cuda(), O))
    got = O.double().cpu().numpy()
    for z in range(400):
        want = mp.newton_schulz(G[z].double().numpy(), 5, *COEF, 1e-7)
        assert np.linalg.norm(got[z] - want) <= NORMWISE * np.linalg.norm(want), z


@pytest.mark.parametrize("M,N", [(1, 70001), (70001, 2)])
def test_very_long_matrices(M, N):
    G = matrix(np.random.default_rng([M, N, 12]), M, N, "f32", "normal")
    O = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    dgt.check(dgt.orthogonalize(G.cuda(), O))
    want = mp.newton_schulz(G.double().numpy(), 5, *COEF, 1e-7)
    assert np.linalg.norm(O.double().cpu().numpy() - want) <= NORMWISE * np.linalg.norm(want)


def test_two_graphs_with_a_workspace_each():
    """Two captured calls replayed on two streams at once."""
    rng = np.random.default_rng(13)
    sets = []
    for M, N in ((256, 256), (260, 2100)):
        G = matrix(rng, M, N, "bf16").cuda()
        want, O = torch.empty_like(G), torch.empty_like(G)
        dgt.check(dgt.orthogonalize(G, want))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):  # the workspace comes from the graph's own pool
            dgt.check(dgt.orthogonalize(G, O))
        sets.append((graph, G, want, O, torch.cuda.Stream()))
    for _ in range(3):
        for _, _, _, O, _ in sets:
            O.zero_()
        torch.cuda.synchronize()
        for graph, _, _, _, stream in sets:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for _, _, want, O, _ in sets:
            assert torch.equal(O, want)
