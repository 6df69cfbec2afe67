"""The forms of the gated and 4-bit kernels that only some sizes take, against plain results that whole numbers
make exact: register-staged tiles of 128 and of 64 rows, rows of fewer than 8 elements, and the 4-bit kernel that shares
the activations of many rows."""

import numpy as np
import pytest
import torch

import dense_gemm_tuning_amd as dgt
import gated_plain as gp
from gpu_util import say
from test_gated_gpu import gen_for, ints, out_like, stored as stored16
from test_w4_gpu import on_gpu, rng_for, whole_weight

pytestmark = pytest.mark.gpu

DT = gp.DT

# 256 tiles of 128 rows and more, and fewer; rows shorter than a 16-byte piece, one element past one, and cut slices
FORWARD = [(1030, 2050, 65), (1030, 2050, 7), (2049, 1027, 130), (70, 70, 5), (65, 3, 9), (129, 300, 71), (64, 65, 1), (3, 200, 15)]
GRADIENT = [(2100, 2001, 65), (2050, 2047, 7), (2050, 2050, 130), (33000, 5, 66), (33000, 7, 3), (70, 5, 130), (100, 7, 3),
            (64, 200, 65), (65, 9, 64), (130, 15, 1), (1, 8, 71)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", FORWARD)
def test_forward_off_16_byte_rows(M, N, K, dtype):
    say("gated", M, N, K, dtype)
    gen = gen_for(M, N, K, 41)
    X, Wg, Wu = (stored16(ints(gen, r, K, top=1), dtype, 1 + K % 2, 1) for r in (M, N, N))
    b = ints(gen, 2, N).cuda()
    H, h_ok = out_like(M, N, dtype, 1)
    G, g_ok = out_like(M, N, dtype, 0, 1)
    U, u_ok = out_like(M, N, dtype, 3)
    dgt.check(dgt.gated(X, Wg, Wu, H, act="relu", bias_g=b[0], bias_u=b[1], G=G, U=U))
    g, u = X.float() @ Wg.float().T + b[0], X.float() @ Wu.float().T + b[1]  # whole numbers: exact
    assert torch.equal(G, g.to(DT[dtype])) and torch.equal(U, u.to(DT[dtype]))
    assert torch.equal(H, (g.clamp(min=0) * u).to(DT[dtype]))
    assert h_ok() and g_ok() and u_ok()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", GRADIENT)
def test_gradient_off_16_byte_rows(M, N, K, dtype):
    gen = gen_for(M, N, K, 43)
    t = DT[dtype]
    dY, Wd = stored16(ints(gen, M, K, top=1), dtype, 1 + K % 2, 1), stored16(ints(gen, K, N, top=1), dtype, 3)
    G, U = stored16(ints(gen, M, N), dtype, 1, 1), stored16(ints(gen, M, N), dtype, 0)
    dh, g, u = dY.float() @ Wd.float(), G.float(), U.float()
    dg, du = dh * u * (g > 0), dh * g.clamp(min=0)
    for place in (False, True):
        say("gated_grad", M, N, K, dtype, "in place" if place else "apart")
        dG, g_ok = (G, None) if place else out_like(M, N, dtype, 1)
        dU, u_ok = (U, None) if place else out_like(M, N, dtype, 0, 3)
        H, h_ok = out_like(M, N, dtype, 2)
        sums = torch.full((2, N), 5.0, device="cuda")
        dgt.check(dgt.gated_grad(dY, Wd, G, U, dG, dU, act="relu", H=H, dbias_g=sums[0], dbias_u=sums[1]))
        assert torch.equal(dG, dg.to(t)) and torch.equal(dU, du.to(t))
        assert torch.equal(H, (g.clamp(min=0) * u).to(t)) and h_ok()
        # whole numbers: sums below 2^24 are exact in any order
        want = torch.stack([dg.double().sum(0), du.double().sum(0)])
        assert want.abs().max() < 2 ** 23
        assert torch.equal(sums.double(), want)
        assert place or (g_ok() and u_ok())


@pytest.mark.parametrize("M,N,K", [(300, 333, 72), (2100, 2101, 64), (300, 5, 64), (2100, 2100, 64)])
def test_gradient_tiles_that_cross_the_last_column(M, N, K):
    """16-byte rows of the product's operands, rows of G, U and the outputs at any pitch: in place and apart."""
    gen = gen_for(M, N, K, 47)
    dY, Wd = ints(gen, M, K, top=1).half().cuda(), stored16(ints(gen, K, N, top=1), "f16", 8 - N % 8)
    G, U = stored16(ints(gen, M, N), "f16", 3, 1), stored16(ints(gen, M, N), "f16", 0)
    dh, g, u = dY.float() @ Wd.float(), G.float(), U.float()
    for place in (False, True):
        dG, dU = (G, U) if place else (out_like(M, N, "f16", 1)[0], out_like(M, N, "f16", 2)[0])
        dgt.check(dgt.gated_grad(dY, Wd, G, U, dG, dU, act="identity"))
        assert torch.equal(dG, (dh * u).half()) and torch.equal(dU, (dh * g).half())


# more than 64 rows, or more than 16 and more than 8192 stored rows: blocks, strips, steps, runs of groups and K's
# pieces that end inside one another
ROWS = [(65, 129, 520), (66, 130, 1003), (100, 257, 2055), (129, 100, 31), (70, 33, 257), (17, 8300, 130), (33, 8212, 263),
        (200, 128, 4104), (80, 1, 1), (65, 300, 9000), (300, 64, 8191)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", ROWS)
def test_w4_many_rows_are_exact_on_whole_numbers(M, N, K, dtype):
    rng = rng_for(M, N, K, 51)
    for group, st, zeros, alpha, beta in ((128, "f16", True, 1.0, 0.0), (64, "bf16", False, 1.5, 0.5), (32, dtype, True, -1.0, 0.0)):
        say("gemm_w4", M, N, K, dtype, group, st, zeros)
        q, s, z = whole_weight(rng, N, K, group, st, zeros)
        z = np.minimum(z, 15)
        X = torch.from_numpy((rng.random((M, K)) < min(1.0, 512 / K)) * rng.integers(-2, 3, (M, K)).astype(np.float32))
        # rows on 16-byte boundaries, NaN behind K
        A = stored16(X, dtype, -K % 8 + 8)
        want = alpha * (X.double().cuda() @ torch.from_numpy(gp.values(q, s, z, group).T.copy()).cuda())
        assert want.abs().max() < 2 ** 22
        C = torch.full((M, N + 1), 4.0, device="cuda")
        b = torch.from_numpy(rng.integers(-8, 9, N).astype(np.float32)).cuda()
        dgt.check(dgt.gemm_w4(A, *on_gpu(q, s, z, zeros, 0), C[:, :N], group=group, alpha=alpha, beta=beta, bias=b))
        assert torch.equal(C[:, :N].double(), want + 4 * beta + b.double())
        assert (C[:, N] == 4.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(65, 65, 520), (17, 4150, 263), (130, 63, 2055), (90, 1, 40)])
def test_w4_gated_many_rows(M, N, K, dtype):
    rng = rng_for(M, N, K, 53)
    for group, zeros in ((128, True), (64, False), (32, True)):
        say("gated_w4", M, N, K, dtype, group, zeros)
        q, s, z = whole_weight(rng, 2 * N, K, group, dtype, False)
        s = s.abs().clamp(max=1)
        if zeros:
            z = rng.integers(6, 10, z.shape).astype(np.uint8)
        X = torch.from_numpy((rng.random((M, K)) < min(1.0, 64 / K)) * rng.integers(-1, 2, (M, K)).astype(np.float32))
        bg, bu = (torch.from_numpy(rng.integers(-8, 9, N).astype(np.float32)).cuda() for _ in range(2))
        p = X.double().cuda() @ torch.from_numpy(gp.values(q, s, z, group).T.copy()).cuda()
        want = (p[:, :N] + bg).clamp(min=0) * (p[:, N:] + bu)
        assert want.abs().max() < 2 ** 22
        H = torch.full((M, N + 1), 77.0, dtype=DT[dtype], device="cuda")
        dgt.check(dgt.gated_w4(stored16(X, dtype, -K % 8 + 8), *on_gpu(q, s, z, zeros, 0), H[:, :N], act="relu", group=group,
                               bias_g=bg, bias_u=bu))
        assert torch.equal(H[:, :N], want.to(DT[dtype]))
        assert (H[:, N] == 77.0).all()


def test_w4_many_rows_without_k():
    none = [torch.empty(40, 0, dtype=t, device="cuda") for t in (torch.uint8, torch.float16, torch.uint8)]
    X = torch.empty(100, 0, dtype=torch.float16, device="cuda")
    H = torch.full((100, 20), 9.0, dtype=torch.float16, device="cuda")
    b = torch.arange(20, dtype=torch.float32, device="cuda")
    dgt.check(dgt.gated_w4(X, *none, H, act="relu", group=64, bias_g=b, bias_u=b * 0 + 2))
    assert torch.equal(H.float(), (2 * b).expand(100, 20))


def test_w4_a_bad_value_stays_in_its_row():
    rng = rng_for(57)
    M, N, K = 70, 200, 304
    W = on_gpu(*whole_weight(rng, N, K, 64, "f16", True), True, 0)
    X = torch.ones(M, K, dtype=torch.float16, device="cuda")
    clean, C = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    dgt.check(dgt.gemm_w4(X, *W, clean, group=64))
    X[3, 7], X[M - 1, K - 1] = float("inf"), float("nan")
    dgt.check(dgt.gemm_w4(X, *W, C, group=64))
    good = [r for r in range(M) if r not in (3, M - 1)]
    assert torch.equal(C[good], clean[good])
    assert torch.isnan(C[M - 1]).all()


def test_w4_many_rows_on_two_streams_and_in_graphs():
    rng = rng_for(59)
    M, N, K = 70, 260, 1000
    q, s, z = gp.quantize(rng.standard_normal((2 * N, K)), 128, torch.bfloat16, True)
    W = on_gpu(q, s, z, True, 0)
    xs = [torch.from_numpy(rng.standard_normal((M, K))).bfloat16().cuda() for _ in range(3)]

    def outs():
        return torch.empty(M, 2 * N, device="cuda"), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")

    def work(x, got):
        dgt.check(dgt.gemm_w4(x, *W, got[0]))
        dgt.check(dgt.gated_w4(x, *W, got[1]))

    want = [outs() for _ in xs]
    for x, w in zip(xs, want):
        work(x, w)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in xs], [outs() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(4):
        for st, x, g in zip(streams, xs, got):
            with torch.cuda.stream(st):
                work(x, g)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    held, out = xs[0].clone(), outs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work(held, out)
    for x, w in list(zip(xs, want)) * 2:
        held.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], w[0]) and torch.equal(out[1], w[1])
        work(x, outs())


@pytest.mark.parametrize("M,N,K", [(400, 2561, 264), (33, 8212, 520), (65, 4100, 263), (513, 130, 1031), (40, 16400, 129), (64, 64, 300)])
def test_w4_tiles_of_the_shared_kernel(M, N, K):
    """Each of its tiles, plain and gated, with strips and blocks of rows that end inside them."""
    rng = rng_for(M, N, K, 61)
    for group in (32, 64, 128):
        say("w4 tiles", M, N, K, group)
        q, s, z = whole_weight(rng, N + N % 2, K, group, "f16", False)
        s = s.abs().clamp(max=1)
        z = rng.integers(6, 10, z.shape).astype(np.uint8)
        X = torch.from_numpy((rng.random((M, K)) < min(1.0, 48 / K)) * rng.integers(-1, 2, (M, K)).astype(np.float32))
        A, W = stored16(X, "bf16", -K % 8), on_gpu(q, s, z, True, 0)
        p = X.double().cuda() @ torch.from_numpy(gp.values(q, s, z, group).T.copy()).cuda()
        C = torch.full((M, len(q) + 1), 4.0, device="cuda")
        dgt.check(dgt.gemm_w4(A, *W, C[:, :-1], group=group))
        assert torch.equal(C[:, :-1].double(), p) and (C[:, -1] == 4.0).all()
        F = len(q) // 2
        H = torch.full((M, F + 1), 77.0, dtype=torch.bfloat16, device="cuda")
        dgt.check(dgt.gated_w4(A, *W, H[:, :F], act="identity", group=group))
        want = p[:, :F] * p[:, F:]
        assert want.abs().max() < 2 ** 22
        assert torch.equal(H[:, :F], want.bfloat16()) and (H[:, F] == 77.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("N", [33, 4097, 8200])
@pytest.mark.parametrize("M,K", [(17, 520), (32, 1032), (33, 72), (64, 2056), (16, 8)])
def test_gated_strips_of_every_width(M, N, K, dtype):
    say("gated strips", M, N, K, dtype)
    gen = gen_for(M, N, K, 67)
    X, Wg, Wu = (stored16(ints(gen, r, K, top=1), dtype, 8) for r in (M, N, N))
    b = ints(gen, 2, N).cuda()
    H, h_ok = out_like(M, N, dtype, 1)
    G, g_ok = out_like(M, N, dtype, 0, 1)
    U, u_ok = out_like(M, N, dtype, 3)
    dgt.check(dgt.gated(X, Wg, Wu, H, act="relu", bias_g=b[0], bias_u=b[1], G=G, U=U))
    g, u = X.float() @ Wg.float().T + b[0], X.float() @ Wu.float().T + b[1]  # whole numbers: exact
    assert torch.equal(G, g.to(DT[dtype])) and torch.equal(U, u.to(DT[dtype]))
    assert torch.equal(H, (g.clamp(min=0) * u).to(DT[dtype]))
    assert h_ok() and g_ok() and u_ok()
