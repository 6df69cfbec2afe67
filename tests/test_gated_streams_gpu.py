"""Gated calls at the same time, captured with workspaces of their own, and with operands and results that are column
ranges of one matrix: each against the same calls one after the other on storage of their own."""

import math

import pytest
import torch

import dense_gemm_tuning_amd as dgt
from gpu_util import say
from test_strips_deep_gpu import packed, whole

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def block(M, N, K, gen):
    """A block's weights, and a step on inputs of its own: forward, gradient with the biases' sums, the workspace allocated by
    the call."""
    W = (torch.randn(2 * N, K, generator=gen, device="cuda") / math.sqrt(K)).to(BF)
    Wd = (torch.randn(K, N, generator=gen, device="cuda") / math.sqrt(N)).to(BF)

    def fresh():
        return [torch.randn(M, K, generator=gen, device="cuda").to(BF) for _ in range(2)]

    def outs():
        return [torch.full((M, c), float("nan"), dtype=BF, device="cuda") for c in (N, 2 * N, 2 * N)] + \
            [torch.full((2, N), float("nan"), device="cuda")]

    def work(x, o, stream=None):
        (X, dY), (H, P, D, s) = x, o
        dgt.check(dgt.gated(X, W[:N], W[N:], H, act="gelu", G=P[:, :N], U=P[:, N:], stream=stream))
        dgt.check(dgt.gated_grad(dY, Wd, P[:, :N], P[:, N:], D[:, :N], D[:, N:], act="gelu", dbias_g=s[0], dbias_u=s[1],
                                 stream=stream))

    return fresh, outs, work


# strips, register-staged tiles (odd K) and DMA tiles of both sizes
SIZES = [(6, 200, 520), (200, 136, 263), (300, 520, 264), (2560, 2560, 128)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_two_streams_at_once(M, N, K):
    gen = torch.Generator(device="cuda").manual_seed(M)
    fresh, outs, work = block(M, N, K, gen)
    xs = [fresh() for _ in range(3)]
    want = [outs() for _ in xs]
    for x, o in zip(xs, want):
        work(x, o)
    streams, got = [torch.cuda.Stream() for _ in xs], [outs() for _ in xs]
    torch.cuda.synchronize()
    say("two streams", M, N, K)
    for turn in range(6):
        for st, x, o in zip(streams, xs, got):
            if turn % 2:
                work(x, o, stream=st)
            else:
                with torch.cuda.stream(st):
                    work(x, o)
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))


@pytest.mark.parametrize("M,N,K", SIZES)
def test_captured_with_the_calls_own_workspace(M, N, K):
    gen = torch.Generator(device="cuda").manual_seed(M + 1)
    fresh, outs, work = block(M, N, K, gen)
    held, got = [fresh() for _ in range(2)], [outs() for _ in range(2)]
    work(held[0], got[0])
    torch.cuda.synchronize()
    graphs = []
    for x, o in zip(held, got):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            work(x, o)
    say("captured", M, N, K)
    for _ in range(3):
        for graph, x, o in zip(graphs, held, got):
            new, want = fresh(), outs()
            for a, b in zip(x, new):
                a.copy_(b)
            graph.replay()
            work(new, want)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(o, want))


@pytest.mark.parametrize("M,N,K", [(7, 200, 520), (40, 136, 263), (130, 264, 135), (300, 300, 72), (2600, 2600, 129)])
def test_column_ranges_of_one_matrix(M, N, K):
    """X, H, G and U side by side in rows on 16-byte boundaries: what a kernel copies behind X's last k are results as
    they are written."""
    gen = torch.Generator(device="cuda").manual_seed(M + 2)
    X, W = whole(gen, M, K), whole(gen, 2 * N, K)
    Wb = torch.full((2 * N, K + -K % 8), float("nan"), dtype=BF, device="cuda")[:, :K]
    Wb.copy_(W)
    g, u = (X @ W.t()).split(N, dim=1)
    want = torch.cat([X, g * u, g, u], dim=1).to(BF)
    A = torch.full((M, K + 3 * N + -(K + 3 * N) % 8), float("nan"), dtype=BF, device="cuda")
    A[:, :K] = X.to(BF)
    say("column ranges", M, N, K)
    dgt.check(dgt.gated(A[:, :K], Wb[:N], Wb[N:], A[:, K:K + N], act="identity", G=A[:, K + N:K + 2 * N],
                        U=A[:, K + 2 * N:K + 3 * N]))
    assert torch.equal(A[:, :K + 3 * N], want) and torch.isnan(A[:, K + 3 * N:]).all()
    # the gradient: dY, dG, dU and H side by side
    dY, Wd = whole(gen, M, K), whole(gen, K, N)
    G, U = whole(gen, M, N, top=3), whole(gen, M, N, top=3)
    Wdb = torch.full((K, N + -N % 8), float("nan"), dtype=BF, device="cuda")[:, :N]
    Wdb.copy_(Wd)
    dh = dY @ Wd
    want = torch.cat([dY, dh * U, dh * G, G * U], dim=1).to(BF)
    A.fill_(float("nan"))
    A[:, :K] = dY.to(BF)
    dgt.check(dgt.gated_grad(A[:, :K], Wdb, G.to(BF), U.to(BF), A[:, K:K + N], A[:, K + N:K + 2 * N], act="identity",
                             H=A[:, K + 2 * N:K + 3 * N]))
    assert torch.equal(A[:, :K + 3 * N], want) and torch.isnan(A[:, K + 3 * N:]).all()


@pytest.mark.parametrize("M,N,K", [(3, 200, 519), (40, 136, 263), (130, 700, 1029), (17, 8200, 255)])
def test_w4_column_ranges_of_one_matrix(M, N, K):
    gen = torch.Generator(device="cuda").manual_seed(M + 3)
    for group in (32, 128):
        W, w = packed(gen, 2 * N, K, group, "bf16", True, 1)
        X = whole(gen, M, K) * (torch.rand(M, K, generator=gen, device="cuda") < 64 / K)
        g, u = (X @ w.t()).split(N, dim=1)
        for width in (-(K + N) % 8, -(K + N) % 8 + 1):  # 16-byte rows, and rows off them
            say("w4 column ranges", M, N, K, group, width)
            A = torch.full((M, K + N + width), float("nan"), dtype=BF, device="cuda")
            A[:, :K] = X.to(BF)
            dgt.check(dgt.gated_w4(A[:, :K], *W, A[:, K:K + N], act="identity", group=group))
            assert torch.equal(A[:, K:K + N], (g * u).to(BF)) and torch.equal(A[:, :K], X.to(BF))
            assert torch.isnan(A[:, K + N:]).all()
