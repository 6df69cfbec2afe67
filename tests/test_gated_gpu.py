"""Gated projections and their gradient on the GPU against the plain 64-bit forms:
bit for bit where every sum is a whole number fp32 holds, else within the bounds
of `gated_plain`; storage, streams, graphs, and a block's forward and backward in a row."""

import math

import numpy as np
import pytest
import torch

import dense_gemm_tuning_amd as dgt
import gated_plain as gp
from gpu_util import say

pytestmark = pytest.mark.gpu

DT = gp.DT


def gen_for(*key):
    return torch.Generator().manual_seed(hash(tuple(map(int, key))) % (1 << 31))


def ints(gen, *shape, top=3):
    return torch.randint(-top, top + 1, shape, generator=gen).float()


def stored(t, dtype, pad, offset=0, fill=float("nan")):
    """t on the GPU as a view of a wider buffer filled with `fill`: `pad` columns more, `offset` elements in."""
    rows, cols = t.shape
    buf = torch.full((rows * (cols + pad) + offset + 8,), fill, dtype=DT[dtype], device="cuda")
    v = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(t)
    return v


def out_like(M, N, dtype, pad, offset=0):
    """An output view and a check that nothing around it was written."""
    buf = torch.full((M * (N + pad) + offset + 8,), 77.0, dtype=DT[dtype], device="cuda")
    v = buf[offset:offset + M * (N + pad)].view(M, N + pad)

    def untouched():
        rest = buf.clone()
        rest[offset:offset + M * (N + pad)].view(M, N + pad)[:, :N] = 77.0
        return bool((rest == 77.0).all())

    return v[:, :N], untouched


# every way a tile, a slice or a strip can end; rows on 16-byte boundaries and off them
SHAPES = [(1, 1, 1), (1, 16, 8), (1, 200, 512), (2, 33, 130), (4, 64, 264), (8, 130, 1000), (15, 17, 31), (16, 128, 256),
          (17, 63, 1024), (31, 64, 2056), (33, 100, 640), (48, 112, 384), (49, 129, 72), (64, 272, 328), (65, 65, 65),
          (100, 127, 128), (128, 128, 96), (129, 300, 200), (255, 64, 160), (256, 256, 128), (257, 129, 264),
          (300, 520, 72), (513, 136, 520)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward_is_exact_on_whole_numbers(M, N, K, dtype):
    """g, u and (act identity or relu) g*u are whole numbers below 2^24, so H, G and U are those rounded once.
    Biases, saving, padding and the offset off 16-byte boundaries alternate with the case."""
    gen = gen_for(M, N, K, len(dtype))
    for pad, offset, bias, save, act in ((0, 0, False, False, "relu"), (8, 0, True, True, "identity"),
                                         (3, 1, True, False, "relu"), (0, 8, False, True, "identity")):
        say("gated", M, N, K, dtype, pad, offset, bias, save, act)
        top = 1 if K > 1024 else 2
        X, Wg, Wu = ints(gen, M, K, top=top), ints(gen, N, K, top=1), ints(gen, N, K, top=top)
        bg, bu = (ints(gen, N).cuda(), ints(gen, N).cuda()) if bias else (None, None)
        h, g, u, _, _ = gp.forward(X, Wg, Wu, bg, bu, act)
        H, h_ok = out_like(M, N, dtype, pad, offset)
        G, g_ok = out_like(M, N, dtype, pad) if save else (None, None)
        U, u_ok = out_like(M, N, dtype, 0, offset) if save else (None, None)
        dgt.check(dgt.gated(stored(X, dtype, pad, offset), stored(Wg, dtype, pad), stored(Wu, dtype, 2 * pad, offset), H,
                            act=act, bias_g=bg, bias_u=bu, G=G, U=U))
        assert torch.equal(H.cpu(), h.to(DT[dtype])) and h_ok()
        if save:
            assert torch.equal(G.cpu(), g.to(DT[dtype])) and g_ok()
            assert torch.equal(U.cpu(), u.to(DT[dtype])) and u_ok()


# sizes whose tiles are the largest: whole ones, cut ones, and K ending inside a slice group
LARGE = [(2304, 2432, 128), (2100, 2100, 128), (2100, 2101, 200), (2900, 3336, 256)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", LARGE)
def test_large_tiles_are_exact_on_whole_numbers(M, N, K, dtype):
    gen = gen_for(M, N, K, 13)
    X, W = ints(gen, M, K, top=2).to(DT[dtype]).cuda(), ints(gen, 2 * N, K, top=2).to(DT[dtype]).cuda()
    b = ints(gen, 2, N).cuda()
    want = (X.float() @ W.float().T) + b.flatten()  # whole numbers below 2^24: exact in fp32
    H = torch.empty(M, N, dtype=DT[dtype], device="cuda")
    P = torch.empty(M, 2 * N, dtype=DT[dtype], device="cuda")
    dgt.check(dgt.gated(X, W[:N], W[N:], H, act="relu", bias_g=b[0], bias_u=b[1], G=P[:, :N], U=P[:, N:]))
    assert torch.equal(P, want.to(DT[dtype]))
    assert torch.equal(H, (want[:, :N].clamp(min=0) * want[:, N:]).to(DT[dtype]))
    dgt.check(dgt.gated(X, W[:N], W[N:], H, act="identity"))
    assert torch.equal(H, ((want - b.flatten())[:, :N] * (want - b.flatten())[:, N:]).to(DT[dtype]))
    # the gradient of the same size: Wd is K x N
    dY, Wd = ints(gen, M, K, top=1).to(DT[dtype]).cuda(), ints(gen, K, N + 8 - N % 8, top=1).to(DT[dtype]).cuda()[:, :N]
    G, U = ints(gen, M, N).to(DT[dtype]).cuda(), ints(gen, M, N).to(DT[dtype]).cuda()
    D = torch.full((M, 2 * N + 8), 77.0, dtype=DT[dtype], device="cuda")
    sums = torch.empty(2, N, device="cuda")
    dgt.check(dgt.gated_grad(dY, Wd, G, U, D[:, :N], D[:, N:2 * N], act="relu", H=H, dbias_g=sums[0], dbias_u=sums[1]))
    dh, g, u = dY.float() @ Wd.float(), G.float(), U.float()
    dg, du = dh * u * (g > 0), dh * g.clamp(min=0)
    assert torch.equal(D[:, :N], dg.to(DT[dtype])) and torch.equal(D[:, N:2 * N], du.to(DT[dtype]))
    assert torch.equal(H, (g.clamp(min=0) * u).to(DT[dtype])) and (D[:, 2 * N:] == 77.0).all()
    assert torch.equal(sums.double(), torch.stack([dg.double().sum(0), du.double().sum(0)]))
    dgt.check(dgt.gated_grad(dY, Wd, G, U, D[:, :N], D[:, N:2 * N], act="identity"))
    assert torch.equal(D[:, :N], (dh * u).to(DT[dtype])) and torch.equal(D[:, N:2 * N], (dh * g).to(DT[dtype]))


def close_forward(H, G, U, X, Wg, Wu, bg, bu, act, dtype, what):
    h, g, u, eg, eu = gp.forward(X, Wg, Wu, bg, bu, act)
    t = DT[dtype]
    # the activation moves by at most its slope's bound (1.13 for these) times g's error
    eh = 1.13 * eg * (u.abs() + eu) + gp.act(g, act).abs() * eu + gp.act_error(g, gp.act(g, act)) * u.abs() + \
        4 * gp.U24 * h.abs()
    for got, want, e, name in ((H, h, eh, "H"), (G, g, eg, "G"), (U, u, eu, "U")):
        if got is not None:
            gp.assert_within(got, want, gp.half_step(want.abs() + e, t) + e, f"{what} {name}")


@pytest.mark.parametrize("act", gp.ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_forward_activations(dtype, act):
    gen = gen_for(len(act), len(dtype))
    for M, N, K, bias in ((3, 70, 264, True), (150, 140, 136, False), (40, 36, 55, True), (260, 260, 1032, True)):
        X = (torch.randn(M, K, generator=gen) * 2).to(DT[dtype])
        Wg, Wu = ((torch.randn(N, K, generator=gen) * 2 / math.sqrt(K)).to(DT[dtype]) for _ in range(2))
        bg, bu = ((torch.randn(N, generator=gen) * 3).cuda() for _ in range(2)) if bias else (None, None)
        H, G, U = (torch.empty(M, N, dtype=DT[dtype], device="cuda") for _ in range(3))
        dgt.check(dgt.gated(X.cuda(), Wg.cuda(), Wu.cuda(), H, act=act, bias_g=bg, bias_u=bu, G=G, U=U))
        close_forward(H, G, U, X, Wg, Wu, bg, bu, act, dtype, f"{act} {M}x{N}x{K}")


@pytest.mark.parametrize("act", gp.ACTS)
def test_activations_over_the_whole_range(act):
    """K = 1 and weights of 1: g is x itself, from tails where the result underflows to large values."""
    x = torch.cat([torch.linspace(-120, 120, 4801), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e30, -1e30])])
    X = x.bfloat16().unsqueeze(1)
    one = torch.ones(1, 1, dtype=torch.bfloat16)
    H, G = (torch.empty(len(x), 1, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dgt.check(dgt.gated(X.cuda(), one.cuda(), one.cuda() * 0.5, H, act=act, G=G))
    want = gp.act(X.double(), act) * X.double() * 0.5
    assert torch.equal(G.cpu(), X)
    e = gp.act_error(torch.clamp(X.double(), -120, 120), want) + 4 * gp.U24 * want.abs() + 1e-37 * X.double().abs()
    gp.assert_within(H, want.bfloat16().double(), gp.half_step(want, torch.bfloat16) * 2 + e, act)


def test_halves_of_one_tensor():
    """Weights as row halves, pre-activations as column halves, as the gradient's products take them."""
    gen = gen_for(5)
    for M, N, K in ((5, 72, 128), (200, 136, 264)):
        X, W = ints(gen, M, K).bfloat16().cuda(), ints(gen, 2 * N, K, top=1).bfloat16().cuda()
        P = torch.empty(M, 2 * N, dtype=torch.bfloat16, device="cuda")
        H = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        dgt.check(dgt.gated(X, W[:N], W[N:], H, act="identity", G=P[:, :N], U=P[:, N:]))
        want = X.double().cpu() @ W.double().cpu().T
        assert torch.equal(P.cpu(), want.bfloat16())
        assert torch.equal(H.cpu(), (want[:, :N] * want[:, N:]).bfloat16())


def test_no_k_leaves_the_biases():
    bg, bu = torch.tensor([1.0, -2.0, 3.0]).cuda(), torch.tensor([2.0, 5.0, -1.0]).cuda()
    X, W = torch.empty(70, 0, dtype=torch.float16, device="cuda"), torch.empty(3, 0, dtype=torch.float16, device="cuda")
    H = torch.full((70, 3), 9.0, dtype=torch.float16, device="cuda")
    dgt.check(dgt.gated(X, W, W, H, act="relu", bias_g=bg, bias_u=bu))
    assert torch.equal(H.cpu(), torch.tensor([2.0, 0.0, -3.0]).half().expand(70, 3))
    dgt.check(dgt.gated(X[:2], W, W, H[:2], act="sigmoid"))
    assert not H[:2].any()
    # and of the gradient: dh is zero, H is still written
    G, U = torch.ones(70, 3, dtype=torch.float16, device="cuda"), torch.full_like(H, 4.0)
    dG, dU, H = (torch.full_like(U, 9.0) for _ in range(3))
    dgt.check(dgt.gated_grad(X, W.t(), G, U, dG, dU, act="relu", H=H))
    assert not dG.any() and not dU.any() and (H == 4.0).all()


@pytest.mark.parametrize("M,N,K", [(4, 64, 128), (70, 200, 136), (300, 300, 264)])
def test_a_bad_value_stays_in_its_row_or_column(M, N, K):
    gen = gen_for(M, N, K)
    X, Wg, Wu = (torch.randn(r, K, generator=gen).bfloat16() for r in (M, N, N))
    clean, H = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dgt.check(dgt.gated(X.cuda(), Wg.cuda(), Wu.cuda(), clean))
    X[M - 1, K - 1] = float("nan")
    Wu[N - 1, 0] = float("inf")
    dgt.check(dgt.gated(X.cuda(), Wg.cuda(), Wu.cuda(), H))
    assert torch.isnan(H[M - 1]).all()
    assert not torch.isfinite(H[:, N - 1]).any()
    assert torch.equal(H[:M - 1, :N - 1], clean[:M - 1, :N - 1])


# ------------------------------------------------------------ the gradient

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gradient_is_exact_on_whole_numbers(M, N, K, dtype):
    gen = gen_for(M, N, K, 7, len(dtype))
    for pad, offset, sums, keep, act in ((0, 0, True, False, "relu"), (8, 0, False, True, "identity"),
                                         (3, 1, True, True, "relu")):
        say("gated_grad", M, N, K, dtype, pad, offset, sums, keep, act)
        dY, Wd = ints(gen, M, K, top=1), ints(gen, K, N, top=1)
        G, U = ints(gen, M, N), ints(gen, M, N)
        dh = dY.double() @ Wd.double()
        a, s = gp.act(G.double(), act), gp.slope(G.double(), act)
        dG, g_ok = out_like(M, N, dtype, pad, offset)
        dU, u_ok = out_like(M, N, dtype, pad)
        H, h_ok = out_like(M, N, dtype, 0, offset) if keep else (None, None)
        sg, su = (torch.full((N,), 5.0, device="cuda") for _ in range(2)) if sums else (None, None)
        dgt.check(dgt.gated_grad(stored(dY, dtype, pad, offset), stored(Wd, dtype, pad, offset), stored(G, dtype, pad),
                                 stored(U, dtype, 0, offset), dG, dU, act=act, H=H, dbias_g=sg, dbias_u=su))
        assert torch.equal(dG.cpu(), (dh * U.double() * s).to(DT[dtype])) and g_ok()
        assert torch.equal(dU.cpu(), (dh * a).to(DT[dtype])) and u_ok()
        if keep:
            assert torch.equal(H.cpu(), (a * U.double()).to(DT[dtype])) and h_ok()
        if sums:  # whole numbers: the sums are exact in any order
            assert torch.equal(sg.cpu().double(), (dh * U.double() * s).sum(0))
            assert torch.equal(su.cpu().double(), (dh * a).sum(0))


@pytest.mark.parametrize("act", gp.ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gradient_against_the_formula_and_differences(dtype, act):
    """Against the formula within the roundings, and against central differences of the 64-bit block."""
    gen = gen_for(len(act), len(dtype), 3)
    t = DT[dtype]
    for M, N, K in ((3, 70, 264), (150, 140, 136), (40, 35, 55), (300, 264, 520)):
        dY = torch.randn(M, K, generator=gen).to(t)
        Wd = (torch.randn(K, N, generator=gen) / math.sqrt(K)).to(t)
        G, U = (2 * torch.randn(M, N, generator=gen)).to(t), torch.randn(M, N, generator=gen).to(t)
        dG, dU, H = (torch.empty(M, N, dtype=t, device="cuda") for _ in range(3))
        sg, su = (torch.empty(N, device="cuda") for _ in range(2))
        dgt.check(dgt.gated_grad(dY.cuda(), Wd.cuda(), G.cuda(), U.cuda(), dG, dU, act=act, H=H, dbias_g=sg,
                                 dbias_u=su))
        g, u = G.double(), U.double()
        dh, e = dY.double() @ Wd.double(), gp.sum_error(dY.double(), Wd.double())
        a, s = gp.act(g, act), gp.slope(g, act)
        # the slope's terms are below 2 + |g| in size
        es = gp.act_error(g, 2 + g.abs())
        eg = e * (u * s).abs() + (dh.abs() + e) * u.abs() * es + 4 * gp.U24 * (dh * u).abs() * (1 + s.abs())
        eu = e * a.abs() + (dh.abs() + e) * gp.act_error(g, a) + 4 * gp.U24 * (dh * a).abs()
        gp.assert_within(dG, dh * u * s, gp.half_step((dh * u * s).abs() + eg, t) + eg, f"{act} dG")
        gp.assert_within(dU, dh * a, gp.half_step((dh * a).abs() + eu, t) + eu, f"{act} dU")
        eh = gp.act_error(g, a) * u.abs() + 4 * gp.U24 * (a * u).abs()
        gp.assert_within(H, a * u, gp.half_step((a * u).abs() + eh, t) + eh, f"{act} H")
        for got, terms, et in ((sg, dh * u * s, eg), (su, dh * a, eu)):  # M additions more
            gp.assert_within(got, terms.sum(0), et.sum(0) + 2 * M * gp.U24 * terms.abs().sum(0), f"{act} sums")
        if act == "relu":
            continue  # a kink has no difference
        step = 1e-5
        for got, plus, minus in ((dG, gp.act(g + step, act) * u, gp.act(g - step, act) * u),
                                 (dU, a * (u + step), a * (u - step))):
            diff = dh * (plus - minus) / (2 * step)
            # the differences' own error: step^2/6 times third derivatives below 2, and cancellation
            tol = gp.half_step(diff.abs() + 1e-5, t) + eg + eu + dh.abs() * (1 + u.abs()) * 1e-9
            gp.assert_within(got, diff, tol, f"{act} differences")


def test_gradient_in_place():
    gen = gen_for(11)
    for M, N, K in ((70, 200, 136), (300, 257, 63), (520, 512, 128)):
        dY, Wd = torch.randn(M, K, generator=gen).half().cuda(), torch.randn(K, N, generator=gen).half().cuda()
        P = torch.randn(M, 2 * N, generator=gen).half().cuda()
        D = torch.empty_like(P)
        dgt.check(dgt.gated_grad(dY, Wd, P[:, :N], P[:, N:], D[:, :N], D[:, N:], act="gelu"))
        dgt.check(dgt.gated_grad(dY, Wd, P[:, :N], P[:, N:], P[:, :N], P[:, N:], act="gelu"))
        assert torch.equal(P, D)
        with pytest.raises(dgt.GemmError):
            dgt.check(dgt.gated_grad(dY, Wd, P[:, :N], P[:, N:], P[:, N:], D[:, :N]))


def test_sums_over_no_rows_are_zero():
    e = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
    sg, su = torch.full((40,), 3.0, device="cuda"), torch.full((40,), 3.0, device="cuda")
    dY, Wd = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda"), torch.ones(16, 40, dtype=torch.bfloat16, device="cuda")
    dgt.check(dgt.gated_grad(dY, Wd, e, e, e, e, dbias_g=sg, dbias_u=su))
    assert not sg.any() and not su.any()


@pytest.mark.parametrize("M,N,K", [(6, 96, 256), (200, 136, 264), (300, 520, 130)])
def test_calls_repeat_bit_for_bit_on_any_stream(M, N, K):
    gen = gen_for(M, N, K, 21)
    X, Wg, Wu = (torch.randn(r, K, generator=gen).bfloat16().cuda() for r in (M, N, N))
    Wd, dY = torch.randn(K, N, generator=gen).bfloat16().cuda(), torch.randn(M, K, generator=gen).bfloat16().cuda()
    runs = []
    torch.cuda.synchronize()
    for how in (None, torch.cuda.Stream(), torch.cuda.Stream().cuda_stream, 0):
        outs = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(6)]
        sums = [torch.empty(N, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        dgt.check(dgt.gated(X, Wg, Wu, outs[0], G=outs[1], U=outs[2], stream=how))
        dgt.check(dgt.gated_grad(dY, Wd, outs[1], outs[2], outs[3], outs[4], H=outs[5], dbias_g=sums[0],
                                 dbias_u=sums[1], stream=how))
        torch.cuda.synchronize()
        runs.append(outs + sums)
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


@pytest.mark.parametrize("M,N,K", [(6, 96, 256), (200, 136, 264)])
def test_captured_calls_replay(M, N, K):
    """Two graphs with workspaces of their own, replayed in turn with eager work between, on new inputs."""
    gen = gen_for(M, N, K, 31)
    t = torch.bfloat16

    def fresh():
        return dict(X=torch.randn(M, K, generator=gen).to(t).cuda(), dY=torch.randn(M, K, generator=gen).to(t).cuda())

    W = torch.randn(2 * N, K, generator=gen).to(t).cuda()
    Wd = torch.randn(K, N, generator=gen).to(t).cuda()
    need = dgt.gemm_gated_grad_workspace_size(M, N)

    def buffers():
        d = dict(H=torch.empty(M, N, dtype=t, device="cuda"), P=torch.empty(M, 2 * N, dtype=t, device="cuda"),
                 D=torch.empty(M, 2 * N, dtype=t, device="cuda"), s=torch.empty(2, N, device="cuda"),
                 ws=torch.empty(need, dtype=torch.uint8, device="cuda"))
        return d

    def work(i, b):
        P, D = b["P"], b["D"]
        dgt.check(dgt.gated(i["X"], W[:N], W[N:], b["H"], G=P[:, :N], U=P[:, N:]))
        dgt.check(dgt.gated_grad(i["dY"], Wd, P[:, :N], P[:, N:], D[:, :N], D[:, N:], dbias_g=b["s"][0],
                                 dbias_u=b["s"][1], workspace=b["ws"]))

    graphs = []
    for _ in range(2):
        i, b = fresh(), buffers()
        work(i, b)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            work(i, b)
        graphs.append((graph, i, b))
    for _ in range(3):
        for graph, i, b in graphs:
            new = fresh()
            for k in new:
                i[k].copy_(new[k])
            graph.replay()
            want = buffers()
            work(new, want)
            torch.cuda.synchronize()
            for k in ("H", "P", "D", "s"):
                assert torch.equal(b[k], want[k]), k


@pytest.mark.parametrize("dtype,act,M,D,F", [("bf16", "silu", 200, 136, 264), ("f16", "gelu", 33, 72, 104)])
def test_block_forward_and_backward(dtype, act, M, D, F):
    """A feed-forward block's training step with the library's calls: forward, second half, and every gradient,
    against 64-bit autograd of the block.  Intermediate 16-bit values (H, G, U, dG, dU, Y's gradient)
    are each rounded once, half a step; through a product of K terms those roundings
    add up like independent errors: normwise a few half steps."""
    gen = gen_for(M, D, F)
    t = DT[dtype]
    X = torch.randn(M, D, generator=gen).to(t)
    W = (torch.randn(2 * F, D, generator=gen) / math.sqrt(D)).to(t)
    Wd = (torch.randn(D, F, generator=gen) / math.sqrt(F)).to(t)
    b = torch.randn(2, F, generator=gen) * 0.5
    dY = torch.randn(M, D, generator=gen).to(t)

    leaves = [v.double().requires_grad_(True) for v in (X, W, Wd, b)]
    x, w, wd, bb = leaves
    g, u = x @ w[:F].T + bb[0], x @ w[F:].T + bb[1]
    f = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[act]
    y = (f(g) * u) @ wd.T
    want = torch.autograd.grad(y, leaves, dY.double())

    dev = dict(X=X.cuda(), W=W.cuda(), Wd=Wd.cuda(), b=b.cuda(), dY=dY.cuda())
    H = torch.empty(M, F, dtype=t, device="cuda")
    P, Dp = (torch.empty(M, 2 * F, dtype=t, device="cuda") for _ in range(2))
    Y, dX = (torch.empty(M, D, device="cuda") for _ in range(2))
    dW, dWd, db = torch.empty(2 * F, D, device="cuda"), torch.empty(D, F, device="cuda"), torch.empty(2, F, device="cuda")
    dgt.check(dgt.gated(dev["X"], dev["W"][:F], dev["W"][F:], H, act=act, bias_g=dev["b"][0], bias_u=dev["b"][1],
                        G=P[:, :F], U=P[:, F:]))
    dgt.check(dgt.gemm(H, dev["Wd"], Y, trans_b=True))
    H2 = torch.empty_like(H)
    dgt.check(dgt.gated_grad(dev["dY"], dev["Wd"], P[:, :F], P[:, F:], Dp[:, :F], Dp[:, F:], act=act, H=H2,
                             dbias_g=db[0], dbias_u=db[1]))
    dgt.check(dgt.gemm(Dp, dev["W"], dX))
    dgt.check(dgt.gemm(Dp, dev["X"], dW, trans_a=True))
    dgt.check(dgt.gemm(dev["dY"], H2, dWd, trans_a=True))
    # G and U feed dG and dU through factors of order one: four roundings at most on a path
    tol = 4 * torch.finfo(t).eps / 2
    for got, ref, name in ((Y, y.detach(), "Y"), (dX, want[0], "dX"), (dW, want[1], "dW"), (dWd, want[2], "dWd"),
                           (db, want[3], "db")):
        rel = ((got.double().cpu() - ref).norm() / ref.norm()).item()
        say(dtype, act, name, rel)
        assert rel <= tol, (name, rel)
