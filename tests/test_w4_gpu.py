"""4-bit weights with group scales on the GPU against the plain 64-bit forms: packing
and reading back bit for bit, products bit for bit where every sum is exactly
representable and within `gated_plain`'s bounds otherwise."""

import math

import numpy as np
import pytest
import torch

import dense_gemm_tuning_amd as dgt
import gated_plain as gp
from gpu_util import say

pytestmark = pytest.mark.gpu

DT = gp.DT


def rng_for(*key):
    return np.random.default_rng(list(map(int, key)))


def weights(rng, rows, K, dtype):
    """Values of very different groups, rounded to dtype: some rows all zero, positive or negative, ties of
    whole scales, groups far below and above 1."""
    x = rng.standard_normal((rows, K)) * 2.0 ** rng.integers(-12, 6, (rows, 1))
    x[rng.random((rows, K)) < 0.1] = 0.0
    ties = rng.random((rows, K)) < 0.1
    x[ties] = rng.integers(-15, 16, ties.sum()) * 0.5
    if rows > 4:
        x[1], x[2], x[3] = 0.0, np.abs(x[2]), -np.abs(x[3])
        x[4] = rng.integers(-7, 8, K) * 0.5  # scales that are whole numbers of halves: many ties
    return torch.from_numpy(x).to(DT[dtype])


def stored(t, pad):
    """A tensor as a view of a wider one."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), 0 if t.dtype is torch.uint8 else float("nan"), dtype=t.dtype)
    wide[:, :t.shape[1]] = t
    return wide.cuda()[:, :t.shape[1]]


PACK = [(1, 1), (1, 32), (3, 31), (5, 33), (2, 64), (7, 127), (6, 128), (9, 129), (5, 511), (6, 513), (33, 1029), (130, 256),
        (8, 4096)]


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,K", PACK)
def test_packing_matches_the_definition(rows, K, dtype, zeros):
    for group in (32, 64, 128):
        for st in ("bf16", "f16"):
            say("pack", rows, K, dtype, zeros, group, st)
            rng = rng_for(rows, K, len(dtype), zeros, group, len(st))
            x = weights(rng, rows, K, dtype)
            q, s, z = gp.quantize(x.double().numpy(), group, DT[st], zeros)
            n = gp.groups(K, group)
            Qw = torch.full((rows, 16 * (-(-K // 32)) + 16), 0xEE, dtype=torch.uint8, device="cuda")
            Sw = torch.full((rows, n + 3), 9.0, dtype=DT[st], device="cuda")
            Zw = torch.full((rows, n + 1), 99, dtype=torch.uint8, device="cuda")
            Q, S, Z = Qw[:, :-16], Sw[:, :n], Zw[:, :n] if zeros else None
            pad = rng.integers(0, 3)
            dgt.check(dgt.quantize_w4(stored(x, int(pad)), Q, S, Z, group=group))
            assert torch.equal(S.cpu(), s) and (Sw[:, n:] == 9.0).all()
            assert torch.equal(Q.cpu(), gp.pack(q)) and (Qw[:, -16:] == 0xEE).all()
            assert (Zw[:, n:] == 99).all()
            if zeros:
                assert np.array_equal(Z.cpu().numpy(), z)
            else:
                assert (Zw == 99).all()
            want = gp.values(q, s, z, group)
            for out in ("f32", "bf16", "f16"):
                Yw = torch.full((rows, K + 2), 5.0, dtype=DT[out], device="cuda")
                dgt.check(dgt.dequantize_w4(Q, S, Z, Yw[:, :K], group=group))
                assert torch.equal(Yw[:, :K].cpu(), torch.from_numpy(want).float().to(DT[out]))
                assert (Yw[:, K:] == 5.0).all()


@pytest.mark.parametrize("st,m", [("f16", 1 + 2.0 ** -11), ("bf16", 1 + 2.0 ** -8)])
def test_scales_are_rounded_twice(st, m):
    """(15 m + 2^-24)/15 lies above m, half way between two scales, by less than fp32 shows: fp32's
    rounding gives m and the tie the even side, 1; a single rounding would go up."""
    x = torch.zeros(3, 32)
    x[0, 3], x[0, 30] = 15 * m, -2.0 ** -24
    x[1] = 2 * x[0]
    Q, S, Z = dgt.w4_empty(3, 32, group=32, scale_dtype=DT[st])
    dgt.check(dgt.quantize_w4(x.cuda(), Q, S, Z, group=32))
    q, s, z = gp.quantize(x.double().numpy(), 32, DT[st], True)
    assert s[:, 0].tolist() == [1.0, 2.0, 0.0] and torch.equal(S.cpu(), s)
    assert torch.equal(Q.cpu(), gp.pack(q)) and np.array_equal(Z.cpu().numpy(), z)


@pytest.mark.parametrize("st", ["bf16", "f16"])
@pytest.mark.parametrize("zeros", [True, False])
def test_unusual_groups(zeros, st):
    """Infinities and NaN stay in their group; scales past the type's largest value, and ones that vanish."""
    x = np.zeros((7, 96))
    x[0, 40] = np.inf
    x[1, 3] = np.nan
    x[2, 90] = -np.inf
    x[3] = np.linspace(-3e38, 3e38, 96)
    x[4] = np.linspace(-1e-44, 1.4e-44, 96)
    x[5] = np.linspace(2e-8, 4e-7, 96)  # FP16's subnormal scales
    x[6] = np.linspace(1e-40, 9e-39, 96)  # BF16's
    x[0, 64:] = x[1, 32:64] = 1.5
    t = torch.from_numpy(x).float()
    q, s, z = gp.quantize(t.double().numpy(), 32, DT[st], zeros)
    Q, S, Z = dgt.w4_empty(7, 96, group=32, scale_dtype=DT[st], zeros=zeros)
    dgt.check(dgt.quantize_w4(t.cuda(), Q, S, Z, group=32))
    assert torch.equal(torch.isnan(S.cpu()), torch.isnan(s))
    assert torch.equal(torch.nan_to_num(S.cpu(), 0), torch.nan_to_num(s, 0))
    assert torch.equal(Q.cpu(), gp.pack(q))
    if zeros:
        assert np.array_equal(Z.cpu().numpy(), z)
    Y = torch.empty(7, 96, device="cuda")
    dgt.check(dgt.dequantize_w4(Q, S, Z, Y, group=32))
    want = torch.from_numpy(gp.values(q, s, z, 32)).float()
    assert torch.equal(torch.isnan(Y.cpu()), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(Y.cpu(), 0), torch.nan_to_num(want, 0))


def whole_weight(rng, rows, K, group, st, zeros):
    """A weight whose products with whole numbers are whole multiples of 1/2, codes past K not zero."""
    n = gp.groups(K, group)
    q = rng.integers(0, 16, (rows, K)).astype(np.uint8)
    s = torch.from_numpy(rng.choice([0.5, 1.0, 2.0, -1.0], (rows, n))).to(DT[st])
    z = rng.integers(0, 16, (rows, n)).astype(np.uint8) if zeros else np.full((rows, n), 8, np.uint8)
    if zeros and rows > 2:
        z[rows // 2] = 255  # a byte, not only a code's range
    return q, s, z


def on_gpu(q, s, z, zeros, pad):
    return stored(gp.pack(q, fill=11), 16 * pad), stored(s, pad), stored(torch.from_numpy(z), pad) if zeros else None


# rows, outputs and depths where strips, blocks, steps and groups end
PRODUCTS = [(1, 1, 1), (1, 16, 32), (1, 17, 31), (2, 15, 33), (3, 64, 128), (4, 100, 127), (5, 33, 129), (8, 130, 256),
            (15, 48, 511), (16, 112, 512), (17, 65, 513), (31, 200, 1000), (32, 16, 1024), (33, 129, 520), (1, 272, 4096),
            (8, 113, 4104), (48, 96, 640), (64, 128, 257), (65, 40, 264), (130, 70, 96), (1, 4100, 64), (20, 4112, 160),
            (1, 9000, 32), (2, 31, 9000)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product_is_exact_on_whole_numbers(M, N, K, dtype):
    rng = rng_for(M, N, K, len(dtype))
    for group, st, zeros, pad, alpha, beta, bias in ((128, "f16", True, 0, 1.0, 0.0, False),
                                                     (64, "bf16", False, 1, 1.5, 0.5, True),
                                                     (32, dtype, True, 3, -1.0, 1.0, False),
                                                     (128, "bf16", False, 8, 2.0, 0.0, True)):
        say("gemm_w4", M, N, K, dtype, group, st, zeros, pad)
        q, s, z = whole_weight(rng, N, K, group, st, zeros)
        X = torch.from_numpy(rng.integers(-2, 3, (M, K)).astype(np.float32)).to(DT[dtype])
        C0 = torch.from_numpy(rng.integers(-8, 9, (M, N)).astype(np.float32))
        b = torch.from_numpy(rng.integers(-8, 9, N).astype(np.float32)) if bias else None
        want = alpha * (X.double() @ torch.from_numpy(gp.values(q, s, z, group).T.copy()))
        want = want + beta * C0.double() if beta else want
        want = want + b.double() if bias else want
        wide = torch.full((M, N + pad), float("nan"), device="cuda")
        if beta:
            wide[:, :N] = C0.cuda()
        dgt.check(dgt.gemm_w4(stored(X, pad), *on_gpu(q, s, z, zeros, pad), wide[:, :N], group=group, alpha=alpha,
                              beta=beta, bias=None if b is None else b.cuda()))
        assert torch.equal(wide[:, :N].cpu().double(), want)
        assert torch.isnan(wide[:, N:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_gated_is_exact_on_whole_numbers(M, N, K, dtype):
    """g and u are whole multiples of 1/2 (of 1/4 their product, below 2^24): H is act(g)*u rounded once."""
    rng = rng_for(M, N, K, 9, len(dtype))
    for group, st, zeros, pad, act, bias in ((128, "f16", True, 0, "identity", False), (64, "bf16", False, 1, "relu", True),
                                             (32, dtype, True, 3, "relu", False)):
        say("gated_w4", M, N, K, dtype, group, st, zeros, pad)
        q, s, z = whole_weight(rng, 2 * N, K, group, st, False)
        s = s.abs().clamp(max=1)
        if zeros:
            z = rng.integers(6, 10, z.shape).astype(np.uint8)
        X = torch.from_numpy((rng.random((M, K)) < min(1.0, 64 / K)) * rng.integers(-1, 2, (M, K)).astype(np.float32))
        X = X.to(DT[dtype])
        bg, bu = (torch.from_numpy(rng.integers(-8, 9, N).astype(np.float32)) for _ in range(2)) if bias else (None, None)
        p = X.double() @ torch.from_numpy(gp.values(q, s, z, group).T.copy())
        g, u = p[:, :N] + (bg.double() if bias else 0), p[:, N:] + (bu.double() if bias else 0)
        want = gp.act(g, act) * u
        assert want.abs().max() < 2 ** 22
        wide = torch.full((M, N + pad), 77.0, dtype=DT[dtype], device="cuda")
        dgt.check(dgt.gated_w4(stored(X, pad), *on_gpu(q, s, z, zeros, pad), wide[:, :N], act=act, group=group,
                               bias_g=None if bg is None else bg.cuda(), bias_u=None if bu is None else bu.cuda()))
        assert torch.equal(wide[:, :N].cpu(), want.to(DT[dtype]))
        assert (wide[:, N:] == 77.0).all()


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K,group", [(1, 300, 2048, 128), (7, 130, 1000, 64), (33, 200, 777, 32), (64, 96, 4096, 128),
                                         (130, 64, 264, 64)])
def test_real_values_are_within_the_sums_bounds(M, N, K, group, dtype, zeros):
    rng = rng_for(M, N, K, group, zeros)
    x = torch.from_numpy(rng.standard_normal((M, K)) * np.exp(0.8 * rng.standard_normal((1, K)))).to(DT[dtype])
    w = rng.standard_normal((2 * N, K)) / math.sqrt(K)
    q, s, z = gp.quantize(w, group, DT[dtype], zeros)
    W = on_gpu(q, s, z, zeros, 0)
    p = x.double() @ torch.from_numpy(gp.values(q, s, z, group).T.copy())
    e = gp.product_error(x, q, s, z, group)
    C = torch.empty(M, 2 * N, device="cuda")
    dgt.check(dgt.gemm_w4(x.cuda(), *W, C, group=group))
    gp.assert_within(C, p, e, "product")
    for act in ("silu", "gelu"):
        H = torch.empty(M, N, dtype=DT[dtype], device="cuda")
        dgt.check(dgt.gated_w4(x.cuda(), *W, H, act=act, group=group))
        g, u = p[:, :N], p[:, N:]
        a = gp.act(g, act)
        eh = 1.13 * e[:, :N] * (u.abs() + e[:, N:]) + a.abs() * e[:, N:] + gp.act_error(g, a) * u.abs() + \
            4 * gp.U24 * (a * u).abs()
        gp.assert_within(H, a * u, gp.half_step((a * u).abs() + eh, DT[dtype]) + eh, act)


@pytest.mark.parametrize("M,N,K", [(1, 40, 300), (33, 130, 512)])
def test_edge_calls(M, N, K):
    rng = rng_for(M, N, K, 77)
    q, s, z = whole_weight(rng, N, K, 64, "f16", True)
    Q, S, Z = on_gpu(q, s, z, True, 0)
    X = torch.ones(M, K, dtype=torch.float16, device="cuda")
    # alpha = 0: the operands are not read (a NaN scale would show), C <- beta*C + bias
    C, b = torch.full((M, N), 4.0, device="cuda"), torch.arange(N, dtype=torch.float32, device="cuda")
    dgt.check(dgt.gemm_w4(X, Q, S * float("nan"), Z, C, group=64, alpha=0.0, beta=0.5, bias=b))
    assert torch.equal(C, (2.0 + b).expand(M, N))
    none = [t[:, :0] for t in (Q, S, Z)]
    dgt.check(dgt.gemm_w4(X[:, :0], *none, C, group=64, bias=b))
    assert torch.equal(C, b.expand(M, N))
    H = torch.full((M, N // 2), 9.0, dtype=torch.float16, device="cuda")
    dgt.check(dgt.gated_w4(X[:, :0], *none, H, group=64, act="relu", bias_g=b[:N // 2], bias_u=b[:N // 2] * 0 + 2))
    assert torch.equal(H.float(), (2 * b[:N // 2]).expand(M, N // 2))
    # a NaN scale stays in its output, a NaN activation in its row, whatever lies past K in the rows
    S2 = S.clone()
    S2[N - 1, -1] = float("nan")
    X2 = X.clone()
    X2[M - 1, K - 1] = float("inf")
    want, C = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    dgt.check(dgt.gemm_w4(X, Q, S, Z, want, group=64))
    dgt.check(dgt.gemm_w4(X2, Q, S2, Z, C, group=64))
    assert torch.isnan(C[:, N - 1]).all() and torch.equal(C[:M - 1, :N - 1], want[:M - 1, :N - 1])
    assert not torch.isfinite(C[M - 1][(q[:, K - 1] != z[:, -1])]).any()
    wide = torch.full((M, K + 9), float("nan"), dtype=torch.float16, device="cuda")
    wide[:, :K] = X
    dgt.check(dgt.gemm_w4(wide[:, :K], Q, S, Z, C, group=64))
    assert torch.equal(C, want)


def test_streams_and_graphs():
    rng = rng_for(3)
    M, N, K = 5, 176, 1000
    q, s, z = gp.quantize(rng.standard_normal((2 * N, K)), 128, torch.bfloat16, True)
    W = on_gpu(q, s, z, True, 0)
    xs = [torch.from_numpy(rng.standard_normal((M, K))).bfloat16().cuda() for _ in range(4)]

    def work(x, C, H, stream=None):
        dgt.check(dgt.gemm_w4(x, *W, C, stream=stream))
        dgt.check(dgt.gated_w4(x, *W, H, stream=stream))

    def outs():
        return torch.empty(M, 2 * N, device="cuda"), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")

    want = []
    for x in xs:
        want.append(outs())
        work(x, *want[-1])
    torch.cuda.synchronize()
    for how in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream, 0):
        got = outs()
        torch.cuda.synchronize()
        work(xs[0], *got, stream=how)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    held = xs[0].clone()
    got = outs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work(held, *got)
    for x, w in list(zip(xs, want)) * 2:
        held.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, w))
        work(x, *outs())


def test_train_then_serve():
    """A block's weights as trained, packed into one operand and served for single tokens: against the 16-bit
    block on the values read back (their rounding to FP16 is half a step of each weight)."""
    gen = torch.Generator().manual_seed(4)
    D, F = 264, 136
    W = torch.randn(2 * F, D, generator=gen).cuda() / math.sqrt(D)
    Wd = torch.randn(D, F, generator=gen).cuda() / math.sqrt(F)
    Q, S, Z = dgt.w4_empty(2 * F, D, group=64)
    Qd, Sd, Zd = dgt.w4_empty(D, F, group=64)
    dgt.check(dgt.quantize_w4(W, Q, S, Z, group=64))
    dgt.check(dgt.quantize_w4(Wd, Qd, Sd, Zd, group=64))
    back, backd = torch.empty(2 * F, D, dtype=torch.float16, device="cuda"), torch.empty(D, F, dtype=torch.float16, device="cuda")
    dgt.check(dgt.dequantize_w4(Q, S, Z, back, group=64))
    dgt.check(dgt.dequantize_w4(Qd, Sd, Zd, backd, group=64))
    # 15 steps span at least the range: half a step off where nothing is cut
    step = S.float().repeat_interleave(64, 1)[:, :D]
    assert ((back.float() - W).abs() <= 0.51 * step + 2 ** -11 * W.abs()).float().mean() > 0.99
    for M in (1, 6):
        X = torch.randn(M, D, generator=gen).half().cuda()
        H, H16 = (torch.empty(M, F, dtype=torch.float16, device="cuda") for _ in range(2))
        Y, Y16 = (torch.empty(M, D, device="cuda") for _ in range(2))
        dgt.check(dgt.gated_w4(X, Q, S, Z, H, group=64))
        dgt.check(dgt.gemm_w4(H, Qd, Sd, Zd, Y, group=64))
        dgt.check(dgt.gated(X, back[:F], back[F:], H16))
        dgt.check(dgt.gemm(H16, backd, Y16, trans_b=True))
        assert ((Y - Y16).norm() / Y16.norm()).item() <= 4 * 2 ** -11
