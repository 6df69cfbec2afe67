"""The gated and 4-bit operators where offsets pass 32 bits: results of more than 2^31 elements, weights of more than
2^32 bytes, rows far apart, many rows of activations.  Whole numbers make the results exact; they are compared whole,
some rows at a time."""

import pytest
import torch

import dense_gemm_tuning_amd as dgt
from gpu_util import say
from test_gated_gpu import stored
from test_strips_deep_gpu import packed, whole

pytestmark = pytest.mark.gpu

BF, F16 = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def memory():
    free, _ = torch.cuda.mem_get_info()
    if free < 60 << 30:
        pytest.skip("needs 60 GB of GPU memory")
    yield
    torch.cuda.empty_cache()


def seeded(n):
    return torch.Generator(device="cuda").manual_seed(n)


def rows_of(M, step=4096):
    return [slice(r, min(r + step, M)) for r in range(0, M, step)]


# 16-byte rows and DMA tiles; rows off those boundaries and register-staged tiles
@pytest.mark.parametrize("K", [64, 9])
def test_gated_and_gradient_of_more_than_2_to_31_elements(K):
    M, N = 70001, 32768
    gen = seeded(K)
    say("gated", M, N, K)
    X, W = whole(gen, M, K).to(BF), whole(gen, 2 * N, K).to(BF)
    H, G, U = (torch.empty(M, N, dtype=BF, device="cuda") for _ in range(3))
    dgt.check(dgt.gated(X, W[:N], W[N:], H, act="relu", G=G, U=U))
    for r in rows_of(M):
        g, u = (X[r].float() @ W.float().t()).split(N, dim=1)
        assert torch.equal(G[r], g.to(BF)) and torch.equal(U[r], u.to(BF)), r
        assert torch.equal(H[r], (g.clamp(min=0) * u).to(BF)), r
    say("gated_grad", M, N, K)
    dY, Wd = whole(gen, M, K).to(BF), whole(gen, K, N + 8 * (K % 8 != 0)).to(BF)[:, :N]
    want = []
    for r in rows_of(M):
        dh, g, u = dY[r].float() @ Wd.float(), G[r].float(), U[r].float()
        want.append(torch.stack([(dh * u * (g > 0)).double().sum(0), (dh * g.clamp(min=0)).double().sum(0)]))
    want = torch.stack(want).sum(0)
    keep = [(r, G[r].clone(), U[r].clone()) for r in (slice(0, 300), slice(M - 300, M))]
    sums = torch.empty(2, N, device="cuda")
    dgt.check(dgt.gated_grad(dY, Wd, G, U, G, U, act="relu", dbias_g=sums[0], dbias_u=sums[1]))  # in place
    for r, g, u in keep:
        dh, g, u = dY[r].float() @ Wd.float(), g.float(), u.float()
        assert torch.equal(G[r], (dh * u * (g > 0)).to(BF)) and torch.equal(U[r], (dh * g.clamp(min=0)).to(BF)), r
    assert want.abs().max() < 2 ** 23  # exact in any order
    assert torch.equal(sums.double(), want)


@pytest.mark.parametrize("M", [3, 20, 64])
def test_gated_strips_over_weights_of_more_than_2_to_32_bytes(M):
    N, K = 270000, 8192
    gen = seeded(M)
    say("gated", M, N, K)
    W = torch.randint(-1, 2, (2 * N, K), generator=gen, device="cuda", dtype=torch.int8).to(F16)
    X = whole(gen, M, K).half()
    H = torch.empty(M, N, dtype=F16, device="cuda")
    dgt.check(dgt.gated(X, W[:N], W[N:], H, act="identity"))
    for c in rows_of(N, 16384):
        g, u = X.float() @ W[:N][c].float().t(), X.float() @ W[N:][c].float().t()
        assert torch.equal(H[:, c], (g * u).half()), c


@pytest.mark.parametrize("M", [5, 40, 300])
def test_gated_rows_far_apart(M):
    """Weights and activations at the widest pitch that the faster kernels take, and one past it."""
    N, K = 130, 264
    gen = seeded(M + 1)
    want = None
    for pitch in ((1 << 24) - 8, 1 << 24):
        say("gated, pitch", M, N, K, pitch)
        wide = [torch.empty(rows * pitch, dtype=BF, device="cuda").view(rows, pitch)[:, :K] for rows in (2 * N, min(M, 40))]
        if want is None:
            X, W = whole(gen, M, K), whole(gen, 2 * N, K)
            want = ((X @ W[:N].t()) * (X @ W[N:].t())).to(BF)
        wide[0].copy_(W)
        Xw = X.to(BF)
        if M <= 40:
            wide[1].copy_(X)
            Xw = wide[1]
        H = torch.empty(M, N, dtype=BF, device="cuda")
        dgt.check(dgt.gated(Xw, wide[0][:N], wide[0][N:], H, act="identity"))
        assert torch.equal(H, want)
        del wide, Xw
        torch.cuda.empty_cache()


@pytest.mark.parametrize("M", [2, 40, 130])
def test_w4_weights_of_more_than_2_to_32_bytes(M):
    N, K = 1100000, 8000
    gen = seeded(M + 2)
    n = -(-K // 128)
    say("gemm_w4", M, N, K)
    Q = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    S = torch.ones(N, n, dtype=F16, device="cuda")
    Z = torch.randint(0, 16, (N, n), generator=gen, device="cuda", dtype=torch.uint8)
    X = whole(gen, M, K)
    C = torch.full((M, N), float("nan"), device="cuda")
    H = torch.full((M, N // 2), float("nan"), dtype=BF, device="cuda")
    dgt.check(dgt.gemm_w4(X.half(), Q, S, Z, C))
    dgt.check(dgt.gated_w4(X.to(BF), Q, S, Z, H, act="relu"))
    for c in rows_of(N, 16384):
        q = torch.stack((Q[c] & 15, Q[c] >> 4), dim=2).flatten(1).float()
        w = q - Z[c].float().repeat_interleave(128, 1)[:, :K]
        assert torch.equal(C[:, c], X @ w.t()), c
    # the sums above are exact: |g|, |u| < 2^24, and their product is rounded twice, in fp32 and then to BF16
    want = (C[:, :N // 2].clamp(min=0) * C[:, N // 2:]).to(BF)
    assert torch.equal(H, want)


@pytest.mark.parametrize("M", [3, 40])
def test_w4_rows_far_apart(M):
    """Codes at the widest pitch there is, scales and zero points millions apart."""
    N, K, group = 264, 520, 64
    gen = seeded(M + 3)
    say("gemm_w4, wide pitches", M, N, K)
    (Q, S, Z), w = packed(gen, N, K, group, "bf16", True, 8)
    far = []
    for t, pitch in ((Q, dgt.MX4_MAX_PITCH), (S, 8500001), (Z, 8500001)):
        v = torch.empty(N * pitch, dtype=t.dtype, device="cuda").view(N, pitch)[:, :t.shape[1]]
        v.copy_(t)
        far.append(v)
    X = whole(gen, M, K)
    C = torch.empty(M, N, device="cuda")
    dgt.check(dgt.gemm_w4(X.to(BF), *far, C, group=group))
    assert torch.equal(C, X @ w.t())
    H = torch.empty(M, N // 2, dtype=BF, device="cuda")
    dgt.check(dgt.gated_w4(X.to(BF), *far, H, act="relu", group=group))
    assert torch.equal(H, (C[:, :N // 2].clamp(min=0) * C[:, N // 2:]).to(BF))
    Y, back = torch.empty(N, K, device="cuda"), torch.empty(N, K, device="cuda")
    dgt.check(dgt.dequantize_w4(*far, Y, group=group))
    assert torch.equal(Y, w)
    dgt.check(dgt.quantize_w4(w, *far, group=group))
    near = [torch.empty_like(t) for t in (Q, S, Z)]
    dgt.check(dgt.quantize_w4(w, *near, group=group))
    for a, b in zip(far, near):
        assert torch.equal(a, b)
    dgt.check(dgt.dequantize_w4(*near, back, group=group))
    dgt.check(dgt.dequantize_w4(*far, Y, group=group))
    assert torch.equal(Y, back)


@pytest.mark.parametrize("pad", [0, 1])
def test_w4_results_of_more_than_2_to_31_elements(pad):
    M, N, K, group = 66000, 33000, 40, 32
    gen = seeded(pad)
    say("gated_w4", M, N, K, pad)
    W, w = packed(gen, 2 * N, K, group, "f16", True, 1)
    X = whole(gen, M, K)
    H = torch.empty(M, N, dtype=F16, device="cuda")
    dgt.check(dgt.gated_w4(stored(X, "f16", pad, pad), *W, H, act="identity", group=group))
    for r in rows_of(M):
        g, u = (X[r] @ w.t()).split(N, dim=1)
        assert torch.equal(H[r], (g * u).half()), r
    C = torch.empty(M, N, device="cuda")
    dgt.check(dgt.gemm_w4(stored(X, "f16", pad, pad), *(t[N:] for t in W), C, group=group))
    for r in rows_of(M):
        assert torch.equal(C[r], X[r] @ w[N:].t()), r


def test_packing_more_than_2_to_31_elements():
    M, K = 66000, 33000
    say("quantize_w4", M, K)
    gen = seeded(9)
    X = torch.empty(M, K, dtype=BF, device="cuda")
    for r in rows_of(M):
        X[r] = torch.randn(X[r].shape, generator=gen, device="cuda").to(BF)
    Q, S, Z = dgt.w4_empty(M, K)
    Y = torch.full((M, K), float("nan"), dtype=BF, device="cuda")
    dgt.check(dgt.quantize_w4(X, Q, S, Z))
    dgt.check(dgt.dequantize_w4(Q, S, Z, Y))
    # the same rows packed by themselves; every element within half a scale and its zero point's
    for r in (slice(0, 100), slice(M // 2, M // 2 + 100), slice(M - 100, M)):
        q, s, z = dgt.w4_empty(100, K)
        y = torch.empty(100, K, dtype=BF, device="cuda")
        dgt.check(dgt.quantize_w4(X[r].clone(), q, s, z))
        dgt.check(dgt.dequantize_w4(q, s, z, y))
        assert torch.equal(q, Q[r]) and torch.equal(s, S[r]) and torch.equal(z, Z[r]) and torch.equal(y, Y[r])
    for r in rows_of(M):
        step = S[r].float().repeat_interleave(128, 1)[:, :K]
        assert ((Y[r].float() - X[r].float()).abs() <= 1.01 * step + 2.0 ** -8 * X[r].float().abs()).all(), r


def test_no_k_and_many_rows():
    """Without weights there is a bias per column, whatever the number of rows."""
    M, N = (1 << 22) + 5, 100
    say("gated_w4 without k", M, N)
    none = [torch.empty(2 * N, 0, dtype=t, device="cuda") for t in (torch.uint8, F16, torch.uint8)]
    X = torch.empty(M, 0, dtype=F16, device="cuda")
    b = torch.arange(N, dtype=torch.float32, device="cuda")
    for dtype in (F16, BF):
        H = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
        dgt.check(dgt.gated_w4(X.to(dtype), *none, H, act="relu", group=64, bias_g=b, bias_u=b * 0 + 2))
        assert torch.equal(H, (2 * b).to(dtype).expand(M, N))
