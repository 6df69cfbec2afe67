"""MX4 operators on the GPU against the plain 64-bit model: quantising and
reading back (bit-exact), products (bit-exact where every partial sum is
exactly representable, else within the fp32 summation bound), strides,
unusual scales, streams and graph capture."""

import numpy as np
import pytest
import torch

import dense_gemm_tuning_amd as dgt
import mx4_plain as mp
from gpu_util import say

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def rng_for(*key):
    return np.random.default_rng(list(map(int, key)))


def activations(rng, M, K, dtype):
    """Values of very different blocks: normal times a block scale of 2^-20 ..
    2^9, some exact ties, zero blocks, negative zeros; rounded to dtype."""
    x = rng.standard_normal((M, K)) * 2.0 ** rng.integers(-12, 10, (M, 1)) * 2.0 ** rng.integers(-8, 1, (1, K))
    x[rng.random((M, K)) < 0.1] = 0.0
    x[rng.random((M, K)) < 0.05] *= -0.0
    ties = rng.random((M, K)) < 0.1
    x[ties] = rng.integers(-20, 21, ties.sum()) * 0.25
    if M > 3:
        x[1] = 0.0
    return torch.from_numpy(x).to(DT[dtype])


def packed(x):
    """Stored operand of float64 values on the GPU, through the plain model."""
    q, s = mp.quantize(x)
    S = np.full((x.shape[0], mp.scale_pitch(x.shape[1])), 255, np.uint8)  # pad bytes are never used
    S[:, :s.shape[1]] = s
    return torch.from_numpy(q).cuda(), torch.from_numpy(S).cuda(), mp.values(q, s, x.shape[1])


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 32), (3, 31), (5, 33), (2, 512), (7, 513), (64, 100),
                                 (33, 1029), (130, 257), (8, 4096)])
def test_quantize_matches_the_definition(M, K, dtype, trans):
    say("quantize", M, K, dtype, trans)
    rng = rng_for(M, K, len(dtype), trans)
    x = activations(rng, M, K, dtype)
    want_q, want_s = mp.quantize(x.double().numpy())
    Q, S = dgt.mx4_empty(M, K)
    Q.fill_(0xEE), S.fill_(0xEE)
    src = x.t().contiguous() if trans else x
    dgt.check(dgt.quantize_mx4(src.cuda(), Q, S, trans=trans))
    assert np.array_equal(S.cpu().numpy()[:, :want_s.shape[1]], want_s)
    assert (S.cpu().numpy()[:, want_s.shape[1]:] == 127).all()
    got = Q.cpu().numpy()
    assert np.array_equal(got & 0x77, want_q & 0x77)   # magnitudes
    nz = [(want_q & 0x07) != 0, (want_q & 0x70) != 0]  # signs of what is not zero
    assert np.array_equal((got & 0x08)[nz[0]], (want_q & 0x08)[nz[0]])
    assert np.array_equal((got & 0x80)[nz[1]], (want_q & 0x80)[nz[1]])
    for out in ("f32", "bf16"):
        Y = torch.full((M, K), float("nan"), dtype=DT[out], device="cuda")
        dgt.check(dgt.dequantize_mx4(Q, S, Y))
        assert np.array_equal(Y.double().cpu().numpy(), mp.values(want_q, want_s, K))


def test_quantize_extremes():
    """Subnormals, the largest values, NaN and infinities, per input type."""
    for dtype in ("f32", "bf16", "f16"):
        t = DT[dtype]
        big, tiny = torch.finfo(t).max, torch.finfo(t).smallest_normal
        x = torch.zeros(8, 64, dtype=torch.float64)
        x[0, :3] = torch.tensor([big, -big, big / 2])
        x[1, :3] = torch.tensor([tiny, tiny / 2, -tiny / 4])
        x[2, 5] = float("nan")
        x[3, 40] = float("-inf")
        x[4, :] = tiny * 3
        x[5, 63] = -0.0
        x[6, 31] = 7.99
        x = x.to(t)
        want_q, want_s = mp.quantize(x.double().numpy())
        Q, S = dgt.mx4_empty(8, 64)
        dgt.check(dgt.quantize_mx4(x.cuda(), Q, S))
        assert np.array_equal(S.cpu().numpy()[:, :2], want_s), dtype
        assert list(want_s[2]) [0] == 255 and want_s[3, 1] == 255
        Y = torch.empty(8, 64, device="cuda")
        dgt.check(dgt.dequantize_mx4(Q, S, Y))
        ref = mp.values(want_q, want_s, 64)
        np.testing.assert_array_equal(Y.double().cpu().numpy(), ref)


def test_dequantize_every_code_and_scale():
    """All 16 codes under all 256 scales; fp16 rounded to nearest even."""
    codes = np.arange(16, dtype=np.uint8).repeat(2)
    row = (codes[0::2] | (codes[1::2] << 4)).astype(np.uint8)
    Q = torch.from_numpy(np.tile(row, (256, 1))).cuda()
    S = torch.zeros(256, 16, dtype=torch.uint8)
    S[:, 0] = torch.arange(256, dtype=torch.uint8)
    S = S.cuda()
    ref = mp.values(Q.cpu().numpy(), S.cpu().numpy(), 32)
    for dtype, t in DT.items():
        Y = torch.empty(256, 32, dtype=t, device="cuda")
        dgt.check(dgt.dequantize_mx4(Q, S, Y))
        want = torch.from_numpy(ref).to(t)
        np.testing.assert_array_equal(Y.double().cpu().numpy(), want.double().numpy(), err_msg=dtype)


@pytest.mark.parametrize("trans", [False, True])
def test_quantize_strided_storage(trans):
    """Padded and misaligned input rows, padded code and scale rows with guard
    bytes that must survive; read back into a padded misaligned output."""
    M, K = 37, 75
    rng = rng_for(3, trans)
    rows, cols = (K, M) if trans else (M, K)
    for dtype, off, pitch in (("bf16", 1, cols + 3), ("f32", 3, cols + 1), ("f16", 8, cols + 5)):
        flat = torch.full((rows * pitch + off,), float("nan"), dtype=DT[dtype], device="cuda")
        X = flat[off:].as_strided((rows, cols), (pitch, 1))
        x = activations(rng, M, K, dtype)
        X.copy_((x.t() if trans else x).cuda())
        qp, sp = mp.code_pitch(K) + 32, mp.scale_pitch(K) + 16
        Qf = torch.full((M + 2, qp), 0xAB, dtype=torch.uint8, device="cuda")
        Sf = torch.full((M + 2, sp), 0xCD, dtype=torch.uint8, device="cuda")
        dgt.check(dgt.quantize_mx4(X, Qf[1:-1], Sf[1:-1], trans=trans))
        want_q, want_s = mp.quantize(x.double().numpy())
        ref = mp.values(want_q, want_s, K)
        yp = K + 7
        Yf = torch.full((M * yp + 1,), -777.0, device="cuda")
        Y = Yf[1:].as_strided((M, K), (yp, 1))
        dgt.check(dgt.dequantize_mx4(Qf[1:-1], Sf[1:-1], Y))
        np.testing.assert_array_equal(Y.double().cpu().numpy(), ref)
        Qc, Sc, Yc = Qf.cpu(), Sf.cpu(), Yf.cpu()
        assert (Qc[0] == 0xAB).all() and (Qc[-1] == 0xAB).all()
        assert (Qc[:, mp.code_pitch(K):] == 0xAB).all()
        assert (Sc[0] == 0xCD).all() and (Sc[-1] == 0xCD).all()
        assert (Sc[:, mp.scale_pitch(K):] == 0xCD).all()
        guard = torch.ones(M * yp + 1, dtype=torch.bool)
        guard[1:].as_strided((M, K), (yp, 1)).fill_(False)
        assert (Yc[guard] == -777.0).all()


SHAPES = [(1, 1, 1), (1, 64, 32), (2, 3, 33), (8, 40, 128), (16, 128, 512), (17, 130, 545), (33, 70, 1024),
          (48, 257, 96), (64, 100, 1000), (64, 300, 2080), (65, 129, 96), (100, 300, 31), (128, 128, 128),
          (130, 257, 640), (256, 256, 512), (300, 520, 1100), (513, 384, 2048), (1030, 770, 288)]


def int_operand(rng, rows, K):
    """Codes of any kind with scales 2^-1 .. 2^2: multiples of 1/4 up to 24."""
    q = rng.integers(0, 256, (rows, mp.code_pitch(K)), dtype=np.uint8)
    flat = np.stack([q & 15, q >> 4], -1).reshape(rows, -1)
    flat[:, K:] = 0
    q = (flat[:, 0::2] | (flat[:, 1::2] << 4)).astype(np.uint8)
    s = np.full((rows, mp.scale_pitch(K)), 255, np.uint8)
    nb = -(-K // 32)
    s[:, :nb] = rng.integers(126, 130, (rows, nb))
    return torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), mp.values(q, s, K)


def small_ints(rng, rows, K):
    return rng.integers(-3, 4, (rows, K)).astype(np.float64)


# Weights of enough columns for strips of 64 and 128 on every compute unit, a
# last strip of one column, K tails of one element, one block and many steps.
WIDE = [(1, 14337, 33), (8, 16400, 160), (16, 28673, 97), (20, 9000, 544), (32, 16500, 300), (40, 17000, 1056),
        (64, 33000, 130), (100, 9000, 320)]

# Few outputs and a long K on small workgroups (16 x 16, 16 x 32, 16 x 64 and
# 32 x 32 outputs), one round of 64 x 64 ones, and tiles of 128 and 256 with
# and without edges and K tails.
MID = [(48, 1024, 2080), (256, 512, 1000), (256, 1024, 333), (64, 4096, 700), (128, 2048, 4100), (128, 4096, 5000),
       (600, 64, 4500), (1030, 40, 9000), (600, 900, 1100), (1024, 768, 1024), (4096, 4096, 96), (3000, 3100, 544),
       (4096, 4096, 512), (4000, 4100, 512)]


# Bit-exact: MX4 operands are multiples of 1/4 of at most 24, so products are
# multiples of 1/16 of at most 576 and every partial sum is below 576 K * 16 <
# 2^24 units for K <= 1820; beyond that the operands' scales are 2^-1 .. 2^0.
@pytest.mark.parametrize("M,N,K", SHAPES + WIDE + MID)
@pytest.mark.parametrize("kind", ["mx4", "bf16", "f16"])
def test_product_exact_values(M, N, K, kind):
    say("product", M, N, K, kind)
    rng = rng_for(M, N, K)
    B, SB, b = int_operand(rng, N, K)
    if K > 1820:
        nb = -(-K // 32)
        SB[:, :nb] = SB[:, :nb].clamp(max=127)
        b = mp.values(B.cpu().numpy(), SB.cpu().numpy(), K)
    if kind == "mx4":
        A, SA, a = int_operand(rng, M, K)
        if K > 1820:
            SA[:, :-(-K // 32)] = SA[:, :-(-K // 32)].clamp(max=127)
            a = mp.values(A.cpu().numpy(), SA.cpu().numpy(), K)
    else:
        a = small_ints(rng, M, K)
        A, SA = torch.from_numpy(a).to(DT[kind]).cuda(), None
    c0 = rng.integers(-8, 9, (M, N)).astype(np.float32)
    bias = rng.integers(-8, 9, N).astype(np.float32)
    ab = a @ b.T
    for alpha, beta, use_bias in ((1.0, 0.0, False), (0.5, -2.0, True), (-1.0, 1.0, False)):
        C = torch.from_numpy(c0).cuda() if beta else torch.full((M, N), float("nan"), device="cuda")
        dgt.check(dgt.gemm_quantized(A, SA, B, SB, C, alpha, beta,
                                     torch.from_numpy(bias).cuda() if use_bias else None))
        want = alpha * ab + (beta * c0 if beta else 0.0) + (bias if use_bias else 0.0)
        got = C.double().cpu().numpy()
        assert np.array_equal(got, want), (alpha, beta, np.argwhere(got != want)[:4], got[got != want][:4],
                                           want[got != want][:4])


@pytest.mark.parametrize("M,N,K", [(8, 200, 4096), (64, 520, 8192), (300, 260, 4000), (1, 33, 8192)])
@pytest.mark.parametrize("kind", ["mx4", "bf16", "f16"])
def test_product_real_values(M, N, K, kind):
    """Normal values in blocks of very different scales: the error of an fp32
    sum of K products in any order is at most (K + 4) * 2^-23 of the sum of
    their magnitudes (2^-23 a step: truncation allowed)."""
    rng = rng_for(M, N, K, 7)
    B, SB, b = packed(rng.standard_normal((N, K)) * 2.0 ** rng.integers(-6, 3, (N, 1)))
    x = rng.standard_normal((M, K)) * np.exp(rng.standard_normal((1, K)))
    if kind == "mx4":
        A, SA, a = packed(x)
    else:
        A, SA = torch.from_numpy(x).to(DT[kind]).cuda(), None
        a = A.double().cpu().numpy()
    C = torch.full((M, N), float("nan"), device="cuda")
    dgt.check(dgt.gemm_quantized(A, SA, B, SB, C))
    got = C.double().cpu().numpy()
    bound = (K + 4) * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)
    err = np.abs(got - a @ b.T)
    assert (err <= bound).all()
    rel = np.linalg.norm(got - a @ b.T) / np.linalg.norm(a @ b.T)
    say(kind, M, N, K, "normwise", rel)
    assert rel <= 1e-5  # the library's gate for fp32 sums
    C2 = torch.empty_like(C)
    dgt.check(dgt.gemm_quantized(A, SA, B, SB, C2))
    assert torch.equal(C, C2)  # run to run


@pytest.mark.parametrize("M,N", [(3, 70), (20, 70), (100, 70), (40, 17000), (64, 6000), (600, 900)])
@pytest.mark.parametrize("kind", ["mx4", "bf16", "f16"])
def test_product_extreme_scales(M, N, kind):
    """NaN blocks reach exactly the outputs they feed; scales near both ends of
    the range with factors that bring the product back into it; f16
    activations against weights far outside f16's range."""
    K = 160
    rng = rng_for(M, N, 11)
    B, SB, _ = int_operand(rng, N, K)
    SB[:, :5] = torch.from_numpy(rng.integers(1, 4, (N, 5), dtype=np.uint8)).cuda()  # 2^-126 ..
    SB[9, 2] = 255
    SB[10, :5] = 0
    b = mp.values(B.cpu().numpy(), SB.cpu().numpy(), K)
    if kind == "mx4":
        A, SA, _ = int_operand(rng, M, K)
        SA[:, :5] = torch.from_numpy(rng.integers(249, 252, (M, 5), dtype=np.uint8)).cuda()
        SA[1, 0] = 255
        a = mp.values(A.cpu().numpy(), SA.cpu().numpy(), K)
        alpha = 1.0
    else:
        # 2^-126-like weights times values below 2^16: sums near 2^-110, scaled up by alpha
        x = rng.standard_normal((M, K)) * 2.0 ** rng.integers(8, 12, (M, 1))
        A, SA = torch.from_numpy(x).to(DT[kind]).cuda(), None
        a = A.double().cpu().numpy()
        alpha = 2.0 ** 100
    C = torch.empty(M, N, device="cuda")
    dgt.check(dgt.gemm_quantized(A, SA, B, SB, C, alpha=alpha))
    got = C.double().cpu().numpy()
    want = alpha * (a @ b.T)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    mag = alpha * (np.abs(np.nan_to_num(a)) @ np.abs(np.nan_to_num(b)).T)
    assert (np.abs(got - want)[ok] <= ((K + 4) * 2.0 ** -23 * mag + alpha * K * 2.0 ** -149)[ok]).all()


def test_infinite_activations_and_zero_codes():
    """An infinite activation meets a zero code as NaN, others as infinity, as
    in the plain product."""
    rng = rng_for(21)
    B, SB, b = int_operand(rng, 40, 64)
    for kind in ("bf16", "f16"):
        a = small_ints(rng, 5, 64)
        a[2, 7] = np.inf
        a[3, 60] = np.nan
        A = torch.from_numpy(a).to(DT[kind]).cuda()
        C = torch.empty(5, 40, device="cuda")
        dgt.check(dgt.gemm_quantized(A, None, B, SB, C))
        with np.errstate(invalid="ignore"):
            want = (a[:, None, :] * b[None]).sum(-1)
        np.testing.assert_array_equal(C.double().cpu().numpy(), want)


@pytest.mark.parametrize("M,N", [(5, 150), (64, 150), (200, 150), (20, 9000), (64, 6000), (600, 900)])
@pytest.mark.parametrize("kind", ["mx4", "bf16", "f16"])
def test_product_strided_storage(M, N, kind):
    """Padded pitches everywhere, misaligned 16-bit rows, NaN and junk behind
    every row, a guard band around C."""
    K = 330
    rng = rng_for(M, N, 5)
    B, SB, b = int_operand(rng, N, K)
    Bf = torch.full((N, B.shape[1] + 48), 0x77, dtype=torch.uint8, device="cuda")
    Bf[:, :B.shape[1]] = B
    Sf = torch.full((N, SB.shape[1] + 32), 255, dtype=torch.uint8, device="cuda")
    Sf[:, :SB.shape[1]] = SB
    cp = N + 5
    Cf = torch.full((M * cp + 3,), -777.0, device="cuda")
    C = Cf[3:].as_strided((M, N), (cp, 1))
    if kind == "mx4":
        A, SA, a = int_operand(rng, M, K)
        Af = torch.full((M, A.shape[1] + 16), 0x77, dtype=torch.uint8, device="cuda")
        Af[:, :A.shape[1]] = A
        w = B.shape[1]
        st = dgt.gemm_mx4(M, N, K, 1.0, Af.data_ptr(), Af.stride(0), SA.data_ptr(), SA.stride(0),
                          Bf.data_ptr(), Bf.stride(0), Sf.data_ptr(), Sf.stride(0), 0.0, C.data_ptr(),
                          cp, 0, torch.cuda.current_stream().cuda_stream)
        assert w == mp.code_pitch(K)
        dgt.check(st)
    else:
        a = small_ints(rng, M, K)
        flat = torch.full((M * (K + 3) + 1,), float("nan"), dtype=DT[kind], device="cuda")
        A = flat[1:].as_strided((M, K), (K + 3, 1))
        A.copy_(torch.from_numpy(a))
        dgt.check(dgt.gemm_quantized(A, None, Bf, Sf, C))
    assert np.array_equal(C.double().cpu().numpy(), a @ b.T)
    guard = torch.ones(M * cp + 3, dtype=torch.bool)
    guard[3:].as_strided((M, N), (cp, 1)).fill_(False)
    assert (Cf.cpu()[guard] == -777.0).all()


def test_alpha_zero_reads_no_operand():
    C = torch.full((70, 9), 2.0, device="cuda")
    bias = torch.arange(9.0, device="cuda")
    dgt.check(dgt.gemm_mx4(70, 9, 64, 0.0, 0, 32, 0, 16, 0, 32, 0, 16, 0.5, C.data_ptr(), 9,
                           bias.data_ptr(), torch.cuda.current_stream().cuda_stream))
    assert torch.equal(C, (1.0 + bias).expand(70, 9))
    dgt.check(dgt.gemm_mx4_a16(1, 70, 9, 0, 1.0, 0, 1, 0, 16, 0, 16, 0.0, C.data_ptr(), 9, 0,
                               torch.cuda.current_stream().cuda_stream))
    assert torch.equal(C, torch.zeros_like(C))


def test_offsets_past_32_bits():
    """Rows more than 2^32 bytes into the codes and into C."""
    pitch = dgt.MX4_MAX_PITCH
    N, K, M = 300, 96, 70
    rng = rng_for(77)
    B, SB, b = int_operand(rng, N, K)
    Bf = torch.empty(N, pitch, dtype=torch.uint8, device="cuda")  # 4.7 GiB
    Bf[:, :B.shape[1]] = B
    A, SA, a = int_operand(rng, M, K)
    for m in (8, M):
        C = torch.empty(m, N, device="cuda")
        dgt.check(dgt.gemm_mx4(m, N, K, 1.0, A.data_ptr(), A.stride(0), SA.data_ptr(), SA.stride(0),
                               Bf.data_ptr(), pitch, SB.data_ptr(), SB.stride(0), 0.0, C.data_ptr(), N, 0,
                               torch.cuda.current_stream().cuda_stream))
        assert np.array_equal(C.double().cpu().numpy(), a[:m] @ b.T)
        X = torch.from_numpy(small_ints(rng, m, K)).to(torch.bfloat16).cuda()
        dgt.check(dgt.gemm_quantized(X, None, Bf, SB, C))
        assert np.array_equal(C.double().cpu().numpy(), X.double().cpu().numpy() @ b.T)
    Y = torch.empty(N, K, device="cuda")
    dgt.check(dgt.dequantize_mx4(Bf, SB, Y))
    assert np.array_equal(Y.double().cpu().numpy(), b)
    Q2 = torch.empty_like(Bf)
    S2 = torch.empty_like(SB)
    dgt.check(dgt.quantize_mx4(Y, Q2, S2))
    Z = torch.empty_like(Y)
    dgt.check(dgt.dequantize_mx4(Q2, S2, Z))
    assert np.array_equal(Z.double().cpu().numpy(), b)


def test_graph_capture_and_streams():
    """quantise -> product captured into a graph and replayed with new inputs,
    and the same calls on two streams at once."""
    M, N, K = 48, 260, 700
    rng = rng_for(31)
    W = torch.from_numpy(rng.standard_normal((N, K))).float().cuda()
    QW, SW = dgt.mx4_empty(N, K)
    dgt.check(dgt.quantize_mx4(W, QW, SW))
    X = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    QX, SX = dgt.mx4_empty(M, K)
    C, D = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")

    def step(stream=None):
        dgt.check(dgt.quantize_mx4(X, QX, SX, stream=stream))
        dgt.check(dgt.gemm_quantized(QX, SX, QW, SW, C, stream=stream))
        dgt.check(dgt.gemm_quantized(X, None, QW, SW, D, stream=stream))

    X.copy_(torch.from_numpy(rng.standard_normal((M, K))))
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(4):
        X.copy_(torch.from_numpy(rng.standard_normal((M, K))))
        g.replay()
        torch.cuda.synchronize()
        got = C.clone(), D.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], C) and torch.equal(got[1], D)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    C2 = torch.empty_like(C)
    dgt.check(dgt.gemm_quantized(QX, SX, QW, SW, C2, stream=side))
    dgt.check(dgt.gemm_quantized(QX, SX, QW, SW, C))
    torch.cuda.synchronize()
    assert torch.equal(C, C2)


def test_training_products_of_a_linear_layer():
    """Y = X W^T, dX = G W, dW = G^T X with operands quantised along each
    product's own summation index, against the formulas in 64 bits; and dX
    against differences of the loss sum(G * Y) in the quantised weights'
    product (linear, so differences of any length are exact up to the fp32 sums)."""
    T, I, O = 96, 160, 72
    rng = rng_for(41)
    X, W, G = (torch.from_numpy(rng.standard_normal(s)).to(torch.bfloat16).cuda()
               for s in ((T, I), (O, I), (T, O)))

    def q(t, trans):
        M, K = t.shape[::-1] if trans else t.shape
        Q, S = dgt.mx4_empty(M, K)
        dgt.check(dgt.quantize_mx4(t, Q, S, trans=trans))
        return Q, S

    def val(t, trans):
        t = t.double().cpu().numpy()
        t = t.T if trans else t
        return mp.values(*mp.quantize(t), t.shape[1])

    for a, ta, b, tb in ((X, False, W, False), (G, False, W, True), (G, True, X, True)):
        (QA, SA), (QB, SB) = q(a, ta), q(b, tb)
        va, vb = val(a, ta), val(b, tb)
        C = torch.empty(va.shape[0], vb.shape[0], device="cuda")
        dgt.check(dgt.gemm_quantized(QA, SA, QB, SB, C))
        bound = (va.shape[1] + 36) * 2.0 ** -23 * (np.abs(va) @ np.abs(vb).T)
        assert (np.abs(C.double().cpu().numpy() - va @ vb.T) <= bound).all()
    # 16-bit activations and the weight as stored: Y(X + d) - Y(X) summed against G is <dX, d>
    QW, SW = q(W, False)
    w = val(W, False)
    g = G.double().cpu().numpy()
    dX = g @ w
    Y0, Y1 = torch.empty(T, O, device="cuda"), torch.empty(T, O, device="cuda")
    d = torch.zeros_like(X)
    d[5, 7], d[50, 100] = 2.0, -4.0
    X1 = (X.float() + d.float()).to(torch.bfloat16)
    dgt.check(dgt.gemm_quantized(X, None, QW, SW, Y0))
    dgt.check(dgt.gemm_quantized(X1, None, QW, SW, Y1))
    diff = (g * (Y1.double() - Y0.double()).cpu().numpy()).sum()
    moved = (X1.double() - X.double()).cpu().numpy()
    scale = (np.abs(g) * ((np.abs(X.double().cpu().numpy()) + np.abs(X1.double().cpu().numpy()))
                          @ np.abs(w).T)).sum()
    assert abs(diff - (dX * moved).sum()) <= (I + 4) * 2.0 ** -23 * scale


@pytest.mark.parametrize("M,N", [(64, 6000), (600, 900), (2, 300)])
def test_products_captured_at_each_form(M, N):
    """Shared strips, tiles and wave-private strips captured together and
    replayed on new operands, with eager work between the replays."""
    K = 640
    rng = rng_for(M, N, 41)
    B, SB, b = int_operand(rng, N, K)
    A, SA, _ = int_operand(rng, M, K)
    X = torch.empty(M, K, dtype=torch.float16, device="cuda")
    C, D = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")

    def step():
        dgt.check(dgt.gemm_quantized(A, SA, B, SB, C))
        dgt.check(dgt.gemm_quantized(X, None, B, SB, D))

    X.zero_()
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        A2, SA2, a = int_operand(rng, M, K)
        A.copy_(A2), SA.copy_(SA2)
        x = small_ints(rng, M, K)
        X.copy_(torch.from_numpy(x))
        C.fill_(float("nan")), D.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(C.double().cpu().numpy(), a @ b.T)
        assert np.array_equal(D.double().cpu().numpy(), x @ b.T)


def test_one_operand_on_both_sides_and_tall_products():
    """A x A^T with one operand given twice; far more rows than tiles of columns."""
    rng = rng_for(42)
    A, SA, a = int_operand(rng, 333, 320)
    C = torch.empty(333, 333, device="cuda")
    dgt.check(dgt.gemm_quantized(A, SA, A, SA, C))
    assert np.array_equal(C.double().cpu().numpy(), a @ a.T)
    M, N, K = 70001, 1, 64
    B, SB, b = int_operand(rng, N, K)
    T, ST, t = int_operand(rng, M, K)
    C = torch.empty(M, N, device="cuda")
    dgt.check(dgt.gemm_quantized(T, ST, B, SB, C))
    assert np.array_equal(C.double().cpu().numpy(), t @ b.T)
    x = small_ints(rng, M, K)
    for dt in (torch.bfloat16, torch.float16):
        dgt.check(dgt.gemm_quantized(torch.from_numpy(x).to(dt).cuda(), None, B, SB, C))
        assert np.array_equal(C.double().cpu().numpy(), x @ b.T)
