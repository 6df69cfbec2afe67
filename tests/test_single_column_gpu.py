"""Single-column operands may have any last stride, which is never used: every
torch-facing call takes them as views and gets the same bits as from packed
copies, writing nothing beside C."""

import pytest
import torch

import dense_gemm_tuning_amd as dgt

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CALLS = {"gemm": dgt.gemm, "split": lambda *a, **k: dgt.gemm_split(*a, splits=2, **k),
         "stream": dgt.gemm_stream}


def column(rows, dtype, gen):
    """A [rows, 1] view with strides (5, 3) of small integers."""
    flat = torch.full((5 * rows + 2,), float("nan"), device="cuda").to(dtype)
    v = flat[2:].as_strided((rows, 1), (5, 3))
    v.copy_(torch.randint(-3, 4, (rows, 1), generator=gen, device="cuda"))
    return v


def full(rows, cols, dtype, gen):
    return torch.randint(-3, 4, (rows, cols), generator=gen, device="cuda").to(dtype)


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(70, 40, 1), (70, 1, 300), (1, 1, 9), (300, 1, 1), (9, 33, 1)])
def test_products_with_single_columns(M, N, K, dtype, call):
    gen = torch.Generator(device="cuda").manual_seed(M + N + K)
    t = DT[dtype]
    for trans_a, trans_b in ((False, False), (True, False), (False, True), (True, True)):
        sa, sb = ((K, M) if trans_a else (M, K)), ((N, K) if trans_b else (K, N))
        A = column(sa[0], t, gen) if sa[1] == 1 else full(*sa, t, gen)
        B = column(sb[0], t, gen) if sb[1] == 1 else full(*sb, t, gen)
        flat = torch.full((5 * M * N + 2,), -7.0, device="cuda")
        C = flat[2:].as_strided((M, 1), (5, 3)) if N == 1 else torch.empty(M, N, device="cuda")
        dgt.check(CALLS[call](A, B, C, trans_a=trans_a, trans_b=trans_b))
        a, b = A.double(), B.double()
        want = torch.mm((a.t() if trans_a else a).contiguous(), (b.t() if trans_b else b).contiguous())
        assert torch.equal(C.double(), want)
        if N == 1:
            C.fill_(-7.0)
            assert (flat == -7.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_batched_with_single_columns(dtype):
    gen = torch.Generator(device="cuda").manual_seed(3)
    nb, M, N, K, t = 3, 50, 20, 1, DT[dtype]
    A = torch.full((nb * 400,), float("nan"), device="cuda").to(t).as_strided((nb, M, 1), (400, 7, 2))
    A.copy_(torch.randint(-3, 4, (nb, M, 1), generator=gen, device="cuda"))
    B = full(nb * K, N, t, gen).view(nb, K, N)
    C = torch.empty(nb, M, N, device="cuda")
    dgt.check(dgt.gemm_batched(A, B, C))
    assert torch.equal(C.double(), A.double() * B.double())
    out = torch.full((nb * 300,), -7.0, device="cuda")
    D = out.as_strided((nb, M, 1), (300, 6, 4))
    x, w = full(nb * M, 64, t, gen).view(nb, M, 64), full(1, 64, t, gen)
    bias = torch.arange(6.0, device="cuda").as_strided((nb, 1), (2, 5))
    dgt.check(dgt.gemm_batched(x, w, D, trans_b=True, bias=bias))
    assert torch.equal(D.double(), (x.double() * w.double()).sum(2, keepdim=True) + bias.double()[:, None])
    D.fill_(-7.0)
    assert (out == -7.0).all()


def test_a_column_that_repeats_one_element_is_refused():
    """Pitch 0 is below the leading dimension's least."""
    A = torch.ones(1, 1, device="cuda").expand(4, 1)
    assert dgt.gemm(A, torch.ones(1, 3, device="cuda"), torch.empty(4, 3, device="cuda")) == dgt.GEMM_ERR_LD
