"""The gradient at the gated projections over the activations' whole range, from tails whose slopes underflow to
the types' largest values, on the register-staged and on the DMA tiles."""

import math

import pytest
import torch

import dense_gemm_tuning_amd as dgt
import gated_plain as gp
from gpu_util import say
from test_gated_gpu import stored

pytestmark = pytest.mark.gpu

DT = gp.DT
TINY = 2.0 ** -126  # fp32's least normal number


def tails(x, name):
    """What of act'(x) and act(x) goes through the exponential or the normal tail, in absolute value: near 1 their
    errors are those of the terms' small parts."""
    a = x.abs()
    if name in ("silu", "sigmoid"):
        t = torch.special.expit(-a)
        return (t * (1 + a), a * t) if name == "silu" else (t, t)
    if name == "gelu":
        t = gp.phi(-a)
        return t + a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi), a * t
    if name == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        t = torch.special.expit(-c * (a + 0.044715 * a ** 3))
        return t * (1 + a * c * (1 + 3 * 0.044715 * a * a)), a * t
    return torch.zeros_like(x), torch.zeros_like(x)


@pytest.mark.parametrize("pad", [0, 7])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", gp.ACTS)
def test_gradient_over_the_whole_range(act, dtype, pad):
    """K = 1 and dY = Wd = U = 1: dG is act'(g), dU and H are act(g).  pad 7: 16-byte rows.

    An exponential's argument is off by (|x| + x^2 + 0.3 |x|^3) roundoffs (see gp.act_error) and a dozen
    operations follow; terms below fp32's normal range, times at most (1 + |x|)(1 + x^2/4), are off by that
    range's end.  From |x| = 120 on every tail is zero in fp32."""
    t = DT[dtype]
    top = [1e4, 6e4] if dtype == "f16" else [1e4, 1e20, 3e35, 5e35, 1e36, 1e38, 3e38, 3.38e38]
    x = torch.cat([torch.linspace(-120, 120, 4801), torch.tensor([0.0, 1e-7] + top), -torch.tensor([0.0, 1e-7] + top)])
    G = x.to(t).unsqueeze(1)
    M = len(x)
    say("gated_grad range", act, dtype, pad)
    dY, Wd, U = stored(torch.ones(M, 1), dtype, pad), stored(torch.ones(1, 1), dtype, pad), stored(torch.ones(M, 1), dtype, 0)
    dG, dU, H = (torch.empty(M, 1, dtype=t, device="cuda") for _ in range(3))
    sums = torch.full((1,), 5.0, device="cuda")
    dgt.check(dgt.gated_grad(dY, Wd, G.cuda(), U, dG, dU, act=act, H=H, dbias_g=sums))
    g = G.double()
    a, s = gp.act(g, act), gp.slope(g, act)
    assert torch.isfinite(s).all() and torch.isfinite(a).all()
    c = g.clamp(-120, 120)
    e = (c.abs() + c ** 2 + 0.3 * c.abs() ** 3 + 16) * gp.U24
    floor = TINY * (1 + c.abs()) * (1 + c * c / 4)
    es, ea = (16 * gp.U24 * v.abs() + e * part + floor for v, part in zip((s, a), tails(c, act)))
    gp.assert_within(dG, s, gp.half_step(s.abs() + es, t) + es, f"{act} dG")
    for got, name in ((dU, "dU"), (H, "H")):
        gp.assert_within(got, a, gp.half_step(a.abs() + ea, t) + ea, f"{act} {name}")
    gp.assert_within(sums, s.sum(0), es.sum(0) + 2 * M * gp.U24 * s.abs().sum(0), f"{act} sum")
