"""Plain 64-bit forms of the gated projections, their gradient and the 4-bit
weights with group scales, on the CPU, written from the definitions in
include/dgt_gemm.h, and the tolerances of the 16-bit results."""

import math

import numpy as np
import torch

ACTS = ("silu", "gelu", "gelu_tanh", "relu", "sigmoid", "identity")
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U24 = 2.0 ** -24  # fp32's unit roundoff


def phi(x):
    """P(normal variable < x); torch.special.ndtr loses the lower tail's digits from about -6 on."""
    return torch.special.erfc(-x * math.sqrt(0.5)) / 2


def act(x, name):
    if name == "silu":
        return x * torch.special.expit(x)
    if name == "gelu":
        return x * phi(x)
    if name == "gelu_tanh":
        return x * torch.special.expit(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))
    if name == "relu":
        return torch.where(x > 0, x, torch.where(x == x, 0.0, x))
    return torch.special.expit(x) if name == "sigmoid" else x.clone()


def slope(x, name):
    if name == "silu":
        s = torch.special.expit(x)
        return s + x * s * torch.special.expit(-x)
    if name == "gelu":
        return phi(x) + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        y = c * (x + 0.044715 * x ** 3)
        return torch.special.expit(y) + x * torch.special.expit(y) * torch.special.expit(-y) * c * (
            1 + 3 * 0.044715 * x ** 2)
    if name == "relu":
        return (x > 0).double()
    if name == "sigmoid":
        return torch.special.expit(x) * torch.special.expit(-x)
    return torch.ones_like(x)


def forward(X, Wg, Wu, bg, bu, name):
    """h, g, u and bounds of the fp32 errors of g and u (see `sum_error`)."""
    X, Wg, Wu = (t.double().cpu() for t in (X, Wg, Wu))
    bg, bu = (torch.zeros(Wg.shape[0], dtype=torch.float64) if b is None else b.double().cpu() for b in (bg, bu))
    g, u = X @ Wg.T + bg, X @ Wu.T + bu
    eg = sum_error(X, Wg.T) + U24 * g.abs() * 2
    eu = sum_error(X, Wu.T) + U24 * u.abs() * 2
    return act(g, name) * u, g, u, eg, eu


def sum_error(A, B):
    """Bound of an fp32 sum's error over K exact products.  Each of the K additions
    is off by at most a unit roundoff (two, where it truncates) of a partial sum, which is at most sum|ab|; the
    signs are independent, so the whole is below 8 sqrt(K) of them but once in 10^14."""
    K = A.shape[1]
    return 8 * math.sqrt(max(K, 1)) * U24 * 2 * (A.abs() @ B.abs())


def act_error(x, y):
    """Bound of act's and its slope's fp32 error where the value is y: the exponential's argument is
    rounded (|x| roundoffs of it, 3|x|^3/10 more for the cubic), erfc's too (x^2 of them), and a dozen
    operations follow, of terms no larger than 1 + |x|."""
    return (x.abs() + x ** 2 + 0.3 * x.abs() ** 3 + 16) * U24 * y.abs()


def half_step(v, dtype):
    """Half a step of the 16-bit type at |v| (its subnormals' step below the normal range)."""
    f = torch.finfo(dtype)
    return torch.clamp(v.abs() * f.eps / 2, min=f.tiny * f.eps / 2)


def assert_within(got, want, bound, what=""):
    """|got - want| <= bound, NaN where want is, infinities alike."""
    got, want = got.double().cpu(), want.double().cpu()
    assert got.shape == want.shape, f"{what}: {tuple(got.shape)} for {tuple(want.shape)}"
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaNs in other places"
    assert torch.equal(got[odd & (want == want)], want[odd & (want == want)]), f"{what}: infinities"
    off = torch.where(odd, torch.zeros_like(want), (got - torch.where(odd, 0.0, want)).abs() - bound)
    off[odd] = 0
    assert not (off > 0).any(), (f"{what}: {int((off > 0).sum())} of {off.numel()} outside, worst at "
                                 f"{int(off.argmax())}: got {got.flatten()[off.argmax()]} want "
                                 f"{want.flatten()[off.argmax()]}")


# ------------------------------------------------- 4-bit weights

def groups(K, group):
    return -(-K // group)


def round_scale(s, dtype):
    """fp64 -> fp32 -> the 16-bit type, both to nearest even, bounded by its largest value."""
    t = torch.from_numpy(np.asarray(s, np.float64)).float().to(dtype)
    top = torch.finfo(dtype).max
    return torch.where(torch.isinf(t), torch.full_like(t, top), t)


def quantize(x, group, dtype, zeros):
    """(codes [rows, K], scales as a 16-bit tensor, zero points) of float64 values."""
    rows, K = x.shape
    n = groups(K, group)
    q = np.zeros((rows, K), np.uint8)
    s = torch.zeros(rows, n, dtype=dtype)
    z = np.full((rows, n), 8, np.uint8)
    for i in range(n):
        part = x[:, i * group:(i + 1) * group]
        bad = ~np.isfinite(part).all(axis=1)
        clean = np.where(bad[:, None], 0.0, part)
        hi, lo = np.maximum(clean.max(axis=1), 0), np.maximum(-clean.min(axis=1), 0)
        s[:, i] = round_scale((hi + lo) / 15 if zeros else np.maximum(hi / 7, lo / 8), dtype)
        unit = s[:, i].double().numpy()
        unit = np.where(unit > 0, unit, 1.0)
        zp = np.minimum(np.rint(lo / unit), 15) if zeros else np.full(rows, 8.0)
        code = np.clip(np.rint(clean / unit[:, None]) + zp[:, None], 0, 15)
        q[:, i * group:(i + 1) * group] = np.where(bad[:, None], 0, code)
        if zeros:
            z[:, i] = np.where(bad, 0, zp)
        s[torch.from_numpy(bad), i] = float("nan")
    return q, s, z


def values(q, s, z, group):
    K = q.shape[1]
    at = np.arange(K) // group
    return s.double().numpy()[:, at] * (q.astype(np.float64) - z.astype(np.float64)[:, at])


def pack(q, fill=0):
    """Stored codes; the places past K in the last 16 bytes get the code `fill`."""
    rows, K = q.shape
    wide = np.full((rows, -(-K // 32) * 32), fill, np.uint8)
    wide[:, :K] = q
    return torch.from_numpy(wide[:, 0::2] | (wide[:, 1::2] << 4))


def product_error(X, q, s, z, group):
    """Bound of the fp32 error of s (sum xq - z sum x) summed over the groups: every sum as in
    `sum_error`, of terms up to |s| |x| (q + z)."""
    at = np.arange(q.shape[1]) // group
    w = np.abs(s.double().numpy())[:, at] * (q.astype(np.float64) + z.astype(np.float64)[:, at])
    return sum_error(X.double().cpu(), torch.from_numpy(w.T.copy()))
