"""Newton-Schulz orthogonalisation in 64 bits on any device: the plain
iteration, and the same with the roundings gemm_orthogonalize documents (FP16
operands of every product, scaled by powers of two; X in two FP16 halves, of
which the products read the first and the term a*X both; the polynomial's
diagonal in 32 bits)."""

import math

import torch

COEF = (3.4445, -4.7750, 2.0315)


def matrix(gen, M, N, kind):
    """float64 [M, N]: 'normal' values; 'rankR', a product of rank R exactly;
    'powerP', singular values 1/i^P; 'lowrank', strong directions over a noise floor."""
    def normal(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float64, device=gen.device)

    n = min(M, N)
    if kind == "normal":
        return normal(M, N)
    if kind == "lowrank":
        r = max(1, n // 8)
        return normal(M, r).mm(normal(r, N)) / math.sqrt(r) + 0.3 * normal(M, N)
    if kind.startswith("rank"):
        r = int(kind[4:])
        return normal(M, r).mm(normal(r, N))
    u, v = (torch.linalg.qr(normal(d, n).cpu())[0].to(gen.device) for d in (M, N))
    i = torch.arange(1, n + 1, dtype=torch.float64, device=gen.device)
    return (u * i ** -float(kind[5:])).mm(v.t().contiguous())


def _step(left, right, a, b, c, s):
    """s -> b*s + c*s*s, and a*left + (that)*right."""
    return a * left + (b * s + c * s.mm(s)).mm(right)


def plain(G, steps=5, a=COEF[0], b=COEF[1], c=COEF[2], eps=1e-7):
    X = G.double()
    tall = X.shape[0] > X.shape[1]
    X = (X.t() if tall else X).contiguous()
    X = X / (torch.linalg.vector_norm(X) + eps)
    for _ in range(steps):
        X = _step(X, X, a, b, c, X.mm(X.t().contiguous()))
    return X.t() if tall else X


def rounded(G, steps=5, a=COEF[0], b=COEF[1], c=COEF[2], eps=1e-7):
    """As `plain` with the documented roundings, before the result's own to bf16."""
    def half(t):
        return t.to(torch.float16).double()

    X = G.double()
    tall = X.shape[0] > X.shape[1]
    X = (X.t() if tall else X).contiguous()
    scale = 2.0 ** round(0.5 * math.log2(X.shape[1]))
    X = X / (torch.linalg.vector_norm(X) + eps) * scale
    for i in range(steps):
        X = X.float().double()
        hi = half(X)
        lo = half(X - hi)
        S = half(4096.0 / scale ** 2 * hi.mm(hi.t().contiguous()))
        B = 1024.0 / 4096.0 * b * S + 1024.0 / 4096.0 ** 2 * c * S.mm(S)
        rest = (B - half(B)).diagonal()[:, None]
        X = a * (hi + lo) + (half(B).mm(hi) + rest * hi) / 1024.0
    return (X.t() if tall else X) / scale


def normwise(x, want):
    return float(torch.linalg.vector_norm(x.double() - want) / torch.linalg.vector_norm(want))


def gate(G, want, steps=5):
    """What a result may be off, normwise: the error that rounding `want` to
    bf16 has, and 1.5 times the error of the documented roundings before it.
    The two are independent, so their squares add.  A kernel that sums in
    another order makes as many roundings of the same size in other places;
    over n elements the norm of n such errors varies by about 0.4 / sqrt(n) of
    itself (an error is even over half a step either way), so 2% is five
    times that from 10,000 elements on."""
    own = 1.02 * normwise(want.to(torch.bfloat16), want)
    return math.sqrt(own ** 2 + (1.5 * normwise(rounded(G, steps), want)) ** 2)
