"""Cases of the operators on a linear layer's weight and activations beyond the plain product: microscaled
4-bit storage (quantising rows or columns, reading back), the products on it, and the orthogonalised update.

Each case is a dict of plain values; `prepare` makes what a caller holds before the call, `run` makes one pass
(in plain torch operations, or with the library's calls where `own` is true), `exact` gives the definition's
values in 64 bits.

The 4-bit format: blocks of 32 consecutive k share a scale 2^(s - 127) (s one byte; 255 stands for NaN), and an
element is 4 bits: a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6.  A row of K elements takes 16 bytes per block
(two elements a byte, the even k in the low half) and 16 bytes of scales per 16 blocks.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ELEM_BYTES = {"f32": 4, "bf16": 2, "f16": 2}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
NS_COEFFICIENTS = (3.4445, -4.7750, 2.0315)
NS_STEPS = 5
NS_EPS = 1e-7


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # a decode step's activations, quantised before a 4-bit product and read back in 16 bits
        dict(name="quant_8x8192_bf16", op="quantize", dtype="bf16", out="bf16", rows=8, cols=8192, trans=False),
        # a master weight [out, in] in fp32 packed for serving, read back in fp32
        dict(name="quant_8192x8192_f32", op="quantize", dtype="f32", out="f32", rows=8192, cols=8192, trans=False),
        # activations stored [tokens, in], blocks along the tokens: the weight-gradient product's operand
        dict(name="quant_trans_6144x4096_bf16", op="quantize", dtype="bf16", out="bf16", rows=6144, cols=4096,
             trans=True),
        # one GPU's share of a decode product, both operands 4-bit
        dict(name="mx4_8x3584x8192", op="product", M=8, N=3584, K=8192, alpha=1.0, beta=0.0, bias=False),
        # the whole weight at a small decode batch: the time to stream it once
        dict(name="mx4_8x28672x8192", op="product", M=8, N=28672, K=8192, alpha=1.0, beta=0.0, bias=False),
        # ragged in every dimension, accumulating into C
        dict(name="mx4_1000_ragged", op="product", M=1000, N=1000, K=1000, alpha=1.5, beta=0.5, bias=False),
        # prefill or training forward of a large layer with its bias
        dict(name="mx4_8192_bias", op="product", M=8192, N=8192, K=8192, alpha=1.0, beta=0.0, bias=True),
        # a single token in 16 bits against 4-bit weights
        dict(name="a16_1x3584x8192_f16", op="product16", dtype="f16", M=1, N=3584, K=8192, alpha=1.0, beta=0.0,
             bias=True),
        # the widest decode batch of the skinny path, 16-bit activations
        dict(name="a16_64x28672x8192_bf16", op="product16", dtype="bf16", M=64, N=28672, K=8192, alpha=1.0,
             beta=0.0, bias=False),
        # one small square weight's update: the time is in the steps, not in the work
        dict(name="orth_256_f32", op="orthogonalize", dtype="f32", batch=1, M=256, N=256),
        # a tall weight (a GPU's share of a layer)
        dict(name="orth_8192x1024_bf16", op="orthogonalize", dtype="bf16", batch=1, M=8192, N=1024),
        # sixteen layers' weights of one shape in one call
        dict(name="orth_16x2048_f32", op="orthogonalize", dtype="f32", batch=16, M=2048, N=2048),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "product16", "orthogonalize"])
    if op == "quantize":
        rows = _log_uniform(rng, 1, 8192)
        cols = _log_uniform(rng, 16, 8192)
        return dict(op=op, dtype=rng.choice(["f32", "bf16", "f16"]), out=rng.choice(["f32", "bf16"]), rows=rows,
                    cols=cols, trans=rng.random() < 0.4)
    if op == "product":
        # half decode batches, half larger ones
        M = _log_uniform(rng, 1, 64) if rng.random() < 0.5 else _log_uniform(rng, 65, 4096)
        N = _log_uniform(rng, 64, 16384 if M <= 64 else 6144)
        K = _log_uniform(rng, 32, 8192)
        beta = rng.choice([0.0, 0.0, 0.5])
        return dict(op=op, M=M, N=N, K=K, alpha=rng.choice([1.0, 1.5]), beta=beta, bias=rng.random() < 0.5)
    if op == "product16":
        M = _log_uniform(rng, 1, 64) if rng.random() < 0.8 else _log_uniform(rng, 65, 300)
        return dict(op=op, dtype=rng.choice(["bf16", "f16"]), M=M, N=_log_uniform(rng, 64, 16384),
                    K=_log_uniform(rng, 32, 8192), alpha=1.0, beta=rng.choice([0.0, 0.0, 0.5]),
                    bias=rng.random() < 0.5)
    batch = rng.choice([1, 1, 1, 2, 4])
    return dict(op=op, dtype=rng.choice(["f32", "bf16", "f16"]), batch=batch, M=_log_uniform(rng, 48, 2600),
                N=_log_uniform(rng, 48, 2600))


# ---------------------------------------------------------- the 4-bit format

def _blocks(k):
    return (k + 31) // 32


def _pack(values, exponents, k):
    """Codes and scales in the stored layout from the elements in units of their scale ([rows, blocks * 32],
    each one of the magnitudes with a sign) and the biased exponents ([rows, blocks])."""
    rows, nb = exponents.shape
    table = torch.tensor(MAGNITUDES, device=values.device)
    code = torch.bucketize(values.abs(), table).to(torch.uint8) | (values.signbit().to(torch.uint8) << 3)
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()
    scales = torch.full((rows, 16 * ((nb + 15) // 16)), 127, dtype=torch.uint8, device=values.device)
    scales[:, :nb] = exponents.to(torch.uint8)
    return codes, scales


def _stored(x):
    """A 4-bit operand as a caller holds it: codes and scales of the fp32 matrix x."""
    rows, k = x.shape
    v, e = _rounded(x.float())
    return _pack(v, e + 127, k)


def _rounded(x):
    """Elements in units of their block's scale, and its exponent: the exponent of the largest magnitude less
    two, each element rounded to the nearest magnitude (ties to the even code), at most 6."""
    rows, k = x.shape
    nb = _blocks(k)
    x = torch.nn.functional.pad(x, (0, 32 * nb - k)).view(rows, nb, 32)
    amax = x.abs().amax(dim=2)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, torch.full_like(amax, -127, dtype=torch.int32))
    e = e.clamp(-127, 127)
    y = torch.ldexp(x, -e.unsqueeze(2))
    mag = y.abs()
    step = torch.where(mag < 2, 0.5, torch.where(mag < 4, 1.0, 2.0))
    mag = (torch.round(mag / step) * step).clamp(max=6.0)
    return torch.copysign(mag, y).view(rows, nb * 32), e


def _values(codes, scales, k):
    """The fp32 values of a stored operand, [rows, k]."""
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=codes.device)
    q = torch.stack((codes & 15, codes >> 4), dim=2).view(codes.shape[0], -1)
    e = scales[:, :_blocks(k)].int() - 127
    v = torch.ldexp(table[q.int()].view(codes.shape[0], -1, 32), e.unsqueeze(2))
    return v.view(codes.shape[0], -1)[:, :k]


# -------------------------------------------------------------- what is held

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _activations(gen, rows, k):
    """Normal values, a few channels much larger than the rest."""
    channel = torch.exp(0.8 * _normal(gen, 1, k))
    return _normal(gen, rows, k) * channel


def _momentum(case, gen):
    """A weight's momentum: a few strong directions over a noise floor, small in absolute size."""
    b, m, n = case["batch"], case["M"], case["N"]
    r = max(1, min(m, n) // 8)
    g = _normal(gen, b, m, r) @ _normal(gen, b, r, n) / math.sqrt(r) + 0.3 * _normal(gen, b, m, n)
    return (1e-3 * g).to(DTYPES[case["dtype"]])


def prepare(case, seed):
    gen = _gen(seed)
    op = case["op"]
    state = dict(case=case)
    if op == "quantize":
        # stored [cols, rows] when the blocks run along the stored columns
        x = _activations(gen, case["rows"], case["cols"])
        if case["rows"] > 4:
            x[case["rows"] // 2] = 0.0  # a padded token
        x = (x.t() if case["trans"] else x).to(DTYPES[case["dtype"]]).contiguous()
        nb = _blocks(case["cols"])
        state["X"] = x
        state["Q"] = torch.empty(case["rows"], 16 * nb, dtype=torch.uint8, device="cuda")
        state["S"] = torch.empty(case["rows"], 16 * ((nb + 15) // 16), dtype=torch.uint8, device="cuda")
        state["Y"] = torch.empty(case["rows"], case["cols"], dtype=DTYPES[case["out"]], device="cuda")
    elif op in ("product", "product16"):
        M, N, K = case["M"], case["N"], case["K"]
        a = _activations(gen, M, K)
        if op == "product":
            state["A"], state["SA"] = _stored(a)
        else:
            state["A"], state["SA"] = a.to(DTYPES[case["dtype"]]), None
        state["B"], state["SB"] = _stored(0.02 * _normal(gen, N, K))
        state["bias"] = _normal(gen, N) if case["bias"] else None
        state["C0"] = _normal(gen, M, N) if case["beta"] else None
        state["C"] = torch.empty(M, N, device="cuda")
    else:
        state["G"] = _momentum(case, gen)
        state["O"] = torch.empty(state["G"].shape, dtype=torch.bfloat16, device="cuda")
    return state


# ------------------------------------------------------------------ one pass

def _plain_product(state):
    case = state["case"]
    K = case["K"]
    a = state["A"].float() if state["SA"] is None else _values(state["A"], state["SA"], K)
    c = case["alpha"] * (a @ _values(state["B"], state["SB"], K).t())
    if case["beta"]:
        c = c + case["beta"] * state["C0"]
    return c if state["bias"] is None else c + state["bias"]


def _plain_orthogonalize(g):
    a, b, c = NS_COEFFICIENTS
    x = g.float()
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2).contiguous() if tall else x
    norm = x.double().square().sum(dim=(1, 2), keepdim=True).sqrt().float()
    x = x / (norm + NS_EPS)
    for _ in range(NS_STEPS):
        gram = x @ x.transpose(1, 2).contiguous()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return (x.transpose(1, 2) if tall else x).to(torch.bfloat16)


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import dense_gemm_tuning_amd as dgt

        if op == "quantize":
            dgt.check(dgt.quantize_mx4(state["X"], state["Q"], state["S"], trans=case["trans"]))
            dgt.check(dgt.dequantize_mx4(state["Q"], state["S"], state["Y"]))
            return state["Y"]
        if op in ("product", "product16"):
            if case["beta"]:
                state["C"].copy_(state["C0"])
            dgt.check(dgt.gemm_quantized(state["A"], state["SA"], state["B"], state["SB"], state["C"],
                                         alpha=case["alpha"], beta=case["beta"], bias=state["bias"]))
            return state["C"]
        dgt.check(dgt.orthogonalize(state["G"], state["O"], steps=NS_STEPS, coefficients=NS_COEFFICIENTS,
                                    eps=NS_EPS))
        return state["O"]
    if op == "quantize":
        x = state["X"].float()
        v, e = _rounded(x.t().contiguous() if case["trans"] else x)
        y = torch.ldexp(v.view(case["rows"], -1, 32), e.unsqueeze(2)).view(case["rows"], -1)
        return y[:, :case["cols"]].to(DTYPES[case["out"]]).contiguous()
    if op in ("product", "product16"):
        return _plain_product(state)
    return _plain_orthogonalize(state["G"])


# ------------------------------------------------------------------ the work

def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        packed = case["rows"] * _blocks(case["cols"]) * 17
        return {"bytes": n * ELEM_BYTES[case["dtype"]] + 2 * packed + n * ELEM_BYTES[case["out"]], "flops": 4 * n}
    if op in ("product", "product16"):
        M, N, K = case["M"], case["N"], case["K"]
        a = M * K * 2 if op == "product16" else M * _blocks(K) * 17
        bytes_ = a + N * _blocks(K) * 17 + 4 * M * N * (2 if case["beta"] else 1) + (4 * N if case["bias"] else 0)
        return {"bytes": bytes_, "flops": 2 * M * N * K}
    # per step: the Gram matrix and its square, half of each (they are symmetric), and the update
    m, n = sorted((case["M"], case["N"]))
    per_step = m * m * n + m * m * m + 2 * m * m * n
    return {"bytes": case["batch"] * m * n * (ELEM_BYTES[case["dtype"]] + 2),
            "flops": case["batch"] * NS_STEPS * per_step}


# ------------------------------------------------------- the definition, 64 bits

def _exact_values(codes, scales, k):
    sign = 1.0 - 2.0 * torch.stack(((codes >> 3) & 1, codes >> 7), dim=2).flatten(1).double()
    c = torch.stack((codes & 7, (codes >> 4) & 7), dim=2).flatten(1).double()
    # code c below 2: c/2; otherwise (1 + mantissa/2) * 2^(exponent - 1)
    exponent, mantissa = torch.floor(c / 2), c % 2
    mag = torch.where(exponent == 0, mantissa / 2, (1 + mantissa / 2) * torch.exp2(exponent - 1))
    scale = torch.exp2(scales[:, :_blocks(k)].double() - 127).repeat_interleave(32, dim=1)
    return (sign * mag * scale)[:, :k]


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = state["X"].double()
        x = x.t().contiguous() if case["trans"] else x
        x = torch.nn.functional.pad(x, (0, -case["cols"] % 32)).view(case["rows"], -1, 32)
        top = x.abs().amax(dim=2, keepdim=True)
        floor = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
        floor = torch.where(torch.exp2(floor) > top, floor - 1, floor)  # log2 rounded up to a whole number
        scale = torch.exp2(torch.where(top > 0, floor - 2, -127.0).clamp(-127, 127))
        # count the midpoints below each magnitude; a tie goes up where the upper code is even
        m = (x / scale).abs()
        code = sum((m > mid).double() if i % 2 == 0 else (m >= mid).double()
                   for i, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)))
        mag = torch.tensor(MAGNITUDES, dtype=torch.float64, device=x.device)[code.long()]
        return (torch.copysign(mag, x) * scale).view(case["rows"], -1)[:, :case["cols"]].contiguous()
    if op in ("product", "product16"):
        K = case["K"]
        a = state["A"].double() if state["SA"] is None else _exact_values(state["A"], state["SA"], K)
        c = case["alpha"] * torch.mm(a, _exact_values(state["B"], state["SB"], K).t().contiguous())
        c = c if state["C0"] is None else c + case["beta"] * state["C0"].double()
        return c if state["bias"] is None else c + state["bias"].double()
    a, b, c = NS_COEFFICIENTS
    out = []
    for g in state["G"].double():
        x = g / (torch.linalg.vector_norm(g) + NS_EPS)
        eye = torch.eye(min(x.shape), dtype=x.dtype, device=x.device)
        for _ in range(NS_STEPS):
            if x.shape[0] <= x.shape[1]:
                s = x.mm(x.t().contiguous())
                x = (a * eye + b * s + c * s.mm(s)).mm(x)
            else:
                s = x.t().contiguous().mm(x)
                x = x.mm(a * eye + b * s + c * s.mm(s))
        out.append(x)
    return torch.stack(out)
