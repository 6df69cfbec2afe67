"""Cases of the feed-forward block of a language model beyond the plain product: the gated projections with
their activation (whole prompts, training steps and single tokens), the gradient at them, and weights held in 4
bits with a scale per group: packing, products of few rows, and the gated projections on them.

Each case is a dict of plain values; `prepare` makes what a caller holds before the call, `run` makes one pass
(in plain torch operations, or with the library's calls where `own` is true), `exact` gives the definition's
values in 64 bits.

The gated projections of x [M, K] with weights stored [N, K]:  g = x Wg^T + bg, u = x Wu^T + bu, h = act(g) u.
Their gradient from dy [M, K] of y = h Wd^T (Wd stored [K, N]):  dh = dy Wd, dg = dh u act'(g), du = dh act(g),
and the sums of dg and du over the rows for the biases.

The 4-bit weights: `group` consecutive k of a row share a 16-bit scale s and a zero point z (8 where none is stored);
an element is s (q - z), q in 0 .. 15.  A row of K elements takes 16 bytes per 32 k, the even k in a byte's low half.
With r the range max(x, 0) - min(x, 0) of a group, s = r/15 and z the whole number nearest to -min(x, 0)/s; without
zero points s = max(max(x)/7, -min(x)/8, 0).  s is rounded to fp32, then to its 16-bit type; q is the whole number nearest
to x/s + z within 0 .. 15, ties of x/s to the even side.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ELEM_BYTES = {"f32": 4, "bf16": 2, "f16": 2}
ACTS = ("silu", "gelu", "gelu_tanh", "relu", "sigmoid", "identity")


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one GPU's share of the projections for a single token
        dict(name="gated_1x3584x8192_f16", op="gated", dtype="f16", act="silu", M=1, N=3584, K=8192, bias=False,
             save=False),
        # a decode batch against both whole weights: the time to stream them
        dict(name="gated_8x28672x8192_bf16", op="gated", dtype="bf16", act="silu", M=8, N=28672, K=8192, bias=False,
             save=False),
        # a ragged training batch: biases, pre-activations kept, rows that start off 16-byte boundaries
        dict(name="gated_1000x1000x1001_bf16", op="gated", dtype="bf16", act="gelu", M=1000, N=1000, K=1001,
             bias=True, save=True),
        # a training step's forward with the pre-activations kept
        dict(name="gated_8192_bf16", op="gated", dtype="bf16", act="silu", M=8192, N=8192, K=8192, bias=False,
             save=True),
        # the gradient of the ragged batch, with the biases' gradients
        dict(name="grad_1000_f16", op="grad", dtype="f16", act="gelu_tanh", M=1000, N=1000, K=1000, bias=True),
        # a training step's gradient, the activations recomputed for the second weight's gradient
        dict(name="grad_8192_bf16", op="grad", dtype="bf16", act="silu", M=8192, N=8192, K=8192, bias=False),
        # a master weight packed for serving and read back
        dict(name="pack_8192x8192_f32", op="pack", dtype="f32", out="f32", scale="f16", zeros=True, group=128,
             rows=8192, cols=8192),
        # a small 16-bit weight, ragged rows, finer groups, no zero points
        dict(name="pack_1000x1000_bf16", op="pack", dtype="bf16", out="bf16", scale="bf16", zeros=False, group=32,
             rows=1000, cols=1000),
        # a single token against one GPU's share of a packed weight
        dict(name="w4_1x3584x8192_bf16", op="w4", dtype="bf16", scale="bf16", zeros=True, group=128, M=1, N=3584,
             K=8192, alpha=1.0, beta=0.0, bias=False),
        # a wide decode batch, with the bias, accumulating
        dict(name="w4_64x28672x8192_f16", op="w4", dtype="f16", scale="f16", zeros=True, group=128, M=64, N=28672,
             K=8192, alpha=1.0, beta=0.5, bias=True),
        # the gated projections for a single token on one GPU's share of packed weights
        dict(name="w4_gated_1x3584x8192_f16", op="w4_gated", dtype="f16", scale="f16", act="silu", zeros=False,
             group=64, M=1, N=3584, K=8192, bias=False),
        # a decode batch against both whole weights, packed
        dict(name="w4_gated_8x28672x8192_bf16", op="w4_gated", dtype="bf16", scale="bf16", act="silu", zeros=True,
             group=128, M=8, N=28672, K=8192, bias=False),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _whole8(rng, n):
    """Mostly the next multiple of 8, as models have them, else any size."""
    return (n + 7) // 8 * 8 if rng.random() < 0.6 else n


def draw(rng):
    op = rng.choice(["gated", "gated", "grad", "pack", "w4", "w4", "w4_gated"])
    dtype = rng.choice(["bf16", "f16"])
    act = rng.choice(["silu", "silu", *ACTS])
    if op in ("gated", "grad"):
        # half decode batches, half larger ones (the gradient: larger ones)
        few = op == "gated" and rng.random() < 0.5
        M = _log_uniform(rng, 1, 64) if few else _log_uniform(rng, 65 if op == "gated" else 1, 4096)
        N = _whole8(rng, _log_uniform(rng, 16, 16384 if few else 8192))
        K = _whole8(rng, _log_uniform(rng, 16, 8192))
        case = dict(op=op, dtype=dtype, act=act, M=M, N=N, K=K, bias=rng.random() < 0.5)
        if op == "gated":
            case["save"] = rng.random() < 0.5
        return case
    group = rng.choice([32, 64, 128])
    scale = rng.choice(["bf16", "f16"])
    zeros = rng.random() < 0.5
    if op == "pack":
        return dict(op=op, dtype=rng.choice(["f32", "bf16", "f16"]), out=rng.choice(["f32", "bf16", "f16"]),
                    scale=scale, zeros=zeros, group=group, rows=_log_uniform(rng, 1, 8192),
                    cols=_whole8(rng, _log_uniform(rng, 16, 8192)))
    M = _log_uniform(rng, 1, 64) if rng.random() < 0.8 else _log_uniform(rng, 65, 300)
    N = _log_uniform(rng, 16, 16384)
    K = _whole8(rng, _log_uniform(rng, 16, 8192))
    case = dict(op=op, dtype=dtype, scale=scale, zeros=zeros, group=group, M=M, N=N, K=K, bias=rng.random() < 0.5)
    if op == "w4":
        case.update(alpha=rng.choice([1.0, 1.5]), beta=rng.choice([0.0, 0.0, 0.5]))
    else:
        case.update(act=act)
    return case


# ---------------------------------------------------------- the 4-bit weights

def _groups(k, group):
    return (k + group - 1) // group


def _grouped(x, group):
    """[rows, groups, group], the last group filled with zeros."""
    rows, k = x.shape
    return torch.nn.functional.pad(x, (0, -k % group)).view(rows, -1, group)


def _quantized(x, group, scale, zeros):
    """Codes [rows, k] (whole numbers), scales and zero points [rows, groups] of the matrix x.  The quotients
    in 64 bits: in 32, one next to a half-way value may be rounded onto it."""
    rows, k = x.shape
    x = _grouped(x, group)
    top = x.amax(dim=2).clamp(min=0).double()
    low = x.amin(dim=2).clamp(max=0).double()
    s = (top - low) / 15 if zeros else torch.maximum(top / 7, -low / 8)
    s = s.float().to(scale)
    s64 = s.double().masked_fill(s == 0, 1.0)
    z = torch.round(-low / s64).clamp(0, 15) if zeros else torch.full_like(low, 8)
    q = torch.empty(rows, x.shape[1] * group, dtype=torch.uint8, device=x.device)
    step = max(1, (1 << 26) // (x.shape[1] * group))
    for r in range(0, rows, step):  # the 64-bit quotients of some rows at a time
        y = torch.round(x[r:r + step].double() / s64[r:r + step].unsqueeze(2)) + z[r:r + step].unsqueeze(2)
        q[r:r + step] = y.clamp(0, 15).flatten(1).to(torch.uint8)
    return q[:, :k], s, z.to(torch.uint8)


def _pack(q):
    """Codes in the stored layout."""
    q = torch.nn.functional.pad(q, (0, -q.shape[1] % 32))
    return (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()


def _weight(w, case):
    """A packed weight as a caller holds it: codes, scales, and zero points or None."""
    q, s, z = _quantized(w, case["group"], DTYPES[case["scale"]], case["zeros"])
    return _pack(q), s, (z if case["zeros"] else None)


def _values(weight, k, group):
    """The fp32 values of a packed weight, [rows, k]."""
    codes, s, z = weight
    q = torch.stack((codes & 15, codes >> 4), dim=2).flatten(1)[:, :k].float()
    z = torch.full_like(s, 8.0, dtype=torch.float32) if z is None else z.float()
    s, z = (t.float().repeat_interleave(group, dim=1)[:, :k] for t in (s, z))
    return s * (q - z)


# -------------------------------------------------------------- what is held

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _activations(gen, rows, k):
    """Normal values, a few channels much larger than the rest."""
    return _normal(gen, rows, k) * torch.exp(0.8 * _normal(gen, 1, k))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    state = dict(case=case)
    if op == "pack":
        x = 0.02 * _activations(gen, case["rows"], case["cols"])
        state["X"] = x.to(DTYPES[case["dtype"]])
        nb, ng = (case["cols"] + 31) // 32, _groups(case["cols"], case["group"])
        state["Q"] = torch.empty(case["rows"], 16 * nb, dtype=torch.uint8, device="cuda")
        state["S"] = torch.empty(case["rows"], ng, dtype=DTYPES[case["scale"]], device="cuda")
        state["Z"] = torch.empty(case["rows"], ng, dtype=torch.uint8, device="cuda") if case["zeros"] else None
        state["Y"] = torch.empty(case["rows"], case["cols"], dtype=DTYPES[case["out"]], device="cuda")
        return state
    dtype = DTYPES[case["dtype"]]
    M, N, K = case["M"], case["N"], case["K"]

    def out(*shape, dtype=dtype):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if op == "grad":
        state["dY"] = _activations(gen, M, K).to(dtype)
        state["Wd"] = (_normal(gen, K, N) / math.sqrt(K)).to(dtype)
        state["G"] = _normal(gen, M, N).to(dtype)
        state["U"] = _normal(gen, M, N).to(dtype)
        state["dG"], state["dU"], state["H"] = out(M, N), out(M, N), out(M, N)
        state["dbias"] = [out(N, dtype=torch.float32) for _ in range(2)] if case["bias"] else [None, None]
        return state
    state["X"] = _activations(gen, M, K).to(dtype)
    state["bias"] = [_normal(gen, N), _normal(gen, N)] if case["bias"] else [None, None]
    if op == "gated":
        state["W"] = [(_normal(gen, N, K) / math.sqrt(K)).to(dtype) for _ in range(2)]
        state["H"] = out(M, N)
        state["G"], state["U"] = (out(M, N), out(M, N)) if case["save"] else (None, None)
    elif op == "w4":
        state["W"] = _weight(_normal(gen, N, K) / math.sqrt(K), case)
        state["C0"] = _normal(gen, M, N) if case["beta"] else None
        state["C"] = out(M, N, dtype=torch.float32)
    else:  # the gate's rows, then the other projection's
        state["W"] = _weight(_normal(gen, 2 * N, K) / math.sqrt(K), case)
        state["H"] = out(M, N)
    return state


# ------------------------------------------------------------------ one pass

def _sigmoid(x):
    t = torch.exp(-x.abs())
    return torch.where(x >= 0, 1 / (1 + t), t / (1 + t))


def _act(x, name):
    if name == "silu":
        return x * _sigmoid(x)
    if name == "gelu":
        return 0.5 * x * torch.erfc(-x * math.sqrt(0.5))
    if name == "gelu_tanh":
        return x * _sigmoid(2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x))
    if name == "relu":
        return x.clamp(min=0)
    return _sigmoid(x) if name == "sigmoid" else x


def _act_grad(x, name):
    if name == "silu":
        return _sigmoid(x) * (1 + x * _sigmoid(-x))
    if name == "gelu":
        return 0.5 * torch.erfc(-x * math.sqrt(0.5)) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        y = c * (x + 0.044715 * x * x * x)
        return _sigmoid(y) * (1 + x * _sigmoid(-y) * c * (1 + 3 * 0.044715 * x * x))
    if name == "relu":
        return (x > 0).to(x.dtype)
    return _sigmoid(x) * _sigmoid(-x) if name == "sigmoid" else torch.ones_like(x)


def _plain_gated(x, wg, wu, bias, act):
    g, u = x @ wg.t(), x @ wu.t()
    if bias[0] is not None:
        g, u = g + bias[0], u + bias[1]
    return _act(g, act) * u, g, u


def _run_own(state, case, op):
    import dense_gemm_tuning_amd as dgt

    if op == "gated":
        dgt.check(dgt.gated(state["X"], *state["W"], state["H"], act=case["act"], bias_g=state["bias"][0],
                            bias_u=state["bias"][1], G=state["G"], U=state["U"]))
        return [state["H"], state["G"], state["U"]] if case["save"] else state["H"]
    if op == "grad":
        dgt.check(dgt.gated_grad(state["dY"], state["Wd"], state["G"], state["U"], state["dG"], state["dU"],
                                 act=case["act"], H=state["H"], dbias_g=state["dbias"][0],
                                 dbias_u=state["dbias"][1]))
        return [state["dG"], state["dU"], state["H"]] + (state["dbias"] if case["bias"] else [])
    if op == "pack":
        dgt.check(dgt.quantize_w4(state["X"], state["Q"], state["S"], state["Z"], group=case["group"]))
        dgt.check(dgt.dequantize_w4(state["Q"], state["S"], state["Z"], state["Y"], group=case["group"]))
        return state["Y"]
    if op == "w4":
        if case["beta"]:
            state["C"].copy_(state["C0"])
        dgt.check(dgt.gemm_w4(state["X"], *state["W"], state["C"], group=case["group"], alpha=case["alpha"],
                              beta=case["beta"], bias=state["bias"][0]))
        return state["C"]
    dgt.check(dgt.gated_w4(state["X"], *state["W"], state["H"], act=case["act"], group=case["group"],
                           bias_g=state["bias"][0], bias_u=state["bias"][1]))
    return state["H"]


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _run_own(state, case, op)
    if op == "pack":
        weight = _weight(state["X"].float(), case)
        return _values(weight, case["cols"], case["group"]).to(DTYPES[case["out"]])
    dtype = DTYPES[case["dtype"]]
    if op == "grad":
        dh = state["dY"].float() @ state["Wd"].float()
        g, u = state["G"].float(), state["U"].float()
        a = _act(g, case["act"])
        dg, du = dh * u * _act_grad(g, case["act"]), dh * a
        sums = [t.sum(dim=0) for t in (dg, du)] if case["bias"] else []
        return [t.to(dtype) for t in (dg, du, a * u)] + sums
    x = state["X"].float()
    if op == "gated":
        outs = _plain_gated(x, state["W"][0].float(), state["W"][1].float(), state["bias"], case["act"])
        return [t.to(dtype) for t in outs] if case["save"] else outs[0].to(dtype)
    w = _values(state["W"], case["K"], case["group"])
    if op == "w4":
        c = case["alpha"] * (x @ w.t())
        if case["beta"]:
            c = c + case["beta"] * state["C0"]
        return c if state["bias"][0] is None else c + state["bias"][0]
    N = case["N"]
    return _plain_gated(x, w[:N], w[N:], state["bias"], case["act"])[0].to(dtype)


# ------------------------------------------------------------------ the work

def _weight_bytes(case, rows, k):
    return rows * (16 * ((k + 31) // 32) + _groups(k, case["group"]) * (3 if case["zeros"] else 2))


def work(case):
    op = case["op"]
    if op == "pack":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (ELEM_BYTES[case["dtype"]] + ELEM_BYTES[case["out"]]) +
                2 * _weight_bytes(case, case["rows"], case["cols"]), "flops": 6 * n}
    M, N, K = case["M"], case["N"], case["K"]
    if op == "gated":
        return {"bytes": 2 * (M * K + 2 * N * K + M * N * (3 if case["save"] else 1)) + (8 * N if case["bias"] else 0),
                "flops": 4 * M * N * K}
    if op == "grad":
        return {"bytes": 2 * (M * K + N * K + 5 * M * N) + (8 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    if op == "w4":
        return {"bytes": 2 * M * K + _weight_bytes(case, N, K) + 4 * M * N * (2 if case["beta"] else 1) +
                (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    return {"bytes": 2 * M * K + _weight_bytes(case, 2 * N, K) + 2 * M * N + (8 * N if case["bias"] else 0),
            "flops": 4 * M * N * K}


# ------------------------------------------------------- the definition, 64 bits

def _exact_act(x, name):
    """The activation and its derivative, from the definitions."""
    x = x.detach().requires_grad_(True)
    with torch.enable_grad():
        if name in ("silu", "sigmoid"):
            y = torch.special.expit(x) * (x if name == "silu" else 1)
        elif name == "gelu":  # x P(normal < x)
            y = x * torch.special.ndtr(x)
        elif name == "gelu_tanh":
            y = 0.5 * x * (1 + torch.tanh((2 / math.pi) ** 0.5 * (x + 0.044715 * x ** 3)))
        else:
            y = torch.relu(x) if name == "relu" else x * 1
        slope, = torch.autograd.grad(y.sum(), x)
    return y.detach(), slope


def _exact_pack(case, x):
    """The stored values, a group at a time from their definition."""
    rows, k, group = x.shape[0], case["cols"], case["group"]
    out = torch.empty(rows, k, dtype=torch.float64, device=x.device)
    for k0 in range(0, k, group):
        part = x[:, k0:k0 + group].double()
        hi = torch.relu(part.max(dim=1, keepdim=True).values)
        lo = torch.relu(-part.min(dim=1, keepdim=True).values)
        s = (hi + lo) / 15 if case["zeros"] else torch.where(hi * 8 > lo * 7, hi / 7, lo / 8)
        s = s.float().to(DTYPES[case["scale"]]).double()
        unit = torch.where(s > 0, s, 1.0)
        z = torch.minimum(torch.round(lo / unit), torch.tensor(15.0, device=x.device)) if case["zeros"] else 8.0
        q = torch.minimum(torch.relu(torch.round(part / unit) + z), torch.tensor(15.0, device=x.device))
        out[:, k0:k0 + group] = s * (q - z)
    return out


def _exact_weight(weight, case):
    codes, s, z = weight
    low = codes % 16
    q = torch.cat((low.unsqueeze(2), ((codes - low) // 16).unsqueeze(2)), dim=2).reshape(codes.shape[0], -1).double()
    at = torch.arange(case["K"], device=codes.device) // case["group"]
    zero = 8.0 if z is None else z.double()[:, at]
    return s.double()[:, at] * (q[:, :case["K"]] - zero)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "pack":
        return _exact_pack(case, state["X"])
    if op == "grad":
        dh = torch.mm(state["dY"].double(), state["Wd"].double())
        y, slope = _exact_act(state["G"].double(), case["act"])
        u = state["U"].double()
        dg, du = dh * slope * u, dh * y
        ones = torch.ones(1, case["M"], dtype=torch.float64, device=dh.device)
        sums = [torch.mm(ones, t)[0] for t in (dg, du)] if case["bias"] else []
        return [dg, du, y * u] + sums
    x = state["X"].double()
    bias = [0.0 if b is None else b.double() for b in state["bias"]]
    if op == "w4":
        c = case["alpha"] * torch.mm(x, _exact_weight(state["W"], case).t().contiguous()) + bias[0]
        return c if state["C0"] is None else c + case["beta"] * state["C0"].double()
    if op == "gated":
        w = [t.double().t().contiguous() for t in state["W"]]
    else:
        both = _exact_weight(state["W"], case)
        w = [both[:case["N"]].t().contiguous(), both[case["N"]:].t().contiguous()]
    g, u = (torch.mm(x, t) + b for t, b in zip(w, bias))
    h = _exact_act(g, case["act"])[0] * u
    return [h, g, u] if op == "gated" and case["save"] else h
