"""Cases for the 8-bit integer operators of served linear layers: what is timed, on which inputs, and the plain forms.

Four kinds of case, each one pass through an operator as a served gated block calls them, in this order:

  norm     the residual's addition s = x + r and its root-mean-square norm s / sqrt(mean(s^2) + eps) * w, in 8 bits;
  gated    h = act(x Wg^T) * (x Wu^T) from x and both weights in 8 bits;
  store    h's rows in 8 bits;
  matmul   y = x W^T from both in 8 bits, in float32 or bfloat16, or the integer sums themselves.

The 8-bit form: integers -127 .. 127 and one float32 scale a row, value = code * scale: a row of activations is a
token, a row of weights an output channel.  With a = max(largest magnitude of the row, 2^-100), code =
round(x * (127 / a)), ties to even, and scale = a / 127, each operation rounded to float32.  The norm's factor is the
same for a whole row: it enters the scale and cancels in the codes, which are those of s * w.
"""

import torch

own = False

LEAST = 2.0 ** -100
TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "int32": torch.int32}


def listed():
    return [
        # one token's gated product on its way to the down projection
        {"name": "store 1x8192 bf16", "kind": "store", "type": "bfloat16", "T": 1, "D": 8192},
        # a large batch of prompts, or a weight matrix
        {"name": "store 8192x8192 f32", "kind": "store", "type": "float32", "T": 8192, "D": 8192},
        # one token before a block
        {"name": "norm 1x4096 bf16", "kind": "norm", "type": "bfloat16", "T": 1, "D": 4096, "residual": True},
        # odd width: rows that start off every vector boundary
        {"name": "norm 1000x1023 f32", "kind": "norm", "type": "float32", "T": 1000, "D": 1023, "residual": True},
        # a large batch of prompts
        {"name": "norm 8192x8192 bf16", "kind": "norm", "type": "bfloat16", "T": 8192, "D": 8192, "residual": True},
        # one token through an ordinary layer: reads the weights
        {"name": "matmul 1x4096x4096 bf16", "kind": "matmul", "type": "bfloat16", "T": 1, "N": 4096, "K": 4096},
        # a batch of sequences, a token each, through a large layer
        {"name": "matmul 24x8192x8192 bf16", "kind": "matmul", "type": "bfloat16", "T": 24, "N": 8192, "K": 8192},
        # a short prompt, odd in every direction
        {"name": "matmul 1000x1023x1025 f32", "kind": "matmul", "type": "float32", "T": 1000, "N": 1023, "K": 1025},
        # a large batch of prompts through a large layer
        {"name": "matmul 8192x8192x8192 bf16", "kind": "matmul", "type": "bfloat16", "T": 8192, "N": 8192, "K": 8192},
        # one token through both projections of a gated block
        {"name": "gated 1x8192x2048 bf16", "kind": "gated", "type": "bfloat16", "act": "silu", "T": 1, "N": 8192,
         "K": 2048},
        # a short prompt, odd in every direction
        {"name": "gated 1000x1023x1025 f32", "kind": "gated", "type": "float32", "act": "gelu", "T": 1000, "N": 1023,
         "K": 1025},
        # a large batch of prompts
        {"name": "gated 8192x8192x4096 bf16", "kind": "gated", "type": "bfloat16", "act": "silu", "T": 8192,
         "N": 8192, "K": 4096},
    ]


def _spread(rng, low, high):
    """A whole number spread over the logarithm of low .. high: as often a size that layers have (4, 5 or 7 times a
    power of two) as an odd one."""
    n = low * (high / low) ** rng.random()
    if n >= 64 and rng.random() < 0.5:
        k = 1
        while 8 * k <= n:
            k *= 2
        n = k * min((4, 5, 7), key=lambda m: abs(m * k - n))
    else:
        n = int(n) | 1
    return max(low, min(high, n))


def draw(rng):
    kind = rng.choice(["store", "norm", "matmul", "matmul", "gated", "gated"])
    while True:
        if kind in ("store", "norm"):
            c = {"kind": kind, "type": rng.choice(["float32", "bfloat16"]), "T": _spread(rng, 1, 16384),
                 "D": _spread(rng, 32, 16384)}
            if kind == "norm":
                c["residual"] = rng.random() < 0.75
            if c["T"] * c["D"] <= 8192 * 8192:
                return c
        else:
            # as often a few tokens as a prompt
            c = {"kind": kind, "type": rng.choice(["float32", "bfloat16"]),
                 "T": _spread(rng, 1, 64) if rng.random() < 0.5 else _spread(rng, 64, 8192),
                 "N": _spread(rng, 32, 16384), "K": _spread(rng, 32, 16384)}
            products = c["T"] * c["N"] * c["K"]
            if kind == "gated":
                c["act"] = rng.choice(["silu", "gelu"])
                products *= 2
            elif products <= 2048 ** 3 and rng.random() < 0.25:
                c["type"] = "int32"
            if products <= 8192 ** 3 and c["N"] * c["K"] <= 8192 * 8192:
                return c


# ---- the 8-bit form in elementary torch operations ---------------------------------------------------------------


def _codes_plain(z):
    """Codes as float32 whole numbers, and the largest magnitudes they were scaled by, of the rows of z."""
    a = z.abs().amax(dim=1).clamp(min=LEAST)
    return (z * (torch.full_like(a, 127.0) / a)[:, None]).round(), a


def _store_plain(x):
    codes, a = _codes_plain(x.float())
    return codes, a / torch.full_like(a, 127.0)


def _bytes(codes):
    """Codes as an int8 matrix whose rows are padded to 16 bytes."""
    T, D = codes.shape
    c = torch.zeros((T, -(-D // 16) * 16), dtype=torch.int8, device=codes.device)
    c[:, :D] = codes
    return c


def _act_plain(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z * (0.5 * (1.0 + torch.erf(z * 0.7071067811865476)))


# ---- cases -------------------------------------------------------------------------------------------------------


def _activations(gen, T, D):
    """Values as a layer sees them: features of different sizes, tokens of different sizes, some outliers."""
    dev = "cuda"
    x = torch.randn((T, D), generator=gen, device=dev)
    x *= torch.exp(0.5 * torch.randn((1, D), generator=gen, device=dev))
    x *= torch.exp(0.3 * torch.randn((T, 1), generator=gen, device=dev))
    loud = torch.randint(0, D, (max(1, D // 128),), generator=gen, device=dev)
    x[:, loud] *= 8.0
    return x


def _weights(gen, N, K):
    w = torch.randn((N, K), generator=gen, device="cuda")
    w *= torch.exp(0.3 * torch.randn((N, 1), generator=gen, device="cuda")) / K ** 0.5
    return w


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = dict(case)
    T = case["T"]
    if case["kind"] in ("store", "norm"):
        D, dtype = case["D"], TYPES[case["type"]]
        s["x"] = _activations(gen, T, D).to(dtype)
        if case["kind"] == "norm":
            s["r"] = (2.0 * _activations(gen, T, D)).to(dtype) if case["residual"] else None
            s["w"] = (1.0 + 0.2 * torch.randn((D,), generator=gen, device="cuda")).to(dtype)
            s["eps"] = 1e-6
        return s
    N, K = case["N"], case["K"]
    codes, s["xs"] = _store_plain(_activations(gen, T, K))
    s["x"] = _bytes(codes)
    for name in ("w", "v") if case["kind"] == "gated" else ("w",):
        codes, s[name + "s"] = _store_plain(_weights(gen, N, K))
        s[name] = _bytes(codes)
    return s


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import dense_fp32_gemm_row_gb300 as g

    if s["kind"] == "store":
        q = g.i8_store(s["x"])
        return {"codes": q.codes[:, : s["D"]], "scales": q.scales}
    if s["kind"] == "norm":
        q, total = g.i8_norm(s["x"], s["w"], residual=s["r"], eps=s["eps"])
        return {"codes": q.codes[:, : s["D"]], "scales": q.scales, "total": total}
    x, w = g.I8(s["x"], s["xs"], s["K"]), g.I8(s["w"], s["ws"], s["K"])
    if s["kind"] == "matmul":
        return g.i8_matmul(x, w, dtype=TYPES[s["type"]])
    return g.i8_gated(x, w, g.I8(s["v"], s["vs"], s["K"]), act=s["act"], dtype=TYPES[s["type"]])


def _run_plain(s):
    if s["kind"] == "store":
        codes, scales = _store_plain(s["x"])
        return {"codes": codes.to(torch.int8), "scales": scales}
    if s["kind"] == "norm":
        total = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
        codes, a = _codes_plain(total * s["w"].float())
        rho = 1.0 / torch.sqrt(total.square().mean(dim=1) + s["eps"])
        return {"codes": codes.to(torch.int8), "scales": a / torch.full_like(a, 127.0) * rho,
                "total": None if s["r"] is None else total.to(s["x"].dtype)}
    K = s["K"]
    if s["type"] == "int32":
        # sums beyond 2^24
        return (s["x"][:, :K].double() @ s["w"][:, :K].double().t()).to(torch.int32)
    x = s["x"][:, :K].float()
    y = x @ s["w"][:, :K].float().t() * s["xs"][:, None] * s["ws"]
    if s["kind"] == "gated":
        y = _act_plain(y, s["act"]) * (x @ s["v"][:, :K].float().t() * s["xs"][:, None] * s["vs"])
    return y.to(TYPES[s["type"]])


def work(case):
    T = case["T"]
    size = 2 if case["type"] == "bfloat16" else 4
    if case["kind"] == "store":
        D = case["D"]
        return {"bytes": size * T * D + T * D + 4 * T, "flops": 3 * T * D}
    if case["kind"] == "norm":
        D = case["D"]
        moved = 3 if case["residual"] else 1
        return {"bytes": moved * size * T * D + size * D + T * D + 4 * T, "flops": 7 * T * D}
    N, K = case["N"], case["K"]
    layers = 2 if case["kind"] == "gated" else 1
    return {"bytes": T * K + layers * N * K + 4 * T + 4 * layers * N + size * T * N, "flops": 2 * layers * T * N * K}


# ---- the same from the definitions, in 64 bits -------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] in ("store", "norm"):
        x = s["x"].double()
        if case["kind"] == "norm":
            total = x + s["r"].double() if case["residual"] else x
            y = total * s["w"].double() * torch.rsqrt((total * total).mean(dim=1, keepdim=True) + s["eps"])
        else:
            y = x
        # no value for the codes: rounding to 8 bits turns a difference in the last place into a whole step
        out = {"codes": None, "scales": torch.amax(torch.abs(y), dim=1) / 127}
        if case["kind"] == "norm":
            out["total"] = total if case["residual"] else None
        return out
    K = case["K"]

    def values(codes, scales):
        return codes[:, :K].double() * scales.double().unsqueeze(1)

    if case["type"] == "int32":
        return s["x"][:, :K].double().mm(s["w"][:, :K].double().T).long().to(torch.int32)
    x = values(s["x"], s["xs"])
    y = torch.mm(x, values(s["w"], s["ws"]).T)
    if case["kind"] == "matmul":
        return y
    gate = y * torch.special.expit(y) if case["act"] == "silu" else y * torch.special.ndtr(y)
    return gate * torch.mm(x, values(s["v"], s["vs"]).T)
