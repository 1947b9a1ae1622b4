"""Cases for the 8-bit activation checkpoint operators: what is timed, on which inputs, and the plain forms.

Three kinds of case, each one pass through the operators as a training step calls them:

  checkpoint   a layer's input X (tokens x features, float32) stored in 8 bits, and restored;
  gated        a gated unit h = act(gate) * up: the forward pass, which keeps gate and up in 8 bits,
               then the backward pass from those and dh (dgate, dup, and h recomputed, in 8 bits again);
  wgrad        the weight gradient dW = X^T dY of a linear layer from X's 8-bit checkpoint.

The 8-bit form: blocks of 32 consecutive columns of a row share a power-of-two scale, one exponent byte E a
block.  int8: value = code * 2^(E - 133); e4m3: value = e4m3(code) * 2^(E - 127); E is the smallest at which the
block's largest magnitude needs no saturation.  Every such value is exactly a bfloat16 number.
"""

import torch

own = False

BLOCK = 32


def listed():
    return [
        # a layer input of a short fine-tuning sequence; the width is no multiple of the block
        {"name": "checkpoint 37x1000 int8", "kind": "checkpoint", "format": "int8", "T": 37, "D": 1000},
        # ragged in both directions, rows that start off every vector boundary
        {"name": "checkpoint 1025x1023 e4m3", "kind": "checkpoint", "format": "e4m3", "T": 1025, "D": 1023},
        # a large layer's input over a full batch
        {"name": "checkpoint 8192x8192 int8", "kind": "checkpoint", "format": "int8", "T": 8192, "D": 8192},
        # one short sequence through a small gated unit: launches count
        {"name": "gated 128x1024 int8", "kind": "gated", "format": "int8", "act": "silu", "T": 128, "F": 1024},
        # odd width: gate and up are the halves of one product, so up starts unaligned
        {"name": "gated 1000x1023 int8", "kind": "gated", "format": "int8", "act": "gelu", "T": 1000, "F": 1023},
        # an ordinary micro-batch
        {"name": "gated 4096x2048 e4m3", "kind": "gated", "format": "e4m3", "act": "gelu", "T": 4096, "F": 2048},
        # the large gated unit over a full batch
        {"name": "gated 8192x8192 int8", "kind": "gated", "format": "int8", "act": "silu", "T": 8192, "F": 8192},
        # weight gradient of one short sequence
        {"name": "wgrad 64x512x512 int8", "kind": "wgrad", "format": "int8", "T": 64, "D": 512, "N": 512},
        # odd in every direction: rows of dY no TMA load can start on
        {"name": "wgrad 1000x1025x1023 e4m3", "kind": "wgrad", "format": "e4m3", "T": 1000, "D": 1025, "N": 1023},
        # a long batch through a small layer: the sum over tokens is the long axis
        {"name": "wgrad 65536x256x256 int8", "kind": "wgrad", "format": "int8", "T": 65536, "D": 256, "N": 256},
        # an ordinary layer and micro-batch
        {"name": "wgrad 4096x2048x2048 e4m3", "kind": "wgrad", "format": "e4m3", "T": 4096, "D": 2048, "N": 2048},
        # the large layer over a full batch
        {"name": "wgrad 8192x8192x8192 int8", "kind": "wgrad", "format": "int8", "T": 8192, "D": 8192, "N": 8192},
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
    kind = rng.choice(["checkpoint", "gated", "wgrad", "wgrad"])
    fmt = rng.choice(["int8", "e4m3"])
    while True:
        if kind == "wgrad":
            c = {"kind": kind, "format": fmt, "T": _spread(rng, 1, 65536), "D": _spread(rng, 32, 8192),
                 "N": _spread(rng, 32, 8192)}
            if c["T"] * c["D"] * c["N"] <= 8192 ** 3 and c["T"] * max(c["D"], c["N"]) <= 8192 * 8192:
                return c
        elif kind == "gated":
            c = {"kind": kind, "format": fmt, "act": rng.choice(["silu", "gelu"]), "T": _spread(rng, 1, 16384),
                 "F": _spread(rng, 32, 16384)}
            if c["T"] * c["F"] <= 8192 * 8192:
                return c
        else:
            c = {"kind": kind, "format": fmt, "T": _spread(rng, 1, 16384), "D": _spread(rng, 32, 16384)}
            if c["T"] * c["D"] <= 8192 * 8192:
                return c


# ---- the 8-bit form in elementary torch operations -------------------------------------------------------------


def _pow2(field):
    """2^(field - 127) as float32, for exponent fields 1 .. 254."""
    return (field << 23).view(torch.float32)


def _store_plain(x, fmt):
    """codes (int32 code values, or e4m3 numbers in float32) and exponent bytes of x, per block of 32 columns."""
    T, D = x.shape
    nb = -(-D // BLOCK)
    xb = torch.nn.functional.pad(x, (0, nb * BLOCK - D)).view(T, nb, BLOCK)
    bits = xb.abs().amax(dim=2).view(torch.int32)
    if fmt == "int8":
        E = ((bits + 0x1FFFF) >> 23).clamp(7, 254)
        codes = (xb * _pow2(260 - E)[:, :, None]).round().clamp(-127, 127)
    else:
        E = (((bits + 0x1FFFFF) >> 23) - 8).clamp(10, 247)
        codes = (xb * _pow2(254 - E)[:, :, None]).to(torch.float8_e4m3fn)
    return codes, E


def _values_plain(codes, E, fmt, D):
    """The float32 values that codes stand for."""
    v = codes.to(torch.float32) * _pow2(E - 6 if fmt == "int8" else E)[:, :, None]
    return v.view(v.shape[0], -1)[:, :D]


def _bytes(codes, E, fmt, D):
    """The same as the two byte tensors that a checkpoint holds: code rows and exponent rows, each padded to 16 bytes."""
    T = codes.shape[0]
    flat = (codes.to(torch.int8) if fmt == "int8" else codes).view(torch.uint8).view(T, -1)
    c = torch.zeros((T, -(-D // 16) * 16), dtype=torch.uint8, device=codes.device)
    c[:, :D] = flat[:, :D]
    e = torch.zeros((T, -(-E.shape[1] // 16) * 16), dtype=torch.uint8, device=codes.device)
    e[:, : E.shape[1]] = E.to(torch.uint8)
    return c, e


def _from_bytes(c, e, fmt, D):
    T, nb = c.shape[0], -(-D // BLOCK)
    pad = torch.nn.functional.pad(c[:, :D], (0, nb * BLOCK - D)).view(T, nb, BLOCK)
    codes = pad.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn)
    return _values_plain(codes, e[:, :nb].to(torch.int32), fmt, D)


def _act_plain(z, act):
    """act(z) and its derivative."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return z * s, s * (1.0 + z * (1.0 - s))
    cdf = 0.5 * (1.0 + torch.erf(z * 0.7071067811865476))
    return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * 0.3989422804014327


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = dict(case)
    T = case["T"]
    if case["kind"] == "checkpoint":
        s["x"] = _activations(gen, T, case["D"])
    elif case["kind"] == "gated":
        # the halves of the one product that gives gate and up
        both = torch.randn((T, 2 * case["F"]), generator=gen, device="cuda")
        both *= 1.5
        s["gate"], s["up"] = both[:, : case["F"]], both[:, case["F"] :]
        s["dh"] = 1e-3 * torch.randn((T, case["F"]), generator=gen, device="cuda")
    else:
        codes, E = _store_plain(_activations(gen, T, case["D"]), case["format"])
        s["codes"], s["scales"] = _bytes(codes, E, case["format"], case["D"])
        s["dy"] = 1e-3 * torch.randn((T, case["N"]), generator=gen, device="cuda")
        s["dy"] *= torch.exp(0.5 * torch.randn((T, 1), generator=gen, device="cuda"))
    return s


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import dense_fp32_gemm_row_gb300 as g

    if s["kind"] == "checkpoint":
        return g.q8_restore(g.q8_store(s["x"], format=s["format"]))
    if s["kind"] == "gated":
        h, gate_q, up_q = g.q8_gated(s["gate"], s["up"], act=s["act"], format=s["format"])
        dgate, dup, h_q = g.q8_gated_backward(gate_q, up_q, s["dh"], act=s["act"])
        return {"h": h, "dgate": dgate, "dup": dup, "h_q": g.q8_restore(h_q, dtype=torch.bfloat16)}
    return g.q8_wgrad(g.Q8(s["codes"], s["scales"], s["D"], s["format"]), s["dy"])


def _run_plain(s):
    fmt = s["format"]
    if s["kind"] == "checkpoint":
        return _values_plain(*_store_plain(s["x"], fmt), fmt, s["D"])
    if s["kind"] == "gated":
        F = s["F"]
        h = _act_plain(s["gate"], s["act"])[0] * s["up"]
        gate = _values_plain(*_store_plain(s["gate"], fmt), fmt, F)
        up = _values_plain(*_store_plain(s["up"], fmt), fmt, F)
        a, da = _act_plain(gate, s["act"])
        h_q = _values_plain(*_store_plain(a * up, fmt), fmt, F)
        return {"h": h, "dgate": s["dh"] * up * da, "dup": s["dh"] * a, "h_q": h_q.to(torch.bfloat16)}
    return _from_bytes(s["codes"], s["scales"], fmt, s["D"]).t() @ s["dy"]


def work(case):
    T = case["T"]
    if case["kind"] == "checkpoint":
        D = case["D"]
        held = T * (D + -(-D // BLOCK))
        return {"bytes": 8 * T * D + 2 * held, "flops": 4 * T * D}
    if case["kind"] == "gated":
        F = case["F"]
        held = T * (F + -(-F // BLOCK))
        # forward: gate, up -> h and two checkpoints; backward: those, dh -> dgate, dup and a third; its values in 16 bits
        return {"bytes": 12 * T * F + 2 * held + 2 * held + 12 * T * F + held + held + 2 * T * F, "flops": 40 * T * F}
    D, N = case["D"], case["N"]
    return {"bytes": T * (D + -(-D // BLOCK)) + 4 * T * N + 4 * D * N, "flops": 2 * T * D * N}


# ---- the same from the definitions, in 64 bits ---------------------------------------------------------------------


def _values_exact(x, fmt):
    """The values x's 8-bit form stands for, from the definition: float64 throughout, exponents by frexp."""
    T, D = x.shape
    nb = -(-D // BLOCK)
    xb = torch.zeros((T, nb * BLOCK), dtype=torch.float64, device=x.device)
    xb[:, :D] = x
    xb = xb.view(T, nb, BLOCK)
    top = xb.abs().amax(dim=2, keepdim=True)
    most, least = (127.0, -126.0) if fmt == "int8" else (448.0, -117.0)
    # the smallest e with top <= most * 2^e
    e = torch.frexp(top / most)[1].to(torch.float64)
    e = torch.where(top <= most * torch.exp2(e - 1.0), e - 1.0, e)
    e = torch.where(top > 0, e, torch.full_like(e, least)).clamp(min=least)
    z = xb / torch.exp2(e)
    if fmt == "int8":
        q = torch.round(z)
    else:
        # four significant bits, down to steps of 2^-9
        step = torch.exp2((torch.frexp(z)[1].to(torch.float64) - 4.0).clamp(min=-9.0))
        q = torch.round(z / step) * step
    return (q * torch.exp2(e)).view(T, -1)[:, :D]


def exact(case, seed):
    s = prepare(case, seed)
    fmt = case["format"]
    if case["kind"] == "checkpoint":
        return _values_exact(s["x"], fmt)
    if case["kind"] == "gated":

        def act(z):
            if case["act"] == "silu":
                p = torch.special.expit(z)
                return z * p, p + z * p * torch.special.expit(-z)
            p = torch.special.ndtr(z)
            return z * p, p + z * torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5

        h = act(s["gate"].double())[0] * s["up"].double()
        gate, up = _values_exact(s["gate"], fmt), _values_exact(s["up"], fmt)
        a, da = act(gate)
        dh = s["dh"].double()
        # no value for h_q: its rounding to 8 bits turns a difference in the last place into a whole step
        return {"h": h, "dgate": dh * up * da, "dup": dh * a, "h_q": None}
    D, nb = case["D"], -(-case["D"] // BLOCK)
    c = s["codes"][:, :D].view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).double()
    scale = torch.exp2(s["scales"][:, :nb].double() - (133.0 if fmt == "int8" else 127.0))
    x = c * scale.repeat_interleave(BLOCK, dim=1)[:, :D]
    return x.t() @ s["dy"].double()
