"""Plain 64-bit forms of the 8-bit checkpoint operators, written from the
format's definition in numpy, for the parity tests."""

from __future__ import annotations

import numpy as np

BLOCK = 32
FORMATS = ("int8", "e4m3")


def _e4m3_table() -> np.ndarray:
    """The 256 numbers of an e4m3 code byte (NaN for 0x7F and 0xFF)."""
    v = np.empty(256)
    for b in range(256):
        exp, man = (b >> 3) & 15, b & 7
        mag = man * 2.0 ** -9 if exp == 0 else (1 + man / 8) * 2.0 ** (exp - 7)
        v[b] = np.nan if (b & 127) == 127 else mag
        if b & 128:
            v[b] = -v[b]
    return v


E4M3 = _e4m3_table()


def _round_e4m3(z: np.ndarray) -> np.ndarray:
    """Code bytes of the e4m3 numbers nearest to z (ties to the even code), |z| <= 448."""
    mags = E4M3[:127]
    hi = np.clip(np.searchsorted(mags, np.abs(z)), 0, 126)
    lo = np.maximum(hi - 1, 0)
    below, above = np.abs(z) - mags[lo], mags[hi] - np.abs(z)
    code = np.where(below < above, lo, np.where(below > above, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(mags[hi] == np.abs(z), hi, code)
    return np.where(np.signbit(z), code + 128, code).astype(np.uint8)


def store(x: np.ndarray, fmt: str):
    """(codes, exponents) of x, as uint8: (rows, cols) and (rows, ceil(cols / 32))."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    xb = np.zeros((rows, nb * BLOCK))
    xb[:, :cols] = x
    xb = xb.reshape(rows, nb, BLOCK)
    bad = ~np.isfinite(xb).all(axis=2)
    fin = np.where(bad[:, :, None], 0.0, xb)
    top = np.abs(fin).max(axis=2)
    most = 127.0 if fmt == "int8" else 448.0
    # the smallest e with top <= most 2^e: ceil(log2(top / most)), exactly
    man, ex = np.frexp(top / most)
    e = np.where(man == 0.5, ex - 1, ex)
    e = np.where(top > 0, e, -1000)
    e = np.clip(e, -126, 121) if fmt == "int8" else np.clip(e, -117, 120)
    z = fin / np.exp2(e.astype(np.float64))[:, :, None]
    if fmt == "int8":
        codes = np.clip(np.rint(z), -127, 127).astype(np.int8).view(np.uint8)
    else:
        codes = _round_e4m3(z)
    codes = np.where(bad[:, :, None], 0, codes).astype(np.uint8)
    exps = np.where(bad, 255, e + (133 if fmt == "int8" else 127)).astype(np.uint8)
    return codes.reshape(rows, -1)[:, :cols].copy(), exps


def values(codes: np.ndarray, exps: np.ndarray, fmt: str) -> np.ndarray:
    """What codes and exponents stand for, in 64 bits."""
    cols = codes.shape[1]
    e = exps.astype(np.float64)
    least = 7 if fmt == "int8" else 10
    scale = np.where(e < least, 0.0, np.exp2(e - (133 if fmt == "int8" else 127)))
    scale = np.where(e == 255, np.nan, scale)
    num = codes.view(np.int8).astype(np.float64) if fmt == "int8" else E4M3[codes]
    return num * np.repeat(scale, BLOCK, axis=1)[:, :cols]


def act(z: np.ndarray, name: str):
    """act(z) and act'(z)."""
    from scipy.special import expit, ndtr

    if name == "silu":
        s = expit(z)
        return z * s, s * (1 + z * expit(-z))
    return z * ndtr(z), ndtr(z) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)


def act_bound(z: np.ndarray, name: str):
    """How far fp32 evaluations of act(z) and act'(z) may be from those, from the error bounds of
    the steps (expf 2 ulp, erfcf 4 ulp, half an ulp a rounding; an error of the argument of erfc
    or exp grows by the z^2 of its relative slope), with the smallest normal number for what
    underflows."""
    a, _ = act(z, name)
    s, tiny = 2.0 ** -23, 2.0 ** -126
    if name == "silu":
        from scipy.special import expit

        return 8 * s * np.abs(a) + tiny * (1 + np.abs(z)), \
            8 * s * expit(z) * (1 + np.abs(z)) + tiny * (1 + np.abs(z))
    from scipy.special import ndtr

    phi = np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    grow = (10 + 2 * z * z) * s
    return grow * np.abs(a) + tiny * (1 + np.abs(z)), \
        grow * (ndtr(z) + np.abs(z) * phi) + tiny * (1 + np.abs(z))


def activations(rng, rows: int, cols: int) -> np.ndarray:
    x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((1, cols)))
    return (x * np.exp(0.5 * rng.standard_normal((rows, 1)))).astype(np.float32)
