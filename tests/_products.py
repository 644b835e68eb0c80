"""Plain 64-bit forms of the 8-bit integer operators and the dense gated feed-forward block (numpy
only), written from their definitions, and the error bounds the tests use."""
import math

import numpy as np

SILU, GELU, GELU_TANH, RELU = 0, 1, 2, 3
ACTS = (SILU, GELU, GELU_TANH, RELU)

_erf = np.vectorize(math.erf, otypes=[np.float64])

BF16 = 2.0 ** -8   # half a step of bf16, relative
F32 = 2.0 ** -24   # half a step of fp32


def quantize_rows(x):
    """(codes int8, scales fp32) of the rows of x (values of bf16, given in any float type)."""
    v = np.asarray(x, np.float64)
    amax = np.abs(v).max(axis=1, keepdims=True)
    bad = ~np.isfinite(v).all(axis=1, keepdims=True)
    amax = np.where(bad, 1.0, np.where(amax > 0, np.maximum(amax, 2.0 ** -110), 0.0))
    safe = np.where(amax > 0, amax, 1.0)
    # 127 v is exact in 64 bits, so a quotient that is a tie comes out as one; rint goes to even
    codes = np.rint(np.where(bad, 0.0, 127.0 * np.where(bad, 0.0, v)) / safe)
    scales = np.where(amax > 0, amax.astype(np.float32) / np.float32(127.0), np.float32(1.0))
    scales = np.where(bad, np.float32(np.nan), scales)
    return codes.astype(np.int8), scales[:, 0].astype(np.float32)


def act(a, g):
    g = np.asarray(g, np.float64)
    if a == SILU:
        return g / (1.0 + np.exp(-g))
    if a == GELU:
        return 0.5 * g * (1.0 + _erf(g / math.sqrt(2.0)))
    if a == GELU_TANH:
        return 0.5 * g * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)))
    return np.maximum(g, 0.0)


def act_grad(a, g):
    g = np.asarray(g, np.float64)
    if a == SILU:
        s = 1.0 / (1.0 + np.exp(-g))
        return s + g * s * (1.0 - s)
    if a == GELU:
        return (0.5 * (1.0 + _erf(g / math.sqrt(2.0)))
                + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi))
    if a == GELU_TANH:
        c = math.sqrt(2.0 / math.pi)
        t = np.tanh(c * (g + 0.044715 * g ** 3))
        return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * g * g)
    return (g > 0).astype(np.float64)


def i8_product(offsets, a, sa, b, sb, rows):
    """{row: values} of the grouped product in 64 bits, [rows, N], NaN where no expert writes."""
    E, N, K = b.shape
    out = np.full((rows, N), np.nan)
    for e in range(E):
        lo, hi = (min(max(int(offsets[e + i]), 0), rows) for i in (0, 1))
        if hi > lo:
            s = a[lo:hi].astype(np.int64) @ b[e].astype(np.int64).T
            out[lo:hi] = s * sa[lo:hi, None].astype(np.float64) * sb[e].astype(np.float64)
    return out


def gated_error(g, u, eg, eu):
    """How far fp32's act(g) u may be from the exact one, g and u off by eg and eu: every activation's
    slope is below 1.2 and |act(g)| <= |g|. Of the activation itself, in half steps of fp32 (F32) of
    |g u|: the argument of the exponential loses up to 4 roundings, each of which moves the
    sigmoid by at most |x| s (1 - s) of itself, with the exponential's own argument product 2 |g|
    more; the exponential 2, 1 + e and the quotient 2, erfc (at most 6 units) 12, the products 3:
    below 24 + 8 |g|."""
    return (1.2 * eg * np.abs(u) + np.abs(g) * eu + 1.2 * eg * eu
            + F32 * (24 + 8 * np.abs(g)) * np.abs(g * u))


def ffn_forward(x, w1, w2, a):
    """(h, A, and the sums of magnitudes behind h) in 64 bits; A is not rounded."""
    h = x @ w1.T
    g, u = np.split(h, 2, axis=1)
    return h, act(a, g) * u, np.abs(x) @ np.abs(w1).T


def ffn_backward(x, w1, w2, H, A, dy, a):
    """(dH, dx, dw1, dw2) in 64 bits from the stored H and A; dH is not rounded."""
    g, u = np.split(H, 2, axis=1)
    da = dy @ w2
    dh = np.concatenate([da * u * act_grad(a, g), da * act(a, g)], axis=1)
    return dh, dh @ w1, dh.T @ x, dy.T @ A
