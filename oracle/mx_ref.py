"""fp64 reference of the 4-bit microscaled layers: rounding to e2m1 with a power-of-two scale per
32 inputs, products of such weights, dense and grouped by expert, and the expert layer of few
tokens.  numpy only; no code is shared with the HIP path."""
import numpy as np

BLOCK = 32


def e2m1_values():
    """Value of each of the 16 codes: sign, 2 exponent bits (bias 1), 1 mantissa bit."""
    v = np.empty(16)
    for c in range(16):
        e, m = (c >> 1) & 3, c & 1
        a = m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)
        v[c] = -a if c & 8 else a
    return v


E2M1 = e2m1_values()


def round_e2m1(v):
    """Codes of the values nearest to fp64 v, ties to the even code; |v| <= 6 after rounding."""
    a = np.abs(np.asarray(v, dtype=np.float64))
    pos = E2M1[:8]
    hi = np.searchsorted(pos, a, side="left").clip(0, 7)
    lo = (hi - 1).clip(0)
    up, down = pos[hi] - a, a - pos[lo]
    pick = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    return (np.where(a >= 6, 7, pick) | np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def scale_codes(top, scaling):
    """E8M0 codes of blocks whose largest magnitude is ``top``."""
    top = np.asarray(top, dtype=np.float64)
    with np.errstate(all="ignore"):
        f, e = np.frexp(top)                              # top = f 2^e, f in [1/2, 1)
        e = e - 3 + (f > 0.75 if scaling == "ceil" else 0)   # 4 = 2^2, 6 = 0.75 * 2^3
        e = np.where(top == 0, -126, np.maximum(e, -126))
    return np.where(np.isfinite(top), e + 127, 255).astype(np.uint8)


def scale_values(codes):
    codes = np.asarray(codes)
    return np.where(codes == 255, np.nan, np.ldexp(1.0, codes.astype(np.int64) - 127))


def ref_quantize(x, scaling):
    """x [rows, cols] -> (codes uint8 [rows, cols], scale codes uint8 [rows, cols / 32])."""
    t = np.asarray(x, dtype=np.float64).reshape(x.shape[0], -1, BLOCK)
    fine = np.isfinite(t).all(axis=2)
    s = scale_codes(np.where(fine, np.abs(np.where(np.isfinite(t), t, 0)).max(axis=2), np.inf), scaling)
    v = np.where(fine[:, :, None], t, 0.0) / np.where(fine, scale_values(s), 1.0)[:, :, None]
    return np.where(fine[:, :, None], round_e2m1(v), 0).astype(np.uint8).reshape(x.shape), s


def pack(codes):
    """Two codes to a byte, the first in the low half."""
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def unpack(q):
    return np.stack([q & 15, q >> 4], axis=-1).reshape(*q.shape[:-1], -1)


def dequantize(codes, scales):
    return E2M1[codes] * np.repeat(scale_values(scales), BLOCK, axis=-1)


def ref_matmul(x, w):
    """(Y, B): the product of values in fp64 and B = sum |x w|, the size its rounding errors go by."""
    with np.errstate(invalid="ignore"):
        return x @ w.T, np.abs(x) @ np.abs(w).T


def ref_grouped(x, w, offsets, row_index=None):
    """(Y, B, written) for experts' weights [E, n, k]; rows that no range covers are NaN."""
    p = x.shape[0] if row_index is None else len(row_index)
    y, b, written = np.full((p, w.shape[1]), np.nan), np.zeros((p, w.shape[1])), np.zeros(p, bool)
    for e in range(w.shape[0]):
        lo = min(max(int(offsets[e]), 0), p)
        hi = min(max(int(offsets[e + 1]), lo), p)
        if hi == lo:
            continue
        r = np.arange(lo, hi) if row_index is None else np.asarray(row_index[lo:hi])
        ok = (r >= 0) & (r < x.shape[0])
        yy, bb = ref_matmul(x[np.where(ok, r, 0)], w[e])
        y[lo:hi], b[lo:hi] = np.where(ok[:, None], yy, 0.0), np.where(ok[:, None], bb, 0.0)
        written[lo:hi] = True
    return y, b, written


def activation(g, kind):
    z = g if kind == "silu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-z)), np.abs(z)


def ref_mlp(x, ids, weights, w1, w2, kind, c1=0.0):
    """(out, size, spread) of the expert layer: size = sum |weight| |W2| |h|; spread = what errors of
    c1 sum |x w| in gate and up, of (4 + |z|) 2^-21 in the activation and of 2^-17 in h (which the
    next product takes in 16 bits) come to at the output.  |act'| <= 1.13 for both activations."""
    tokens, d = x.shape
    inner = w2.shape[2]
    out, size, spread = np.zeros((tokens, d)), np.zeros((tokens, d)), np.zeros((tokens, d))
    for t in range(tokens):
        for e, w in zip(ids[t], weights[t]):
            if not 0 <= e < w1.shape[0]:
                continue
            y, b = ref_matmul(x[t:t + 1], w1[e])
            g, u, bg, bu = y[0, :inner], y[0, inner:], b[0, :inner], b[0, inner:]
            a, z = activation(g, kind)
            off = c1 * (1.13 * bg * np.abs(u) + bu * np.abs(a)) + np.abs(a * u) * ((4 + z) * 2.0 ** -21 + 2.0 ** -17)
            out[t] += float(w) * (w2[e] @ (a * u))
            size[t] += abs(float(w)) * (np.abs(w2[e]) @ np.abs(a * u))
            spread[t] += abs(float(w)) * (np.abs(w2[e]) @ off)
    return out, size, spread
