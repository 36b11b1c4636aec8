"""fp64 reference of the block-scaled 8-bit layers: rounding to e4m3 with a scale per block of
128 inputs, and the products of such operands, dense and grouped by expert.  numpy only; no
code is shared with the HIP path."""
import numpy as np

BLOCK = 128


def e4m3_values():
    """Value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and
    0xff are NaN, there is no infinity."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = np.ldexp(m / 8, -6) if e == 0 else np.ldexp(1 + m / 8, e - 7)
        v[c] = np.nan if (c & 127) == 127 else (-a if c & 128 else a)
    return v


E4M3 = e4m3_values()


def round_e4m3(v):
    """Codes of the values nearest to fp64 v, ties to the even code; |v| <= 448 after rounding."""
    a = np.abs(np.asarray(v, dtype=np.float64))
    pos = E4M3[:127]
    hi = np.searchsorted(pos, a, side="left").clip(0, 126)
    lo = (hi - 1).clip(0)
    up, down = pos[hi] - a, a - pos[lo]
    pick = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    pick = np.where(pos[hi] == a, hi, pick)
    return (pick | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def block_scales(top, e8m0):
    """Scales (fp64 holding fp32 values) of blocks whose largest magnitude is ``top``."""
    top = np.asarray(top, dtype=np.float64)
    with np.errstate(all="ignore"):
        if e8m0:
            f, e = np.frexp(top)                     # top = f 2^e, f in [1/2, 1)
            s = np.where(top == 0, 0.0, np.ldexp(1.0, e - 9 + (f > 0.875)))   # 448 = 0.875 * 2^9
        else:
            s = (top / 448.0).astype(np.float32).astype(np.float64)
    s = np.maximum(s, 2.0 ** -126)
    return np.where(np.isfinite(top), s, np.nan)


def ref_quantize(x, block_rows, e8m0):
    """x [rows, cols] -> (codes uint8, scales fp64 [row blocks, col blocks])."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    rb, cb = -(-rows // block_rows), -(-cols // BLOCK)
    codes, scales = np.zeros((rows, cols), np.uint8), np.empty((rb, cb))
    for i in range(rb):
        for j in range(cb):
            t = x[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK]
            top = np.max(np.abs(t)) if np.all(np.isfinite(t)) else np.inf
            s = scales[i, j] = block_scales(top, e8m0)
            if np.isfinite(s):
                codes[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK] = round_e4m3(t / s)
    return codes, scales


def dequantize(codes, scales, block_rows):
    s = np.repeat(np.repeat(scales, block_rows, 0)[:codes.shape[0]], BLOCK, 1)[:, :codes.shape[1]]
    return E4M3[codes] * s


def ref_matmul(xq, xs, wq, ws):
    """(Y, B): the product in fp64 and B = sum |x w|, the size its rounding errors go by."""
    x, w = dequantize(xq, xs, 1), dequantize(wq, ws, BLOCK)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def ref_grouped(xq, xs, wq, ws, offsets, row_index=None):
    """(Y, B, written) for experts' weights [E, n, k]; rows that no range covers are NaN."""
    p = xq.shape[0] if row_index is None else len(row_index)
    n = wq.shape[1]
    y, b, written = np.full((p, n), np.nan), np.zeros((p, n)), np.zeros(p, bool)
    for e in range(wq.shape[0]):
        lo = min(max(int(offsets[e]), 0), p)
        hi = min(max(int(offsets[e + 1]), lo), p)
        if hi == lo:
            continue
        r = np.arange(lo, hi) if row_index is None else np.asarray(row_index[lo:hi])
        ok = (r >= 0) & (r < xq.shape[0])
        yy, bb = ref_matmul(xq[np.where(ok, r, 0)], xs[np.where(ok, r, 0)], wq[e], ws[e])
        y[lo:hi], b[lo:hi] = np.where(ok[:, None], yy, 0.0), np.where(ok[:, None], bb, 0.0)
        written[lo:hi] = True
    return y, b, written
