"""Plain forms of the FP8 block-scaled operators in 64 bits (NumPy / torch on
the CPU), for the tests.

The quantizers' definition is FP32 arithmetic (scale = b / 448, r = 448 / b,
code = E4M3(x * r)), so their codes and scales have one right value each and are
compared bit for bit.  Everything else is compared with FP64 within bounds that
the tests derive.
"""
import numpy as np
import torch


def e4m3_code(p):
    """E4M3 bytes of FP32 values, to nearest even, |p| <= 464, sign of zero kept; NaN -> 0x7F."""
    p = np.asarray(p, dtype=np.float32)
    v = np.abs(p.astype(np.float64))
    nan = np.isnan(v)
    v = np.where(nan, 0.0, np.minimum(v, 448.0))
    _, e = np.frexp(v)                                    # v = m * 2^e, m in [0.5, 1)
    step = np.exp2(np.maximum(e - 4, -9).astype(np.float64))
    n = np.rint(v / step) * step                          # rint: ties to even
    _, e = np.frexp(n)
    normal = n >= 2.0 ** -6
    mant = np.where(normal, n / np.exp2((e - 1).astype(np.float64)) * 8 - 8, n * 512)
    code = np.where(normal, (e - 1 + 7) * 8, 0) + mant
    code = code.astype(np.int64) | np.where(np.signbit(p), 0x80, 0)
    return np.where(nan, 0x7F, code).astype(np.uint8)


def e4m3_value(codes):
    c = np.asarray(codes).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (8 + m) * np.exp2(e.astype(np.float64) - 10), m * 2.0 ** -9)
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


def quantize(x, rows, cols):
    """(codes u8, scales f32 [row block, column block]) of FP32 x [R, C] in blocks of rows x cols."""
    x = np.asarray(x, dtype=np.float32)
    r, c = x.shape
    nr, nc = -(-r // rows), -(-c // cols)
    big = np.zeros((nr * rows, nc * cols), np.float32)
    big[:r, :c] = x
    big = big.reshape(nr, rows, nc, cols)
    with np.errstate(invalid="ignore", divide="ignore"):
        amax = np.abs(big).max((1, 3))                    # NaN propagates
        zero = amax < np.float32(2.0 ** -100)
        scale = np.where(zero, np.float32(0), amax / np.float32(448)).astype(np.float32)
        factor = np.where(zero, np.float32(0), np.float32(448) / amax).astype(np.float32)
        prod = big * factor[:, None, :, None]
    return e4m3_code(prod.reshape(nr * rows, nc * cols)[:r, :c]), scale


def rows_quantize(x):
    c, s = quantize(x, 1, 128)
    return c, np.ascontiguousarray(s.T)


def columns_quantize(x):
    return quantize(x, 128, 1)


def tiles_quantize(x):
    return quantize(x, 128, 128)


def value(codes, scales, kind):
    """FP64 values of codes with scales as the library lays them out (torch or NumPy)."""
    codes, scales = (t.cpu().numpy() if isinstance(t, torch.Tensor) else np.asarray(t) for t in (codes, scales))
    s = scales.astype(np.float64)
    r, c = codes.shape
    ri, ci = np.arange(r), np.arange(c)
    s = s[ci // 128][:, ri].T if kind == "rows" else s[ri // 128] if kind == "columns" else s[ri // 128][:, ci // 128]
    return e4m3_value(codes.view(np.uint8)) * s


def silu(g):
    return g / (1 + np.exp(-g))


def gated_grads(dh, gate, up):
    """(dgate, dup, h) in FP64."""
    s = 1 / (1 + np.exp(-gate))
    return dh * up * s * (1 + gate * (1 - s)), dh * gate * s, gate * s * up
