"""Plain numpy reference of the 8-bit rows, the residual norm, the integer product and the gated block, in 64 bits where the
definition is in real numbers and in rounded fp32 operations where it says so."""
import numpy as np

FLOOR = np.float32(2.0 ** -100)


def bf16(x):
    """fp32 rounded to bf16 (nearest even), as fp32."""
    x = np.ascontiguousarray(x, np.float32)
    b = x.view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), r).reshape(x.shape)


def quantize(v):
    """Codes int8, scales fp32 and the rows' largest magnitudes of v [n, K] fp32."""
    v = np.asarray(v, np.float32)
    top = np.abs(v).max(1)
    bad = ~np.isfinite(top)
    a = np.maximum(np.where(bad, np.float32(1), top), FLOOR).astype(np.float32)
    with np.errstate(invalid="ignore"):
        q = np.rint(127.0 * v.astype(np.float64) / a.astype(np.float64)[:, None])
    q = np.where(bad[:, None], 0, q).astype(np.int8)
    return q, np.where(bad, np.float32(np.nan), a / np.float32(127)).astype(np.float32), np.where(bad, np.float32(np.nan), a)


def norm(h, r, gain, eps):
    """s (fp32), the codes, and in 64 bits the scales and the normalised rows."""
    s = np.asarray(h, np.float32) if r is None else np.asarray(h, np.float32) + np.asarray(r, np.float32)
    v = s if gain is None else s * np.asarray(gain, np.float32)
    q, _, a = quantize(v)
    with np.errstate(invalid="ignore", divide="ignore"):
        rho = 1.0 / np.sqrt((s.astype(np.float64) ** 2).mean(1) + np.float64(np.float32(eps)))
        return s, q, a.astype(np.float64) * rho / 127.0, v.astype(np.float64) * rho[:, None]


def product(xq, xs, wq, ws):
    """fp32: (float(exact integer sum) * xs) * ws, each operation rounded."""
    acc = np.rint(xq.astype(np.float64) @ wq.astype(np.float64).T)     # (exact: far below 2^53)
    return (acc.astype(np.int64).astype(np.float32) * np.asarray(xs, np.float32)[:, None]) * np.asarray(ws, np.float32)[None]


def gated(g, u):
    """SiLU(g) u in 64 bits of fp32 g and u."""
    g, u = g.astype(np.float64), u.astype(np.float64)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u
