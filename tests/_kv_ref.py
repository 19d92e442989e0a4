"""Plain numpy reference of the 4-bit paged KV cache (encoding, layout, rotation) and of attention over it, written from the
definitions in include/moe.h and sharing no code with the kernels. The encoders' arithmetic is fp32 as the call defines it, so
bytes are compared exactly; attention is in 64 bits."""
from __future__ import annotations

import numpy as np

MXFP4, INT4 = 1, 2
F = np.float32
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
GRID = [F(6) / F(7), F(0.9), F(0.95), F(1), F(1.05), F(1.1)]


def bf16(a) -> np.ndarray:
    """fp32 -> the nearest bf16 value (ties to even), as fp32"""
    u = np.ascontiguousarray(a, F).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16
    return np.where(np.isnan(a), a, r.astype(np.uint32).view(F).reshape(np.shape(a)))


def sub_bytes(fmt, D):
    return 16 * D + D * (1 if fmt == MXFP4 else 2)


def encode_row(fmt, x):
    """[D] fp32 -> codes [D], scales [D / 32] (E8M0 or bf16 bits)"""
    codes, scales = [], []
    x = np.clip(np.where(np.isnan(x), F(0), x).astype(F), F(-2.0 ** 64), F(2.0 ** 64))
    for w in x.reshape(-1, 32):
        amax = np.max(np.abs(w))
        if fmt == MXFP4:
            k = -126
            while k < 127 and float(amax) > 6.0 * 2.0 ** k:
                k += 1
            u = w.astype(np.float64) * 2.0 ** -k
            mag = np.abs(u)[:, None]
            d = np.abs(mag - E2M1[:8])
            best = d.min(1, keepdims=True)
            near = d == best
            # ties between two neighbouring codes go to the even one
            c = np.array([[i for i in range(8) if row[i]] for row in near], dtype=object)
            c = np.array([v[0] if len(v) == 1 else [i for i in v if i % 2 == 0][0] for v in c])
            codes.append(c + 8 * np.signbit(w))
            scales.append(k + 127)
        else:
            am = max(amax, F(1e-8))
            best = None
            for g in GRID:
                s = F(F(am * g) / F(7))
                q = np.clip(np.rint((w / s).astype(F)), -8, 7).astype(F)
                e = (w - (q * s).astype(F)).astype(F)
                m = (e * e).astype(F)
                for h in (16, 8, 4, 2, 1):
                    m = (m[:h] + m[h:2 * h]).astype(F)
                if best is None or m[0] < best[0]:
                    best = (m[0], q, s)
            codes.append(best[1].astype(int) & 15)
            scales.append(int(bf16(np.array([best[2]], F)).view(np.uint32)[0] >> 16))
    return np.concatenate(codes).astype(np.uint8), np.array(scales)


def put(fmt, D, sub, slot, kc, ks, vc, vs):
    """Writes one token's codes and scales into a sub-block (uint8 array), nibble by nibble."""
    nb, sb = D // 32, 1 if fmt == MXFP4 else 2

    def nibble(byte, hi, c):
        sub[byte] = (sub[byte] & (0x0F if hi else 0xF0)) | (int(c) << (4 if hi else 0))

    for d in range(D):
        b, n = divmod(d, 32)
        nibble(slot * (D // 2) + ((n // 8) * nb + b) * 4 + (n % 8) // 2, n % 2, kc[d])
        word = 8 * D + ((((slot // 8) * 8 + n // 4) * 4 + (slot % 8) // 2) * nb + b) * 4
        j = n % 4
        if fmt == MXFP4:
            nibble(word + j, slot % 2, vc[d])
        else:
            nibble(word + 2 * (slot % 2) + j // 2, j % 2, vc[d])
    for at, s in ((16 * D, ks), (16 * D + 16 * nb * sb, vs)):
        for b in range(nb):
            for y in range(sb):
                sub[at + (slot * nb + b) * sb + y] = (int(s[b]) >> (8 * y)) & 255


def get(fmt, D, sub):
    """K and V [16, D] in 64 bits of one sub-block"""
    nb, sb = D // 32, 1 if fmt == MXFP4 else 2
    K, V = np.zeros((16, D)), np.zeros((16, D))
    d = np.arange(D)
    b, n, j = d // 32, d % 32, d % 4
    val = (lambda c: E2M1[c]) if fmt == MXFP4 else (lambda c: np.where(c > 7, c.astype(float) - 16, c))
    for i in range(16):
        sc = []
        for at in (16 * D, 16 * D + 16 * nb * sb):
            raw = sub[at + i * nb * sb: at + (i + 1) * nb * sb]
            if fmt == MXFP4:
                with np.errstate(over="ignore"):
                    sc.append(np.where(raw == 0, 0.0, np.where(raw == 255, np.nan, 2.0 ** (raw.astype(float) - 127))))
            else:
                with np.errstate(invalid="ignore"):
                    sc.append((raw.view(np.uint16).astype(np.uint32) << 16).view(F).astype(float))
        kb = sub[i * (D // 2) + ((n // 8) * nb + b) * 4 + (n % 8) // 2].astype(int)
        with np.errstate(invalid="ignore"):
            K[i] = val((kb >> (4 * (n % 2))) & 15) * sc[0][b]
        word = 8 * D + ((((i // 8) * 8 + n // 4) * 4 + (i % 8) // 2) * nb + b) * 4
        if fmt == MXFP4:
            vc = (sub[word + j].astype(int) >> (4 * (i % 2))) & 15
        else:
            vc = (sub[word + 2 * (i % 2) + j // 2].astype(int) >> (4 * (j % 2))) & 15
        with np.errstate(invalid="ignore"):
            V[i] = val(vc) * sc[1][b]
    return K, V


def rotate(x, cos, sin, R, inter):
    """[D] fp32, one position's cos / sin [R / 2]; every operation rounded to fp32"""
    y = x.astype(F).copy()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if inter else (slice(0, R // 2), slice(R // 2, R))
    xa, xb = x[a].astype(F), x[b].astype(F)
    y[a] = (xa * cos).astype(F) - (xb * sin).astype(F)
    y[b] = (xb * cos).astype(F) + (xa * sin).astype(F)
    return y


def sequence_kv(fmt, D, pages, table_row, page_tokens, h, length):
    """K, V [length, D] of KV head h; pages uint8 [n, Hkv, page_tokens / 16, bytes]"""
    ks, vs = [], []
    for s in range((length + 15) // 16):
        p, i = divmod(s * 16, page_tokens)
        K, V = get(fmt, D, pages[table_row[p], h, i // 16])
        ks.append(K)
        vs.append(V)
    return np.concatenate(ks)[:length], np.concatenate(vs)[:length]


def attend(q, K, V, scale, pos, window):
    """One row: (out, lse, sum p |v|, sum |q k| scale of the largest key) in 64 bits; zeros and -inf if it sees nothing"""
    lo = max(0, pos - window + 1) if window else 0
    if pos < lo:
        return np.zeros(K.shape[1] if len(K) else q.shape[0]), -np.inf, 0.0, 0.0
    k, v = K[lo:pos + 1], V[lo:pos + 1]
    x = (k @ q) * scale
    m = x.max()
    p = np.exp(x - m)
    l = p.sum()
    p = p / l
    return p @ v, m + np.log(l), p @ np.abs(v), float((np.abs(k) @ np.abs(q)).max() * abs(scale))
