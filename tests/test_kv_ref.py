"""Pins of the numpy reference of the 4-bit KV cache against the CPU oracle's block formats and closed forms."""
import numpy as np
import pytest

import oracle
from tests import _kv_ref as R


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("D", [64, 128])
def test_encoder_matches_the_block_formats(fmt, D):
    """MXFP4: the oracle's codes and exponents bit for bit. INT4: the same candidates; where the pairwise and the sequential
    sums of squares choose differently, the two errors differ by rounding only."""
    rng = np.random.default_rng(D + fmt)
    x = (rng.standard_normal((40, D)) * np.exp(rng.standard_normal((40, 1)) * 3)).astype(np.float32)
    x[0] = 0
    x[1, ::2] = -0.0
    x[2] *= 1e-30
    ref = oracle.encode(fmt, x).reshape(40, D // 32, -1)
    for i in range(40):
        c, s = R.encode_row(fmt, x[i])
        c = c.reshape(-1, 32)
        codes = (c[:, 0::2] << 4) | c[:, 1::2]
        for b in range(D // 32):
            if fmt == 1:
                assert np.array_equal(ref[i, b, 1:], codes[b]) and ref[i, b, 0] == s[b]
            else:
                assert np.array_equal(ref[i, b, :16], codes[b]) and (ref[i, b, 16:].view(np.uint16)[0] == s[b])


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("D", [64, 128])
def test_layout_round_trip_touches_only_the_token(fmt, D):
    rng = np.random.default_rng(7)
    sub = rng.integers(0, 256, R.sub_bytes(fmt, D), dtype=np.uint8)
    seen = np.zeros(sub.size * 2, bool)
    vals = {}
    for slot in rng.permutation(16):
        x = rng.standard_normal((2, D)).astype(np.float32)
        enc = [R.encode_row(fmt, v) for v in x]
        before = sub.copy()
        R.put(fmt, D, sub, slot, *enc[0], *enc[1])
        changed = np.stack([(sub ^ before) & 15, (sub ^ before) >> 4], 1).reshape(-1) != 0
        assert not np.any(changed & seen), "a token's nibbles are its own"
        seen |= changed
        vals[slot] = enc
    K, V = R.get(fmt, D, sub)
    for slot, enc in vals.items():
        for got, (c, s) in ((K[slot], enc[0]), (V[slot], enc[1])):
            sc = 2.0 ** (s - 127.0) if fmt == 1 else (s.astype(np.uint32) << 16).view(np.float32).astype(float)
            code = R.E2M1[c] if fmt == 1 else np.where(c > 7, c.astype(float) - 16, c)
            assert np.array_equal(got, code * np.repeat(sc, 32))


def test_rotation_is_a_rotation():
    rng = np.random.default_rng(3)
    x = rng.standard_normal(64).astype(np.float32)
    a = rng.uniform(0, 6, 16)
    c, s = np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)
    for inter in (False, True):
        y = R.rotate(x, c, s, 32, inter)
        assert np.array_equal(y[32:], x[32:]) and abs(np.linalg.norm(y) - np.linalg.norm(x)) < 1e-5
        pair = (y[0], y[1]) if inter else (y[0], y[16])
        src = (x[0], x[1]) if inter else (x[0], x[16])
        assert np.allclose(complex(*pair), complex(*src) * complex(c[0], s[0]), atol=1e-6)


def test_attention_closed_forms():
    K = np.zeros((5, 64))
    V = np.arange(5 * 64, dtype=float).reshape(5, 64)
    q = np.ones(64)
    o, lse, _, _ = R.attend(q, K, V, 0.3, 3, 0)             # equal scores: the mean of the visible values
    assert np.allclose(o, V[:4].mean(0)) and np.isclose(lse, np.log(4))
    o, lse, _, _ = R.attend(q, K, V, 0.3, 4, 2)             # a window of two keys
    assert np.allclose(o, V[3:5].mean(0)) and np.isclose(lse, np.log(2))
    o, lse, _, _ = R.attend(q, K, V, 0.3, -1, 0)
    assert not o.any() and lse == -np.inf
