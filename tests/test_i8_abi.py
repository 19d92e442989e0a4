"""Host side of the 8-bit calls, without a GPU: workspace sizes and every refusal that precedes a launch."""
import ctypes as C

import numpy as np
import pytest

from tests import _i8_ref as ref


@pytest.fixture(scope="module")
def m():
    from bit_moe_decode_gb300 import build
    build.build()
    import bit_moe_decode_gb300 as mod
    mod.lib()
    return mod


class Mem:
    """256-byte aligned host addresses (only for checks that precede any launch)"""

    def __init__(self):
        self.buf = (C.c_uint8 * 65536)()
        self.base = C.addressof(self.buf) + (-C.addressof(self.buf)) % 256

    def __call__(self, off=0):
        return self.base + off


P = Mem()


def rows(m, **kw):
    a = dict(rows=4, cols=64, stride=64, q=P(), scale=P())
    a.update(kw)
    return C.byref(m.moe_i8_rows_t(a["rows"], a["cols"], a["stride"], a["q"], a["scale"]))


BAD_ROWS = [(dict(q=None), 1), (dict(scale=None), 1), (dict(q=P(8)), 1), (dict(scale=P(2)), 1), (dict(rows=0), 2), (dict(rows=-1), 2),
            (dict(rows=(1 << 22) + 1), 2), (dict(cols=0), 2), (dict(cols=8), 2), (dict(cols=72, stride=80), 2),
            (dict(cols=131072, stride=131072), 2), (dict(stride=48), 1), (dict(stride=72), 1)]


def test_workspace_bytes(m):
    assert m.lib().moe_i8_workspace_bytes(rows(m), 1) >= 256
    assert m.lib().moe_i8_workspace_bytes(rows(m), 0) == 0
    assert m.lib().moe_i8_workspace_bytes(None, 1) == 0
    for bad, _ in BAD_ROWS:
        assert m.lib().moe_i8_workspace_bytes(rows(m, **bad), 1) == 0, bad


def test_rows_calls_refuse(m, monkeypatch):
    L = m.lib()

    def quantize(type=0, src=P(), stride=64, dst=None):
        return L.moe_i8_quantize(type, src, stride, dst or rows(m), None)

    for bad, st in BAD_ROWS:
        assert quantize(dst=rows(m, **bad)) == st, bad
        assert L.moe_i8_values(rows(m, **bad), P(), None) == st, bad
    assert L.moe_i8_quantize(0, P(), 64, None, None) == 1
    for bad in (dict(type=2), dict(type=-1), dict(src=None), dict(src=P(8)), dict(stride=63), dict(stride=66), dict(type=1, stride=68)):
        assert quantize(**bad) == 1, bad
    assert L.moe_i8_values(rows(m), None, None) == 1
    assert L.moe_i8_values(rows(m), P(8), None) == 1
    for name, call in (("i8_quantize", quantize), ("i8_values", lambda: L.moe_i8_values(rows(m), P(), None))):
        monkeypatch.setenv("MOE_FAULT", name)
        assert call() == 8


def test_norm_refuses(m, monkeypatch):
    L = m.lib()

    def norm(xq="new", **kw):
        a = dict(T=4, H=64, ht=0, rt=1, h=P(), hs=64, r=P(), rs=64, gain=P(), eps=1e-6, ho=P(), hos=64, x=P())
        a.update(kw)
        c = m.moe_norm_t(*[a[k] for k in ("T", "H", "ht", "rt", "h", "hs", "r", "rs", "gain", "eps", "ho", "hos", "x")])
        return L.moe_rms_norm_i8(C.byref(c), rows(m) if xq == "new" else xq, None)

    assert L.moe_rms_norm_i8(None, rows(m), None) == 1
    for bad in (dict(h=None), dict(ht=2), dict(rt=3), dict(h=P(4)), dict(r=P(8)), dict(gain=P(4)), dict(ho=P(2)), dict(x=P(2)), dict(hs=60),
                dict(hs=65), dict(rs=68), dict(rs=56), dict(hos=32), dict(x=None, xq=None)):
        assert norm(**bad) == 1, bad
    for bad in (dict(T=0), dict(T=5), dict(H=80, hs=80, rs=80, hos=80), dict(H=8), dict(H=72, hs=80), dict(H=32784, hs=1 << 16, xq=None),
                dict(eps=-1.0), dict(eps=float("nan"))):
        assert norm(**bad) == 2, bad
    for bad, st in BAD_ROWS:
        assert norm(xq=rows(m, **bad)) == st, bad
    monkeypatch.setenv("MOE_FAULT", "norm_i8")
    assert norm() == 8


def test_products_refuse(m, monkeypatch):
    L = m.lib()

    def matmul(x=None, w=None, base=None, bs=0, y=P(), ys=8, yb=None, ybs=0, ws=P(), n=1 << 24):
        return L.moe_i8_matmul(x or rows(m), w or rows(m, rows=8), base, bs, y, ys, yb, ybs, ws, n, None)

    def gated(x=None, g=None, u=None, y=P(), ys=8, yb=None, ybs=0, ws=P(), n=1 << 24):
        return L.moe_i8_gated(x or rows(m), g or rows(m, rows=8), u or rows(m, rows=8), y, ys, yb, ybs, ws, n, None)

    for call in (matmul, gated):
        for bad in (dict(y=None), dict(ws=None), dict(ws=P(128)), dict(y=P(2)), dict(ys=7), dict(yb=P(1), ybs=8), dict(yb=P(), ybs=7)):
            assert call(**bad) == 1, bad
        assert call(n=255) == 5
        assert call(x=rows(m, cols=48)) == 2
        for bad, st in BAD_ROWS:
            assert call(x=rows(m, **bad)) == st, bad
    for bad, st in BAD_ROWS:
        assert matmul(w=rows(m, **bad)) == st, bad
        assert gated(g=rows(m, **bad)) == st, bad
        assert gated(u=rows(m, **bad)) == st, bad
    assert matmul(base=P(2), bs=8) == 1 and matmul(base=P(), bs=7) == 1
    assert gated(u=rows(m, rows=9)) == 2 and gated(u=rows(m, rows=8, cols=48)) == 2
    assert L.moe_i8_gated(rows(m), rows(m, rows=8), None, P(), 8, None, 0, P(), 1 << 24, None) == 1
    assert L.moe_i8_matmul(None, rows(m), None, 0, P(), 8, None, 0, P(), 1 << 24, None) == 1
    assert L.moe_i8_matmul(rows(m), None, None, 0, P(), 8, None, 0, P(), 1 << 24, None) == 1
    for name, call in (("i8_matmul", matmul), ("i8_gated", gated)):
        monkeypatch.setenv("MOE_FAULT", name)
        assert call() == 8


def test_reference_closed_forms():
    """The reference itself: known rows, borders to the even code, rows of zeros, NaN and infinities."""
    q, s, _ = ref.quantize(np.array([[127, -127, 1, 0.5, 1.5, 2.5, -0.5, -1.5], [0] * 8, [np.nan] + [1] * 7, [np.inf] + [1] * 7], np.float32))
    assert q[0].tolist() == [127, -127, 1, 0, 2, 2, 0, -2] and s[0] == 1.0
    assert not q[1:].any() and s[1] == np.float32(2.0 ** -100) / np.float32(127) and np.isnan(s[2:]).all()
    h = np.array([[3.0, 4.0] * 8], np.float32)
    s, q, scale, x = ref.norm(h, None, None, 0.0)
    assert np.allclose(x, h / np.sqrt(12.5)) and np.allclose(q * scale[:, None], x, atol=scale[0] / 2)
    y = ref.product(np.array([[127] * 16], np.int8), [2.0], np.array([[-127] * 16], np.int8), [0.5])
    assert y[0, 0] == -127 * 127 * 16
    assert ref.bf16(np.float32(1 + 2.0 ** -8)) == 1.0 and ref.bf16(np.float32(1 + 3 * 2.0 ** -8)) == np.float32(1 + 2.0 ** -6)
    assert ref.gated(np.float32([0.0, 100.0]), np.float32([2.0, 2.0])).tolist() == [0.0, 200.0]
