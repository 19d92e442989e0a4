"""Host side of the KV cache and logits calls, without a GPU: page sizes, and every refusal that precedes a launch."""
import ctypes as C

import pytest


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
        return C.c_void_p(self.base + off)


def test_page_bytes(m):
    # 16 tokens: K and V codes 8 D bytes each, 16 D / 32 scales of 1 or 2 bytes each
    for fmt, sb in ((1, 1), (2, 2)):
        for D in (64, 128):
            for h in (1, 3, 8):
                for page in (16, 48, 64, 1024):
                    assert m.moe_kv_page_bytes(fmt, D, h, page) == h * (page // 16) * (16 * D + 2 * 16 * (D // 32) * sb)
    for bad in ((3, 128, 8, 16), (4, 128, 8, 16), (1, 96, 8, 16), (1, 128, 0, 16), (1, 128, 257, 16), (1, 128, 8, 8),
                (1, 128, 8, 24), (1, 128, 8, 1040)):
        assert m.moe_kv_page_bytes(*bad) == 0


def test_kv_calls_refuse(m, monkeypatch):
    L, p = m.lib(), Mem()

    def cache(**kw):
        a = dict(fmt=1, D=128, h=2, page=16, n=4, stride=2 * 2176, ptr=p())
        a.update(kw)
        return C.byref(m.moe_kv_cache_t(a["fmt"], a["D"], a["h"], a["page"], a["n"], a["stride"], a["ptr"]))

    def batch(**kw):
        a = dict(n=2, t=3, q=2, stride=4, qs=p(), sl=p(), bt=p())
        a.update(kw)
        return C.byref(m.moe_kv_batch_t(a["n"], a["t"], a["q"], a["stride"], a["qs"], a["sl"], a["bt"]))

    big = 1 << 26
    def attn(c=None, b=None, q=p(), qs=512, hq=4, scale=0.1, window=0, out=p(), lse=None, ws=p(), n=big):
        return L.moe_kv_attention(c or cache(), b or batch(), q, qs, hq, scale, window, out, lse, ws, n, None)

    def append(c=None, b=None, k=p(), ks=256, v=p(), vs=256, q=p(), qs=512, hq=4, qo=p(), cos=p(), sin=p(), R=64, rows=9, ws=p(), n=256):
        return L.moe_kv_append(c or cache(), b or batch(), k, ks, v, vs, q, qs, hq, qo, cos, sin, R, rows, 0, ws, n, None)

    def read(c=None, b=None, k=p(), v=p(), ws=p(), n=256):
        return L.moe_kv_read(c or cache(), b or batch(), k, v, ws, n, None)

    for call in (attn, append, read):
        assert call(c=cache(fmt=3)) == 3
        assert call(c=cache(D=96)) == 2 and call(c=cache(page=24)) == 2 and call(c=cache(h=0)) == 2
        assert call(c=cache(n=0)) == 2 and call(c=cache(stride=2 * 2176 - 16)) == 2 and call(c=cache(stride=2 * 2176 + 8)) == 2
        assert call(c=cache(ptr=None)) == 1 and call(c=cache(ptr=p(8))) == 1
        assert call(b=batch(n=0)) == 2 and call(b=batch(n=1025)) == 2 and call(b=batch(t=0)) == 2 and call(b=batch(q=0)) == 2
        assert call(b=batch(stride=0)) == 2 and call(b=batch(stride=1 << 26)) == 2
        assert call(b=batch(qs=None)) == 1 and call(b=batch(sl=None)) == 1 and call(b=batch(bt=None)) == 1 and call(b=batch(sl=p(2))) == 1
        assert call(ws=None) == 1 and call(ws=p(16)) == 1 and call(n=128) == 5
    assert attn(q=None) == 1 and attn(q=p(8)) == 1 and attn(out=None) == 1 and attn(out=p(2)) == 1 and attn(lse=p(2)) == 1
    assert attn(hq=3) == 2 and attn(hq=0) == 2 and attn(qs=504) == 2 and attn(qs=516) == 2 and attn(window=-1) == 2
    assert attn(scale=float("nan")) == 1 and attn(scale=float("inf")) == 1
    assert attn(b=batch(q=9)) == 2 and attn(b=batch(q=8), hq=34, qs=34 * 128) == 2
    assert append(k=None) == 1 and append(v=p(8)) == 1 and append(qo=None) == 1 and append(cos=None) == 1 and append(sin=p(4)) == 1
    assert append(ks=255) == 2 and append(vs=248) == 2 and append(qs=504) == 2 and append(hq=0) == 2
    assert append(R=4) == 2 and append(R=136) == 2 and append(R=-8) == 2 and append(rows=0) == 2
    assert read(k=None, v=None) == 1 and read(k=p(4)) == 1
    ws_bytes = L.moe_kv_workspace_bytes
    assert ws_bytes(cache(), batch(), 4) >= 256 and ws_bytes(cache(), batch(), 3) == 0 and ws_bytes(cache(D=32), batch(), 4) == 0
    for site, call in (("kv_attention", attn), ("kv_append", append), ("kv_read", read)):
        monkeypatch.setenv("MOE_FAULT", site)
        assert call() == 8


def test_logits_call_refuses(m, monkeypatch):
    L, p = m.lib(), Mem()

    def call(probs=p(1024), top=p(), **kw):
        a = dict(type=0, n=2, rows=2, V=100, logits=p(), stride=100, params=p(), counts=p(), draft=p(), bs=p(), bi=p(), bv=p(),
                 allowed=p(), as_=4)
        a.update(kw)
        s = m.moe_logits_t(a["type"], a["n"], a["rows"], a["V"], a["logits"], a["stride"], a["params"], a["counts"], a["draft"],
                           a["bs"], a["bi"], a["bv"], a["allowed"], a["as_"])
        return L.moe_logits_probs(C.byref(s), probs, top, None)

    assert L.moe_logits_probs(None, p(), None, None) == 1
    assert call(logits=None) == 1 and call(params=None) == 1 and call(probs=None) == 1 and call(type=2) == 1
    assert call(logits=p(2)) == 1 and call(type=1, logits=p(1)) == 1 and call(probs=p(2)) == 1 and call(top=p(1)) == 1
    assert call(counts=p(2)) == 1 and call(bi=None) == 1 and call(bv=None) == 1
    assert call(n=0) == 2 and call(rows=0) == 2 and call(rows=65) == 2 and call(n=40000) == 2
    assert call(V=0) == 2 and call(V=(1 << 22) + 1, stride=1 << 23, as_=1 << 18) == 2 and call(stride=99) == 2 and call(as_=3) == 2
    assert call(probs=p(), logits=p(), stride=104) == 1 and call(probs=p(), logits=p(), type=1) == 1     # in place: fp32, dense
    monkeypatch.setenv("MOE_FAULT", "logits")
    assert call() == 8
