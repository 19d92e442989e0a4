"""Append to and read from the 4-bit paged KV cache against the numpy reference: page bytes and the rotated q bit for bit,
nothing else in the pages touched, read-back equal to the decoded bytes; device data out of range is recorded and stays in
bounds; the calls' refusals."""
import numpy as np
import pytest
import torch

from tests import _kv_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def m():
    import bit_moe_decode_gb300 as mod
    return mod


def make_pages(rng, fmt, D, Hkv, page, n_pages, extra=0):
    """Random bytes, with `extra` more after each page (the page stride)."""
    nbytes = Hkv * (page // 16) * R.sub_bytes(fmt, D)
    return rng.integers(0, 256, (n_pages, nbytes + extra), dtype=np.uint8), nbytes


def table_for(rng, lens, page, n_pages):
    need = [-(-int(n) // page) for n in lens]
    perm = rng.permutation(n_pages)[:sum(need)]
    table = np.full((len(lens), max(need + [1]) + 1), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table


def batch_of(m, ql, lens, table, tokens=None):
    start = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)  # noqa: E731
    return m.KvBatch(d(start), d(lens), d(table), tokens=int(tokens or start[-1]), max_q=max(int(max(ql)), 1))


def sub_view(pages, fmt, D, Hkv, page):
    n = Hkv * (page // 16) * R.sub_bytes(fmt, D)
    return pages[:, :n].reshape(pages.shape[0], Hkv, page // 16, -1)


def reference_append(fmt, D, Hkv, page, pages, table, ql, lens, k, v, q, cos, sin, inter):
    want = pages.copy()
    view = want[:, :Hkv * (page // 16) * R.sub_bytes(fmt, D)].reshape(want.shape[0], Hkv, page // 16, -1).copy()
    Rd = 2 * cos.shape[1] if cos is not None else 0
    q_out = None if q is None else np.zeros_like(q)
    t = 0
    for b, n in enumerate(ql):
        for j in range(n):
            pos = lens[b] - n + j
            turn = (lambda x: R.rotate(x, cos[max(pos, 0)], sin[max(pos, 0)], Rd, inter)) if Rd else (lambda x: x)
            if q is not None:
                for h in range(q.shape[1]):
                    q_out[t, h] = R.bf16(turn(q[t, h]))
            if pos >= 0:
                p, i = divmod(pos, page)
                for h in range(Hkv):
                    R.put(fmt, D, view[table[b, p], h, i // 16], pos % 16, *R.encode_row(fmt, turn(k[t, h])),
                          *R.encode_row(fmt, v[t, h]))
            t += 1
    want[:, :view[0].size] = view.reshape(want.shape[0], -1)
    return want, q_out


CASES = [
    # fmt, D, Hkv, Hq, page, rows, lengths after, rope, interleaved
    (1, 128, 2, 4, 16, [1], [1], 128, False),
    (1, 128, 1, 3, 32, [1, 1, 1], [16, 17, 2], 64, True),         # one token: either half of a shared byte
    (1, 64, 3, 3, 48, [3, 1, 8, 2], [3, 0, 50, 49], 64, False),    # a padding slot in between
    (1, 64, 1, 1, 16, [33, 4], [40, 5], 32, True),
    (2, 128, 2, 4, 16, [2, 1], [2, 100], 128, True),
    (2, 64, 2, 6, 64, [5, 0, 7], [64, 30, 70], 0, False),          # a sequence without new tokens
    (2, 128, 1, 1, 1024, [8], [1030], 8, False),
]


@pytest.mark.parametrize("case", CASES, ids=["%s-D%d-p%d-%s" % ("mxfp4" if c[0] == 1 else "int4", c[1], c[4], c[5]) for c in CASES])
def test_append_and_read(m, case):
    fmt, D, Hkv, Hq, page, ql, lens, rope, inter = case
    rng = np.random.default_rng(sum(lens) * 7 + D + fmt)
    pages, nbytes = make_pages(rng, fmt, D, Hkv, page, sum(-(-n // page) for n in lens) + 2, extra=48)
    table = table_for(rng, lens, page, pages.shape[0])
    T = sum(ql)
    x = R.bf16((rng.standard_normal((T, Hq + 2 * Hkv + 1, D)) * np.exp(rng.standard_normal((T, 1, 1)))).astype(np.float32))
    n = max(max(lens), 1)
    ang = np.arange(n)[:, None] * 100.0 ** (-np.arange(0, max(rope, 2), 2) / max(rope, 2))
    cos, sin = (np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)) if rope else (None, None)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:Hq + 2 * Hkv]
    want, q_want = reference_append(fmt, D, Hkv, page, pages, table, ql, lens, k, v, q, cos, sin, inter)

    dev = torch.from_numpy(x).to(DEV).to(torch.bfloat16)             # q, k, v as slices of one wider tensor
    cache = m.KvCache(fmt, D, Hkv, page, pages=torch.from_numpy(pages).to(DEV))
    batch = batch_of(m, ql, lens, table)
    ws = cache.workspace(batch, Hq)
    q_out = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=DEV)
    up = (lambda a: None if a is None else torch.from_numpy(a).to(DEV))  # noqa: E731
    m.moe_kv_append(cache, batch, dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:Hq + 2 * Hkv], q=dev[:, :Hq], q_out=q_out, cos=up(cos), sin=up(sin),
                    interleaved=inter, ws=ws)
    torch.cuda.synchronize()
    assert m.moe_get_device_status(ws) == 0
    got = cache.pages.cpu().numpy()
    assert np.array_equal(got, want), "page bytes differ at %s" % np.argwhere(got != want)[:5].tolist()
    assert np.array_equal(q_out.float().cpu().numpy().view(np.uint32), q_want.astype(np.float32).view(np.uint32))

    ko = torch.full((T, Hkv, D), float("nan"), device=DEV)
    vo = torch.full((T, Hkv, D), float("nan"), device=DEV)
    m.moe_kv_read(cache, batch, ko, vo, ws=ws)
    torch.cuda.synchronize()
    view = sub_view(want, fmt, D, Hkv, page)
    t = 0
    for b, nq in enumerate(ql):
        for j in range(nq):
            pos = lens[b] - nq + j
            for h in range(Hkv):
                K, V = R.get(fmt, D, view[table[b, pos // page], h, pos % page // 16]) if pos >= 0 else (np.zeros((16, D)),) * 2
                assert np.array_equal(ko[t, h].cpu().numpy().astype(float), K[pos % 16])
                assert np.array_equal(vo[t, h].cpu().numpy().astype(float), V[pos % 16])
            t += 1
    m.moe_kv_read(cache, batch, None, vo, ws=ws)       # either output alone


@pytest.mark.parametrize("fmt", [1, 2])
def test_append_of_unusual_values(m, fmt):
    """Zeros, negative zeros, subnormals, the largest bf16, infinities and NaN: clamped and encoded as defined."""
    D, Hkv, page, T = 64, 1, 16, 6
    x = np.zeros((T, 2, D), np.float32)
    x[1] = -0.0
    x[2] = 1e-39
    x[3, :, ::3] = 3.3e38
    x[4, :, ::2], x[4, :, 1::2] = np.inf, 1.0
    x[5] = np.linspace(-4, 4, 2 * D).reshape(2, D)
    x[5, :, 7], x[5, :, 40] = np.nan, -np.inf
    x = np.where(np.isfinite(x), R.bf16(np.where(np.isfinite(x), x, 0)), x).astype(np.float32)
    rng = np.random.default_rng(0)
    pages, _ = make_pages(rng, fmt, D, Hkv, page, 1)
    table = np.zeros((1, 1), np.int32)
    want, _ = reference_append(fmt, D, Hkv, page, pages, table, [T], [T], x[:, :1], x[:, 1:], None, None, None, False)
    cache = m.KvCache(fmt, D, Hkv, page, pages=torch.from_numpy(pages).to(DEV))
    batch = batch_of(m, [T], [T], table)
    ws = cache.workspace(batch, 1)
    dev = torch.from_numpy(x).to(DEV).to(torch.bfloat16)
    m.moe_kv_append(cache, batch, dev[:, :1], dev[:, 1:], ws=ws)
    torch.cuda.synchronize()
    assert np.array_equal(cache.pages.cpu().numpy(), want)


def test_append_token_by_token_equals_append_at_once(m):
    """A prompt appended in one call, in pieces, and one token at a time fills the pages with the same bytes; q_out may be q."""
    D, Hkv, Hq, page, n = 128, 2, 4, 32, 45
    rng = np.random.default_rng(5)
    pages, _ = make_pages(rng, 1, D, Hkv, page, 3)
    table = np.array([[2, 0]], np.int32)
    x = torch.from_numpy(rng.standard_normal((n, Hq + 2 * Hkv, D)).astype(np.float32)).to(DEV).to(torch.bfloat16)
    ang = torch.arange(n, device=DEV)[:, None] * torch.rand(1, D // 2, device=DEV)
    cos, sin = ang.cos(), ang.sin()
    results = []
    for piece in (n, 7, 1):
        cache = m.KvCache(1, D, Hkv, page, pages=torch.from_numpy(pages).to(DEV))
        qs = []
        for i in range(0, n, piece):
            c = min(piece, n - i)
            batch = batch_of(m, [c], [i + c], table)
            ws = cache.workspace(batch, Hq)
            q = x[i:i + c, :Hq].contiguous()
            m.moe_kv_append(cache, batch, x[i:i + c, Hq:Hq + Hkv], x[i:i + c, Hq + Hkv:], q=q, q_out=q, cos=cos, sin=sin, ws=ws)
            qs.append(q)
        results.append((cache.pages.cpu(), torch.cat(qs).cpu()))
    for p, q in results[1:]:
        assert torch.equal(p, results[0][0]) and torch.equal(q, results[0][1])


def test_device_data_out_of_range_is_recorded(m):
    """Page ids, lengths and rows that the host cannot check: status MOE_ERR_INVALID_ARG, no write anywhere."""
    D, Hkv, page = 64, 1, 16
    rng = np.random.default_rng(1)
    x = torch.zeros(2, 1, D, dtype=torch.bfloat16, device=DEV)
    good = dict(ql=[1, 1], lens=[3, 20], table=np.array([[0, 1], [2, 3]], np.int32))
    bad = [dict(good, table=np.array([[4, 1], [2, 3]], np.int32)), dict(good, table=np.array([[-1, 1], [2, 3]], np.int32)),
           dict(good, lens=[33, 20]), dict(good, lens=[-5, 20])]
    for i, c in enumerate([good] + bad):
        pages, _ = make_pages(rng, 1, D, Hkv, page, 4)
        cache = m.KvCache(1, D, Hkv, page, pages=torch.from_numpy(pages).to(DEV))
        batch = batch_of(m, **c)
        ws = cache.workspace(batch, 1)
        m.moe_kv_append(cache, batch, x, x, ws=ws)
        assert m.moe_get_device_status(ws) == (1 if i else 0)
        got = cache.pages.cpu().numpy()
        untouched = [0] if i in (1, 2) else [0, 1] if i > 2 else []
        for p in untouched:
            assert np.array_equal(got[p], pages[p])
        assert not np.array_equal(got[3], pages[3])          # the other sequence's token is there
    # a rotation table shorter than the positions; rows beyond the call's tensors
    cache = m.KvCache(1, D, Hkv, page, n_pages=4)
    batch = batch_of(m, **good)
    ws = cache.workspace(batch, 1)
    cos = torch.ones(5, 4, device=DEV)
    m.moe_kv_append(cache, batch, x, x, cos=cos, sin=cos, ws=ws)
    assert m.moe_get_device_status(ws) == 1
    batch.c.n_tokens = 1
    m.moe_kv_append(cache, batch, x[:1], x[:1], ws=ws)
    assert m.moe_get_device_status(ws) == 0                   # only row 0 is run, and it is in order
    batch.q_start.copy_(torch.tensor([0, 2, 1], dtype=torch.int32))
    m.moe_kv_append(cache, batch, x[:1], x[:1], ws=ws)
    assert m.moe_get_device_status(ws) == 1


def test_append_refusals(m):
    D, Hkv, page = 64, 2, 16
    cache = m.KvCache(1, D, Hkv, page, n_pages=2)
    batch = batch_of(m, [1], [1], np.zeros((1, 1), np.int32))
    ws = cache.workspace(batch, 2)
    x = torch.zeros(1, 2 * Hkv + 2, D + 8, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(1, Hkv, D, dtype=torch.bfloat16, device=DEV)
    t = torch.ones(4, 6, device=DEV)
    with pytest.raises(m.MoeError) as e:
        m.moe_kv_append(cache, batch, k, k, cos=t, sin=t, ws=ws)                 # R = 12 is no multiple of 8
    assert e.value.status == 2
    with pytest.raises(m.MoeError) as e:
        m.moe_kv_append(cache, batch, k, k, cos=t[:0], sin=t[:0], ws=ws)
    assert e.value.status in (1, 2)
    with pytest.raises(m.MoeError) as e:
        m.moe_kv_append(cache, batch, k, k, ws=ws[:128])
    assert e.value.status == 5
    flat = torch.zeros(Hkv * D + 8, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(m.MoeError) as e:
        m.moe_kv_append(cache, batch, flat[4:4 + Hkv * D].view(1, Hkv, D), k, ws=ws)   # 8-byte aligned only
    assert e.value.status == 1
    with pytest.raises(AssertionError):
        m.moe_kv_append(cache, batch, x[:, :Hkv, :D], k, ws=ws)                  # heads are not contiguous
    for bad in ((3, 64, 1, 16), (1, 96, 1, 16), (1, 64, 0, 16), (1, 64, 1, 24), (1, 64, 1, 2048)):
        assert m.moe_kv_page_bytes(*bad) == 0
        with pytest.raises(m.MoeError):
            m.KvCache(*bad, n_pages=1)
    cache.c.page_stride = 8
    with pytest.raises(m.MoeError) as e:
        m.moe_kv_read(cache, batch, torch.zeros(1, Hkv, D, device=DEV), None, ws=ws)
    assert e.value.status == 2
