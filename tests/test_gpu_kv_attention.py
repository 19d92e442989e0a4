"""Attention over the 4-bit paged KV cache against 64 bits.

Bounds, per element: the output is rounded to bf16 (2^-8 relative covers the half step and the edge of a binade), each
weight times its value scale once to binary16 (2^-11 of sum p |v|, padded to 2^-10 for the joined parts), and a score is off
by at most eps = (D + 16) 2^-24 sum |q k| scale + 2^-21 |x| through fp32 sums, which moves the output by 2 eps sum p |v| and
lse by eps; the fp32 sums of p add (keys / 8 + 64) 2^-24."""
import numpy as np
import pytest
import torch

from tests import _kv_ref as R
from tests.test_gpu_kv_cache import DEV, batch_of, make_pages, sub_view, table_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import bit_moe_decode_gb300 as mod
    return mod


def fill(rng, fmt, D, Hkv, page, pages, table, lens, kscale=1.0, vscale=None):
    """Plausible blocks at every position of every sequence, drawn directly as codes and scales; the rest stays random."""
    view = sub_view(pages, fmt, D, Hkv, page)
    nb, sb = D // 32, 1 if fmt == R.MXFP4 else 2
    for b, n in enumerate(lens):
        for s in range(-(-int(n) // 16)):
            p, i = divmod(s * 16, page)
            for h in range(Hkv):
                sub = view[table[b, p], h, i // 16]
                keep = n - s * 16
                fresh = rng.integers(0, 256, sub.size, dtype=np.uint8)
                if keep >= 16:
                    sub[:16 * D] = fresh[:16 * D]
                else:
                    sub[:16 * D] = fresh[:16 * D]      # codes are finite whatever they are
                for at, sc in ((16 * D, kscale), (16 * D + 16 * nb * sb, 1.0)):
                    vals = 0.4 * sc * np.exp(0.4 * rng.standard_normal((16, nb)))
                    if at != 16 * D and vscale is not None:
                        vals = vals * vscale(b, s * 16 + np.arange(16))[:, None]
                    if fmt == R.MXFP4:
                        raw = np.clip(np.rint(np.log2(vals)) + 127, 1, 190).astype(np.uint8)
                    else:
                        raw = (R.bf16(vals.astype(np.float32)).view(np.uint32) >> 16).astype(np.uint16).view(np.uint8).reshape(16, -1)
                    rows = min(16, keep)               # scales past the end stay random: NaN and huge ones among them
                    sub[at:at + 16 * nb * sb].reshape(16, -1)[:rows] = raw.reshape(16, -1)[:rows]
    pages[:, :view[0].size] = view.reshape(pages.shape[0], -1)


def check(m, fmt, D, Hkv, Hq, page, ql, lens, window=0, scale=None, seed=0, kscale=1.0, vscale=None, qmul=1.0, extra=0, stream=None):
    rng = np.random.default_rng(seed + sum(lens) + 13 * D + fmt)
    pages, _ = make_pages(rng, fmt, D, Hkv, page, sum(-(-n // page) for n in lens) + 2, extra=extra)
    table = table_for(rng, lens, page, pages.shape[0])
    pages = pages.copy()
    fill(rng, fmt, D, Hkv, page, pages, table, lens, kscale, vscale)
    T, scale = sum(ql), scale if scale is not None else D ** -0.5
    q = R.bf16((qmul * rng.standard_normal((T, Hq, D))).astype(np.float32))
    cache = m.KvCache(fmt, D, Hkv, page, pages=torch.from_numpy(pages).to(DEV))
    batch = batch_of(m, ql, lens, table)
    ws = cache.workspace(batch, Hq)
    wide = torch.zeros(T, Hq + 1, D, dtype=torch.bfloat16, device=DEV)
    wide[:, :Hq] = torch.from_numpy(q).to(DEV)
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, Hq), float("nan"), device=DEV)
    torch.cuda.synchronize()
    for _ in range(2):      # a workspace serves call after call
        m.moe_kv_attention(cache, batch, wide[:, :Hq], scale, out, lse=lse, window=window, ws=ws, stream=stream)
    torch.cuda.synchronize()
    first = out.clone(), lse.clone()
    torch.cuda.synchronize()
    m.moe_kv_attention(cache, batch, wide[:, :Hq], scale, out, lse=lse, window=window, ws=ws, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(first[0], out) and torch.equal(first[1], lse), "the same call gives the same bits"
    assert m.moe_get_device_status(ws) == 0
    o, z = out.float().cpu().numpy().astype(float), lse.cpu().numpy().astype(float)
    view = sub_view(pages, fmt, D, Hkv, page)
    worst, t, group = 0.0, 0, Hq // Hkv
    for b, n in enumerate(ql):
        for h in range(Hkv):
            K, V = R.sequence_kv(fmt, D, view, table[b], page, h, lens[b]) if lens[b] else (np.zeros((0, D)),) * 2
            for j in range(n):
                pos = lens[b] - n + j
                for g in range(group):
                    row = t + j, h * group + g
                    ref, rl, pv, qk = R.attend(q[row].astype(float), K, V, scale, pos, window)
                    if rl == -np.inf:
                        assert not o[row].any() and z[row] == -np.inf
                        continue
                    eps = (D + 16) * 2.0 ** -24 * qk + 2.0 ** -21 * (abs(rl) + 1) + (lens[b] / 8 + 64) * 2.0 ** -24
                    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + 2 * eps) * pv + 1e-30
                    worst = max(worst, float(np.max(np.abs(o[row] - ref) / bound)), abs(z[row] - rl) / eps)
        t += n
    assert worst <= 1.0, "error / bound %.3g" % worst
    return worst


@pytest.mark.parametrize("fmt", [1, 2], ids=["mxfp4", "int4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [31], [32], [33], [63], [65], [129], [517]], ids=lambda v: str(v[0]))
def test_decode_lengths(m, fmt, D, lens):
    check(m, fmt, D, 2, 8, 16, [1], lens)


@pytest.mark.parametrize("fmt", [1, 2], ids=["mxfp4", "int4"])
@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 9, 12, 16])
@pytest.mark.parametrize("T", [1, 3, 8])
def test_groups_and_rows(m, fmt, group, T):
    """Every number of query rows a KV head, from 1 to 128."""
    check(m, fmt, 128, 2, 2 * group, 32, [T, T], [77, T])


@pytest.mark.parametrize("fmt,D", [(1, 64), (2, 128), (1, 128), (2, 64)])
@pytest.mark.parametrize("page", [16, 48, 64, 1024])
def test_ragged_batch(m, fmt, D, page):
    """Lengths from none to hundreds, rows from none to five, padding slots, sequences shorter than their rows."""
    check(m, fmt, D, 3, 6, page, [1, 2, 0, 5, 1, 1, 4, 3], [300, 2, 40, 161, 0, 1, 2, 1000], extra=16)


@pytest.mark.parametrize("fmt", [1, 2], ids=["mxfp4", "int4"])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 33, 100, 5000])
def test_window(m, fmt, window):
    check(m, fmt, 128, 1, 4, 16, [3, 1, 8], [260, 99, 41], window=window)


def test_window_leaves_earlier_pages_alone(m):
    """Pages wholly before the window may have been given away: their table entries are not read."""
    D, page, n, w = 64, 16, 200, 40
    rng = np.random.default_rng(2)
    pages, _ = make_pages(rng, 1, D, 1, page, 13)
    table = np.arange(13, dtype=np.int32)[None]
    fill(rng, 1, D, 1, page, pages, table, [n])
    cache = m.KvCache(1, D, 1, page, pages=torch.from_numpy(pages).to(DEV))
    q = torch.randn(2, 4, D, device=DEV).to(torch.bfloat16)
    outs = []
    for gone in (False, True):
        t = table.copy()
        if gone:
            t[0, :(n - 2 - w + 1) // page] = -1
        batch = batch_of(m, [2], [n], t)
        ws = cache.workspace(batch, 4)
        out = torch.empty(2, 4, D, dtype=torch.bfloat16, device=DEV)
        m.moe_kv_attention(cache, batch, q, 0.125, out, window=w, ws=ws)
        assert m.moe_get_device_status(ws) == 0
        outs.append(out)
    assert torch.equal(*outs)


@pytest.mark.parametrize("fmt", [1, 2], ids=["mxfp4", "int4"])
def test_many_sequences(m, fmt):
    rng = np.random.default_rng(9)
    lens = [int(v) for v in rng.integers(0, 200, 130)]
    check(m, fmt, 64, 2, 2, 16, [1] * 130, lens)


@pytest.mark.parametrize("fmt", [1, 2], ids=["mxfp4", "int4"])
@pytest.mark.parametrize("rows", [(8, 1), (1, 1), (4, 8), (8, 4)])
def test_long_context(m, fmt, rows):
    """One sequence over all of the GPU: its parts are joined across CTAs."""
    group, T = rows
    check(m, fmt, 128, 1, group, 64, [T], [9001])


def test_scores_large_and_small(m):
    """A softmax of one key, of equal keys, a zero query, and scores of hundreds."""
    for kscale, qmul in ((30.0, 30.0), (1e-3, 1e-3), (1.0, 0.0), (1.0, 1e4)):
        check(m, 1, 128, 1, 4, 32, [2], [300], kscale=kscale, qmul=qmul)
        check(m, 2, 64, 1, 4, 32, [2], [300], kscale=kscale, qmul=qmul)


@pytest.mark.parametrize("fmt", [1, 2], ids=["mxfp4", "int4"])
@pytest.mark.parametrize("size", [2.0 ** 40, 2.0 ** 20, 2.0 ** -20, 2.0 ** -60])
def test_values_of_very_different_size(m, fmt, size):
    """Some tokens' values are many powers of two larger or smaller than the others', early, late and alone in a block: the
    bound goes by sum p |v| of the row, so it holds whichever tokens a row weighs."""
    for where in (lambda pos: pos < 3, lambda pos: pos % 97 == 50, lambda pos: pos > 200, lambda pos: pos >= 0):
        check(m, fmt, 128, 1, 4, 16, [3], [333], vscale=lambda b, pos: np.where(where(pos), size, 1.0), kscale=3.0, qmul=2.0)


def test_cache_of_more_than_four_gigabytes(m):
    """Page offsets beyond 2^32 bytes."""
    D, Hkv, page, fmt = 128, 8, 64, 1
    nbytes = m.moe_kv_page_bytes(fmt, D, Hkv, page)
    n_pages = (5 << 30) // nbytes
    rng = np.random.default_rng(4)
    small, _ = make_pages(rng, fmt, D, Hkv, page, 4)
    table = np.arange(4, dtype=np.int32)[None]
    fill(rng, fmt, D, Hkv, page, small, table, [250])
    q = torch.randn(1, 32, D, device=DEV).to(torch.bfloat16)
    outs = []
    for big in (False, True):
        pages = torch.zeros((n_pages if big else 4, nbytes), dtype=torch.uint8, device=DEV)
        ids = np.array([[n_pages - 1, 3, n_pages - 2, n_pages // 2]], np.int32) if big else table
        pages[torch.from_numpy(ids[0].astype(np.int64)).to(DEV)] = torch.from_numpy(small).to(DEV)
        cache = m.KvCache(fmt, D, Hkv, page, pages=pages)
        batch = batch_of(m, [1], [250], ids)
        ws = cache.workspace(batch, 32)
        out = torch.empty(1, 32, D, dtype=torch.bfloat16, device=DEV)
        k = torch.randn(1, Hkv, D, device=DEV, generator=torch.Generator(DEV).manual_seed(1)).to(torch.bfloat16)
        m.moe_kv_append(cache, batch, k, k, ws=ws)
        m.moe_kv_attention(cache, batch, q, 0.1, out, ws=ws)
        assert m.moe_get_device_status(ws) == 0
        outs.append(out.cpu())
        del pages, cache
    assert torch.equal(*outs)


def test_side_stream_and_graph(m):
    """On another stream, and replayed from a graph after the lengths have grown in place."""
    s = torch.cuda.Stream()
    check(m, 1, 128, 2, 8, 32, [1, 4], [100, 300], stream=s)
    D, Hkv, Hq, page = 64, 1, 4, 16
    cache = m.KvCache(2, D, Hkv, page, n_pages=8)
    batch = batch_of(m, [1], [1], np.arange(8, dtype=np.int32)[None])
    ws = cache.workspace(batch, Hq)
    x = torch.zeros(1, Hq + 2, D, dtype=torch.bfloat16, device=DEV)
    q = torch.empty(1, Hq, D, dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(q)

    def step():
        m.moe_kv_append(cache, batch, x[:, Hq:Hq + 1], x[:, Hq + 1:], q=x[:, :Hq], q_out=q, ws=ws, stream=torch.cuda.current_stream())
        m.moe_kv_attention(cache, batch, q, 0.125, out, ws=ws, stream=torch.cuda.current_stream())

    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    data = torch.randn(40, Hq + 2, D, device=DEV).to(torch.bfloat16)
    for i in range(40):
        x.copy_(data[i:i + 1])
        batch.seq_len.fill_(i + 1)
        g.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    pages = cache.pages.clone()
    cache.pages.zero_()
    whole = batch_of(m, [40], [40], np.arange(8, dtype=np.int32)[None])
    m.moe_kv_append(cache, whole, data[:, Hq:Hq + 1], data[:, Hq + 1:], ws=ws)
    step()
    torch.cuda.synchronize()
    assert torch.equal(replayed, out) and torch.equal(pages, cache.pages)
    assert m.moe_get_device_status(ws) == 0


def test_device_data_out_of_range(m):
    """Counts as an empty sequence (zeros, -inf) or reads page 0, and is recorded; the others are not touched by it."""
    D, page = 64, 16
    rng = np.random.default_rng(3)
    pages, _ = make_pages(rng, 1, D, 1, page, 6)
    table = np.array([[0, 1], [2, 3], [4, 5]], np.int32)
    fill(rng, 1, D, 1, page, pages, table, [20, 30, 32])
    cache = m.KvCache(1, D, 1, page, pages=torch.from_numpy(pages).to(DEV))
    q = torch.randn(3, 2, D, device=DEV).to(torch.bfloat16)

    def run(lens, tab, ql=(1, 1, 1), max_q=None):
        batch = batch_of(m, list(ql), lens, tab)
        if max_q:
            batch.c.max_q = max_q
        ws = cache.workspace(batch, 2)
        out = torch.full((3, 2, D), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((3, 2), 7.0, device=DEV)
        m.moe_kv_attention(cache, batch, q, 0.125, out, lse=lse, ws=ws)
        st = m.moe_get_device_status(ws)
        m.moe_workspace_init(ws)
        return out.float().cpu(), lse.cpu(), st

    ref, ref_lse, st = run([20, 30, 32], table)
    assert st == 0
    for lens, tab in (([20, 33, 32], table), ([20, -1, 32], table)):
        out, lse, st = run(lens, tab)
        assert st == 1 and not out[1].any() and torch.isneginf(lse[1]).all()
        assert torch.equal(out[[0, 2]], ref[[0, 2]]) and torch.equal(lse[[0, 2]], ref_lse[[0, 2]])
    bad = table.copy()
    bad[1, 1] = 6
    out, lse, st = run([20, 30, 32], bad)
    assert st == 1 and torch.isfinite(out).all() and torch.equal(out[[0, 2]], ref[[0, 2]])
    out, lse, st = run([20, 30], table[:2], ql=(2, 1), max_q=1)     # more rows than max_q
    assert st == 1 and not out[:2].any() and torch.equal(out[2], run([20, 30], table[:2], ql=(2, 1))[0][2])


def test_refusals(m):
    D, page = 64, 16
    cache = m.KvCache(1, D, 2, page, n_pages=2)
    batch = batch_of(m, [1], [1], np.zeros((1, 1), np.int32))
    ws = cache.workspace(batch, 4)
    q = torch.zeros(1, 4, D, dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(q)

    def status(**kw):
        a = dict(cache=cache, batch=batch, q=q, scale=0.1, out=out, ws=ws)
        a.update(kw)
        with pytest.raises(m.MoeError) as e:
            m.moe_kv_attention(**a)
        return e.value.status

    q3 = torch.zeros(1, 3, D, dtype=torch.bfloat16, device=DEV)
    assert status(q=q3, out=torch.empty_like(q3)) == 2                    # 3 query heads over 2 KV heads
    assert status(window=-1) == 2
    assert status(scale=float("nan")) == 1 and status(scale=float("inf")) == 1
    assert status(ws=ws[:64]) == 5
    assert status(ws=ws[16:]) in (1, 5)
    batch.c.max_q = 9
    assert status() == 2
    batch.c.max_q = 8
    q40 = torch.zeros(1, 40, D, dtype=torch.bfloat16, device=DEV)
    assert status(q=q40, out=torch.empty_like(q40)) == 2                  # 8 x 20 query rows a KV head
    batch.c.max_q, batch.c.n_seqs = 1, 1025
    assert status() == 2
    batch.c.n_seqs, cache.c.n_pages = 1, 0
    assert status() == 2
