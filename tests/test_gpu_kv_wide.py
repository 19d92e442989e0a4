"""Attention of more than 16 query rows a KV head, where the block table leaves room for long sequences: these calls go to the
tensor cores first, and what that kernel's binary16 windows cannot hold is done again. Bounds as in
test_gpu_kv_attention.py."""
import numpy as np
import pytest
import torch

from tests import _kv_ref as R
from tests import test_gpu_kv_attention as A
from tests.test_gpu_kv_cache import DEV, batch_of, table_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import bit_moe_decode_gb300 as mod
    return mod


@pytest.fixture(autouse=True)
def long_table(monkeypatch):
    """Block tables with room for 2048 keys; entries that no sequence reaches are -1."""
    def wide(rng, lens, page, n_pages):
        t = table_for(rng, lens, page, n_pages)
        return np.concatenate([t, np.full((t.shape[0], max(0, -(-2048 // page) - t.shape[1])), -1, np.int32)], 1)
    monkeypatch.setattr(A, "table_for", wide)


@pytest.mark.parametrize("fmt", [1, 2], ids=["mxfp4", "int4"])
@pytest.mark.parametrize("group,T", [(17, 1), (6, 3), (8, 4), (11, 3), (5, 7), (8, 8), (9, 8), (32, 4)])
def test_rows(m, fmt, group, T):
    A.check(m, fmt, 128 if group % 2 else 64, 1, group, 16, [T], [200 + group])


@pytest.mark.parametrize("fmt,D", [(1, 64), (2, 128), (1, 128), (2, 64)])
@pytest.mark.parametrize("n", [4, 15, 16, 17, 127, 128, 129, 255, 257, 640])
def test_lengths(m, fmt, D, n):
    A.check(m, fmt, D, 1, 8, 16, [4], [n])


@pytest.mark.parametrize("fmt,D", [(1, 128), (2, 64)])
@pytest.mark.parametrize("page", [16, 48, 1024])
def test_ragged_batch(m, fmt, D, page):
    """Sequences of fewer new tokens than the largest (rows that are not there), empty ones, and ones of a single key."""
    A.check(m, fmt, D, 2, 16, page, [8, 1, 0, 3, 1, 8, 1], [700, 1, 0, 130, 0, 8, 400], extra=32)


@pytest.mark.parametrize("fmt", [1, 2], ids=["mxfp4", "int4"])
@pytest.mark.parametrize("window", [1, 100, 248, 255, 256, 257, 500])
def test_window(m, fmt, window):
    """With 128 rows a window of 256 - 8 and more goes to the tensor cores."""
    A.check(m, fmt, 64, 1, 16, 16, [8, 5], [700, 300], window=window)


def test_window_of_a_layer(m):
    A.check(m, 2, 128, 2, 12, 32, [3, 3, 2], [2500, 1100, 90], window=1024)


def test_many_sequences(m):
    lens = [int(v) for v in np.random.default_rng(3).integers(4, 150, 90)]
    A.check(m, 1, 64, 2, 16, 16, [4] * 90, lens)


@pytest.mark.parametrize("fmt", [1, 2], ids=["mxfp4", "int4"])
@pytest.mark.parametrize("group,T", [(8, 3), (8, 8)])
def test_long_context(m, fmt, group, T):
    A.check(m, fmt, 128, 1, group, 64, [T], [9001])


def test_scores_large_and_small(m):
    for kscale, qmul in ((30.0, 30.0), (1e-3, 1e-3), (1.0, 0.0), (1.0, 1e4), (1.0, 6.0)):
        A.check(m, 1, 128, 1, 8, 32, [4], [300], kscale=kscale, qmul=qmul)
        A.check(m, 2, 64, 1, 8, 32, [4], [300], kscale=kscale, qmul=qmul)


@pytest.mark.parametrize("fmt", [1, 2], ids=["mxfp4", "int4"])
@pytest.mark.parametrize("size", [2.0 ** 40, 2.0 ** 7, 2.0 ** -9, 2.0 ** -60])
def test_values_of_very_different_size(m, fmt, size):
    for where in (lambda pos: pos < 3, lambda pos: pos % 97 == 50, lambda pos: pos > 200, lambda pos: pos >= 0):
        A.check(m, fmt, 128, 1, 8, 16, [3], [333], vscale=lambda b, pos: np.where(where(pos), size, 1.0), kscale=3.0, qmul=2.0)


def test_one_sequence_of_several_is_done_again(m):
    """Only the second has values beyond the window; the marks are gone afterwards (the calls inside repeat)."""
    A.check(m, 1, 128, 2, 16, 16, [4, 4, 4], [300, 260, 500],
            vscale=lambda b, pos: np.where((b == 1) & (pos > 200), 2.0 ** 30, 1.0))


def test_graph(m):
    """Replayed from a graph as the lengths grow in place from one key to several tiles."""
    D, Hq, page = 64, 8, 16
    cache = m.KvCache(1, D, 1, page, n_pages=32)
    table = np.concatenate([np.arange(32, dtype=np.int32), np.full(96, -1, np.int32)])[None]
    batch = batch_of(m, [3], [3], table)
    ws = cache.workspace(batch, Hq)
    gen = torch.Generator(DEV).manual_seed(2)
    data = torch.randn(402, Hq + 2, D, device=DEV, generator=gen).to(torch.bfloat16)
    m.moe_kv_append(cache, batch_of(m, [402], [402], table), data[:, Hq:Hq + 1], data[:, Hq + 1:], ws=ws)
    q, out = data[:3, :Hq].contiguous(), torch.empty(3, Hq, D, dtype=torch.bfloat16, device=DEV)
    m.moe_kv_attention(cache, batch, q, 0.125, out, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_kv_attention(cache, batch, q, 0.125, out, ws=ws, stream=torch.cuda.current_stream())
    for n in (3, 100, 128, 129, 402):
        batch.seq_len.fill_(n)
        g.replay()
        torch.cuda.synchronize()
        again = out.clone()
        torch.cuda.synchronize()
        m.moe_kv_attention(cache, batch, q, 0.125, out, ws=ws)
        torch.cuda.synchronize()
        assert torch.equal(again, out) and torch.isfinite(out.float()).all()
    assert m.moe_get_device_status(ws) == 0
