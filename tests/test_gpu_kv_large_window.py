"""Windows near the largest 32-bit number, which callers pass for "none": the same bits as without a window, over sequences that are
shorter than their new tokens, empty, and long, on both attention kernels. Bounds as in test_gpu_kv_attention.py."""
import numpy as np
import pytest
import torch

from tests import test_gpu_kv_attention as A
from tests.test_gpu_kv_cache import DEV, batch_of, make_pages, table_for

pytestmark = pytest.mark.gpu
LARGE = [(1 << 30) - 1, 1 << 30, (1 << 31) - 8, (1 << 31) - 1]


@pytest.fixture(scope="module")
def m():
    import bit_moe_decode_gb300 as mod
    return mod


@pytest.mark.parametrize("fmt", [1, 2], ids=["mxfp4", "int4"])
@pytest.mark.parametrize("group,room", [(2, 0), (4, 0), (8, 2048), (16, 2048)])
def test_same_as_none(m, fmt, group, room):
    D, Hkv, page = 64, 2, 16
    Hq, ql, lens = Hkv * group, [4, 4, 8, 1, 4, 3], [1, 0, 2, 1, 4, 300]
    rng = np.random.default_rng(group)
    pages, _ = make_pages(rng, fmt, D, Hkv, page, sum(-(-n // page) for n in lens) + 2)
    pages = pages.copy()
    table = table_for(rng, lens, page, pages.shape[0])
    table = np.concatenate([table, np.full((len(lens), max(0, -(-room // page) - table.shape[1])), -1, np.int32)], 1)
    A.fill(rng, fmt, D, Hkv, page, pages, table, lens)
    cache = m.KvCache(fmt, D, Hkv, page, pages=torch.from_numpy(pages).to(DEV))
    batch = batch_of(m, ql, lens, table)
    ws = cache.workspace(batch, Hq)
    q = torch.from_numpy(rng.standard_normal((sum(ql), Hq, D)).astype(np.float32)).to(DEV).to(torch.bfloat16)
    outs = []
    for window in [0] + LARGE:
        out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), device=DEV)
        m.moe_kv_attention(cache, batch, q, 0.125, out, lse=lse, window=window, ws=ws)
        torch.cuda.synchronize()
        assert m.moe_get_device_status(ws) == 0
        outs.append((out, lse))
    for out, lse in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])


@pytest.mark.parametrize("window", LARGE)
def test_values(m, window):
    A.check(m, 1, 64, 1, 8, 16, [4, 8, 2], [1, 3, 200], window=window)
