"""One workspace, sized for the largest batch, serves batches of other sizes in any order."""
import numpy as np
import pytest
import torch

from tests import test_gpu_kv_attention as A
from tests.test_gpu_kv_cache import DEV, batch_of, make_pages, table_for

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [1, 2], ids=["mxfp4", "int4"])
def test_shared_by_batches(fmt):
    import bit_moe_decode_gb300 as m
    D, Hkv, Hq, page = 64, 2, 16, 16
    rng = np.random.default_rng(5)
    lens = [int(v) for v in rng.integers(60, 700, 60)]
    pages, _ = make_pages(rng, fmt, D, Hkv, page, sum(-(-n // page) for n in lens) + 2)
    pages = pages.copy()
    table = table_for(rng, lens, page, pages.shape[0])
    # (room for 2048 keys, so that four new tokens, 32 rows a KV head, go to the tensor cores)
    table = np.concatenate([table, np.full((60, 128 - table.shape[1]), -1, np.int32)], 1)
    A.fill(rng, fmt, D, Hkv, page, pages, table, lens)
    cache = m.KvCache(fmt, D, Hkv, page, pages=torch.from_numpy(pages).to(DEV))
    batches = []
    for n, T in ((2, 1), (60, 4), (7, 4), (60, 1), (1, 8), (33, 2), (60, 4)):
        batch = batch_of(m, [T] * n, lens[:n], table[:n])
        q = torch.from_numpy(rng.standard_normal((n * T, Hq, D)).astype(np.float32)).to(DEV).to(torch.bfloat16)
        batches.append((batch, q))
    shared = cache.workspace(batch_of(m, [8] * 60, lens, table), Hq)
    for batch, q in batches:
        outs = []
        for ws in (cache.workspace(batch, Hq), shared, shared):
            out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), device=DEV)
            m.moe_kv_attention(cache, batch, q, 0.125, out, lse=lse, ws=ws)
            torch.cuda.synchronize()
            assert m.moe_get_device_status(ws) == 0
            outs.append((out, lse))
        for out, lse in outs[1:]:
            assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])
