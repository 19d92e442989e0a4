"""What a workspace holds after device errors: a call with device data out of range leaves it ready; whatever a call that ran out of
time left in it (counters, marks, parts), moe_workspace_init makes it ready again."""
import numpy as np
import pytest
import torch

from tests.test_gpu_kv_cache import DEV, batch_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group,T", [(4, 1), (8, 8)])
def test_ready_after_errors(group, T):
    import bit_moe_decode_gb300 as m
    D, Hkv, page, lens = 64, 2, 16, [900, 40, 301]
    cache = m.KvCache(1, D, Hkv, page, n_pages=100)
    table, at = np.full((3, 128), -1, np.int32), 0
    for b, n in enumerate(lens):
        table[b, :-(-n // page)] = np.arange(at, at - (-n // page))
        at += -(-n // page)
    batch, whole = batch_of(m, [T] * 3, lens, table), batch_of(m, lens, lens, table)
    gen = torch.Generator(DEV).manual_seed(4)
    x = torch.randn(sum(lens), 2 * Hkv, D, device=DEV, generator=gen).to(torch.bfloat16)
    q = torch.randn(3 * T, Hkv * group, D, device=DEV, generator=gen).to(torch.bfloat16)
    ws = cache.workspace(batch, Hkv * group)
    m.moe_kv_append(cache, whole, x[:, :Hkv], x[:, Hkv:], ws=ws)

    def attend(w=ws):
        out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), device=DEV)
        m.moe_kv_attention(cache, batch, q, D ** -0.5, out, lse=lse, ws=w)
        torch.cuda.synchronize()
        return out, lse, m.moe_get_device_status(w)

    want = attend()
    assert want[2] == 0
    good = batch.block_table.clone()
    batch.block_table[0, 20] = 100                     # no such page
    assert attend()[2] == 1
    batch.block_table.copy_(good)
    batch.seq_len[1] = 128 * page + 1                  # longer than the table
    assert attend()[2] == 1
    batch.seq_len[1] = lens[1]
    again = attend()
    assert again[2] == 0 and torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    ws.fill_(0x5A)
    m.moe_workspace_init(ws)
    again = attend()
    assert again[2] == 0 and torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
