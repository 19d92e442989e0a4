"""Nothing outside the outputs, the pages and the workspace is written: each lies between two bands of a byte pattern."""
import numpy as np
import pytest
import torch

from tests.test_gpu_kv_cache import DEV, batch_of

pytestmark = pytest.mark.gpu
BAND = 4096


def guarded(bands, shape, dtype):
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    raw = torch.full((n + 2 * BAND + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    off = BAND + (-(raw.data_ptr() + BAND)) % 256
    bands.append((raw, off, n))
    raw[off:off + n] = 0
    return raw[off:off + n].view(dtype).view(shape)


@pytest.mark.parametrize("fmt", [1, 2], ids=["mxfp4", "int4"])
@pytest.mark.parametrize("D,Hkv,Hq,T,lens", [(128, 2, 6, 1, [5, 40, 1]), (64, 1, 32, 3, [700, 3, 2049]), (64, 3, 24, 8, [300, 8])])
def test_cache_and_attention(fmt, D, Hkv, Hq, T, lens):
    import bit_moe_decode_gb300 as m
    page, n, bands = 32, len(lens), []
    need = sum(-(-v // page) for v in lens)
    pages = guarded(bands, (need, m.moe_kv_page_bytes(fmt, D, Hkv, page)), torch.uint8)
    cache = m.KvCache(fmt, D, Hkv, page, pages=pages)
    table, at = np.full((n, 70), -1, np.int32), 0
    for b, v in enumerate(lens):
        k = -(-v // page)
        table[b, :k] = np.arange(at, at + k)
        at += k
    gen = torch.Generator(DEV).manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(torch.bfloat16)  # noqa: E731
    whole = batch_of(m, lens, lens, table)
    ws = guarded(bands, (m.moe_kv_workspace_bytes(cache, whole, Hq),), torch.uint8)
    q_out = guarded(bands, (sum(lens), Hq, D), torch.bfloat16)
    x = rand(sum(lens), Hq + 2 * Hkv, D)
    m.moe_kv_append(cache, whole, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], q=x[:, :Hq], q_out=q_out, ws=ws)
    k, v = (guarded(bands, (sum(lens), Hkv, D), torch.float32) for _ in range(2))
    m.moe_kv_read(cache, whole, k, v, ws=ws)
    new = [min(T, v) for v in lens]
    batch = batch_of(m, new, lens, table)
    ws2 = guarded(bands, (m.moe_kv_workspace_bytes(cache, batch, Hq),), torch.uint8)
    out, lse = guarded(bands, (sum(new), Hq, D), torch.bfloat16), guarded(bands, (sum(new), Hq), torch.float32)
    for window in (0, 100):
        m.moe_kv_attention(cache, batch, rand(sum(new), Hq, D), D ** -0.5, out, lse=lse, window=window, ws=ws2)
    torch.cuda.synchronize()
    assert m.moe_get_device_status(ws) == 0 and m.moe_get_device_status(ws2) == 0
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    for raw, off, size in bands:
        assert (raw[:off] == 0xA5).all() and (raw[off + size:] == 0xA5).all()


@pytest.mark.parametrize("S,rows,V", [(1, 1, 1), (3, 4, 1001), (2, 1, 40003)])
def test_probabilities(S, rows, V):
    import bit_moe_decode_gb300 as m
    bands = []
    probs, top = guarded(bands, (S * rows, V), torch.float32), guarded(bands, (S * rows,), torch.int32)
    x = torch.randn(S * rows, V, generator=torch.Generator(DEV).manual_seed(1), device=DEV)
    m.moe_logits_probs(x, torch.tensor([[1.0, 0.0, 0.0, 0.7]], device=DEV).repeat(S, 1), probs, rows_per_seq=rows, top=top)
    torch.cuda.synchronize()
    assert (probs.sum(1) - 1).abs().max() < 1e-4 and (top == x.argmax(1)).all()
    for raw, off, size in bands:
        assert (raw[:off] == 0xA5).all() and (raw[off + size:] == 0xA5).all()
