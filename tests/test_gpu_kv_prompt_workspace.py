"""A workspace made for a prompt's batch serves the decode steps that follow, with the bits of one made for them."""
import numpy as np
import pytest
import torch

from tests.test_gpu_kv_cache import DEV, batch_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,T", [(2, 1), (8, 4), (34, 7)])
def test_prompt_then_decode(Hq, T):
    import bit_moe_decode_gb300 as m
    D, Hkv, page, n = 64, 2, 16, 300
    cache = m.KvCache(1, D, Hkv, page, n_pages=20)
    table = np.concatenate([np.arange(20, dtype=np.int32), np.full(108, -1, np.int32)])[None]
    prompt, step = batch_of(m, [n], [n], table), batch_of(m, [T], [n], table)
    ws = cache.workspace(prompt, Hq)
    gen = torch.Generator(DEV).manual_seed(3)
    x = torch.randn(n, Hq + 2 * Hkv, D, device=DEV, generator=gen).to(torch.bfloat16)
    m.moe_kv_append(cache, prompt, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], ws=ws)
    outs = []
    for w in (ws, cache.workspace(step, Hq)):
        out = torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
        m.moe_kv_attention(cache, step, x[:T, :Hq], D ** -0.5, out, ws=w)
        torch.cuda.synchronize()
        assert m.moe_get_device_status(w) == 0
        outs.append(out)
    assert torch.equal(*outs) and torch.isfinite(outs[0].float()).all()
