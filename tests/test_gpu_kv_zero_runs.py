"""Runs of tokens whose values (or one block of them) are zero, or far smaller than the others', in batches where a warp streams many
units of keys: the tokens before and after keep their share. Against 64 bits over the values that moe_kv_read gives; bounds as in
test_gpu_kv_attention.py."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_kv_cache import DEV, batch_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import bit_moe_decode_gb300 as mod
    return mod


def check(m, fmt, D, Hkv, group, T, S, n, edit, room=0, kscale=1.0, seed=0):
    """S sequences of n keys; edit(k, v) changes their fp32 [S, n, Hkv, D] before they are appended."""
    page, Hq = 32, Hkv * group
    g = torch.Generator(DEV).manual_seed(seed + n)
    k, v = (torch.randn(S, n, Hkv, D, device=DEV, generator=g) for _ in range(2))
    k *= kscale
    edit(k, v)
    per = -(-n // page)
    table = np.full((S, max(per, -(-room // page))), -1, np.int32)
    table[:, :per] = np.random.default_rng(seed).permutation(S * per).reshape(S, per)
    cache = m.KvCache(fmt, D, Hkv, page, n_pages=S * per)
    whole, step = batch_of(m, [n] * S, [n] * S, table), batch_of(m, [T] * S, [n] * S, table)
    ws = cache.workspace(whole, Hq)
    m.moe_kv_append(cache, whole, *(x.reshape(S * n, Hkv, D).to(torch.bfloat16) for x in (k, v)), ws=ws)
    m.moe_kv_read(cache, whole, k.view(S * n, Hkv, D), v.view(S * n, Hkv, D), ws=ws)
    q = torch.randn(S * T, Hq, D, device=DEV, generator=g).to(torch.bfloat16)
    step_ws = cache.workspace(step, Hq)
    out, lse = torch.full_like(q, float("nan")), torch.full((S * T, Hq), float("nan"), device=DEV)
    m.moe_kv_attention(cache, step, q, D ** -0.5, out, lse=lse, ws=step_ws)
    torch.cuda.synchronize()
    assert m.moe_get_device_status(ws) == 0 and m.moe_get_device_status(step_ws) == 0
    worst = 0.0
    for s in range(S):
        K, V = (x[s].double().transpose(0, 1) for x in (k, v))                              # [Hkv, n, D]
        Q, o, z = (x[s * T:(s + 1) * T].double().reshape(T, Hkv, group, -1).permute(1, 0, 2, 3) for x in (q, out, lse))
        hide = torch.arange(n, device=DEV) > torch.arange(n - T, n, device=DEV)[:, None]
        x = (torch.einsum("htgd,hsd->htgs", Q, K) * D ** -0.5).masked_fill(hide[None, :, None], -math.inf)
        qk = torch.einsum("htgd,hsd->htgs", Q.abs(), K.abs()).amax(-1) * D ** -0.5
        rl, p = torch.logsumexp(x, -1), torch.softmax(x, -1)
        ref, pv = torch.einsum("htgs,hsd->htgd", p, V), torch.einsum("htgs,hsd->htgd", p, V.abs())
        eps = (D + 16) * 2.0 ** -24 * qk + 2.0 ** -21 * (rl.abs() + 1) + (n / 8 + 64) * 2.0 ** -24
        bound = 2.0 ** -8 * ref.abs() + (2.0 ** -10 + 2 * eps[..., None]) * pv + 1e-30
        assert bool(torch.isfinite(o).all() and torch.isfinite(z).all())
        worst = max(worst, float(((o - ref).abs() / bound).max()), float(((z[..., 0] - rl).abs() / eps).max()))
    assert worst <= 1.0, "error / bound %.3g" % worst


SHAPES = [(4, 1, 96, 4, 0), (8, 2, 80, 4, 0), (8, 4, 96, 2, 2048), (16, 8, 40, 2, 2048)]   # group, T, S, Hkv, room


@pytest.mark.parametrize("fmt", [1, 2], ids=["mxfp4", "int4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group,T,S,Hkv,room", SHAPES)
def test_zero_values(m, fmt, D, group, T, S, Hkv, room):
    """From every sequence's start, in its middle or to its end; all blocks, or one of the second head's"""
    n = 1000

    def edit(k, v):
        rng = np.random.default_rng(1)
        for s in range(S):
            first = int(rng.integers(0, n - 100))
            first, last = [(0, 150), (first, first + int(rng.integers(40, 400))), (700, n - T)][s % 3]
            v[s, first:last, 0] = 0
            v[s, first:last, 1, :32] = 0

    check(m, fmt, D, Hkv, group, T, S, n, edit, room)


@pytest.mark.parametrize("fmt", [1, 2], ids=["mxfp4", "int4"])
@pytest.mark.parametrize("group,T,S,Hkv,room", SHAPES)
@pytest.mark.parametrize("size", [2.0 ** -20, 2.0 ** -60])
@pytest.mark.parametrize("kscale", [1.0, 16.0])
def test_runs_of_tiny_values(m, fmt, group, T, S, Hkv, room, size, kscale):
    """Values far below the others' in whole units, also where (at the larger scores) their weights go down to 2^-100."""
    n = 1000

    def edit(k, v):
        v[::2, 100:300] *= size
        v[1::2, 500:] *= size

    check(m, fmt, 64, Hkv, group, T, S, n, edit, room, kscale)
