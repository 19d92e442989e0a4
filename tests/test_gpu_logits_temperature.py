"""Temperatures at the ends of their range: infinity leaves the uniform distribution over the tokens that are allowed and not at
-inf; the largest finite ones come near it. (x / T differs from 0 by at most 2^-100 there, the sum is of ones: 2^-20 covers
rounding.)"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 5, 1000, 1001, 32768, 50001, 300001])
@pytest.mark.parametrize("temperature", [float("inf"), 3.4e38])
def test_hot(dtype, V, temperature):
    import bit_moe_decode_gb300 as m
    rng = np.random.default_rng(V)
    x = torch.from_numpy((3 * rng.standard_normal((4, V + 3))).astype(np.float32)).to(dtype)[:, :V]
    x[1, V // 2] = float("-inf")
    x[2, V // 3] = float("nan")
    ok = rng.random((4, V)) < 0.7
    ok[:, 0] = True
    ok[0] = True
    words = (V + 31) // 32
    bits = np.zeros((4, words * 32), bool)
    bits[:, :V] = ok
    allowed = torch.from_numpy(np.packbits(bits, axis=-1, bitorder="little").view(np.int32)).to(DEV)
    par = torch.tensor([[1.0, 0.0, 0.0, temperature]] * 4, device=DEV)
    probs, top = torch.full((4, V), float("nan"), device=DEV), torch.full((4,), -7, dtype=torch.int32, device=DEV)
    m.moe_logits_probs(x.to(DEV), par, probs, allowed=allowed, top=top)
    torch.cuda.synchronize()
    v = x.double().numpy()
    v = np.where(np.isnan(v) | ~ok, -np.inf, v)
    for r in range(4):
        n = int((v[r] > -np.inf).sum())
        want = (v[r] > -np.inf) / max(n, 1)
        assert np.all(np.abs(probs[r].double().cpu().numpy() - want) <= 2.0 ** -20 * want)
        assert int(top[r]) == (int(np.argmax(v[r])) if n else -1)
