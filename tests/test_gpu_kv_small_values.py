"""Values that are all small (2^-6 to 2^-40 of 1) over few keys: an output's relative accuracy does not depend on their common size,
also where only keys of small weight have a code in a dimension. Bounds as in test_gpu_kv_attention.py."""
import numpy as np
import pytest

from tests import test_gpu_kv_attention as A
from tests.test_gpu_kv_cache import table_for

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [1, 2], ids=["mxfp4", "int4"])
@pytest.mark.parametrize("size", [2.0 ** 20, 1.0, 2.0 ** -6, 2.0 ** -9, 2.0 ** -11, 2.0 ** -40])
@pytest.mark.parametrize("group,T,room", [(4, 1, 0), (4, 4, 0), (8, 4, 2048)])
def test_few_keys(monkeypatch, fmt, size, group, T, room):
    import bit_moe_decode_gb300 as m
    monkeypatch.setattr(A, "table_for", lambda r, lens, page, n: np.concatenate(
        [table_for(r, lens, page, n), np.full((len(lens), -(-room // page)), -1, np.int32)], 1))
    lens = [5 + b % 9 for b in range(48)]
    A.check(m, fmt, 64, 2, 2 * group, 16, [T] * 48, lens, vscale=lambda b, pos: np.where(pos >= 0, size, 0.0), kscale=2.0, qmul=1.5)
