"""A workspace for batches of up to some size serves every smaller one: its size never shrinks as the batch grows. No GPU."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def m():
    from bit_moe_decode_gb300 import build
    build.build()
    import bit_moe_decode_gb300 as mod
    mod.lib()
    return mod


@pytest.mark.parametrize("fmt", [1, 2], ids=["mxfp4", "int4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 16, 17, 33, 64, 65, 100, 128])
def test_grows_with_the_rows(m, fmt, D, group):
    cache = C.byref(m.moe_kv_cache_t(fmt, D, 2, 16, 1, 0, None))

    def size(max_q):
        return m.lib().moe_kv_workspace_bytes(cache, C.byref(m.moe_kv_batch_t(4, 4, max_q, 1, None, None, None)), 2 * group)

    sizes = [size(n) for n in (1, 2, 3, 4, 5, 6, 7, 8, 9, 16, 100, 5000, 1 << 30)]
    assert sizes[0] > 256 and sizes == sorted(sizes), sizes


def test_beyond_attention(m):
    """More than 128 query heads a KV head: attention takes no batch, append and read need the status word."""
    cache = C.byref(m.moe_kv_cache_t(1, 128, 2, 16, 1, 0, None))
    for max_q in (1, 8, 100):
        assert m.lib().moe_kv_workspace_bytes(cache, C.byref(m.moe_kv_batch_t(4, 4, max_q, 1, None, None, None)), 2 * 129) == 256
