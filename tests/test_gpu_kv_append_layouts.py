"""Appends whose rows are spread over the lanes in the other ways: rotated parts of which a half is no multiple of 8, heads that
do not fill a warp, prompts long enough that a warp takes several rows in turn."""
import pytest

from tests import test_gpu_kv_cache as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import bit_moe_decode_gb300 as mod
    return mod


CASES = [
    # fmt, D, Hkv, Hq, page, new tokens, lengths after, rotated, interleaved
    (1, 128, 1, 1, 16, [3], [9], 8, False),
    (1, 64, 3, 6, 32, [2, 5], [2, 40], 24, False),
    (1, 128, 2, 2, 16, [4, 1], [4, 18], 120, False),
    (1, 64, 1, 3, 16, [7], [7], 24, True),
    (1, 128, 3, 9, 64, [6], [70], 16, False),
    (1, 64, 5, 5, 16, [1, 2], [1, 33], 48, False),
    (1, 64, 2, 6, 32, [700, 3], [700, 60], 64, False),
    (2, 64, 2, 6, 32, [700, 3], [700, 60], 64, False),
]


@pytest.mark.parametrize("case", CASES, ids=["%s-D%d-h%d-r%d%s" % ("mxfp4" if c[0] == 1 else "int4", c[1], c[2], c[7], "i" * c[8]) for c in CASES])
def test_append_and_read(m, case):
    C.test_append_and_read(m, case)
