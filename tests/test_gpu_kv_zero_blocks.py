"""Keys and values that are zero in some blocks, or altogether: their blocks have the smallest scale, far from the others'.
Bounds as in test_gpu_kv_attention.py."""
import numpy as np
import pytest

from tests import _kv_ref as R
from tests import test_gpu_kv_attention as A
from tests.test_gpu_kv_cache import sub_view, table_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import bit_moe_decode_gb300 as mod
    return mod


@pytest.mark.parametrize("fmt", [1, 2], ids=["mxfp4", "int4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group,T", [(4, 1), (8, 2), (8, 4), (8, 8)])
def test_zero_blocks(m, monkeypatch, fmt, D, group, T):
    """A tenth of the tokens is zero; of the others a tenth has one block of zeros in K or V."""
    nb, sb = D // 32, 1 if fmt == R.MXFP4 else 2
    fill, rng = A.fill, np.random.default_rng(D + fmt)

    def with_zeros(rng_, fmt_, D_, Hkv, page, pages, table, lens, *args):
        fill(rng_, fmt_, D_, Hkv, page, pages, table, lens, *args)
        view = sub_view(pages, fmt, D, Hkv, page)
        for b, n in enumerate(lens):
            for s in range(n):
                whole, some = rng.random() < 0.1, rng.random() < 0.1
                if not (whole or some):
                    continue
                p, i = divmod(s, page)
                for h in range(Hkv):
                    sub, slot = view[table[b, p], h, i // 16], i % 16
                    for blk in range(nb) if whole else [int(rng.integers(nb))]:
                        for is_v in ((False, True) if whole else (rng.random() < 0.5,)):
                            at = 16 * D + (16 * nb * sb if is_v else 0) + (slot * nb + blk) * sb
                            # the encoders' scale of a block of zeros: the smallest (MXFP4), 1e-8 times a candidate / 7 (INT4)
                            sub[at:at + sb] = np.frombuffer(b"\x01" if sb == 1 else b"\xa8\x30", np.uint8)
                            if is_v:
                                for r in range(8):
                                    w = 8 * D + ((((slot >> 3) * 8 + r) * 4 + ((slot >> 1) & 3)) * nb + blk) * 4
                                    if fmt == R.MXFP4:
                                        sub[w:w + 4] &= 0x0F if slot & 1 else 0xF0
                                    else:
                                        sub[w + 2 * (slot & 1):w + 2 * (slot & 1) + 2] = 0
                            else:
                                for c in range(4):
                                    w = slot * (D // 2) + (c * nb + blk) * 4
                                    sub[w:w + 4] = 0
        pages[:, :view[0].size] = view.reshape(pages.shape[0], -1)

    monkeypatch.setattr(A, "fill", with_zeros)
    monkeypatch.setattr(A, "table_for", lambda r, lens, page, n: np.concatenate(
        [table_for(r, lens, page, n), np.full((len(lens), 64), -1, np.int32)], 1))
    A.check(m, fmt, D, 1, group, 32, [T, T], [333, 1100])
