"""examples/verify_step.py: append, attention, experts, probabilities and acceptance as one decoding step."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "verify_step.py")
    spec = importlib.util.spec_from_file_location("verify_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("seqs,drafts", [(2, 3), (1, 7), (8, 0)])
def test_generates(ex, seqs, drafts):
    """The lengths follow what was accepted, and the same seeds give the same tokens."""
    runs = []
    for _ in range(2):
        d = ex.Decoder(seqs, drafts)
        out = d.generate(list(range(5, 5 + seqs)), 12)
        assert all(0 <= t < d.V for o in out for t in o)
        assert all(12 + 1 <= len(o) <= 12 * (1 + drafts) + 1 for o in out)
        assert d.seq_len.tolist() == [len(o) - 1 for o in out]       # (the last token is not in the cache yet)
        assert d.counts.sum(1).tolist() == [len(o) - 1 for o in out]
        runs.append(out)
    assert runs[0] == runs[1]


def test_verified_rows_see_what_single_rows_see(ex):
    """The tokens that a run with drafts produced, fed one by one to a decoder without drafts, put the same keys and values
    into the first layer's cache (they depend on the tokens and their positions alone)."""
    d = ex.Decoder(2, 3)
    out = d.generate([11, 12], 10)
    one = ex.Decoder(2, 0)
    # the same weights: the drafts change neither the generator's order nor the shapes drawn from it
    assert torch.equal(one.embed, d.embed) and torch.equal(one.layers[1]["router"], d.layers[1]["router"])
    n = min(len(o) for o in out) - 1
    for t in range(n):
        one.seq_len += 1
        one.forward(torch.tensor([o[t] for o in out], device="cuda"))
    kv = []
    for dec in (d, one):
        m, cache = ex.m, dec.layers[0]["cache"]
        start = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
        batch = m.KvBatch(start, torch.full((2,), n, dtype=torch.int32, device="cuda"), dec.batch.block_table, tokens=2 * n, max_q=n)
        k, v = (torch.empty(2 * n, dec.kv_heads, dec.D, device="cuda") for _ in range(2))
        m.moe_kv_read(cache, batch, k, v, ws=cache.workspace(batch, dec.heads))
        torch.cuda.synchronize()
        kv.append((k, v))
    # (a projection's row may round differently in a product of 8 rows and one of 2; few codes lie that near to a tie)
    for a, b in zip(*kv):
        same = (a == b).float().mean().item()
        assert same > 0.98, same
