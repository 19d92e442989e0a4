"""Logits to probabilities against 64 bits, `top` against the same fp32 steps in numpy.

Bound of a probability p: the steps before the softmax round at most 6 times at magnitude X = the row's largest finite |x|
(before or after a step) and the division by the temperature once more, so an exponent is off by at most
d = 8 2^-24 X / temperature (doubled for the row maximum's own error); exp and the sums add 2^-20: |error| <= p (2 d + 2^-20) +
2^-126 (below the smallest normal number fp32 may flush)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
F = np.float32


@pytest.fixture(scope="module")
def m():
    import bit_moe_decode_gb300 as mod
    return mod


def steps(x, dt, rep, pres, freq, c, bias, allowed):
    """The steps up to the mask in type dt, with the largest magnitude met."""
    x = np.where(np.isnan(x), -np.inf, x).astype(dt)
    top = [np.max(np.abs(x[np.isfinite(x)]), initial=0)]
    with np.errstate(over="ignore", invalid="ignore"):
        if c is not None:
            y = np.where(x > 0, x / dt(rep), x * dt(rep)).astype(dt)
            top.append(np.max(np.abs(y[np.isfinite(y)]), initial=0))
            y = (y - (dt(freq) * c.astype(dt)).astype(dt)).astype(dt)
            y = (y - dt(pres)).astype(dt)
            x = np.where(c > 0, y, x)
            top.append(np.max(np.abs(x[np.isfinite(x)]), initial=0) + abs(pres))
        if bias is not None:
            x = (x + bias.astype(dt)).astype(dt)
            top.append(np.max(np.abs(x[np.isfinite(x)]), initial=0))
    if allowed is not None:
        x = np.where(allowed, x, -np.inf).astype(dt)
    return x, float(max(top))


def check(m, S, rows, V, dtype="f32", counts=True, draft=True, bias=5, mask=False, seed=0, edit=None, params=None, stride=0, inplace=False):
    rng = np.random.default_rng(seed + V + 1000 * rows)
    n = S * rows
    x = (3 * rng.standard_normal((n, V))).astype(F)
    par = np.stack([1 + 0.5 * rng.random(S), 0.5 * rng.random(S), 0.3 * rng.random(S), 0.3 + rng.random(S)], 1).astype(F)
    if params is not None:
        par[:] = params
    if edit:
        edit(x, par)
    if dtype == "bf16":
        xt = torch.from_numpy(x).to(torch.bfloat16)
        x = xt.float().numpy()
    else:
        xt = torch.from_numpy(x)
    wide = torch.full((n, V + stride), 99.0, dtype=xt.dtype)
    wide[:, :V] = xt
    cnt = np.zeros((S, V), np.int32)
    for s in range(S):
        np.add.at(cnt[s], rng.integers(0, V, 40), 1)
    d = rng.integers(0, V, (S, max(rows - 1, 1))).astype(np.int32)
    if rows > 2:
        d[0, 1] = d[0, 0]                 # a draft repeated, and ids outside the vocabulary
        d[-1, 0] = V
        d[-1, rows - 2] = -1
    nb = min(bias, V)
    ids = np.stack([rng.choice(V, nb, replace=False) for _ in range(S)]).astype(np.int32) if nb else None
    vals = (2 * rng.standard_normal((S, nb))).astype(F) if nb else None
    words = (V + 31) // 32 + (1 if stride else 0)
    ok = rng.random((n, V)) < 0.5 if mask else None
    bits = np.zeros((n, words * 32), bool)
    if mask:
        if n > 2:
            ok[1] = False
            ok[2] = False
            ok[2, V - 1] = True
        bits[:, :V] = ok
        bits[:, V:] = True                # bits past the vocabulary mean nothing
    packed = np.packbits(bits.reshape(n, -1, 32), axis=-1, bitorder="little").reshape(n, -1).view(np.int32)
    dv = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    logits = wide.to(DEV)[:, :V]
    guard = torch.full((n * V + 64,), 5.0, device=DEV)
    probs = logits if inplace else guard[32:32 + n * V].view(n, V)
    top = torch.full((n,), -7, dtype=torch.int32, device=DEV)
    start = np.arange(S + 1, dtype=np.int32) * nb
    m.moe_logits_probs(logits, dv(par), probs, rows_per_seq=rows, counts=dv(cnt) if counts else None,
                       draft=dv(d) if counts and draft and rows > 1 else None,
                       bias=(dv(start), dv(ids.reshape(-1)), dv(vals.reshape(-1))) if nb else None, allowed=dv(packed) if mask else None, top=top)
    torch.cuda.synchronize()
    assert bool((guard[:32] == 5).all() and (guard[32 + n * V:] == 5).all())
    got, gtop = probs.cpu().numpy().astype(float), top.cpu().numpy()
    for r in range(n):
        s, j = divmod(r, rows)
        rep, pres, freq, temp = par[s]
        c = None
        if counts:
            c = cnt[s].copy()
            if draft and rows > 1:
                for t in d[s, :j]:
                    if 0 <= t < V:
                        c[t] += 1
        b = None
        if nb:
            b = np.zeros(V, F)
            b[ids[s]] = vals[s]
        args = (rep, pres, freq, c, b, ok[r] if mask else None)
        y32, X = steps(x[r], F, *args)
        y, _ = steps(x[r], np.float64, *args)
        mx = y32.max()
        want_top = -1 if mx == -np.inf else int(np.argmax(y32))
        assert gtop[r] == want_top, (r, gtop[r], want_top)
        if mx == -np.inf:
            ref = np.zeros(V)
        elif not temp > 0:
            ref = np.zeros(V)
            ref[want_top] = 1
        elif mx == np.inf:
            ref = (y32 == np.inf) / np.sum(y32 == np.inf)
        else:
            z = y / float(temp)
            ref = np.exp(z - z.max())
            ref /= ref.sum()
        dd = 16 * 2.0 ** -24 * X / float(temp) if temp > 0 else 0.0
        bound = ref * (2 * dd + 2.0 ** -20) + 2.0 ** -126
        assert np.all(np.abs(got[r] - ref) <= bound), (r, float(np.max(np.abs(got[r] - ref) / bound)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 31, 33, 257, 4096, 32768, 50001])
def test_vocabularies(m, dtype, V):
    check(m, 2, 1, V, dtype, mask=V > 2, bias=min(5, V))


@pytest.mark.parametrize("rows", [2, 3, 8])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_rows_count_their_drafts(m, rows, dtype):
    check(m, 3, rows, 1003, dtype, mask=True, bias=40)


@pytest.mark.parametrize("V", [131071, 262144, 300001, 1 << 20])
def test_large_vocabularies(m, V):
    check(m, 1, 2, V, "f32", mask=True, bias=100)
    check(m, 2, 1, V, "bf16", mask=False, bias=0, draft=False)


def test_many_rows(m):
    check(m, 400, 1, 517, mask=True)
    check(m, 100, 8, 2000, "bf16")


@pytest.mark.parametrize("off", ["counts", "bias", "all"])
def test_steps_left_out(m, off):
    check(m, 2, 3, 777, counts=off == "bias", bias=0 if off in ("bias", "all") else 7, mask=off == "counts")


@pytest.mark.parametrize("stride", [1, 3, 64])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_row_strides(m, stride, dtype):
    check(m, 3, 1, 999, dtype, stride=stride, mask=True)


def test_in_place(m):
    check(m, 3, 2, 5000, inplace=True, mask=True)
    check(m, 1, 1, 400000, inplace=True, mask=True)


def test_greedy_and_ties(m):
    def edit(x, par):
        x[:] = np.round(x)           # many equal logits: the first of the largest
        par[:, 3] = 0
    check(m, 4, 2, 3000, edit=edit, bias=0, counts=False)
    check(m, 4, 2, 3000, edit=edit, mask=True)


def test_infinities_nan_and_lowest_values(m):
    low = np.finfo(F).min

    def edit(x, par):
        x[0, ::3] = -np.inf
        x[1, ::5] = np.nan
        x[2, :] = low                # a mask of the type's lowest value over everything: uniform
        x[3, 7], x[3, 90] = np.inf, np.inf
        x[4, :] = -np.inf
        x[5, :] = low
        x[5, 11] = 0.0
        x[6, :] = np.nan
        x[7, 5:] = np.finfo(F).max
    check(m, 8, 1, 300, edit=edit, counts=False, bias=0)
    check(m, 8, 1, 300, edit=edit, counts=True, bias=3, mask=True, params=[1.0, 0.0, 0.0, 1.0])
    check(m, 8, 1, 70000, edit=edit, counts=False, bias=0)


@pytest.mark.parametrize("params", [[1, 0, 0, 1], [2, 0, 0, 1], [1, 1.5, 0, 1], [1, 0, 0.7, 1], [0.5, -1, -0.2, 3.0], [1.2, 0.3, 0.2, 1e-3]])
def test_parameters(m, params):
    check(m, 3, 4, 2049, params=params)


def test_feeds_acceptance(m):
    """The rows are what moe_spec_accept takes: a one-hot row of a greedy sequence keeps exactly the drafts it would make."""
    V, K = 1000, 3
    x = torch.randn(K + 1, V, device=DEV)
    best = x.argmax(1).int()
    p = torch.empty(K + 1, V, device=DEV)
    par = torch.tensor([[1.0, 0, 0, 0]], device=DEV)
    m.moe_logits_probs(x, par, p, rows_per_seq=K + 1)
    q = torch.full((K, V), 1.0 / V, device=DEV)
    draft = best[:K].clone()
    draft[2] = (draft[2] + 1) % V
    res = torch.empty(2, dtype=torch.int32, device=DEV)
    m.moe_spec_accept(p, q, K, V, draft, torch.full((K + 1,), 0.5, device=DEV), res)
    assert res.tolist() == [2, int(best[2])]


def test_refusals(m):
    x = torch.zeros(4, 100, device=DEV)
    par = torch.ones(2, 4, device=DEV)
    p = torch.empty(4, 100, device=DEV)

    def status(**kw):
        a = dict(logits=x, params=par, probs=p, rows_per_seq=2)
        a.update(kw)
        with pytest.raises(m.MoeError) as e:
            m.moe_logits_probs(**a)
        return e.value.status

    assert status(allowed=torch.zeros(4, 3, dtype=torch.int32, device=DEV)) == 2      # 3 words for 100 tokens
    big = torch.zeros(65, 8, device=DEV)
    assert status(logits=big, params=par[:1], probs=torch.empty(65, 8, device=DEV), rows_per_seq=65) == 2
    with pytest.raises(AssertionError):
        m.moe_logits_probs(x, par, p, rows_per_seq=3)
    with pytest.raises(AssertionError):
        m.moe_logits_probs(x, par, p[:3], rows_per_seq=2)
