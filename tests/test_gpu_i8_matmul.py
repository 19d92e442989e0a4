"""moe_i8_matmul and moe_i8_gated against the reference: the product bit for bit (the integer sum is exact and every further
operation is one rounding), for all sizes of tokens, channels and depth; the gated block within its derived bound."""
import numpy as np
import pytest
import torch

from tests import _i8_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def m():
    import bit_moe_decode_gb300 as mod
    return mod


def codes(rows, cols, seed, kind="uniform"):
    g = np.random.default_rng(seed)
    if kind == "uniform":
        q = g.integers(-128, 128, (rows, cols))
    elif kind == "normal":
        q = np.clip(np.rint(g.standard_normal((rows, cols)) * 30), -127, 127)
    elif kind == "near":                             # sums of 1024 products just below 2^24, whose last bit counts
        q = g.integers(125, 128, (rows, cols)) * np.where(g.random((rows, 1)) < 0.3, -1, 1)
    else:                                            # the largest sums there are, of both signs
        q = np.where(g.random((rows, 1)) < 0.5, -128, 127) * np.ones((1, cols))
    return q.astype(np.int8), np.exp2(g.uniform(-12, 4, rows)).astype(np.float32)


def device_rows(m, q, scale, pad=0):
    t = torch.full((q.shape[0] + 1, q.shape[1] + pad), 99, dtype=torch.int8, device=DEV)
    t[:-1, :q.shape[1]] = torch.from_numpy(q).to(DEV)
    return m.I8Rows(q=t[:-1, :q.shape[1]], scale=torch.from_numpy(scale).to(DEV))


class Out:
    """A [T, N] output (or base) in wider rows at an odd offset, and a check that nothing beside it was written."""

    def __init__(self, T, N, dtype, pad=3, off=1):
        self.raw = torch.full((T + 2, N + pad + off), 7.0, dtype=dtype, device=DEV)
        self.t = self.raw[1:T + 1, off:off + N]
        self.T, self.N, self.off = T, N, off

    def intact(self):
        c = self.raw.clone()
        c[1:self.T + 1, self.off:self.off + self.N] = 7
        return bool((c == 7).all())


def check_matmul(m, T, N, K, kind="uniform", pad=0, seed=0):
    xq, xs = codes(T, K, seed + 1, kind)
    wq, ws = codes(N, K, seed + 2, kind)
    x, w = device_rows(m, xq, xs, pad), device_rows(m, wq, ws, 2 * pad)
    want = ref.product(xq, xs, wq, ws)
    wsp = w.workspace(T)
    y, yb = Out(T, N, torch.float32), Out(T, N, torch.bfloat16, pad=0, off=0)
    m.moe_i8_matmul(x, w, y=y.t, y_bf16=yb.t, ws=wsp)
    assert m.moe_get_device_status(wsp) == 0
    assert np.array_equal(y.t.cpu().numpy(), want)
    assert np.array_equal(yb.t.float().cpu().numpy(), ref.bf16(want))
    assert y.intact() and yb.intact()
    base = np.random.default_rng(seed).standard_normal((T, N)).astype(np.float32) * np.abs(want).mean()
    b = Out(T, N, torch.float32, pad=0)
    b.t.copy_(torch.from_numpy(base))
    yb2 = Out(T, N, torch.bfloat16)
    m.moe_i8_matmul(x, w, y_bf16=yb2.t, base=b.t, ws=wsp)
    m.moe_i8_matmul(x, w, y=b.t, base=b.t, ws=wsp)           # in place
    assert np.array_equal(b.t.cpu().numpy(), base + want)
    assert np.array_equal(yb2.t.float().cpu().numpy(), ref.bf16(base + want))
    assert b.intact() and yb2.intact()
    return x, w, want


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 64, 65, 100, 127, 129, 200, 256, 257, 300, 520])
@pytest.mark.parametrize("N,K", [(1, 16), (70, 144), (513, 1040)])
def test_matmul_sizes(m, T, N, K):
    check_matmul(m, T, N, K, pad=16 * (T % 3))


@pytest.mark.parametrize("T,N,K", [(1, 6144, 4096), (3, 131071, 64), (8, 4096, 4096), (11, 333, 8208), (40, 1000, 12288), (150, 640, 4112),
                                   (1000, 384, 2064), (2049, 127, 1024), (129, 4097, 128), (1, 1, 131056), (40, 3, 131056)])
def test_matmul_shapes(m, T, N, K):
    check_matmul(m, T, N, K, kind="normal")


@pytest.mark.parametrize("T,N,K", [(1, 64, 4096), (8, 100, 8208), (16, 64, 131056), (17, 40, 65552), (70, 130, 16384), (260, 260, 8192),
                                   (300, 129, 131056)])
def test_matmul_largest_sums(m, T, N, K):
    """Sums up to 2^31: exact integers far beyond what fp32 holds."""
    check_matmul(m, T, N, K, kind="largest")


@pytest.mark.parametrize("T", [1, 8, 12, 30, 64, 100, 300, 520])
@pytest.mark.parametrize("N,K", [(300, 1024), (200, 1920), (40, 2048), (1000, 4096)])
def test_matmul_sums_near_the_limit(m, T, N, K):
    check_matmul(m, T, N, K, kind="near")


@pytest.mark.parametrize("T,N,K", [(1000, 512, 512), (1500, 700, 1024), (2000, 128, 128), (12000, 65, 80), (200, 2000, 336), (16, 2048, 4096),
                                   (17, 3000, 1040), (32, 700, 2064), (31, 5000, 528), (25, 100, 1280), (32, 1, 32)])
def test_matmul_small_products(m, T, N, K):
    check_matmul(m, T, N, K, pad=16, seed=T)


def test_tokens_do_not_depend_on_each_other(m):
    """A row alone, in a batch of 8 and in a prompt has the same bits."""
    x, w, want = check_matmul(m, 300, 200, 4096, kind="normal")
    for n in (1, 5, 16, 90, 256):
        y = torch.empty(n, 200, device=DEV)
        m.moe_i8_matmul(x.first(n), w, y=y, ws=w.workspace(n))
        assert np.array_equal(y.cpu().numpy(), want[:n])


def gated_bound(g, u, want):
    """exp to 2 units in the last place, a sum, a reciprocal and two products: below 2^-20 relative. exp(-g) overflows below g =
    -88.7, where SiLU is under 2^-121."""
    return 2.0 ** -20 * np.abs(want) + 2.0 ** -121 * np.abs(u) + 2.0 ** -149


def check_gated(m, T, N, K, kind="normal", pad=0, small=2.0 ** -8):
    (xq, xs), (gq, gs), (uq, us) = codes(T, K, 1, kind), codes(N, K, 2, kind), codes(N, K, 3, kind)
    xs, gs = xs * np.float32(small), gs * np.float32(small)          # (so that the gates are not all saturated)
    x, wg, wu = device_rows(m, xq, xs, pad), device_rows(m, gq, gs, pad), device_rows(m, uq, us)
    g, u = ref.product(xq, xs, gq, gs), ref.product(xq, xs, uq, us)
    want = ref.gated(g, u)
    wsp = wg.workspace(T)
    y, yb = Out(T, N, torch.float32), Out(T, N, torch.bfloat16, pad=0)
    m.moe_i8_gated(x, wg, wu, y=y.t, y_bf16=yb.t, ws=wsp)
    assert m.moe_get_device_status(wsp) == 0
    got = y.t.cpu().numpy()
    assert np.all(np.abs(got - want) <= gated_bound(g, u, want))
    assert np.array_equal(yb.t.float().cpu().numpy(), ref.bf16(got))
    assert y.intact() and yb.intact()
    yb2 = Out(T, N, torch.bfloat16)
    m.moe_i8_gated(x, wg, wu, y_bf16=yb2.t, ws=wsp)
    assert torch.equal(yb2.t, yb.t) and yb2.intact()
    n = max(1, T // 3)
    one = torch.empty(n, N, device=DEV)
    m.moe_i8_gated(x.first(n), wg, wu, y=one, ws=wsp)
    assert torch.equal(one, y.t[:n])


@pytest.mark.parametrize("T", [1, 4, 8, 9, 16, 17, 40, 64, 65, 128, 129, 260])
@pytest.mark.parametrize("N,K", [(1, 16), (65, 208), (300, 1104)])
def test_gated_sizes(m, T, N, K):
    check_gated(m, T, N, K, pad=16 * (T % 2))


@pytest.mark.parametrize("T,N,K", [(1, 2048, 4096), (8, 11008, 4096), (48, 1500, 4096), (333, 640, 2064), (1500, 130, 512)])
def test_gated_shapes(m, T, N, K):
    check_gated(m, T, N, K)


@pytest.mark.parametrize("T,N,K", [(300, 1024, 512), (900, 333, 1040), (4000, 33, 64), (16, 2048, 2048), (30, 2500, 1040), (20, 9, 2064)])
def test_gated_small_products(m, T, N, K):
    check_gated(m, T, N, K, pad=16)


@pytest.mark.parametrize("T", [1, 8, 20, 200])
def test_gated_largest_sums(m, T):
    """Gates far beyond exp's range on both sides give u g, or zero."""
    check_gated(m, T, 50, 16384, kind="largest", small=1.0)


def test_gate_and_up_of_one_tensor(m):
    """Both weights as halves of one matrix, and the same weights twice."""
    T, N, K = 20, 96, 512
    (xq, xs), (q, s) = codes(T, K, 5, "normal"), codes(2 * N, K, 6, "normal")
    xs = xs * np.float32(2.0 ** -8)
    x, both = device_rows(m, xq, xs), device_rows(m, q, s)
    gate, up = both.first(N), m.I8Rows(q=both.q[N:], scale=both.scale[N:].clone())
    for u_rows, lo in ((up, N), (gate, 0)):
        y = torch.empty(T, N, device=DEV)
        m.moe_i8_gated(x, gate, u_rows, y=y, ws=gate.workspace(T))
        g, u = ref.product(xq, xs, q[:N], s[:N]), ref.product(xq, xs, q[lo:lo + N], s[lo:lo + N])
        want = ref.gated(g, u)
        assert np.all(np.abs(y.cpu().numpy() - want) <= gated_bound(g, u, want))


@pytest.mark.parametrize("T", [3, 40, 300])
def test_nan_scales_stay_in_their_rows(m, T):
    """A token or a channel of scale NaN (a row that held NaN or an infinity) makes its outputs NaN, and no others."""
    (xq, xs), (wq, ws) = codes(T, 64, 1), codes(37, 64, 2)
    xs[1], ws[5] = np.nan, np.nan
    x, w = device_rows(m, xq, xs), device_rows(m, wq, ws)
    want = ref.product(xq, xs, wq, ws)
    y, yg = torch.empty(T, 37, device=DEV), torch.empty(T, 37, device=DEV)
    m.moe_i8_matmul(x, w, y=y, ws=w.workspace(T))
    m.moe_i8_gated(x, w, w, y=yg, ws=w.workspace(T))
    assert np.array_equal(y.cpu().numpy(), want, equal_nan=True)
    bad = torch.from_numpy(np.isnan(want))
    assert torch.equal(torch.isnan(yg.cpu()), bad)


@pytest.mark.parametrize("T", [1, 8, 24, 140, 300])
def test_in_a_graph_and_on_two_streams(m, T):
    """Captured calls follow their inputs; calls on two streams, each with a workspace of its own."""
    N, K = 320, 2064
    (wq, ws) = codes(N, K, 9, "normal")
    w = device_rows(m, wq, ws)
    wsp = w.workspace(T)
    x = m.I8Rows(T, K)
    y, h = torch.empty(T, N, device=DEV), torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    x.q.zero_()
    x.scale.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_i8_matmul(x, w, y=y, ws=wsp)
        m.moe_i8_gated(x, w, w, y_bf16=h, ws=wsp)
    for seed in (1, 2):
        xq, xs = codes(T, K, seed, "normal")
        x.q.copy_(torch.from_numpy(xq))
        x.scale.copy_(torch.from_numpy(xs))
        graph.replay()
        assert np.array_equal(y.cpu().numpy(), ref.product(xq, xs, wq, ws))
    torch.cuda.synchronize()
    want_h = h.clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(y), torch.empty_like(h), w.workspace(T)] for _ in streams]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, (a, b, own) in zip(streams, outs):
            with torch.cuda.stream(s):
                m.moe_i8_matmul(x, w, y=a, ws=own)
                m.moe_i8_gated(x, w, w, y_bf16=b, ws=own)
    torch.cuda.synchronize()
    for a, b, own in outs:
        assert torch.equal(a, y) and torch.equal(b, want_h) and m.moe_get_device_status(own) == 0


@pytest.mark.parametrize("T,N,K,gated", [(1, 6144, 4096, False), (8, 16384, 4096, False), (8, 4096, 2048, True), (5, 4096, 6144, False),
                                          (30, 8192, 4096, False), (200, 4096, 4096, True), (12, 4096, 4096, False), (30, 2048, 3200, False),
                                          (16, 2048, 2048, True), (900, 512, 1024, False), (400, 512, 512, True)])
def test_many_launches_one_after_another(m, T, N, K, gated):
    """Weights from memory each time (three sets, more than the cache holds together with what lies between), always the same bits."""
    x = device_rows(m, *codes(T, K, 1, "normal"))
    sets = [[device_rows(m, *codes(N, K, 10 * i + j, "normal")) for j in range(2 if gated else 1)] for i in range(3)]
    flush = torch.empty(1 << 27, dtype=torch.uint8, device=DEV)
    wsp = sets[0][0].workspace(T)

    def run(w, y):
        if gated:
            m.moe_i8_gated(x, *w, y=y, ws=wsp)
        else:
            m.moe_i8_matmul(x, w[0], y=y, ws=wsp)
    first = [torch.empty(T, N, device=DEV) for _ in sets]
    for w, y in zip(sets, first):
        run(w, y)
    for i in range(60):
        if i % 5 == 0:
            flush.fill_(i)
        y = torch.empty(T, N, device=DEV)
        run(sets[i % 3], y)
        assert torch.equal(y, first[i % 3]), i
    assert m.moe_get_device_status(wsp) == 0


def test_products_refuse(m):
    x, w = m.I8Rows(4, 64), m.I8Rows(8, 64)
    ws = w.workspace(4)
    with pytest.raises(m.MoeError):
        m.moe_i8_matmul(x, w, ws=ws)
    with pytest.raises(m.MoeError):
        m.moe_i8_matmul(x, m.I8Rows(8, 80), y=torch.empty(4, 8, device=DEV), ws=ws)
    with pytest.raises(AssertionError):
        m.moe_i8_matmul(x, w, y=torch.empty(4, 9, device=DEV), ws=ws)
    with pytest.raises(m.MoeError):
        m.moe_i8_gated(x, w, m.I8Rows(9, 64), y=torch.empty(4, 8, device=DEV), ws=ws)


WIDE = [(40, 40004, 128), (64, 20008, 512), (100, 9000, 512), (200, 2996, 1040), (300, 10004, 256), (600, 4100, 2064), (30, 33000, 1024), (64, 4096, 4096)]


@pytest.mark.parametrize("T,N,K", WIDE)
def test_matmul_aligned_outputs(m, T, N, K):
    """Rows that four channels at a time can be written to, N not a multiple of a group's channels: each output alone and all
    together, onto a base of their own and in place, with nothing written between the rows."""
    (xq, xs), (wq, ws) = codes(T, K, 1, "normal"), codes(N, K, 2, "normal")
    x, w = device_rows(m, xq, xs), device_rows(m, wq, ws)
    want = ref.product(xq, xs, wq, ws)
    wsp = w.workspace(T)
    base = np.random.default_rng(3).standard_normal((T, N)).astype(np.float32) * np.abs(want).mean()
    y, b = Out(T, N, torch.float32, pad=8, off=0), Out(T, N, torch.float32, pad=4, off=0)
    h = Out(T, N, torch.bfloat16, pad=4, off=0)
    m.moe_i8_matmul(x, w, y=y.t, ws=wsp)
    m.moe_i8_matmul(x, w, y_bf16=h.t, ws=wsp)
    assert np.array_equal(y.t.cpu().numpy(), want) and np.array_equal(h.t.float().cpu().numpy(), ref.bf16(want))
    assert y.intact() and h.intact()
    b.t.copy_(torch.from_numpy(base))
    m.moe_i8_matmul(x, w, y=y.t, y_bf16=h.t, base=b.t, ws=wsp)
    m.moe_i8_matmul(x, w, y=b.t, base=b.t, ws=wsp)
    for o in (y, b):
        assert np.array_equal(o.t.cpu().numpy(), base + want) and o.intact()
    assert np.array_equal(h.t.float().cpu().numpy(), ref.bf16(base + want)) and h.intact()
    assert m.moe_get_device_status(wsp) == 0


@pytest.mark.parametrize("T,N,K", [(40, 20004, 128), (64, 10008, 512), (100, 4500, 512), (200, 1500, 1040), (300, 5004, 256), (600, 2052, 2064)])
def test_gated_aligned_outputs(m, T, N, K):
    (xq, xs), (gq, gs), (uq, us) = codes(T, K, 1, "normal"), codes(N, K, 2, "normal"), codes(N, K, 3, "normal")
    xs, gs = xs * np.float32(2.0 ** -8), gs * np.float32(2.0 ** -8)
    x, gate, up = device_rows(m, xq, xs), device_rows(m, gq, gs), device_rows(m, uq, us)
    g, u = ref.product(xq, xs, gq, gs), ref.product(xq, xs, uq, us)
    want = ref.gated(g, u)
    wsp = gate.workspace(T)
    y, h = Out(T, N, torch.float32, pad=4, off=0), Out(T, N, torch.bfloat16, pad=4, off=0)
    m.moe_i8_gated(x, gate, up, y=y.t, ws=wsp)
    m.moe_i8_gated(x, gate, up, y_bf16=h.t, ws=wsp)
    got = y.t.cpu().numpy()
    assert np.all(np.abs(got - want) <= gated_bound(g, u, want))
    assert np.array_equal(h.t.float().cpu().numpy(), ref.bf16(got))
    y2, odd = Out(T, N, torch.float32), Out(T, N, torch.bfloat16)          # the same bits a channel a thread
    m.moe_i8_gated(x, gate, up, y=y2.t, y_bf16=odd.t, ws=wsp)
    assert torch.equal(y2.t, y.t) and torch.equal(odd.t, h.t)
    assert y.intact() and h.intact() and y2.intact() and odd.intact() and m.moe_get_device_status(wsp) == 0
