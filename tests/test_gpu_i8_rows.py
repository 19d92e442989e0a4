"""moe_i8_quantize, moe_i8_values and moe_rms_norm_i8 against the reference: codes and quantising scales bit for bit, the norm's
scales and rows within their few fp32 roundings, every type, strides, borders between codes, extreme and non-finite rows."""
import numpy as np
import pytest
import torch

from tests import _i8_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module")
def m():
    import bit_moe_decode_gb300 as mod
    return mod


def data(T, K, seed=0):
    """Rows of very different sizes, exact borders between codes among them, and zeros."""
    g = np.random.default_rng(seed + T * 7 + K)
    v = g.standard_normal((T, K)).astype(np.float32) * np.exp2(g.integers(-12, 12, (T, 1))).astype(np.float32)
    if T > 2:
        v[1] = 0
        v[2] = (g.integers(-254, 255, K) * 0.5).astype(np.float32)       # with the largest 127: halves are ties
        v[2, 0] = 127
    return v


def wide(a, pad, dtype=torch.float32):
    """The array on the device in rows of a wider tensor that holds NaN beside them."""
    t = torch.full((a.shape[0], a.shape[1] + pad), float("nan"), dtype=dtype, device=DEV)
    t[:, :a.shape[1]] = torch.from_numpy(a).to(DEV).to(dtype)
    return t[:, :a.shape[1]]


def guarded_rows(m, T, K, pad=0):
    """I8Rows whose codes have a pattern around them, and a check that it still stands."""
    raw = torch.full((T + 2, K + pad + 32), 77, dtype=torch.int8, device=DEV)
    sraw = torch.full((T + 8,), 5.0, device=DEV)
    rows = m.I8Rows(q=raw[1:T + 1, 16:16 + K], scale=sraw[4:T + 4])

    def intact():
        c = raw.clone()
        c[1:T + 1, 16:16 + K] = 77
        return bool((c == 77).all()) and bool((sraw[:4] == 5).all()) and bool((sraw[T + 4:] == 5).all())
    return rows, intact


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,K,pad", [(1, 16, 0), (5, 64, 16), (3, 4096, 0), (130, 272, 8), (4, 7184, 0), (3, 8208, 0), (3, 16400, 24),
                                     (2, 32768, 0), (2, 32784, 0), (1, 131056, 0)])
def test_quantize_and_values(m, T, K, pad, dtype):
    src = wide(data(T, K), pad, dtype)
    rows, intact = guarded_rows(m, T, K, pad // 16 * 16)
    m.moe_i8_quantize(src, rows)
    out = torch.empty(T, K, device=DEV)
    m.moe_i8_values(rows, out)
    q, scale, _ = ref.quantize(src.float().cpu().numpy())
    assert np.array_equal(rows.q.cpu().numpy(), q)
    assert np.array_equal(rows.scale.cpu().numpy(), scale)
    assert np.array_equal(out.cpu().numpy(), q.astype(np.float32) * scale[:, None])
    assert intact()


def test_quantize_borders(m):
    """Values on both sides of each border between two codes, and on it, for maxima with long mantissas."""
    g = np.random.default_rng(3)
    out = []
    for a in (1.0, 127.0, 3.0e-30, 1.7e38, *g.uniform(1, 2, 8)):
        a = np.float32(a)
        b = ((np.arange(-127, 127) + 0.5) / 127.0 * np.float64(a)).astype(np.float32)
        row = np.concatenate([b, np.nextafter(b, np.float32(np.inf)), np.nextafter(b, np.float32(-np.inf)), [a, -a]])
        out.append(np.pad(row, (0, -len(row) % 16)))
    v = np.stack(out).astype(np.float32)
    rows = m.I8Rows.of(torch.from_numpy(v).to(DEV))
    q, scale, _ = ref.quantize(v)
    assert np.array_equal(rows.q.cpu().numpy(), q) and np.array_equal(rows.scale.cpu().numpy(), scale)


def test_quantize_extreme_rows(m):
    v = np.ones((9, 32), np.float32)
    v[0, 5], v[1, 31], v[2, 0] = np.nan, np.inf, -np.inf
    v[3] = 1e-45
    v[4] = 2.0 ** -101
    v[5] = 3.4e38
    v[6] = 0
    v[7] = -0.0
    rows = m.I8Rows.of(torch.from_numpy(v).to(DEV))
    q, scale, _ = ref.quantize(v)
    assert np.array_equal(rows.q.cpu().numpy(), q) and np.array_equal(rows.scale.cpu().numpy(), scale, equal_nan=True)
    assert np.isnan(scale[:3]).all() and not q[:4].any() and q[5].all()


TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("h,r,gain", [("f32", None, False), ("f32", "f32", True), ("f32", "bf16", True), ("bf16", None, True),
                                      ("bf16", "f32", False), ("bf16", "bf16", True)])
@pytest.mark.parametrize("T,K,pad", [(1, 16, 0), (7, 80, 16), (3, 4096, 0), (40, 1040, 8), (3, 8208, 8), (2, 16400, 0), (2, 32768, 0)])
def test_norm(m, T, K, pad, h, r, gain):
    """Codes and sums bit for bit. The scale: the sum of squares has at most 4 * 8 sequential roundings and 10 of the tree, halved by
    the root, then 5 more; the bf16 row one more and its own half step."""
    eps = 1e-6
    rng = np.random.default_rng(K)
    hd = wide(data(T, K, 1), pad, TYPES[h])
    rd = None if r is None else wide(data(T, K, 2), pad // 2 // 8 * 8, TYPES[r])
    gd = torch.from_numpy((1 + 0.3 * rng.standard_normal(K)).astype(np.float32)).to(DEV) if gain else None
    xq, intact = guarded_rows(m, T, K)
    x = torch.empty(T, K, dtype=torch.bfloat16, device=DEV)
    h_out = torch.full((T, K + pad), 9.0, dtype=TYPES[h], device=DEV)
    m.moe_rms_norm_i8(hd, xq, r=rd, gain=gd, eps=eps, h_out=h_out[:, :K], x_bf16=x)
    s, q, scale, xn = ref.norm(hd.float().cpu().numpy(), None if rd is None else rd.float().cpu().numpy(),
                               None if gd is None else gd.cpu().numpy(), eps)
    got_s = h_out[:, :K].float().cpu().numpy()
    assert np.array_equal(got_s, s if h == "f32" else ref.bf16(s))
    assert bool((h_out[:, K:] == 9).all()) and intact()
    assert np.array_equal(xq.q.cpu().numpy(), q)
    assert np.all(np.abs(xq.scale.cpu().numpy() - scale) <= 26 * U * np.abs(scale))
    assert np.all(np.abs(x.float().cpu().numpy() - xn) <= (2.0 ** -8 + 30 * U) * np.abs(xn) + 2.0 ** -133)
    # without the other outputs, in place, and a row alone: the same bits
    x2, xq2, h2 = torch.empty_like(x), m.I8Rows(T, K), hd.clone()
    m.moe_rms_norm_i8(h2, None, r=rd, gain=gd, eps=eps, h_out=h2, x_bf16=x2)
    assert torch.equal(x, x2) and torch.equal(h2, h_out[:, :K])
    m.moe_rms_norm_i8(hd, xq2, r=rd, gain=gd, eps=eps)
    assert torch.equal(xq2.q, xq.q) and torch.equal(xq2.scale, xq.scale)
    t = T - 1
    one = m.I8Rows(1, K)
    m.moe_rms_norm_i8(hd[t:], one, r=None if rd is None else rd[t:], gain=gd, eps=eps)
    assert torch.equal(one.q[0], xq.q[t]) and torch.equal(one.scale[0], xq.scale[t])


@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6, 1.0])
def test_norm_extreme_rows(m, eps):
    """Squares that overflow or vanish, rows of zeros, NaN and infinities."""
    rng = np.random.default_rng(1)
    h = np.stack([rng.standard_normal(512) * f for f in (1e30, 1e-30, 1e-36, 1e19, 1e-19, 2.0 ** -50, 1, 1)]).astype(np.float32)
    h[6, 7], h[7, 9] = np.nan, -np.inf
    h = np.concatenate([h, np.zeros((1, 512), np.float32)])
    xq, x = m.I8Rows(9, 512), torch.empty(9, 512, dtype=torch.bfloat16, device=DEV)
    m.moe_rms_norm_i8(torch.from_numpy(h).to(DEV), xq, eps=eps, x_bf16=x)
    s, q, scale, xn = ref.norm(h, None, None, eps)
    got, gx = xq.scale.cpu().numpy(), x.float().cpu().numpy()
    assert np.array_equal(xq.q.cpu().numpy(), q)
    assert np.all(np.abs(got[:6] - scale[:6]) <= 26 * U * scale[:6] + 2.0 ** -148)
    assert np.all(np.abs(gx[:6] - xn[:6]) <= (2.0 ** -8 + 30 * U) * np.abs(xn[:6]) + 2.0 ** -133)
    assert np.isnan(got[6:8]).all() and np.isnan(gx[6]).all()
    if eps > 0:
        assert np.all(gx[8] == 0) and np.isfinite(got[8])


def test_rows_on_a_stream_and_in_a_graph(m):
    """A captured norm follows its inputs; the stream's order is kept."""
    T, K = 6, 4096
    h, r = torch.zeros(T, K, device=DEV), torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)
    xq, x = m.I8Rows(T, K), torch.empty(T, K, dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        m.moe_rms_norm_i8(h, xq, r=r, h_out=h, x_bf16=x)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_rms_norm_i8(h, xq, r=r, x_bf16=x)
        m.moe_i8_quantize(x, xq)
    for seed in (1, 2):
        h.copy_(torch.from_numpy(data(T, K, seed)))
        r.copy_(torch.from_numpy(data(T, K, seed + 5)))
        graph.replay()
        q, scale, _ = ref.quantize(x.float().cpu().numpy())
        assert np.array_equal(xq.q.cpu().numpy(), q) and np.array_equal(xq.scale.cpu().numpy(), scale)


def test_rows_refuse(m):
    h = torch.zeros(4, 64, device=DEV)
    xq = m.I8Rows(4, 64)
    with pytest.raises(m.MoeError):
        m.moe_rms_norm_i8(h, None)
    with pytest.raises(m.MoeError):
        m.moe_rms_norm_i8(h, m.I8Rows(3, 64))
    with pytest.raises(m.MoeError):
        m.moe_i8_quantize(torch.zeros(4, 66, device=DEV)[:, 2:], xq)      # rows that are not aligned
    with pytest.raises(AssertionError):
        m.moe_i8_quantize(torch.zeros(4, 64, dtype=torch.float16, device=DEV), xq)
    with pytest.raises(m.MoeError):
        m.I8Rows.of(torch.zeros(4, 40, device=DEV))
