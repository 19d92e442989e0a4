"""The 8-bit calls as a layer runs them, one after another, each held to the reference of what it was given; in the verify step
(examples/verify_step.py with the dense half in 8 bits); in a graph; and nothing written beside outputs and workspaces."""
import importlib.util
import os

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


@pytest.fixture(scope="module")
def ex():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "verify_step.py")
    spec = importlib.util.spec_from_file_location("verify_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


class Dense:
    """norm -> product -> (a stand-in for attention: the first H of the product's outputs) -> quantize -> product onto the stream ->
    norm -> gated -> quantize -> product onto the stream."""

    def __init__(self, m, T, H, I, seed=0):
        g = torch.Generator(DEV).manual_seed(seed)
        self.m, self.T, self.H, self.I = m, T, H, I

        def weight(n, k):
            return m.I8Rows.of(torch.randn(n, k, generator=g, device=DEV) / k ** 0.5)
        self.wqkv, self.wout, self.wg, self.wu, self.wd = weight(2 * H, H), weight(H, H), weight(I, H), weight(I, H), weight(H, I)
        self.gain = [1 + 0.1 * torch.randn(H, generator=g, device=DEV) for _ in range(2)]
        self.x1, self.x2, self.a8, self.act8 = m.I8Rows(T, H), m.I8Rows(T, H), m.I8Rows(T, H), m.I8Rows(T, I)
        self.h = [torch.empty(T, H, device=DEV) for _ in range(3)]
        self.qkv, self.act = torch.empty(T, 2 * H, dtype=torch.bfloat16, device=DEV), torch.empty(T, I, dtype=torch.bfloat16, device=DEV)
        self.ws = max((w.workspace(T) for w in (self.wqkv, self.wd)), key=torch.numel)

    def run(self, h, r):
        m, h0, h1, h2 = self.m, *self.h
        m.moe_rms_norm_i8(h, self.x1, r=r, gain=self.gain[0], h_out=h0)
        m.moe_i8_matmul(self.x1, self.wqkv, y_bf16=self.qkv, ws=self.ws)
        m.moe_i8_quantize(self.qkv[:, :self.H], self.a8)
        m.moe_i8_matmul(self.a8, self.wout, y=h1, base=h0, ws=self.ws)
        m.moe_rms_norm_i8(h1, self.x2, gain=self.gain[1])
        m.moe_i8_gated(self.x2, self.wg, self.wu, y_bf16=self.act, ws=self.ws)
        m.moe_i8_quantize(self.act, self.act8)
        m.moe_i8_matmul(self.act8, self.wd, y=h2, base=h1, ws=self.ws)

    def check(self, h, r):
        def rows(x):
            return x.q.cpu().numpy(), x.scale.cpu().numpy()
        h0, h1, h2 = (t.cpu().numpy() for t in self.h)
        s, q, scale, _ = ref.norm(h.cpu().numpy(), r.float().cpu().numpy(), self.gain[0].cpu().numpy(), 1e-6)
        assert np.array_equal(h0, s) and np.array_equal(rows(self.x1)[0], q)
        assert np.all(np.abs(rows(self.x1)[1] - scale) <= 26 * U * scale)
        assert np.array_equal(self.qkv.float().cpu().numpy(), ref.bf16(ref.product(*rows(self.x1), *rows(self.wqkv))))
        q, sc, _ = ref.quantize(self.qkv[:, :self.H].float().cpu().numpy())
        assert np.array_equal(rows(self.a8)[0], q) and np.array_equal(rows(self.a8)[1], sc)
        assert np.array_equal(h1, h0 + ref.product(q, sc, *rows(self.wout)))
        _, q, scale, _ = ref.norm(h1, None, self.gain[1].cpu().numpy(), 1e-6)
        assert np.array_equal(rows(self.x2)[0], q)
        g, u = ref.product(*rows(self.x2), *rows(self.wg)), ref.product(*rows(self.x2), *rows(self.wu))
        want = ref.gated(g, u)
        act = self.act.float().cpu().numpy()
        assert np.all(np.abs(act - want) <= (2.0 ** -8 + 2.0 ** -19) * np.abs(want) + 2.0 ** -120)
        q, sc, _ = ref.quantize(act)
        assert np.array_equal(rows(self.act8)[0], q) and np.array_equal(rows(self.act8)[1], sc)
        assert np.array_equal(h2, h1 + ref.product(q, sc, *rows(self.wd)))
        assert self.m.moe_get_device_status(self.ws) == 0


def stream(T, H, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randn(T, H, generator=g, device=DEV), torch.randn(T, H, generator=g, device=DEV).bfloat16()


@pytest.mark.parametrize("T", [1, 5, 8, 9, 33, 64, 65, 130, 300])
@pytest.mark.parametrize("H,I", [(512, 768), (1040, 2064)])
def test_layer(m, T, H, I):
    d = Dense(m, T, H, I)
    h, r = stream(T, H, 1)
    d.run(h, r)
    d.check(h, r)


@pytest.mark.parametrize("T", [1, 20, 200])
def test_layer_in_a_graph(m, T):
    """Captured once, replayed with other inputs, several layers' calls in flight behind each other."""
    d = Dense(m, T, 512, 1024)
    h, r = stream(T, 512, 2)
    d.run(h, r)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            d.run(h, r)
    for seed in (3, 4):
        a, b = stream(T, 512, seed)
        h.copy_(a)
        r.copy_(b)
        graph.replay()
        graph.replay()
        d.check(h, r)


def test_rows_of_a_layer_do_not_depend_on_the_batch(m):
    """The layer's outputs for the first tokens of a prompt, and of each of them alone: the same bits."""
    H, I = 512, 768
    big = Dense(m, 150, H, I)
    h, r = stream(150, H, 5)
    big.run(h, r)
    for n in (1, 8, 40, 100):
        d = Dense(m, n, H, I)
        d.run(h[:n].contiguous(), r[:n].contiguous())
        assert torch.equal(d.h[2], big.h[2][:n]), n


@pytest.mark.parametrize("seqs,drafts", [(2, 3), (1, 7), (8, 0)])
def test_verify_step(ex, seqs, drafts):
    """The lengths follow what was accepted, and the same seeds give the same tokens."""
    runs = []
    for _ in range(2):
        d = ex.Decoder(seqs, drafts, dense8=True)
        out = d.generate(list(range(5, 5 + seqs)), 12)
        assert all(0 <= t < d.V for o in out for t in o)
        assert all(12 + 1 <= len(o) <= 12 * (1 + drafts) + 1 for o in out)
        assert d.seq_len.tolist() == [len(o) - 1 for o in out]
        runs.append(out)
    assert runs[0] == runs[1]


GUARD = 4096


@pytest.mark.parametrize("T,N,K", [(1, 300, 512), (9, 300, 1040), (16, 4096, 1024), (40, 700, 4096), (64, 4096, 2064), (65, 300, 512), (128, 300, 2064),
                                   (129, 520, 1040), (300, 100, 64), (700, 600, 4112)])
@pytest.mark.parametrize("gated", [False, True])
def test_workspace_and_outputs_keep_their_bounds(m, T, N, K, gated):
    """Workspaces of exactly the size asked for, and outputs, between guard bands."""
    g = torch.Generator(DEV).manual_seed(1)
    x, w, u = (m.I8Rows.of(torch.randn(n, K, generator=g, device=DEV)) for n in (T, N, N))
    size = m.moe_i8_workspace_bytes(w, T)
    raw = torch.full((size + 2 * GUARD + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    lo = GUARD + (-(raw.data_ptr() + GUARD)) % 256
    ws = raw[lo:lo + size]
    m.moe_workspace_init(ws)
    out = torch.full((T * N + 2 * GUARD,), 7.0, device=DEV)
    y = out[GUARD:GUARD + T * N].view(T, N)
    for _ in range(2):
        if gated:
            m.moe_i8_gated(x, w, u, y=y, ws=ws)
        else:
            m.moe_i8_matmul(x, w, y=y, ws=ws)
    assert m.moe_get_device_status(ws) == 0
    assert bool((raw[:lo] == 0xA5).all()) and bool((raw[lo + size:] == 0xA5).all())
    assert bool((out[:GUARD] == 7).all()) and bool((out[GUARD + T * N:] == 7).all())
    with pytest.raises(m.MoeError):
        m.moe_i8_matmul(x, w, y=y, ws=ws[:size - 1])


@pytest.mark.parametrize("T", [2, 20, 70])
def test_rows_far_apart(m, T):
    """Row strides that take offsets past 32 bits: weights, tokens and outputs."""
    K, N, far = 256, 5, 1 << 30
    g = np.random.default_rng(T)
    xq, wq = g.integers(-127, 128, (T, K)).astype(np.int8), g.integers(-127, 128, (N, K)).astype(np.int8)
    xs, ws = g.uniform(0.5, 2, T).astype(np.float32), g.uniform(0.5, 2, N).astype(np.float32)
    wbuf = torch.empty((N - 1) * far + K, dtype=torch.int8, device=DEV)
    wt = torch.as_strided(wbuf, (N, K), (far, 1))
    wt.copy_(torch.from_numpy(wq))
    stride = far // 16
    ybuf = torch.empty((T - 1) * stride + N, device=DEV)
    y = torch.as_strided(ybuf, (T, N), (stride, 1))
    x, w = m.I8Rows(q=torch.from_numpy(xq).to(DEV), scale=torch.from_numpy(xs).to(DEV)), m.I8Rows(q=wt, scale=torch.from_numpy(ws).to(DEV))
    wsp = w.workspace(T)
    m.moe_i8_matmul(x, w, y=y, ws=wsp)
    assert np.array_equal(y.cpu().numpy(), ref.product(xq, xs, wq, ws))
    m.moe_i8_gated(w.first(3), x, x, y=torch.empty(3, T, device=DEV), ws=x.workspace(3))     # tokens with that stride
    assert m.moe_get_device_status(wsp) == 0


@pytest.mark.parametrize("T,K", [(300, 8192), (600, 12288)])
def test_heavy_and_light_tokens_in_one_call(m, T, K):
    """Tokens whose codes are all +-127 (sums far beyond 2^24) beside tokens that are nearly zero, tile by tile and mixed."""
    N = 200
    g = np.random.default_rng(K)
    xq = g.integers(-3, 4, (T, K)).astype(np.int8)
    xq[T // 2:T // 2 + 40] = 127
    xq[T - 1] = -127
    wq = np.where(g.random((N, 1)) < 0.5, -127, 127) * np.ones((1, K))
    wq = np.where(np.arange(N)[:, None] % 3 == 0, g.integers(-127, 128, (N, K)), wq).astype(np.int8)
    xs, ws = np.ones(T, np.float32), np.ones(N, np.float32)
    x, w = (m.I8Rows(q=torch.from_numpy(q).to(DEV), scale=torch.from_numpy(s).to(DEV)) for q, s in ((xq, xs), (wq, ws)))
    y = torch.empty(T, N, device=DEV)
    m.moe_i8_matmul(x, w, y=y, ws=w.workspace(T))
    assert np.array_equal(y.cpu().numpy(), ref.product(xq, xs, wq, ws))


def test_many_tokens(m):
    """More tokens than 16 bits count, of few channels."""
    T, N, K = 70001, 40, 64
    g = np.random.default_rng(0)
    xq, wq = g.integers(-127, 128, (T, K)).astype(np.int8), g.integers(-127, 128, (N, K)).astype(np.int8)
    xs, ws = g.uniform(0.5, 2, T).astype(np.float32), g.uniform(0.5, 2, N).astype(np.float32)
    x, w = (m.I8Rows(q=torch.from_numpy(q).to(DEV), scale=torch.from_numpy(s).to(DEV)) for q, s in ((xq, xs), (wq, ws)))
    y = torch.empty(T, N, device=DEV)
    m.moe_i8_matmul(x, w, y=y, ws=w.workspace(T))
    assert np.array_equal(y.cpu().numpy(), ref.product(xq, xs, wq, ws))


@pytest.mark.parametrize("T,K,N", [(1, 1024, 700), (20, 512, 512), (60, 2048, 900), (200, 1040, 300), (300, 512, 2000), (1000, 256, 256)])
@pytest.mark.parametrize("graph", [False, True])
def test_calls_behind_each_other_share_their_buffers(m, T, K, N, graph):
    """Launches overlap: each call's codes, outputs and workspace are written again by the calls right behind it (ours and torch's),
    and what was computed in between is what each call computes alone."""
    g = torch.Generator(DEV).manual_seed(T)
    src = [torch.randn(T, K, generator=g, device=DEV) for _ in range(3)]
    w, v = m.I8Rows.of(torch.randn(N, K, generator=g, device=DEV)), m.I8Rows.of(torch.randn(N, K, generator=g, device=DEV))
    x8, h8, y, h = m.I8Rows(T, K), m.I8Rows(T, K), torch.empty(T, N, device=DEV), torch.empty(T, K, device=DEV)
    ws = w.workspace(T)
    keep = torch.empty(24, 2, T, N, device=DEV)

    def step(i, wait):
        m.moe_i8_quantize(src[i % 3], x8)
        wait()
        m.moe_i8_matmul(x8, w, y=y, ws=ws)
        wait()
        m.moe_i8_quantize(src[(i + 1) % 3], x8)          # behind the product that read x8
        wait()
        m.moe_i8_matmul(x8, v, y=y, base=y, ws=ws)       # onto the product before it
        wait()
        keep[i, 0].copy_(y)
        wait()
        m.moe_rms_norm_i8(src[i % 3], h8, r=src[(i + 2) % 3], h_out=h)
        wait()
        h.mul_(0.5)
        wait()
        m.moe_rms_norm_i8(h, h8, h_out=h)
        wait()
        m.moe_i8_gated(h8, w, v, y=y, ws=ws)
        wait()
        keep[i, 1].copy_(y)
        wait()
    for i in range(3):
        step(i, torch.cuda.synchronize)
    want = keep[:3].clone()
    keep.zero_()
    torch.cuda.synchronize()
    if graph:
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            for i in range(24):
                step(i, lambda: None)
        cg.replay()
        keep.zero_()
        cg.replay()
    else:
        for i in range(24):
            step(i, lambda: None)
    torch.cuda.synchronize()
    assert m.moe_get_device_status(ws) == 0
    for i in range(24):
        assert torch.equal(keep[i], want[i % 3]), i


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("T", [4, 100, 400])
def test_calls_on_streams_that_wait_for_each_other(m, T, graph):
    """A call behind an event of another stream, whose kernels are still under way, and one behind two streams."""
    K, N = 1024, 768
    g = torch.Generator(DEV).manual_seed(T)
    src, w, v = torch.randn(T, K, generator=g, device=DEV), *(m.I8Rows.of(torch.randn(N, K, generator=g, device=DEV)) for _ in range(2))
    big = torch.randn(4096, 4096, generator=g, device=DEV)
    x, x8, z8 = torch.zeros(T, K, device=DEV), m.I8Rows(T, K), m.I8Rows(T, N)
    y, z, out = (torch.zeros(T, N, device=DEV) for _ in range(3))
    ws, ws2 = w.workspace(T), v.workspace(T)
    side = torch.cuda.Stream()

    def run():
        main = torch.cuda.current_stream()
        big.mul_(1.0)                                    # something long before it
        torch.mul(src, 2.0, out=x)
        m.moe_i8_quantize(x, x8)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            m.moe_i8_matmul(x8, v, y=z, ws=ws2)
            big.add_(0.0)
            m.moe_i8_quantize(z, z8)
        m.moe_i8_matmul(x8, w, y=y, ws=ws)
        main.wait_stream(side)
        m.moe_i8_values(z8, out)
        out.add_(y)
        m.moe_i8_matmul(x8, w, y=out, base=out, ws=ws2)
    run()
    torch.cuda.synchronize()
    q, sc, _ = ref.quantize((2 * src).cpu().numpy())
    a = ref.product(q, sc, w.q.cpu().numpy(), w.scale.cpu().numpy())
    b = ref.product(q, sc, v.q.cpu().numpy(), v.scale.cpu().numpy())
    zq, zs, _ = ref.quantize(b)
    want = torch.from_numpy((zq.astype(np.float32) * zs[:, None] + a) + a)
    assert torch.equal(out.cpu(), want)
    if graph:
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            run()
    for _ in range(20):
        for t in (x, y, z, out):
            t.zero_()
        cg.replay() if graph else run()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want)
    assert m.moe_get_device_status(ws) == 0 and m.moe_get_device_status(ws2) == 0


@pytest.mark.parametrize("T", [1, 8, 20, 64, 100])
@pytest.mark.parametrize("N,K", [(768, 1024), (100, 208), (4096, 4096)])
def test_weights_written_right_before_their_product(m, T, N, K):
    """Weights that the kernel before a product writes, time after time in the same place."""
    g = torch.Generator(DEV).manual_seed(T + N)
    x = m.I8Rows.of(torch.randn(T, K, generator=g, device=DEV))
    src = [torch.randn(N, K, generator=g, device=DEV) for _ in range(3)]
    w, ws, y = m.I8Rows(N, K), m.I8Rows(N, K).workspace(T), torch.empty(3, 2, T, N, device=DEV)
    want = torch.empty_like(y)
    for i in range(3):
        v = m.I8Rows.of(src[i])
        torch.cuda.synchronize()
        m.moe_i8_matmul(x, v, y=want[i, 0], ws=ws)
        m.moe_i8_gated(x, v, v, y=want[i, 1], ws=ws)
        torch.cuda.synchronize()
    for _ in range(10):
        for i in range(3):
            m.moe_i8_quantize(src[i], w)
            m.moe_i8_matmul(x, w, y=y[i, 0], ws=ws)
            m.moe_i8_quantize(src[(i + 1) % 3], w)
            m.moe_i8_quantize(src[i], w)
            m.moe_i8_gated(x, w, w, y=y[i, 1], ws=ws)
        assert torch.equal(y, want)
        y.zero_()
    assert m.moe_get_device_status(ws) == 0
