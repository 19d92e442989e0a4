"""Measured cases of the dense half of a layer in 8 bits: what stands around the attention and the routed experts.

Four operators:
  norm       moe_rms_norm_i8: the residual's addition, RMS norm with a gain, the result in bf16 and in 8 bits with a scale
             for each token (and moe_i8_values, which returns the values that the 8 bits stand for);
  quantize   moe_i8_quantize: rows of activations or weights to 8 bits with a scale each (and moe_i8_values);
  matmul     moe_i8_matmul: product of 8-bit integers with scales for each token and each output channel;
  gated      moe_i8_gated: SiLU(x Wg) * (x Wu), both projections, the activation and the product.

`own` chooses between the framework's calls and their plain form (elementary torch operations in 32 bits).

8 bits: a row of K values v (fp32) with a = max |v| has the codes q = 127 v / a, rounded to the nearest (ties to even; in 64
bits here, as 32 would move values next to a border), and one fp32 scale a / 127; it stands for q * scale. The norm's v are
the stream's sums as fp32 holds them, times the gain, rounded to fp32; its 1 / rms is in the scale alone.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
FLOOR = 2.0 ** -100      # a row's largest magnitude counts as this much at least


def listed():
    return [
        # one user's next token: latency
        dict(name="norm 1x4096", op="norm", T=1, K=4096, h="f32", r="bf16", gain=True, pad=0),
        # a prompt of 8192 tokens, the experts' fp32 sum added to the stream
        dict(name="norm 8192x4096", op="norm", T=8192, K=4096, h="f32", r="f32", gain=True, pad=0),
        # a ragged serving step of a model with a bf16 stream, r a slice of a wider projection
        dict(name="norm 333x7168", op="norm", T=333, K=7168, h="bf16", r="bf16", gain=True, pad=64),
        # attention's output of a verify batch before the output projection
        dict(name="quantize 64x4096", op="quantize", T=64, K=4096, src="bf16", pad=0),
        # the weights of a vocabulary's projection, once when a model is loaded
        dict(name="quantize 32768x4096", op="quantize", T=32768, K=4096, src="f32", pad=0),
        # q, k and v of one user's next token: latency
        dict(name="matmul 1x4096x6144", op="matmul", T=1, K=4096, N=6144, y="bf16", base=False, pad=0),
        # logits of a verify step of eight rows
        dict(name="matmul 8x4096x32768", op="matmul", T=8, K=4096, N=32768, y="f32", base=False, pad=0),
        # the output projection of a serving batch (an odd number of tokens), added to the stream
        dict(name="matmul 201x4096x4096", op="matmul", T=201, K=4096, N=4096, y="f32", base=True, pad=0),
        # q, k and v of a prompt
        dict(name="matmul 4096x4096x6144", op="matmul", T=4096, K=4096, N=6144, y="bf16", base=False, pad=0),
        # the shared expert, one token: latency
        dict(name="gated 1x4096x2048", op="gated", T=1, K=4096, N=2048, y="bf16", pad=0),
        # a dense layer of a serving batch
        dict(name="gated 48x4096x11008", op="gated", T=48, K=4096, N=11008, y="bf16", pad=0),
        # a dense layer of a prompt of odd length
        dict(name="gated 3333x4096x11008", op="gated", T=3333, K=4096, N=11008, y="bf16", pad=0),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "matmul", "matmul", "gated", "gated"])
    pad = rng.choice([0, 0, 16, 80])     # rows that are slices of wider ones
    if op in ("norm", "quantize"):
        K = 16 * _logint(rng, 4, 1024)
        T = _logint(rng, 1, max(1, min(32768, (1 << 25) // K)))
        if op == "norm":
            return dict(op=op, T=T, K=K, h=rng.choice(["f32", "f32", "bf16"]), r=rng.choice(["none", "f32", "bf16"]),
                        gain=rng.random() < 0.7, pad=pad)
        return dict(op=op, T=T, K=K, src=rng.choice(["f32", "bf16"]), pad=pad)
    K = 16 * _logint(rng, 4, 768)
    N = _logint(rng, 1, max(64, min(32768, (1 << 27) // K)))
    T = _logint(rng, 1, max(8, min(8192, int(2.9e11 / (K * N)))))
    T = min(T, max(1, (1 << 26) // N))
    if op == "gated":
        N = max(1, N // 2)
        return dict(op=op, T=T, K=K, N=N, y=rng.choice(["bf16", "bf16", "f32"]), pad=pad)
    return dict(op=op, T=T, K=K, N=N, y=rng.choice(["bf16", "f32"]), base=rng.random() < 0.3, pad=pad)


_SIZE = {"f32": 4, "bf16": 2, "none": 0}
_TYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def work(case):
    T, K, op = case["T"], case["K"], case["op"]
    if op == "norm":
        h, r = _SIZE[case["h"]], _SIZE[case["r"]]
        # h, r and the gain read; the sum, bf16 and the codes with their scales written
        return {"bytes": T * K * (2 * h + r + 2 + 1) + T * 4 + (K * 4 if case["gain"] else 0), "flops": 8 * T * K}
    if op == "quantize":
        return {"bytes": T * K * (_SIZE[case["src"]] + 1) + T * 4, "flops": 4 * T * K}
    N = case["N"]
    weights = (2 if op == "gated" else 1) * N
    base = 4 * T * N if case.get("base") else 0
    return {"bytes": T * K + 4 * T + weights * (K + 4) + T * N * _SIZE[case["y"]] + base, "flops": 2 * T * K * weights}


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 2654435761 % (1 << 62) + 1)


def _rows(t, pad):
    """The same values in rows of a wider tensor (pad elements more)."""
    if not pad:
        return t
    wide = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=DEV)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _activations(g, T, K):
    """Tokens of differing size with a few strong channels, as the stream of a model has them."""
    x = torch.randn(T, K, generator=g, device=DEV)
    x[:, ::61] *= 6.0
    return x * torch.exp(0.7 * torch.randn(T, 1, generator=g, device=DEV))


def _codes(x):
    """Codes and scales of rows, as a model's weights or a token's activations come to the product."""
    q, a = _plain_values(x)
    return q.to(torch.int8), (a / 127.0).squeeze(1).contiguous()


def _weights(g, N, K):
    return _codes(torch.randn(N, K, generator=g, device=DEV) * (K ** -0.5) * torch.exp(0.3 * torch.randn(N, 1, generator=g, device=DEV)))


def prepare(case, seed):
    g = _gen(seed)
    T, K, op, pad = case["T"], case["K"], case["op"], case["pad"]
    s = dict(case=case)
    if op == "norm":
        s["h"] = _rows(_activations(g, T, K).to(_TYPE[case["h"]]), 0)
        s["r"] = None if case["r"] == "none" else _rows((0.5 * torch.randn(T, K, generator=g, device=DEV)).to(_TYPE[case["r"]]), pad)
        s["gain"] = 1.0 + 0.2 * torch.randn(K, generator=g, device=DEV) if case["gain"] else None
        s.update(h_out=torch.empty(T, K, dtype=_TYPE[case["h"]], device=DEV), x=torch.empty(T, K, dtype=torch.bfloat16, device=DEV))
    elif op == "quantize":
        s["src"] = _rows(_activations(g, T, K).to(_TYPE[case["src"]]), pad)
    if op in ("norm", "quantize"):
        s.update(q=torch.empty(T, K, dtype=torch.int8, device=DEV), scale=torch.empty(T, device=DEV),
                 values=torch.empty(T, K, device=DEV))
        return s
    N = case["N"]
    q, scale = _codes(_activations(g, T, K))
    s["x"] = (_rows(q, pad), scale)
    s["w"] = [_weights(g, N, K) for _ in range(2 if op == "gated" else 1)]
    s["y"] = torch.empty(T, N + pad, dtype=_TYPE[case["y"]], device=DEV)[:, :N]
    s["base"] = torch.randn(T, N, generator=g, device=DEV) if case.get("base") else None
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "quantize": _own_quantize, "matmul": _own_matmul, "gated": _own_gated}[op](state)
    return {"norm": _plain_norm, "quantize": _plain_quantize, "matmul": _plain_matmul, "gated": _plain_gated}[op](state)


def _kept(s):
    """What a program keeps: the descriptors of its 8-bit rows and the workspace; made at the first pass."""
    if "kept" not in s:
        import bit_moe_decode_gb300 as m
        if s["case"]["op"] in ("norm", "quantize"):
            s["kept"] = (m, m.I8Rows(q=s["q"], scale=s["scale"]))
        else:
            w = [m.I8Rows(q=q, scale=scale) for q, scale in s["w"]]
            s["kept"] = (m, m.I8Rows(q=s["x"][0], scale=s["x"][1]), w, w[0].workspace(s["case"]["T"]))
    return s["kept"]


def _own_norm(s):
    m, xq = _kept(s)
    m.moe_rms_norm_i8(s["h"], xq, r=s["r"], gain=s["gain"], eps=EPS, h_out=s["h_out"], x_bf16=s["x"])
    m.moe_i8_values(xq, s["values"])
    return {"h": s["h_out"], "x": s["x"], "values": s["values"]}


def _own_quantize(s):
    m, xq = _kept(s)
    m.moe_i8_quantize(s["src"], xq)
    m.moe_i8_values(xq, s["values"])
    return {"values": s["values"]}


def _own_matmul(s):
    m, x, w, ws = _kept(s)
    y = s["y"]
    if y.dtype == torch.float32:
        m.moe_i8_matmul(x, w[0], y=y, base=s["base"], ws=ws)
    else:
        m.moe_i8_matmul(x, w[0], y_bf16=y, base=s["base"], ws=ws)
    return {"y": y}


def _own_gated(s):
    m, x, w, ws = _kept(s)
    y = s["y"]
    if y.dtype == torch.float32:
        m.moe_i8_gated(x, w[0], w[1], y=y, ws=ws)
    else:
        m.moe_i8_gated(x, w[0], w[1], y_bf16=y, ws=ws)
    return {"y": y}


def _plain_values(v):
    a = v.abs().amax(1, keepdim=True).clamp_min(FLOOR)
    return torch.round(v.double() * 127.0 / a.double()).float(), a


def _plain_norm(s):
    h = s["h"].float()
    if s["r"] is not None:
        h = h + s["r"].float()
    v = h if s["gain"] is None else h * s["gain"]
    rho = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    q, a = _plain_values(v)
    return {"h": h.to(s["h"].dtype), "x": (v * rho).to(torch.bfloat16), "values": q * (a * rho / 127.0)}


def _plain_quantize(s):
    q, a = _plain_values(s["src"].float())
    return {"values": q * (a / 127.0)}


def _plain_product(s, w):
    (q, scale), (wq, wscale) = s["x"], w
    return (q.float() @ wq.float().T) * scale[:, None] * wscale


def _plain_matmul(s):
    y = _plain_product(s, s["w"][0])
    if s["base"] is not None:
        y = y + s["base"]
    return {"y": y.to(s["y"].dtype)}


def _plain_gated(s):
    g, u = (_plain_product(s, w) for w in s["w"])
    return {"y": (g / (1.0 + torch.exp(-g)) * u).to(s["y"].dtype)}


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "quantize": _exact_quantize, "matmul": _exact_matmul, "gated": _exact_gated}[case["op"]](s)


def _exact_rows(v, factor):
    """The values that 8 bits of the rows of v stand for, times factor [T, 1]: 127 steps to the largest."""
    top = torch.linalg.vector_norm(v, ord=math.inf, dim=1, keepdim=True).clamp_min(FLOOR)
    return torch.round(127 * v / top) * (top * factor / 127)


def _exact_norm(s):
    h = s["h"].double()
    if s["r"] is not None:
        h = h + s["r"].double()
    factor = (h.square().sum(1, keepdim=True) / h.shape[1] + EPS).rsqrt()
    g = 1.0 if s["gain"] is None else s["gain"].double()
    held = (h.float().double() * g).float().double()          # what is quantised: the sum and its product as fp32 holds them
    return {"h": h, "x": h * g * factor, "values": _exact_rows(held, factor)}


def _exact_quantize(s):
    v = s["src"].double()
    return {"values": _exact_rows(v, torch.ones(v.shape[0], 1, dtype=torch.float64, device=DEV))}


def _exact_product(x, w):
    """Rows in blocks, the integers' sums in 64 bits (exact: below 2^53)."""
    (q, scale), (wq, wscale) = x, w
    right = wq.double().t().contiguous()
    return torch.cat([torch.mm(q[i:i + 512].double(), right) * torch.outer(scale[i:i + 512].double(), wscale.double())
                      for i in range(0, q.shape[0], 512)])


def _exact_matmul(s):
    y = _exact_product(s["x"], s["w"][0])
    return {"y": y if s["base"] is None else y + s["base"].double()}


def _exact_gated(s):
    g, u = (_exact_product(s["x"], w) for w in s["w"])
    return {"y": g * torch.sigmoid(g) * u}
