"""Measured cases of the operators around a verify step: the 4-bit paged KV cache (append with rotation, attention)
and the processing of logits into the probabilities that speculative acceptance reads.

Three operators:
  append     moe_kv_append: rotary positions on q and k, K and V encoded to 4-bit blocks in their pages (and
             moe_kv_read, which returns the values that the new tokens' blocks stand for);
  attention  moe_kv_attention: attention of 1..8 new tokens of each sequence over its 4-bit paged cache;
  probs      moe_logits_probs: penalties for repeated tokens, biases, an allowed-token mask, temperature, softmax.

`own` chooses between the framework's calls and their plain form (elementary torch operations in 32 bits).

The cache. A page holds page_tokens tokens of every KV head; for each head it is a run of 16-token sub-blocks. One
sub-block: K codes, V codes, K scales, V scales. A row of D values is nb = D / 32 blocks of 32 values with a scale each
(MXFP4: one E8M0 byte and E2M1 codes; INT4: a bf16 scale and two's-complement codes).
  K codes: token i's D / 2 bytes at i D / 2, as 32-bit words (c, b), c = 0..3 outer, b = 0..nb-1 inner; nibble n of
           word (c, b) is the code of dimension 32 b + 8 c + n.
  V codes: 32-bit words (g, r, c, b), g = 0..1, r = 0..7, c = 0..3, b = 0..nb-1, with the codes of tokens 8 g + 2 c and
           8 g + 2 c + 1 at dimensions 32 b + 4 r + j, j = 0..3. MXFP4: byte j, the even token in its low nibble and
           the odd one in its high nibble. INT4: nibble j for the even token, nibble 4 + j for the odd one.
  scales:  token-major, nb a token.
"""
import math
import random

import torch

own = False

MXFP4, INT4 = 1, 2
DEV = "cuda"
GRID = (6.0 / 7.0, 0.9, 0.95, 1.0, 1.05, 1.1)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
CLAMP = 2.0 ** 64        # the cache saturates at this magnitude
VOCAB = 32768            # the vocabulary of this framework's hash-routed layers


def listed():
    return [
        # one token of one sequence: the step of a single user's decode, all latency
        dict(name="append 1x1", op="append", fmt=MXFP4, B=1, q=1, ragged=False, ctx=1000, Hq=32, Hkv=8, D=128,
             page=16, rope=128, inter=False),
        # the drafts and the committed token of 48 sequences before a verify sweep, partial interleaved rotation
        dict(name="append 48x8", op="append", fmt=INT4, B=48, q=8, ragged=True, ctx=5000, Hq=32, Hkv=4, D=128,
             page=64, rope=64, inter=True),
        # prompts of four users (16381 tokens in all at the most), D = 64, one KV head a query head
        dict(name="append 4x5459", op="append", fmt=MXFP4, B=4, q=5459, ragged=True, ctx=0, Hq=16, Hkv=16, D=64,
             page=32, rope=64, inter=False),
        # one user's early decode step: latency
        dict(name="decode 1x517", op="attention", fmt=MXFP4, B=1, q=1, ragged=False, len=517, Hq=32, Hkv=8, D=128,
             page=16, window=0),
        # a serving batch of decodes, ragged, with a padding slot
        dict(name="decode 64x8192", op="attention", fmt=MXFP4, B=64, q=1, ragged=True, len=8192, Hq=32, Hkv=4, D=128,
             page=64, window=0),
        # one user's long context (an odd length), bytes from many pages for one row of queries
        dict(name="decode 1x262143", op="attention", fmt=INT4, B=1, q=1, ragged=False, len=262143, Hq=32, Hkv=8, D=128,
             page=128, window=0),
        # verify of 7 drafts and the committed token over long contexts: 64 query rows a KV head
        dict(name="verify8 16x32768", op="attention", fmt=MXFP4, B=16, q=8, ragged=True, len=32768, Hq=64, Hkv=8, D=128,
             page=64, window=0),
        # a large batch of short chats, one query head a KV head
        dict(name="decode 256x600", op="attention", fmt=INT4, B=256, q=1, ragged=True, len=600, Hq=16, Hkv=16, D=64,
             page=16, window=0),
        # verify of 2 drafts in a layer with a sliding window, six query heads a KV head
        dict(name="verify3 33x20000 w1024", op="attention", fmt=INT4, B=33, q=3, ragged=True, len=20000, Hq=48, Hkv=8,
             D=128, page=32, window=1024),
        # one sequence's next token: latency
        dict(name="probs 1x32768", op="probs", S=1, rows=1, V=VOCAB, dtype="f32", counts=True, bias=16, mask=False),
        # a verify step of 4 sequences, 8 rows each, under a grammar
        dict(name="probs 4x8x32768", op="probs", S=4, rows=8, V=VOCAB, dtype="bf16", counts=True, bias=100, mask=True),
        # a large batch over a large, odd vocabulary
        dict(name="probs 256x131071", op="probs", S=256, rows=1, V=131071, dtype="f32", counts=True, bias=100, mask=True),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "probs"])
    fmt = rng.choice([MXFP4, INT4])
    D = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "probs":
        V = _logint(rng, 1000, 150000)
        rows = rng.choice([1, 1, 2, 5, 8])
        S = _logint(rng, 1, max(1, min(256, 33000000 // (V * rows))))
        return dict(op=op, S=S, rows=rows, V=V, dtype=rng.choice(["f32", "bf16"]), counts=rng.random() < 0.8,
                    bias=rng.choice([0, 3, 100]), mask=rng.random() < 0.6)
    Hkv = rng.choice([1, 2, 4, 8, 16])
    if op == "append":
        q = rng.choice([1, 1, 3, 8, _logint(rng, 9, 4000)])
        B = _logint(rng, 1, max(1, min(256, 4000 // q)))
        Hq = Hkv * rng.choice([1, 2, 4])
        return dict(op=op, fmt=fmt, B=B, q=q, ragged=rng.random() < 0.7, ctx=_logint(rng, 1, 6000) - 1, Hq=Hq, Hkv=Hkv,
                    D=D, page=page, rope=rng.choice([0, 32, D]), inter=rng.random() < 0.5)
    q = rng.choice([1, 1, 1, 2, 4, 7, 8])
    group = rng.choice([1, 2, 3, 4, 6, 8, 16])
    B = _logint(rng, 1, 256)
    most = 1.0e6 / (Hkv * B) * (8.0 / max(8, group * q)) * 2.0
    length = _logint(rng, 1, int(max(64, min(131072, most))))
    return dict(op=op, fmt=fmt, B=B, q=q, ragged=rng.random() < 0.7, len=length, Hq=Hkv * group, Hkv=Hkv, D=D, page=page,
                window=rng.choice([0, 0, 0, 100, 4096]))


# ------------------------------------------------------------------------------------------------ sizes of a case
def _lens(case):
    """(new tokens, sequence length after them) of each sequence; the same for every seed. A ragged batch of 8 or more
    ends with a padding slot: one row, an empty sequence."""
    B, q = case["B"], case["q"]
    r = random.Random(B * 7919 + q * 31 + case.get("len", case.get("ctx", 0)))
    ql, sl = [], []
    for b in range(B):
        n = q if (not case["ragged"] or b == 0) else r.randint(max(1, q // 2), q)
        if case["op"] == "append":
            ctx = case["ctx"] if (not case["ragged"] or b == 0) else r.randint(0, case["ctx"])
            length = ctx + n
        else:
            length = case["len"] if (not case["ragged"] or b == 0) else int(case["len"] * (0.05 + 0.95 * r.random()))
            length = max(length, n)
        ql.append(n)
        sl.append(length)
    if case["ragged"] and B >= 8:
        ql[-1], sl[-1] = 1, 0
    return ql, sl


def _sub_bytes(fmt, D):
    return 16 * D + 32 * (D // 32) * (1 if fmt == MXFP4 else 2)


def work(case):
    if case["op"] == "probs":
        n = case["S"] * case["rows"] * case["V"]
        b = n * (4 if case["dtype"] == "f32" else 2) + n * 4 + case["S"] * case["rows"] * 4
        b += (case["S"] * case["V"] * 4 if case["counts"] else 0) + (n // 8 if case["mask"] else 0)
        return {"bytes": b + case["S"] * case["bias"] * 8, "flops": 8 * n}
    ql, sl = _lens(case)
    T, D, Hq, Hkv = sum(ql), case["D"], case["Hq"], case["Hkv"]
    per_key = Hkv * _sub_bytes(case["fmt"], D) // 16
    if case["op"] == "append":
        kv = T * Hkv * D * 2
        # read q, k, v (2 bytes) and the tables; write q and the blocks; read them back, write K and V in 32 bits
        return {"bytes": 2 * T * Hq * D * 2 + kv * 2 + T * case["rope"] * 4 + 2 * T * per_key + kv * 4, "flops": 6 * T * D * (Hq + 2 * Hkv)}
    keys = pairs = 0
    for n, length in zip(ql, sl):
        lo = max(0, length - n + 1 - case["window"]) if case["window"] else 0
        keys += max(0, length - lo)
        for j in range(n):
            top = length - n + j + 1
            pairs += max(0, min(top, case["window"]) if case["window"] else top)
    return {"bytes": keys * per_key + T * Hq * D * 4 + T * Hq * 4, "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------------------------------------ 4-bit blocks
def _encode(fmt, x):
    """[..., D] fp32 -> codes [..., D] uint8, scales [..., D/32] (uint8 E8M0, or bf16 bits as int16)."""
    x = torch.nan_to_num(x, nan=0.0, posinf=CLAMP, neginf=-CLAMP).clamp(-CLAMP, CLAMP)
    w = x.reshape(*x.shape[:-1], -1, 32)
    amax = w.abs().amax(-1, keepdim=True)
    if fmt == MXFP4:
        bits = amax.view(torch.int32)
        e = ((bits >> 23) - 2 + ((bits & 0x7FFFFF) > 0x400000)).clamp(1, 254)
        # w 2^(127 - e) by two exact powers of two (one alone can lie outside fp32's range)
        h = (127 - e) >> 1
        v = w * ((h + 127) << 23).view(torch.float32) * ((127 - e - h + 127) << 23).view(torch.float32)
        a = v.abs()
        c = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8) + (a >= 1.75).to(torch.uint8)
             + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8) + (a > 5.0).to(torch.uint8))
        c = c | (torch.signbit(v).to(torch.uint8) << 3)
        return c.reshape(x.shape), e.squeeze(-1).to(torch.uint8)
    grid = torch.tensor(GRID, dtype=torch.float32, device=x.device)
    seven = torch.full((1,), 7.0, device=x.device)                          # (by a number, torch multiplies by 1/7)
    s = amax.clamp_min(1e-8) * grid / seven                                 # [..., nb, 6]
    q = torch.round(w.unsqueeze(-2) / s.unsqueeze(-1)).clamp(-8, 7)         # [..., nb, 6, 32]
    d = w.unsqueeze(-2) - q * s.unsqueeze(-1)
    m = d * d
    m = m[..., :16] + m[..., 16:]                                           # pairwise, so that the order is fixed
    m = m[..., :8] + m[..., 8:]
    m = m[..., :4] + m[..., 4:]
    m = m[..., :2] + m[..., 2:]
    m = m[..., 0] + m[..., 1]
    first = torch.where(m == m.amin(-1, keepdim=True), torch.arange(6, device=x.device), 6).amin(-1, keepdim=True)
    s = s.gather(-1, first)
    q = q.gather(-2, first.unsqueeze(-1).expand(*first.shape, 32)).squeeze(-2)
    return (q.to(torch.int8) & 15).to(torch.uint8).reshape(x.shape), s.squeeze(-1).to(torch.bfloat16).view(torch.int16)


def _scale_f32(fmt, s):
    if fmt == MXFP4:
        return (s.to(torch.int32) << 23).view(torch.float32)   # e = 0 is zero
    return s.view(torch.bfloat16).float()


def _decode(fmt, codes, scales):
    """Codes [..., D] uint8 and scales [..., D/32] -> fp32 values."""
    t = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device) if fmt == MXFP4 else \
        torch.tensor([float(v if v < 8 else v - 16) for v in range(16)], dtype=torch.float32, device=codes.device)
    v = t[codes.to(torch.int32)].reshape(*codes.shape[:-1], -1, 32)
    return (v * _scale_f32(fmt, scales).unsqueeze(-1)).reshape(codes.shape)


def _k_bytes(codes):
    """[..., D] codes of one token -> its D / 2 bytes."""
    w = codes.reshape(*codes.shape[:-1], -1, 4, 4, 2).transpose(-4, -3)      # (c, b, byte, nibble)
    return (w[..., 0] | (w[..., 1] << 4)).reshape(*codes.shape[:-1], -1)


def _unpack(fmt, D, sub):
    """Sub-blocks [N, bytes] -> K codes, K scales, V codes, V scales of [N, 16 tokens, ...]."""
    N, nb, half = sub.shape[0], D // 32, 8 * D
    k = sub[:, :half].reshape(N, 16, 4, nb, 4)
    k = torch.stack([k & 15, k >> 4], -1).permute(0, 1, 3, 2, 4, 5).reshape(N, 16, D)
    v = sub[:, half:2 * half].reshape(N, 2, 8, 4, nb, 4)                     # g r c b byte
    v = torch.stack([v & 15, v >> 4], -1)                                    # and nibble
    if fmt == MXFP4:
        v = v.permute(0, 1, 3, 6, 4, 2, 5)                                   # byte = j, nibble = parity
    else:
        v = v.reshape(N, 2, 8, 4, nb, 2, 2, 2).permute(0, 1, 3, 5, 4, 2, 6, 7)   # byte = (parity, j / 2), nibble = j % 2
    v = v.reshape(N, 16, D)                                                  # token (g c parity), dimension (b r j)
    sc = sub[:, 2 * half:]
    if fmt == INT4:
        sc = sc.contiguous().view(torch.int16)
    sc = sc.reshape(N, 2, 16, nb)
    return k, sc[:, 0], v, sc[:, 1]


def _v_words(D, slot):
    """Byte offsets [T, 8 (r), nb] of the V words that hold tokens' codes in their sub-blocks; slot [T] in 0..15."""
    nb, dev = D // 32, slot.device
    g, c = slot >> 3, (slot >> 1) & 3
    word = ((g[:, None] * 8 + torch.arange(8, device=dev)) * 4 + c[:, None])[:, :, None] * nb + torch.arange(nb, device=dev)
    return 8 * D + word * 4


def _store(fmt, D, pages, page, sub, slot, kc, ks, vc, vs):
    """Writes tokens' codes and scales [T, Hkv, ...] into pages [n, Hkv, page / 16, bytes]."""
    T, Hkv, nb, dev = kc.shape[0], kc.shape[1], D // 32, pages.device
    at = (page[:, None, None], torch.arange(Hkv, device=dev)[None, :, None], sub[:, None, None])
    pages[at + ((slot[:, None] * (D // 2) + torch.arange(D // 2, device=dev))[:, None],)] = _k_bytes(kc)
    c = vc.reshape(T, Hkv, nb, 8, 4).transpose(2, 3)                         # (r, b, j)
    if fmt == MXFP4:                                                         # a byte is shared with the token's neighbour
        place = _v_words(D, slot)[..., None] + torch.arange(4, device=dev)
        odd = slot & 1
        e, o = (odd == 0).nonzero().squeeze(1), odd.nonzero().squeeze(1)
        to = (at[0][e], at[1], at[2][e]) + (place[e].flatten(1)[:, None],)
        pages[to] = (pages[to] & 240) | c[e].flatten(2)
        to = (at[0][o], at[1], at[2][o]) + (place[o].flatten(1)[:, None],)
        pages[to] = (pages[to] & 15) | (c[o].flatten(2) << 4)
    else:
        place = _v_words(D, slot)[..., None] + 2 * (slot & 1)[:, None, None, None] + torch.arange(2, device=dev)
        pages[at + (place.flatten(1)[:, None],)] = (c[..., 0::2] | (c[..., 1::2] << 4)).flatten(2)
    w = nb * (1 if fmt == MXFP4 else 2)
    at_s = 16 * D + slot[:, None] * w + torch.arange(w, device=dev)
    pages[at + (at_s[:, None],)] = ks.contiguous().view(torch.uint8).reshape(T, Hkv, w)
    pages[at + ((at_s + 16 * w)[:, None],)] = vs.contiguous().view(torch.uint8).reshape(T, Hkv, w)


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 2654435761 % (1 << 62) + 1)


def _kv_values(g, T, Hkv, D):
    """K with a few strong channels, as keys have, and V with tokens of differing size."""
    k = torch.randn(T, Hkv, D, generator=g, device=DEV)
    k[..., ::29] *= 4.0
    v = torch.randn(T, Hkv, D, generator=g, device=DEV) * torch.exp(0.5 * torch.randn(T, Hkv, 1, generator=g, device=DEV))
    return k, v


def _pool(case, g, sl):
    """Pages of random bytes (what is past a sequence's end is left over from others), and a block table."""
    page, Hkv, D = case["page"], case["Hkv"], case["D"]
    need = [-(-n // page) for n in sl]
    n_pages = sum(need) + 3
    pages = torch.randint(0, 256, (n_pages, Hkv, page // 16, _sub_bytes(case["fmt"], D)), dtype=torch.uint8, generator=g, device=DEV)
    perm = torch.randperm(n_pages, generator=g, device=DEV, dtype=torch.int32)
    table = torch.full((len(sl), max(max(need), 1) + 2), -1, dtype=torch.int32)
    at = 0
    perm = perm.cpu()
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return pages, table.to(DEV)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "probs":
        return _prepare_probs(case, g)
    ql, sl = _lens(case)
    T, fmt, D, Hq, Hkv, page = sum(ql), case["fmt"], case["D"], case["Hq"], case["Hkv"], case["page"]
    pages, table = _pool(case, g, sl)
    start = torch.tensor([0] + ql).cumsum(0).to(torch.int32).to(DEV)
    s = dict(case=case, pages=pages, table=table, start=start, lens=torch.tensor(sl, dtype=torch.int32, device=DEV), T=T,
             max_q=max(ql))
    if case["op"] == "append":
        # q, k and v are parts of one projection's output, as a layer has them
        qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV).to(torch.bfloat16)
        s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], q_out=torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV),
                 k_out=torch.empty(T, Hkv, D, device=DEV), v_out=torch.empty(T, Hkv, D, device=DEV))
        R = case["rope"]
        if R:
            n = max(sl)
            a = torch.arange(n, dtype=torch.float64)[:, None] * (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R))
            s.update(cos=a.cos().float().to(DEV), sin=a.sin().float().to(DEV))
    else:
        flat = torch.arange(len(sl), device=DEV).repeat_interleave(torch.tensor(sl, device=DEV))
        pos = torch.cat([torch.arange(n, device=DEV) for n in sl])
        step = max(1, (1 << 25) // (Hkv * D) // (8 if fmt == INT4 else 1))
        for i in range(0, flat.numel(), step):
            b, p = flat[i:i + step], pos[i:i + step]
            k, v = _kv_values(g, b.numel(), Hkv, D)
            _store(fmt, D, pages, table[b, p // page].long(), p % page // 16, p % 16, *_encode(fmt, k), *_encode(fmt, v))
        q = (1.5 * torch.randn(T, Hq, D, generator=g, device=DEV)).to(torch.bfloat16)
        s.update(q=q, out=torch.empty_like(q), lse=torch.empty(T, Hq, device=DEV), scale=D ** -0.5)
    return s


def _prepare_probs(case, g):
    S, rows, V = case["S"], case["rows"], case["V"]
    R = S * rows
    x = 3.0 * torch.randn(R, V, generator=g, device=DEV)
    x = x.to(torch.float32 if case["dtype"] == "f32" else torch.bfloat16)
    u = torch.rand(S, 4, generator=g, device=DEV)
    s = dict(case=case, logits=x, probs=torch.empty(R, V, device=DEV), top=torch.empty(R, dtype=torch.int32, device=DEV),
             counts=None, draft=None, allowed=None, bias=None)
    # repetition, presence and frequency penalties and the temperature of each sequence; every seventh is greedy
    par = torch.stack([1.0 + 0.3 * u[:, 0], 0.6 * u[:, 1], 0.4 * u[:, 2], 0.4 + u[:, 3]], 1)
    par[6::7, 3] = 0.0
    s["params"] = par.contiguous()
    if case["counts"]:
        c = torch.zeros(S, V, dtype=torch.int32, device=DEV)
        ids = (V * torch.rand(S, 700, generator=g, device=DEV) ** 3).long().clamp_max(V - 1)   # frequent tokens repeat
        c.scatter_add_(1, ids, torch.ones_like(ids, dtype=torch.int32))
        s["counts"] = c
        if rows > 1:
            s["draft"] = (V * torch.rand(S, rows - 1, generator=g, device=DEV) ** 3).int().clamp_max(V - 1)
    if case["bias"]:
        n = min(case["bias"], V)
        ids = torch.rand(S, V, generator=g, device=DEV).topk(n, 1).indices.int()
        s["bias"] = (torch.arange(S + 1, dtype=torch.int32, device=DEV) * n, ids.reshape(-1).contiguous(),
                     2.0 * torch.randn(S * n, generator=g, device=DEV))
    if case["mask"]:
        words = -(-V // 32)
        m = torch.randint(-(1 << 31), 1 << 31, (R, words), generator=g, device=DEV, dtype=torch.int64)
        few = torch.randint(-(1 << 31), 1 << 31, (R, words), generator=g, device=DEV, dtype=torch.int64) & m
        m[1::2] = few[1::2]              # a grammar's states allow some tokens, or few
        if R > 2:
            m[2] = 0                     # a state that allows none
        s["allowed"] = m.to(torch.int32)
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "attention": _own_attention, "probs": _own_probs}[op](state)
    return {"append": _plain_append, "attention": _plain_attention, "probs": _plain_probs}[op](state)


def _kv(state):
    """The cache, the batch and the workspace that a program keeps; made at the first pass."""
    if "kv" not in state:
        import bit_moe_decode_gb300 as m
        c = state["case"]
        cache = m.KvCache(c["fmt"], c["D"], c["Hkv"], c["page"], pages=state["pages"])
        batch = m.KvBatch(state["start"], state["lens"], state["table"], tokens=state["T"], max_q=state["max_q"])
        ws = cache.workspace(batch, c["Hq"])
        state["kv"] = (m, cache, batch, ws)
    return state["kv"]


def _own_append(s):
    m, cache, batch, ws = _kv(s)
    m.moe_kv_append(cache, batch, s["k"], s["v"], q=s["q"], q_out=s["q_out"], cos=s.get("cos"), sin=s.get("sin"),
                    interleaved=s["case"]["inter"], ws=ws)
    m.moe_kv_read(cache, batch, s["k_out"], s["v_out"], ws=ws)
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _own_attention(s):
    m, cache, batch, ws = _kv(s)
    m.moe_kv_attention(cache, batch, s["q"], s["scale"], s["out"], lse=s["lse"], window=s["case"]["window"], ws=ws)
    return {"out": s["out"], "lse": s["lse"]}


def _own_probs(s):
    import bit_moe_decode_gb300 as m
    m.moe_logits_probs(s["logits"], s["params"], s["probs"], rows_per_seq=s["case"]["rows"], counts=s["counts"], draft=s["draft"],
                       bias=s["bias"], allowed=s["allowed"], top=s["top"])
    return {"probs": s["probs"], "top": s["top"]}


def _tokens(s):
    """(sequence, position, order among the sequence's new tokens) of every new token."""
    start, lens = s["start"].long(), s["lens"].long()
    t = torch.arange(s["T"], device=DEV)
    b = torch.searchsorted(start, t, right=True) - 1
    n = start[b + 1] - start[b]
    return b, lens[b] - n + (t - start[b]), t - start[b]


def _rotate(x, cos, sin, inter):
    R = 2 * cos.shape[-1]
    c, n = cos[:, None], sin[:, None]
    if inter:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        return torch.cat([torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2), x[..., R:]], -1)
    a, b = x[..., :R // 2], x[..., R // 2:R]
    return torch.cat([a * c - b * n, b * c + a * n, x[..., R:]], -1)


def _plain_append(s):
    c = s["case"]
    fmt, D, page = c["fmt"], c["D"], c["page"]
    b, pos, _ = _tokens(s)
    there = pos >= 0                     # a padding slot's row has no place in the cache
    at = pos.clamp_min(0)
    q, k = s["q"].float(), s["k"].float()
    if c["rope"]:
        cos, sin = s["cos"][at], s["sin"][at]
        q, k = _rotate(q, cos, sin, c["inter"]), _rotate(k, cos, sin, c["inter"])
    kc, ks = _encode(fmt, k)
    vc, vs = _encode(fmt, s["v"].float())
    i = there.nonzero().squeeze(1)
    p = s["table"][b[i], at[i] // page].long()
    _store(fmt, D, s["pages"], p, at[i] % page // 16, at[i] % 16, kc[i], ks[i], vc[i], vs[i])
    keep = there[:, None, None]
    return {"q": q.to(torch.bfloat16), "k": torch.where(keep, _decode(fmt, kc, ks), 0.0), "v": torch.where(keep, _decode(fmt, vc, vs), 0.0)}


def _plain_attention(s):
    c = s["case"]
    fmt, D, Hq, Hkv, page, B = c["fmt"], c["D"], c["Hq"], c["Hkv"], c["page"], c["B"]
    group, Q = Hq // Hkv, s["max_q"]
    table = s["table"][:, :-2].clamp_min(0).long()
    L = table.shape[1] * page
    # the cache of every sequence, dequantised: [B, Hkv, L, D]
    sub = s["pages"][table].transpose(1, 2).reshape(-1, _sub_bytes(fmt, D))
    kc, ks, vc, vs = _unpack(fmt, D, sub)
    key = torch.arange(L, device=DEV)
    there = (key < s["lens"][:, None])[:, None, :, None]
    k = torch.where(there, _decode(fmt, kc, ks).reshape(B, Hkv, L, D), 0.0)
    v = torch.where(there, _decode(fmt, vc, vs).reshape(B, Hkv, L, D), 0.0)
    del sub, kc, ks, vc, vs
    # the new tokens, padded to Q rows a sequence: [B, Hkv, Q group, D]
    b, pos, j = _tokens(s)
    q = torch.zeros(B, Q, Hq, D, device=DEV)
    q[b, j] = s["q"].float()
    q = q.reshape(B, Q, Hkv, group, D).transpose(1, 2).reshape(B, Hkv, Q * group, D)
    x = (q @ k.transpose(-1, -2)) * s["scale"]
    top = torch.full((B, Q), -1, dtype=torch.long, device=DEV)
    top[b, j] = pos
    row = top.repeat_interleave(group, 1)[:, None, :, None]
    seen = key <= row
    if c["window"]:
        seen = seen & (key > row - c["window"])
    x = x.masked_fill(~seen, -math.inf)
    most = x.amax(-1, keepdim=True)
    p = torch.exp(x - most.clamp_min(-3e38))
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / total.clamp_min(1e-38)
    lse = torch.where(total > 0, most + torch.log(total), -math.inf)
    o = o.reshape(B, Hkv, Q, group, D).transpose(1, 2).reshape(B, Q, Hq, D)[b, j]
    lse = lse.reshape(B, Hkv, Q, group).transpose(1, 2).reshape(B, Q, Hq)[b, j]
    return {"out": o.to(torch.bfloat16), "lse": lse}


def _plain_probs(s):
    c = s["case"]
    S, rows, V = c["S"], c["rows"], c["V"]
    seq = torch.arange(S, device=DEV).repeat_interleave(rows)
    rep, presence, frequency, temperature = s["params"][seq].unsqueeze(-1).unbind(1)
    x = s["logits"].float()
    x = torch.where(torch.isnan(x), -math.inf, x)
    if s["counts"] is not None:
        n = s["counts"][seq]
        if s["draft"] is not None:       # row j has seen the drafts before it
            d = s["draft"].long().repeat_interleave(rows, 0)
            j = torch.arange(rows, device=DEV).repeat(S)
            n = n.scatter_add(1, d, (torch.arange(rows - 1, device=DEV) < j[:, None]).to(n.dtype))
        y = torch.where(n > 0, torch.where(x > 0, x / rep, x * rep), x)
        y = y - frequency * n.float()
        x = torch.where(n > 0, y - presence, x)
    if s["bias"] is not None:
        n = s["bias"][1].numel() // S
        x = x.scatter_add(1, s["bias"][1].long().reshape(S, n)[seq], s["bias"][2].reshape(S, n)[seq])
    if s["allowed"] is not None:
        v = torch.arange(V, device=DEV)
        ok = (s["allowed"][:, v // 32] >> (v % 32)) & 1
        x = torch.where(ok != 0, x, -math.inf)
    most = x.amax(-1, keepdim=True)
    top = torch.where(x == most, torch.arange(V, device=DEV, dtype=torch.int32), V).amin(-1)
    t = torch.where(temperature > 0, temperature, 1.0)
    e = torch.where(most == math.inf, (x == math.inf).float(), torch.exp(x / t - (most / t).clamp_min(-3e38)))
    p = e / e.sum(-1, keepdim=True).clamp_min(1e-38)
    p = torch.where(temperature > 0, p, (torch.arange(V, device=DEV) == top[:, None]).float())
    none = most == -math.inf
    return {"probs": torch.where(none, 0.0, p), "top": torch.where(none.squeeze(1), -1, top).to(torch.int32)}


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "probs": _exact_probs}[case["op"]](case, s)


def _exact_blocks(fmt, x):
    """The values that 4-bit blocks of x [..., D] (64 bits) stand for."""
    w = x.clamp(-CLAMP, CLAMP).reshape(-1, 32)
    amax = w.abs().amax(1, keepdim=True)
    if fmt == MXFP4:
        k = torch.ceil(torch.log2((amax / 6).clamp_min(2.0 ** -200))).clamp(-126, 127)
        k = torch.where(amax > 6 * torch.exp2(k), k + 1, torch.where(amax <= 6 * torch.exp2(k - 1), k - 1, k)).clamp_min(-126)
        u = (w / torch.exp2(k)).abs()
        # E2M1 has steps of 0.5 below 2, 1 below 4, then 2; torch.round takes a tie to the even multiple
        r = torch.where(u < 2, torch.round(u * 2) / 2, torch.where(u < 4, torch.round(u), (torch.round(u / 2) * 2).clamp_max(6)))
        return (torch.sign(w) * r * torch.exp2(k)).reshape(x.shape)
    best = torch.full_like(amax, math.inf)
    out = torch.zeros_like(w)
    for g in GRID:
        sc = amax.clamp_min(1e-8) * g / 7
        q = torch.round(w / sc).clamp(-8, 7)
        err = ((w - q * sc) ** 2).sum(1, keepdim=True)
        out = torch.where(err < best, q * sc.to(torch.float32).to(torch.bfloat16).double(), out)
        best = torch.minimum(best, err)
    return out.reshape(x.shape)


def _exact_read(fmt, D, sub):
    """K and V [N 16, D] in 64 bits of sub-blocks [N, bytes], each value from its place by the layout's definition."""
    nb = D // 32
    i, d = torch.arange(16, device=DEV)[:, None], torch.arange(D, device=DEV)[None]
    b, n = d // 32, d % 32
    z = sub.long()
    kn = (z[:, i * (D // 2) + ((n // 8) * nb + b) * 4 + n % 8 // 2] >> (4 * (n % 2))) & 15
    at = 8 * D + ((((i // 8) * 8 + n // 4) * 4 + i % 8 // 2) * nb + b) * 4
    if fmt == MXFP4:
        vn = (z[:, at + n % 4] >> (4 * (i % 2))) & 15
        first = 16 * D + i * nb + b
        size = [torch.where(z[:, first + 16 * nb * w] > 0, torch.exp2(z[:, first + 16 * nb * w].double() - 127), 0.0) for w in (0, 1)]
        sign, e, m = [[f(c) for c in (kn, vn)] for f in (lambda c: 1.0 - 2.0 * (c >> 3), lambda c: (c >> 1) & 3, lambda c: (c & 1).double())]
        k, v = (sign[w] * torch.where(e[w] > 0, torch.exp2(e[w].double() - 1) * (1 + m[w] / 2), m[w] / 2) for w in (0, 1))
    else:
        vn = (z[:, at + (i % 2) * 2 + n % 4 // 2] >> (4 * (n % 2))) & 15
        first = 16 * D + (i * nb + b) * 2
        size = [((z[:, first + 32 * nb * w] + 256 * z[:, first + 32 * nb * w + 1]) << 16).int().view(torch.float32).double() for w in (0, 1)]
        k, v = ((c - 16 * (c > 7)).double() for c in (kn, vn))
    return (k * size[0]).reshape(-1, D), (v * size[1]).reshape(-1, D)


def _exact_append(case, s):
    ql, sl = _lens(case)
    pos = torch.cat([torch.arange(n - q, n) for q, n in zip(ql, sl)])
    q, k, v = (s[n].double() for n in "qkv")
    R = case["rope"]
    if R:
        at = pos.clamp_min(0).to(DEV)
        z = torch.complex(s["cos"].double(), s["sin"].double())[at][:, None]

        def turn(x):
            y = x.clone()
            a, b = (slice(0, R, 2), slice(1, R, 2)) if case["inter"] else (slice(0, R // 2), slice(R // 2, R))
            w = torch.complex(x[..., a].contiguous(), x[..., b].contiguous()) * z
            y[..., a], y[..., b] = w.real, w.imag
            return y
        q, k = turn(q), turn(k)
    keep = (pos >= 0).to(DEV).double()[:, None, None]
    return {"q": q, "k": _exact_blocks(case["fmt"], k) * keep, "v": _exact_blocks(case["fmt"], v) * keep}


def _exact_attention(case, s):
    ql, sl = _lens(case)
    fmt, D, Hq, Hkv, page = case["fmt"], case["D"], case["Hq"], case["Hkv"], case["page"]
    group = Hq // Hkv
    if sum(sl) * Hq * case["q"] * D > 1.2e11:
        return None
    out = torch.zeros(s["T"], Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((s["T"], Hq), -math.inf, dtype=torch.float64, device=DEV)
    t = 0
    for b, (n, length) in enumerate(zip(ql, sl)):
        if length:
            own_pages = s["pages"][s["table"][b, :-(-length // page)].long()]
            for h in range(Hkv):
                k, v = (x[:length] for x in _exact_read(fmt, D, own_pages[:, h].reshape(-1, own_pages.shape[-1])))
                q = s["q"][t:t + n, h * group:(h + 1) * group].double()
                x = torch.einsum("jgd,ld->jgl", q, k) * s["scale"]
                at = torch.arange(length, device=DEV)
                top = torch.arange(length - n, length, device=DEV)[:, None]
                hide = at > top
                if case["window"]:
                    hide = hide | (at <= top - case["window"])
                x = x.masked_fill(hide[:, None], -math.inf)
                lse[t:t + n, h * group:(h + 1) * group] = torch.logsumexp(x, -1)
                out[t:t + n, h * group:(h + 1) * group] = torch.einsum("jgl,ld->jgd", torch.softmax(x, -1), v)
        t += n
    return {"out": out, "lse": lse}


def _exact_probs(case, s):
    S, rows, V = case["S"], case["rows"], case["V"]
    probs = torch.zeros(S * rows, V, dtype=torch.float64, device=DEV)
    for r in range(S * rows):
        i, j = divmod(r, rows)
        rep, presence, frequency, temperature = s["params"][i].double().tolist()
        x = s["logits"][r].double()
        if s["counts"] is not None:
            n = s["counts"][i].double()
            for d in (s["draft"][i, :j].tolist() if s["draft"] is not None else []):
                n[d] += 1
            hit = n > 0
            x = torch.where(hit, torch.where(x > 0, x / rep, x * rep) - frequency * n - presence, x)
        if s["bias"] is not None:
            a, b = s["bias"][0][i:i + 2].tolist()
            x[s["bias"][1][a:b].long()] += s["bias"][2][a:b].double()
        if s["allowed"] is not None:
            bits = (s["allowed"][r][:, None] >> torch.arange(32, device=DEV)) & 1
            x = x.masked_fill(bits.reshape(-1)[:V] == 0, -math.inf)
        if x.max() > -math.inf:
            if temperature > 0:
                probs[r] = torch.softmax(x / temperature, 0)
            else:
                probs[r, int(torch.argmax(x))] = 1.0
    return {"probs": probs, "top": None}
