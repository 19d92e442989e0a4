"""Speculative decoding with the library's calls: the verify step of a small routed-MoE decoder with random weights.

Per step each sequence brings its last token and K drafts. In every layer their keys and values are appended to the 4-bit
paged cache (rotated on the way), the new rows attend to it, and the routed experts serve all rows in one sweep; after the
last layer the logits become probabilities (penalties, temperature) and moe_spec_accept keeps the drafts that the model
agrees with. Rejected tokens stay in the cache past the sequence's length and are overwritten by the next step.

    python examples/verify_step.py --seqs 2 --drafts 3 --steps 20
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_moe_decode_gb300 as m  # noqa: E402


class Decoder:
    def __init__(self, seqs=2, drafts=3, layers=2, H=512, I=256, E=8, k=2, heads=8, kv_heads=2, D=64, vocab=1024, max_len=512,
                 fmt=None, temperature=0.8, seed=0, device="cuda"):
        rows = seqs * (1 + drafts)
        assert rows <= 8, "the experts' verify sweep takes up to 8 rows"
        self.S, self.K, self.R, self.H, self.E, self.k, self.V, self.D = seqs, drafts, rows, H, E, k, vocab, D
        self.heads, self.kv_heads, self.max_len, self.dev = heads, kv_heads, max_len, device
        g = torch.Generator(device).manual_seed(seed)
        self.gen = torch.Generator(device).manual_seed(seed + 1)

        def rand(*shape, dtype=torch.bfloat16):
            return (torch.randn(*shape, generator=g, device=device) / shape[-1] ** 0.5).to(dtype)

        self.embed, self.head = rand(vocab, H) * H ** 0.5, rand(vocab, H)
        # what follows a token on its own: the drafter knows only this, the model adds what its layers say
        self.bigram = 2.0 * torch.randn(vocab, vocab, generator=g, device=device)
        self.layers = []
        page = 32
        per_seq = -(-(max_len + 8) // page)
        table = torch.randperm(seqs * per_seq, generator=g, device=device).to(torch.int32).reshape(seqs, per_seq).contiguous()
        start = torch.arange(0, rows + 1, 1 + drafts, dtype=torch.int32, device=device)
        self.seq_len = torch.zeros(seqs, dtype=torch.int32, device=device)
        self.batch = m.KvBatch(start, self.seq_len, table, tokens=rows, max_q=1 + drafts)
        for _ in range(layers):
            layer = m.Layer(m.MOE_FMT_MXFP4, H, I, E, layout=m.MOE_LAYOUT_TC, device=device)
            layer.pack(m.MOE_SRC_F32, rand(E, I, H, dtype=torch.float32), rand(E, I, H, dtype=torch.float32),
                       rand(E, H, I, dtype=torch.float32))
            self.layers.append(dict(
                qkv=rand((heads + 2 * kv_heads) * D, H), out=rand(H, heads * D), router=rand(E, H, dtype=torch.float16),
                experts=layer, cache=m.KvCache(fmt or m.MOE_FMT_MXFP4, D, kv_heads, page, n_pages=seqs * per_seq, device=device)))
        self.ws = layer.workspace(rows, k)
        self.kv_ws = self.layers[0]["cache"].workspace(self.batch, heads)
        angle = torch.arange(max_len + 8, device=device)[:, None] * 10000.0 ** (-torch.arange(0, D, 2, device=device) / D)
        self.cos, self.sin = angle.cos().contiguous(), angle.sin().contiguous()
        self.params = torch.tensor([[1.1, 0.0, 0.05, temperature]], device=device).repeat(seqs, 1).contiguous()
        self.counts = torch.zeros(seqs, vocab, dtype=torch.int32, device=device)
        self.draft = torch.zeros(seqs, drafts, dtype=torch.int32, device=device) if drafts else None
        self.idx = torch.empty(rows, k, dtype=torch.int32, device=device)
        self.w = torch.empty(rows, k, device=device)
        self.y = torch.empty(rows, H, device=device)
        self.x = torch.empty(rows, H, dtype=torch.bfloat16, device=device)
        self.q = torch.empty(rows, heads, D, dtype=torch.bfloat16, device=device)
        self.attn = torch.empty_like(self.q)
        self.probs = torch.empty(rows, vocab, device=device)
        self.result = torch.empty(seqs, 2, dtype=torch.int32, device=device)

    def forward(self, tokens):
        """Logits [rows, V] of the rows' next tokens; seq_len holds the lengths with these rows."""
        h = self.embed[tokens].float()
        for lay in self.layers:
            m.moe_rms_norm_bf16(h, self.R, self.H, 1e-6, self.x)
            qkv = (self.x @ lay["qkv"].T).view(self.R, -1, self.D)
            a, b = self.heads, self.heads + self.kv_heads
            m.moe_kv_append(lay["cache"], self.batch, qkv[:, a:b], qkv[:, b:], q=qkv[:, :a], q_out=self.q, cos=self.cos,
                            sin=self.sin, ws=self.kv_ws)
            m.moe_kv_attention(lay["cache"], self.batch, self.q, self.D ** -0.5, self.attn, ws=self.kv_ws)
            h += (self.attn.view(self.R, -1) @ lay["out"].T).float()
            m.moe_rms_norm_bf16(h, self.R, self.H, 1e-6, self.x)
            m.moe_route_topk(lay["router"], self.x, self.R, self.H, self.E, self.k, None, None, 0, self.idx, self.w)
            m.moe_expert_ffn_verify(lay["experts"], self.x, self.R, self.idx, self.w, self.k, self.y, ws=self.ws)
            h += self.y
        m.moe_rms_norm_bf16(h, self.R, self.H, 1e-6, self.x)
        return (self.x @ self.head.T).float() + self.bigram[tokens]

    def step(self, last):
        """last [S]: each sequence's last token, not yet in the cache. Returns per sequence the tokens that follow it."""
        S, K, V = self.S, self.K, self.V
        tok, dist = last, []
        for j in range(K):                         # the drafter proposes from its own distribution q
            dist.append(self.bigram[tok].softmax(-1))
            tok = torch.multinomial(dist[-1], 1, generator=self.gen)[:, 0]
            self.draft[:, j] = tok
        rows = torch.cat([last[:, None], self.draft.long()], 1) if K else last[:, None]
        before = self.seq_len.clone()
        self.seq_len += 1 + K
        self.counts.scatter_add_(1, last[:, None], torch.ones_like(last[:, None], dtype=torch.int32))
        logits = self.forward(rows.reshape(-1))
        m.moe_logits_probs(logits, self.params, self.probs, rows_per_seq=1 + K, counts=self.counts, draft=self.draft)
        u = torch.rand(S, K + 1, generator=self.gen, device=self.dev)
        q = torch.stack(dist, 1).contiguous() if K else [None] * S
        for s in range(S):
            m.moe_spec_accept(self.probs[s * (1 + K):(s + 1) * (1 + K)], q[s], K, V, self.draft[s] if K else None, u[s], self.result[s])
        kept = self.result.tolist()
        for s, (n, _) in enumerate(kept):
            for j in range(n):
                self.counts[s, self.draft[s, j]] += 1
        self.seq_len.copy_(before + 1 + self.result[:, 0])
        return [self.draft[s, :n].tolist() + [t] if K else [t] for s, (n, t) in enumerate(kept)]

    def generate(self, first, steps):
        out = [[t] for t in first]
        for _ in range(steps):
            if int(self.seq_len.max()) + 1 + self.K > self.max_len:
                break
            for s, new in enumerate(self.step(torch.tensor([o[-1] for o in out], device=self.dev))):
                out[s] += new
        for ws in (self.ws, self.kv_ws):
            if m.moe_get_device_status(ws) != 0:
                raise RuntimeError("device status not OK")
        return out


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--seqs", type=int, default=2)
    ap.add_argument("--drafts", type=int, default=3)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--temperature", type=float, default=0.8)
    a = ap.parse_args()
    d = Decoder(a.seqs, a.drafts, temperature=a.temperature)
    t0 = time.time()
    out = d.generate([7 + s for s in range(a.seqs)], a.steps)
    n = sum(len(o) - 1 for o in out)
    print("%d tokens in %d steps of %d sequences (%.2f per step), %.2f s" % (n, a.steps, a.seqs, n / a.seqs / a.steps, time.time() - t0))
    for o in out:
        print(o)


if __name__ == "__main__":
    main()
