"""A small decoder that runs a whole decode step on this library.

Every projection is a quantized product (``qmm_forward_fused``, ``qmm_forward``);
between them ``qmm_qk_norm_rope`` norms and rotates queries and keys into the
paged cache, ``qmm_paged_attention`` attends over it, and after the last
projection ``qmm_sample`` chooses the tokens. Residuals, the layers' norms and
the gate are plain torch. Weights are random: the point is how the calls fit
together, for a prompt, for one token at a time, for several drafted rows of a
verify step, and captured into a graph.

    python examples/decode_step.py
"""
from __future__ import annotations

import sys
from dataclasses import dataclass
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parents[1]))

import affine_group_quantized_qmm_amd as qmm  # noqa: E402

BITS, G = 4, 32


@dataclass
class Config:
    layers: int = 2
    hidden: int = 512
    heads: int = 8
    kv_heads: int = 2
    head_dim: int = 64
    rotary: int = 32
    ffn: int = 1024
    vocab: int = 2048
    pages: int = 64
    page_size: int = 16
    max_pages: int = 16    # of one sequence
    window: int = 0        # of the odd layers; 0: all tokens
    sinks: int = 0
    eps: float = 1e-6


def random_weight(N: int, K: int, gen, dev):
    """(packed words, scales, biases) of an [N, K] matrix with values around zero."""
    codes = torch.randint(0, 1 << BITS, (N, K), generator=gen, dtype=torch.uint8).to(dev)
    scales = (torch.rand(N, K // G, generator=gen) * 0.01 + 0.005).half()
    biases = (-7.5 * scales.float()).half()  # the codes' middle
    return qmm.qmm_pack(codes, BITS), scales.to(dev), biases.to(dev)


class Decoder:
    def __init__(self, c: Config, seed: int = 0, device: str = "cuda"):
        g = torch.Generator().manual_seed(seed)
        self.c, self.dev = c, torch.device(device)
        D = c.head_dim

        def w(N, K):
            return random_weight(N, K, g, self.dev)
        self.embedding = torch.randn(c.vocab, c.hidden, generator=g).to(self.dev)
        self.layers = [dict(q=w(c.heads * D, c.hidden), k=w(c.kv_heads * D, c.hidden), v=w(c.kv_heads * D, c.hidden),
                            o=w(c.hidden, c.heads * D), gate=w(c.ffn, c.hidden), up=w(c.ffn, c.hidden),
                            down=w(c.hidden, c.ffn),
                            q_norm=(1 + 0.1 * torch.randn(D, generator=g)).to(self.dev),
                            k_norm=(1 + 0.1 * torch.randn(D, generator=g)).to(self.dev)) for _ in range(c.layers)]
        self.head = w(c.vocab, c.hidden)
        self.inv_freq = (1e4 ** (-torch.arange(0, c.rotary, 2).double() / c.rotary)).float().to(self.dev)
        shape = (c.pages, c.kv_heads, c.page_size, D)
        self.caches = [(torch.zeros(shape, dtype=torch.float16, device=self.dev),
                        torch.zeros(shape, dtype=torch.float16, device=self.dev)) for _ in range(c.layers)]

    def norm(self, x):
        return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + self.c.eps)).half()

    def logits(self, tokens, batch) -> torch.Tensor:
        """fp32 [T, vocab] of the rows `tokens` [T], whose keys and values join the cache."""
        c, T, D = self.c, tokens.shape[0], self.c.head_dim
        x = self.embedding[tokens.long()]
        for i, p in enumerate(self.layers):
            q, k, v = qmm.qmm_forward_fused(self.norm(x), [p["q"], p["k"], p["v"]], BITS, G)
            kc, vc = self.caches[i]
            q = qmm.qmm_qk_norm_rope(q.view(T, c.heads, D), k.view(T, c.kv_heads, D), v.view(T, c.kv_heads, D),
                                     p["q_norm"], p["k_norm"], batch.positions, self.inv_freq, batch.slots, kc, vc,
                                     eps=c.eps)
            a = qmm.qmm_paged_attention(q, kc, vc, batch.block_table, batch.context_lens, batch.row_starts,
                                        batch.max_rows, batch.max_context, window=c.window if i % 2 else 0,
                                        sinks=c.sinks)
            x = x + qmm.qmm_forward(a.view(T, c.heads * D), *p["o"], BITS, G)
            gate, up = qmm.qmm_forward_fused(self.norm(x), [p["gate"], p["up"]], BITS, G)
            x = x + qmm.qmm_forward((torch.nn.functional.silu(gate) * up).half(), *p["down"], BITS, G)
        return qmm.qmm_forward(self.norm(x), *self.head, BITS, G)

    def step(self, tokens, batch, u, **sampling) -> torch.Tensor:
        """One token for each row."""
        return qmm.qmm_sample(self.logits(tokens, batch), u, **sampling)


class Batch:
    """Where the rows of a call stand: `rows[b]` new rows after `past[b]` tokens
    of each sequence b, whose pages are `pages[b]`."""

    def __init__(self, c: Config, pages, past, rows, device="cuda"):
        def ints(v):
            return torch.tensor(v, dtype=torch.int32, device=device)
        positions, slots, starts = [], [], [0]
        for pg, p, n in zip(pages, past, rows):
            for t in range(p, p + n):
                positions.append(t)
                slots.append(pg[t // c.page_size] * c.page_size + t % c.page_size)
            starts.append(starts[-1] + n)
        self.positions, self.slots, self.row_starts = ints(positions), ints(slots), ints(starts)
        self.context_lens = ints([p + n for p, n in zip(past, rows)])
        self.block_table = ints([list(pg) + [-1] * (c.max_pages - len(pg)) for pg in pages])
        self.max_rows = max(rows)
        self.max_context = c.max_pages * c.page_size


def main() -> None:
    c = Config()
    model = Decoder(c)
    pages = [list(range(0, 16)), list(range(16, 32))]
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, c.vocab, (n,), generator=g, dtype=torch.int32) for n in (37, 20)]
    past = [0, 0]
    rows = [len(p) for p in prompts]
    u = torch.rand(sum(rows), generator=g).cuda()
    out = model.step(torch.cat(prompts).cuda(), Batch(c, pages, past, rows), u,
                     temperature=torch.full_like(u, 0.8), top_p=torch.full_like(u, 0.9))
    last = out[[rows[0] - 1, sum(rows) - 1]]
    text = [[int(t)] for t in last]
    past = rows
    for _ in range(8):
        u = torch.rand(2, generator=g).cuda()
        last = model.step(last, Batch(c, pages, past, [1, 1]), u, temperature=torch.full_like(u, 0.8),
                          top_p=torch.full_like(u, 0.9))
        past = [p + 1 for p in past]
        for t, n in zip(text, last.tolist()):
            t.append(n)
    print("tokens:", text)


if __name__ == "__main__":
    main()
