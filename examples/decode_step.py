"""A small decoder that runs a whole decode step on this library.

Every projection is a quantized product (``qmm_forward_fused``, ``qmm_forward``);
between them ``qmm_qk_norm_rope`` norms and rotates queries and keys into the
paged cache, ``qmm_paged_attention`` attends over it, and after the last
projection ``qmm_sample`` chooses the tokens. With ``cache_bits`` the cache holds
8- or 4-bit codes (``qmm_qk_norm_rope_quant``, ``qmm_paged_attention_quant``); with
``adapters`` each row may have a low-rank adapter of its own beside the
projections (``qmm_lora``); ``qmm_logprobs`` reports what the chosen tokens'
probabilities were. Residuals, the layers' norms and the gate are plain torch. Weights are random: the point is how the calls fit
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
    cache_bits: int = 0    # 8 or 4: a cache of codes; 0: of fp16 rows
    cache_group: int = 32
    adapters: int = 0      # beside q, k, v and the output projection
    rank: int = 8


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
        shape = (c.pages, c.kv_heads, c.page_size)

        def cache():  # rows, or (codes, scales and biases)
            if c.cache_bits == 0:
                return (torch.zeros(*shape, D, dtype=torch.float16, device=self.dev),)
            return tuple(torch.zeros(*shape, n, dtype=torch.int32, device=self.dev)
                         for n in (D * c.cache_bits // 32, D // c.cache_group))
        self.caches = [cache() + cache() for _ in range(c.layers)]
        # (A [n, r, K], B [n, N, r]) of each projection that has adapters, and their scales.
        sizes = dict(q=(c.heads * D, c.hidden), k=(c.kv_heads * D, c.hidden), v=(c.kv_heads * D, c.hidden),
                     o=(c.hidden, c.heads * D))
        self.adapters = [{m: ((torch.randn(c.adapters, c.rank, K, generator=g) * K ** -0.5).half().to(self.dev),
                              (torch.randn(c.adapters, N, c.rank, generator=g) * 0.2).half().to(self.dev))
                          for m, (N, K) in sizes.items()} for _ in range(c.layers if c.adapters else 0)]
        self.adapter_scales = torch.rand(c.adapters, generator=g).to(self.dev) + 0.5

    def norm(self, x):
        return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + self.c.eps)).half()

    def adapted(self, layer, names, x, ys, batch):
        """The products `ys` of `x` with what each row's adapter adds to them."""
        if self.c.adapters == 0 or batch.adapters is None:
            return ys
        return qmm.qmm_lora(x, [self.adapters[layer][m] for m in names], batch.adapters, ys, scales=self.adapter_scales)

    def logits(self, tokens, batch) -> torch.Tensor:
        """fp32 [T, vocab] of the rows `tokens` [T], whose keys and values join the cache."""
        c, T, D = self.c, tokens.shape[0], self.c.head_dim
        x = self.embedding[tokens.long()]
        for i, p in enumerate(self.layers):
            h = self.norm(x)
            q, k, v = self.adapted(i, "qkv", h, qmm.qmm_forward_fused(h, [p["q"], p["k"], p["v"]], BITS, G), batch)
            new = (q.view(T, c.heads, D), k.view(T, c.kv_heads, D), v.view(T, c.kv_heads, D), p["q_norm"], p["k_norm"],
                   batch.positions, self.inv_freq, batch.slots, *self.caches[i])
            where = (batch.block_table, batch.context_lens, batch.row_starts, batch.max_rows, batch.max_context)
            seen = dict(window=c.window if i % 2 else 0, sinks=c.sinks)
            if c.cache_bits:
                q = qmm.qmm_qk_norm_rope_quant(*new, c.cache_bits, c.cache_group, eps=c.eps)
                a = qmm.qmm_paged_attention_quant(q, *self.caches[i], c.cache_bits, c.cache_group, *where, **seen)
            else:
                q = qmm.qmm_qk_norm_rope(*new, eps=c.eps)
                a = qmm.qmm_paged_attention(q, *self.caches[i], *where, **seen)
            a = a.view(T, c.heads * D)
            x = x + self.adapted(i, "o", a, [qmm.qmm_forward(a, *p["o"], BITS, G)], batch)[0]
            gate, up = qmm.qmm_forward_fused(self.norm(x), [p["gate"], p["up"]], BITS, G)
            x = x + qmm.qmm_forward((torch.nn.functional.silu(gate) * up).half(), *p["down"], BITS, G)
        return qmm.qmm_forward(self.norm(x), *self.head, BITS, G)

    def step(self, tokens, batch, u, **sampling) -> torch.Tensor:
        """One token for each row."""
        return qmm.qmm_sample(self.logits(tokens, batch), u, **sampling)

    def step_with_logprobs(self, tokens, batch, u, top_n: int = 0, **sampling):
        """One token for each row, and qmm_logprobs of it."""
        logits = self.logits(tokens, batch)
        chosen = qmm.qmm_sample(logits, u, **sampling)
        return chosen, qmm.qmm_logprobs(logits, chosen, top_n)


class Batch:
    """Where the rows of a call stand: `rows[b]` new rows after `past[b]` tokens
    of each sequence b, whose pages are `pages[b]`, under `adapters[b]` (-1: none)."""

    def __init__(self, c: Config, pages, past, rows, device="cuda", adapters=None):
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
        self.adapters = None if adapters is None else ints([i for i, n in zip(adapters, rows) for _ in range(n)])
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

    # The same prompts over a cache of 8-bit codes, the second under an adapter.
    c = Config(cache_bits=8, adapters=2)
    model = Decoder(c)
    rows = [len(p) for p in prompts]
    u = torch.zeros(sum(rows), device="cuda")
    chosen, (logprobs, ranks, entropy, top_tokens, _) = model.step_with_logprobs(
        torch.cat(prompts).cuda(), Batch(c, pages, [0, 0], rows, adapters=[-1, 1]), u, top_n=3,
        temperature=torch.zeros_like(u))
    for b, row in enumerate((rows[0] - 1, sum(rows) - 1)):
        print(f"sequence {b}: token {int(chosen[row])}, log probability {float(logprobs[row]):.2f}, rank "
              f"{int(ranks[row])}, entropy {float(entropy[row]):.2f}, likeliest {top_tokens[row].tolist()}")


if __name__ == "__main__":
    main()
