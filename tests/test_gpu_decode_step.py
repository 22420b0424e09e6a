"""The example decoder: the products and the operators between them as a decode
step runs them. Its logits against a plain 64-bit decoder that computes the
whole sequence at once from the dequantized weights, and its ways of running
(prompt, single tokens, verify rows, a captured graph) against each other."""
import numpy as np
import pytest
import torch

from tests import _gpu, _step

pytestmark = pytest.mark.gpu


def example():
    _gpu.dev()
    from examples import decode_step
    return decode_step


def dense(weight, K):
    """[N, K] in 64 bits of (words, scales, biases), code by code."""
    words, scales, biases = (t.cpu() for t in weight)
    w = words.numpy().view(np.uint32)
    codes = np.stack([(w >> (4 * j)) & 15 for j in range(8)], -1).reshape(w.shape[0], K).astype(np.float64)
    return codes * np.repeat(_step.f64(scales), 32, 1) + np.repeat(_step.f64(biases), 32, 1)


def plain_logits(model, tokens):
    """A whole sequence in 64 bits, with the 16-bit roundings of what the step
    hands from call to call left out."""
    c, D = model.c, model.c.head_dim
    inv = model.inv_freq.double().cpu().numpy()
    x = _step.f64(model.embedding)[tokens]
    n = len(tokens)

    def norm(v):
        return v / np.sqrt((v * v).mean(-1, keepdims=True) + c.eps)
    for i, p in enumerate(model.layers):
        h = norm(x)
        q, k, v = (h @ dense(p[m], c.hidden).T for m in ("q", "k", "v"))
        q, k, v = q.reshape(n, c.heads, D), k.reshape(n, c.kv_heads, D), v.reshape(n, c.kv_heads, D)
        for t in range(n):
            for hh in range(c.heads):
                q[t, hh], _ = _step.rope_head(q[t, hh], _step.f64(p["q_norm"]), t, inv, c.eps, 0.0, False)
            for hh in range(c.kv_heads):
                k[t, hh], _ = _step.rope_head(k[t, hh], _step.f64(p["k_norm"]), t, inv, c.eps, 0.0, False)
        a = np.zeros((n, c.heads, D))
        for t in range(n):
            see = _step.visible_tokens(t, c.window if i % 2 else 0, c.sinks)
            for hh in range(c.heads):
                kv = hh // (c.heads // c.kv_heads)
                s = k[see, kv] @ q[t, hh] / np.sqrt(D)
                w = np.exp(s - s.max())
                a[t, hh] = w / w.sum() @ v[see, kv]
        x = x + a.reshape(n, -1) @ dense(p["o"], c.heads * D).T
        h = norm(x)
        gate, up = h @ dense(p["gate"], c.hidden).T, h @ dense(p["up"], c.hidden).T
        x = x + (gate / (1 + np.exp(-gate)) * up) @ dense(p["down"], c.ffn).T
    return norm(x) @ dense(model.head, c.hidden).T


@pytest.mark.parametrize("window,sinks", [(0, 0), (11, 2)])
def test_logits_against_plain_decoder(window, sinks):
    ex = example()
    c = ex.Config(window=window, sinks=sinks)
    model = ex.Decoder(c, seed=3)
    tokens = np.random.default_rng(4).integers(0, c.vocab, 50)
    got = model.logits(torch.tensor(tokens, dtype=torch.int32, device="cuda"), ex.Batch(c, [range(9, 25)], [0], [50]))
    want = plain_logits(model, tokens)
    # Each of the two layers rounds seven times to fp16 (two norms, q, k, v, the
    # attention, the gated product), the end once: 15 roundings of 2^-11 that a
    # product of random signs carries on without enlarging them in the 2-norm,
    # each at most doubled by the norm and the softmax after it.
    rel = np.linalg.norm(_step.f64(got) - want) / np.linalg.norm(want)
    assert rel < 15 * 2 * 2.0 ** -11, rel


def test_prompt_steps_and_verify_rows_agree():
    """The same sequence as one prompt, token by token and in verify steps of
    five rows gives the same greedy tokens."""
    ex = example()
    c = ex.Config()
    prompt = torch.randint(0, c.vocab, (21,), generator=torch.Generator().manual_seed(5), dtype=torch.int32).cuda()
    pages = [[3, 40, 7, 12, 30, 1]]
    greedy = dict(temperature=torch.zeros(1, device="cuda"))
    u = torch.zeros(1, device="cuda")
    model = ex.Decoder(c, seed=6)
    model.logits(prompt[:-1], ex.Batch(c, pages, [0], [20]))
    token, text = prompt[-1:], []
    for i in range(20):
        token = model.step(token, ex.Batch(c, pages, [20 + i], [1]), u, **greedy)
        text.append(token)
    text = torch.cat(text)
    whole = torch.cat((prompt, text[:-1]))
    model = ex.Decoder(c, seed=6)
    all_at_once = model.logits(whole, ex.Batch(c, pages, [0], [40]))[20:].argmax(-1)
    model = ex.Decoder(c, seed=6)
    model.logits(whole[:20], ex.Batch(c, pages, [0], [20]))
    rows = [model.logits(whole[t:t + 5], ex.Batch(c, pages, [t], [5])).argmax(-1) for t in range(20, 40, 5)]
    # near ties aside (different kernels sum in other orders), the same tokens
    assert (all_at_once.int() == text).float().mean() >= 0.9
    assert (torch.cat(rows).int() == text).float().mean() >= 0.9


def test_captured_step():
    """A decode step of two sequences in a graph: every replay equals the eager
    step on the same inputs."""
    ex = example()
    c = ex.Config()
    model = ex.Decoder(c, seed=7)
    pages = [list(range(10)), list(range(20, 30))]
    prompt = torch.randint(0, c.vocab, (40,), generator=torch.Generator().manual_seed(8), dtype=torch.int32).cuda()
    model.logits(prompt, ex.Batch(c, pages, [0, 0], [25, 15]))
    batch = ex.Batch(c, pages, [25, 15], [1, 1])
    token = torch.tensor([5, 9], dtype=torch.int32, device="cuda")
    u = torch.tensor([0.3, 0.8], device="cuda")
    sampling = dict(temperature=torch.ones(2, device="cuda"), top_p=torch.full((2,), 0.9, device="cuda"))
    model.step(token, batch, u, **sampling)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = model.step(token, batch, u, **sampling)
    for i in range(4):
        nxt = ex.Batch(c, pages, [26 + i, 16 + i], [1, 1])
        for n in ("positions", "slots", "context_lens"):
            getattr(batch, n).copy_(getattr(nxt, n))
        eager = model.step(token, batch, u, **sampling).clone()
        torch.cuda.synchronize()
        out.fill_(-7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), f"replay {i}"
        token.copy_(out)
        u.copy_(torch.rand(2))
