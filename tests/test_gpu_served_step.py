"""The example decoder as a server of many users runs it: a cache of codes, an
adapter for each sequence, and the log probabilities of the tokens. Its logits against
a plain 64-bit decoder, and its ways of running against each other."""
import numpy as np
import pytest
import torch

from tests import _logprobs, _quant, _step
from tests.test_gpu_decode_step import dense, example

pytestmark = pytest.mark.gpu


def through_codes(y, bits, G):
    """What the cache gives back for rows y [n, H, D]."""
    codes, s, b, _ = _quant.quantize(y, bits, G)
    return (codes * np.repeat(s, G, -1) + np.repeat(b, G, -1)).astype(np.float16).astype(np.float64)


def plain_logits(model, tokens, adapter):
    """A whole sequence in 64 bits, keys and values through the cache's codes, with the
    16-bit roundings of what the step hands from call to call left out."""
    c, D = model.c, model.c.head_dim
    inv = model.inv_freq.double().cpu().numpy()
    x = _step.f64(model.embedding)[tokens]
    n = len(tokens)

    def norm(v):
        return v / np.sqrt((v * v).mean(-1, keepdims=True) + c.eps)

    def product(i, m, h):
        y = h @ dense(model.layers[i][m], h.shape[1]).T
        if adapter >= 0:
            a, b = (_step.f64(t[adapter]) for t in model.adapters[i][m])
            y = y + float(model.adapter_scales[adapter]) * (h @ a.T @ b.T)
        return y
    for i, p in enumerate(model.layers):
        h = norm(x)
        q, k, v = (product(i, m, h).reshape(n, -1, D) for m in "qkv")
        for y, w in ((q, "q_norm"), (k, "k_norm")):
            for t in range(n):
                for hh in range(y.shape[1]):
                    y[t, hh], _ = _step.rope_head(y[t, hh], _step.f64(p[w]), t, inv, c.eps, 0.0, False)
        k, v = (through_codes(y, c.cache_bits, c.cache_group) for y in (k, v))
        a = np.zeros((n, c.heads, D))
        for t in range(n):
            for hh in range(c.heads):
                kv = hh // (c.heads // c.kv_heads)
                s = k[:t + 1, kv] @ q[t, hh] / np.sqrt(D)
                w = np.exp(s - s.max())
                a[t, hh] = w / w.sum() @ v[:t + 1, kv]
        x = x + product(i, "o", a.reshape(n, -1))
        h = norm(x)
        gate, up = h @ dense(p["gate"], c.hidden).T, h @ dense(p["up"], c.hidden).T
        x = x + (gate / (1 + np.exp(-gate)) * up) @ dense(p["down"], c.ffn).T
    return norm(x) @ dense(model.head, c.hidden).T


@pytest.mark.parametrize("bits", [8, 4])
def test_logits_against_plain_decoder(bits):
    """Two sequences with adapters and one without in one call."""
    ex = example()
    c = ex.Config(cache_bits=bits, adapters=3)
    model = ex.Decoder(c, seed=3)
    rows, adapters = [30, 1, 19], [2, -1, 0]
    tokens = np.random.default_rng(4).integers(0, c.vocab, sum(rows))
    batch = ex.Batch(c, [range(9, 25), range(5), range(30, 46)], [0, 0, 0], rows, adapters=adapters)
    got = model.logits(torch.tensor(tokens, dtype=torch.int32, device="cuda"), batch)
    at = 0
    for n, adapter in zip(rows, adapters):
        want = plain_logits(model, tokens[at:at + n], adapter)
        # 15 roundings to fp16, as over a cache of rows, each at most doubled by the norm and the
        # softmax after it. Besides, an error e before the codes (in standard deviations of k or
        # v) moves a share e / step of the values to the neighbouring code, which is off by a
        # whole step: sqrt(e * step) in the 2-norm, for k and v of two layers. e is at most a
        # layer's 7 roundings, doubled likewise; a step is the range of 32 values, 4.5 standard
        # deviations, over the levels.
        e, step = 7 * 2 * 2.0 ** -11, 4.5 / (2 ** bits - 1)
        bound = 15 * 2 * 2.0 ** -11 + 4 * np.sqrt(e * step)
        rel = np.linalg.norm(_step.f64(got[at:at + n]) - want) / np.linalg.norm(want)
        assert rel < bound, (adapter, rel, bound)
        at += n


@pytest.mark.parametrize("bits", [8, 4])
def test_rows_without_an_adapter(bits):
    """Rows without an adapter have exactly the logits of a decoder that has none, also
    next to rows that have one."""
    ex = example()
    plain, c = ex.Config(cache_bits=bits), ex.Config(cache_bits=bits, adapters=2)
    tokens = torch.randint(0, c.vocab, (24,), generator=torch.Generator().manual_seed(5), dtype=torch.int32).cuda()
    pages = [range(10), range(20, 30)]
    none = ex.Decoder(c, seed=6).logits(tokens, ex.Batch(c, pages, [0, 0], [13, 11], adapters=[-1, -1]))
    assert torch.equal(none, ex.Decoder(plain, seed=6).logits(tokens, ex.Batch(plain, pages, [0, 0], [13, 11])))
    both = ex.Decoder(c, seed=6).logits(tokens, ex.Batch(c, pages, [0, 0], [13, 11], adapters=[-1, 1]))
    assert torch.equal(both[:13], none[:13])
    assert not torch.equal(both[13:], none[13:])


def test_captured_step():
    """A step of two sequences with adapters, over codes, with log probabilities, in
    a graph: every replay equals the eager step on the same inputs."""
    ex = example()
    c = ex.Config(cache_bits=4, adapters=2)
    model = ex.Decoder(c, seed=7)
    pages = [list(range(10)), list(range(20, 30))]
    prompt = torch.randint(0, c.vocab, (40,), generator=torch.Generator().manual_seed(8), dtype=torch.int32).cuda()
    model.logits(prompt, ex.Batch(c, pages, [0, 0], [25, 15], adapters=[1, 0]))
    batch = ex.Batch(c, pages, [25, 15], [1, 1], adapters=[1, 0])
    token = torch.tensor([5, 9], dtype=torch.int32, device="cuda")
    u = torch.tensor([0.3, 0.8], device="cuda")
    sampling = dict(temperature=torch.ones(2, device="cuda"), top_p=torch.full((2,), 0.9, device="cuda"))
    model.step_with_logprobs(token, batch, u, 4, **sampling)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, report = model.step_with_logprobs(token, batch, u, 4, **sampling)
    for i in range(4):
        nxt = ex.Batch(c, pages, [26 + i, 16 + i], [1, 1], adapters=[i % 2, -1])
        for n in ("positions", "slots", "context_lens", "adapters"):
            getattr(batch, n).copy_(getattr(nxt, n))
        chosen, eager = model.step_with_logprobs(token, batch, u, 4, **sampling)
        chosen, eager = chosen.clone(), [t.clone() for t in eager]
        torch.cuda.synchronize()
        for t in (out, *report):
            t.fill_(-7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, chosen), f"replay {i}"
        assert all(torch.equal(a, b) for a, b in zip(report, eager)), f"replay {i}"
        token.copy_(out)
        u.copy_(torch.rand(2))


def test_log_probabilities_of_the_chosen_tokens():
    ex = example()
    c = ex.Config(cache_bits=8, adapters=1)
    model = ex.Decoder(c, seed=9)
    tokens = torch.randint(0, c.vocab, (9,), generator=torch.Generator().manual_seed(2), dtype=torch.int32).cuda()
    batch = ex.Batch(c, [range(4)], [0], [9], adapters=[0])
    logits = model.logits(tokens, batch)
    chosen, report = model.step_with_logprobs(tokens, batch, torch.zeros(9, device="cuda"), 3,
                                              temperature=torch.zeros(9, device="cuda"))
    assert torch.equal(chosen.long(), logits.argmax(-1))
    assert report[1].tolist() == [0] * 9 and torch.equal(report[3][:, 0], chosen)
    for m in range(9):
        lp, rank, entropy, top, top_lp = _logprobs.reference(_step.f64(logits[m]), int(chosen[m]), 3)
        tol, tol_entropy = _logprobs.bounds(_step.f64(logits[m]), c.vocab)
        assert abs(float(report[0][m]) - lp) <= tol + abs(lp) * 2.0 ** -24
        assert abs(float(report[2][m]) - entropy) <= tol_entropy + entropy * 2.0 ** -24
