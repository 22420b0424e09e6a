"""qmm_qk_norm_rope_quant and qmm_quant_cache_read against the plain 64-bit form:
values, which no arithmetic precedes, to the bit; keys within half a step."""
import numpy as np
import pytest
import torch

from tests import _gpu, _quant, _step
from tests.test_gpu_qk_norm_rope import problem

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def caches(p, bits, G, fill=0x2C00):
    """Four tensors over the problem's pool; scales and biases of 2^-4 where nothing is written."""
    pool, Hkv, page, D = p["k_cache"].shape
    words = torch.full((pool, Hkv, page, D * bits // 32), 0x35A1C7E2, dtype=torch.int32)
    sb = torch.full((pool, Hkv, page, D // G), fill | fill << 16, dtype=torch.int32)
    return [t.clone().to(_gpu.dev()) for t in (words, sb, words, sb)]


def run(p, bits, G, cs=None, **kw):
    qmm, dev = _gpu.lib(), _gpu.dev()
    d = {n: t.to(dev) for n, t in p.items()}
    cs = caches(p, bits, G) if cs is None else cs
    out = qmm.qmm_qk_norm_rope_quant(d["q"], d["k"], d["v"], d["q_weight"], d["k_weight"], d["positions"], d["inv_freq"],
                                     d["slots"], *cs, bits, G, **kw)
    torch.cuda.synchronize()
    return out, cs


def check(p, bits, G, dtype=BF16, eps=1e-6, weight_offset=0.0, interleaved=False):
    out, cs = run(p, bits, G, dtype=dtype, eps=eps, weight_offset=weight_offset, interleaved=interleaved)
    before = caches(p, bits, G)
    (qo, qb), (kr, kb), (vr, _) = _step.rope_reference(
        *(_step.f64(p[n]) for n in ("q", "k", "v", "q_weight", "k_weight")), p["positions"].numpy(),
        p["inv_freq"].double().numpy(), p["slots"].numpy(), np.full(p["k_cache"].shape, np.nan),
        np.full(p["v_cache"].shape, np.nan), eps, weight_offset, interleaved)
    _step.assert_rounded(out, qo, qb, "q")
    pool, Hkv, page, D = p["k_cache"].shape
    wrote = np.zeros((pool, page), bool)
    for s in p["slots"].tolist():
        if 0 <= s < pool * page:
            wrote[s // page, s % page] = True
    at = np.broadcast_to(wrote[:, None, :], (pool, Hkv, page))
    for new, old in zip(cs, before):  # other places are as they were
        assert torch.equal(new.cpu()[torch.from_numpy(~at)], old.cpu()[torch.from_numpy(~at)])
    # values: the format's words to the bit; codes but for places within 2^-13 of a border (documented: 2^-14)
    y = vr[at]
    codes, s, b, place = _quant.quantize(y, bits, G)
    gc, gs, gb = (x[at] for x in _quant.unpack(cs[2], cs[3], bits, G))
    assert np.array_equal(gs, s, equal_nan=True) and np.array_equal(gb, b)
    border = np.abs(place - np.floor(place) - 0.5) < 2.0 ** -13
    assert ((gc == codes) | border).all() and (np.abs(gc.astype(int) - codes) <= 1).all()
    # keys: within half a step of the 64-bit value, 32-bit arithmetic and the number's rounding added
    k = _quant.numbers(cs[0], cs[1], bits, G)[at]
    _, ks, _ = (x[at] for x in _quant.unpack(cs[0], cs[1], bits, G))
    y, bound = kr[at], kb[at]
    fine = np.isfinite(y)
    y = np.clip(y, -_quant.MOST, _quant.MOST)
    step = np.repeat(ks, G, -1)
    tol = step * (0.5 + 2.0 ** -13) + bound + np.maximum(np.abs(k) * 2.0 ** -11, 2.0 ** -25)
    assert (np.abs(k - y) <= tol)[fine].all()
    # and no coarser than the range asks: a step past (max - min) / levels by 2^-10 of it, the bias's
    # rounding (2^-10 of the minimum, 2^-24 at least) and the arithmetic
    levels = 2 ** bits - 1
    g, gbnd = y.reshape(*y.shape[:-1], -1, G), bound.reshape(*y.shape[:-1], -1, G)
    widest = (g.max(-1) - g.min(-1) + 2 * gbnd.max(-1) + np.abs(g.min(-1)) * 2.0 ** -10 + 2.0 ** -24) / levels
    ok = np.isfinite(g).all(-1)
    assert (ks <= widest * (1 + 2.0 ** -10) + 2.0 ** -24)[ok].all()
    return out, cs


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D,R,G", [(32, 32, 32), (64, 64, 64), (64, 16, 32), (96, 96, 32), (128, 128, 128), (128, 64, 64),
                                   (160, 32, 32), (192, 64, 64), (256, 64, 64), (256, 256, 128), (256, 0, 32)])
def test_heads_and_groups(D, R, G, bits, interleaved):
    check(problem(5, 3, 2, D, R, F32, F16, 16, seed=D + R), bits, G, interleaved=interleaved)


@pytest.mark.parametrize("din,dtype", [(F32, F16), (BF16, BF16), (F16, F16), (BF16, F16), (F16, BF16)])
def test_types(din, dtype):
    check(problem(6, 4, 2, 128, 64, din, F16, 16, seed=1), 8, 32, dtype=dtype)


@pytest.mark.parametrize("M,Hq,Hkv,page", [(1, 24, 4, 16), (1, 1, 1, 1), (2, 48, 8, 17), (37, 7, 1, 100), (600, 3, 1, 32)])
def test_rows_and_pages(M, Hq, Hkv, page):
    check(problem(M, Hq, Hkv, 64, 32, F32, F16, page, seed=M), 4, 64, weight_offset=1.0, eps=1e-5)


def test_padding_and_slots_past_the_cache():
    p = problem(9, 2, 2, 64, 64, F32, F16, 5, seed=2)
    total = p["k_cache"].shape[0] * 5
    p["slots"][[1, 4, 6, 8]] = torch.tensor([-1, total, (1 << 31) - 1, -(1 << 31)], dtype=torch.int32)
    check(p, 8, 32)


@pytest.mark.parametrize("bits", [4, 8])
def test_ranges(bits):
    """Groups of zeros, of one value, without spread around a number, tiny, large,
    past the largest, and of one sign."""
    p = problem(12, 1, 1, 64, 0, F32, F16, 16, seed=3)
    v = p["v"]
    v[0] = 0
    v[1] = 0.3
    v[2] = 7.0 + torch.arange(64) * 2.0 ** -20
    v[3] *= 1e-8
    v[4] *= 1e-30
    v[5] *= 5e4
    v[6] = v[6] * 1e30
    v[7, :, 3], v[7, :, 40] = float("inf"), float("-inf")
    v[8] = v[8].abs() + 1
    v[9] = -v[9].abs() - 100
    v[10] = -2.0 ** -26
    v[11, :, ::2], v[11, :, 1::2] = 65280.0, -65280.0
    _, cs = check(p, bits, 32)
    assert np.isfinite(_quant.numbers(cs[2], cs[3], bits, 32)).all()


def test_nan_stays_in_its_group():
    p = problem(3, 2, 2, 64, 32, F32, F16, 16, seed=4)
    _, clean = check(p, 8, 32)
    p["v"][1, 0, 40] = float("nan")
    p["k"][2, 1, 3] = float("nan")  # a key's norm carries it through its head
    _, cs = run(p, 8, 32, dtype=F16)
    values = [_quant.numbers(cs[i], cs[i + 1], 8, 32) for i in (0, 2)]
    before = [_quant.numbers(clean[i], clean[i + 1], 8, 32) for i in (0, 2)]
    s = p["slots"].tolist()
    assert np.isnan(values[1][s[1] // 16, 0, s[1] % 16, 32:]).all()
    before[1][s[1] // 16, 0, s[1] % 16, 32:] = np.nan
    assert np.isnan(values[0][s[2] // 16, 1, s[2] % 16]).all()
    before[0][s[2] // 16, 1, s[2] % 16] = np.nan
    for a, b in zip(values, before):
        assert np.array_equal(a, b, equal_nan=True)


def test_views_of_a_fused_projection():
    p = problem(7, 4, 2, 64, 64, F32, F16, 16, seed=6)
    want, cs = check(p, 4, 32)
    fused = torch.full((7, 8 * 64 + 16), float("nan"), device=_gpu.dev())
    at, views = 8, {}
    for n, h in (("q", 4), ("k", 2), ("v", 2)):
        fused[:, at:at + h * 64] = p[n].flatten(1).to(fused)
        views[n] = fused[:, at:at + h * 64].unflatten(1, (h, 64))
        at += h * 64
    out, got = run(dict(p, **views), 4, 32, dtype=BF16)
    assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(got, cs))


@pytest.mark.parametrize("bits,G,D,Hkv,page", [(8, 64, 256, 4, 16), (4, 32, 128, 8, 17), (4, 128, 128, 1, 1), (8, 32, 32, 1, 5),
                                               (4, 32, 96, 3, 16), (8, 64, 192, 5, 7)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_read(bits, G, D, Hkv, page, dtype):
    """Any words, in any order of slots, some twice and some outside: the numbers to the bit."""
    g = np.random.default_rng(D + page)
    pages = 9
    words = [torch.from_numpy(g.integers(-2 ** 31, 2 ** 31, (pages, Hkv, page, D * bits // 32), dtype=np.int32)) for _ in range(2)]
    pairs = []
    for _ in range(2):
        s, b = g.standard_normal((2, pages, Hkv, page, D // G)) * np.exp(g.uniform(-12, 5, (pages, Hkv, page, D // G)))
        s[0, 0, 0, 0], b[-1, 0, -1, 0] = np.nan, np.inf
        pairs.append(_quant.pack(np.zeros((1, 32), int), s, b, 8)[1])
    slots = torch.from_numpy(g.integers(-3, pages * page + 3, 41, dtype=np.int32))
    slots[5] = slots[4]
    slots[6], slots[7] = 2 ** 31 - 1, -2 ** 31
    dev = _gpu.dev()
    got = _gpu.lib().qmm_quant_cache_read(*(t.to(dev) for t in (words[0], pairs[0], words[1], pairs[1])), bits, G,
                                          slots.to(dev), dtype=dtype)
    for out, w, p in zip(got, words, pairs):
        values = _quant.numbers(w, p, bits, G)
        want = np.zeros((41, Hkv, D))
        for m, s in enumerate(slots.tolist()):
            if 0 <= s < pages * page:
                want[m] = values[s // page, :, s % page]
        want = torch.from_numpy(want).to(dtype)
        torch.testing.assert_close(out.cpu(), want, rtol=0, atol=0, equal_nan=True)


def test_graph_replays_and_streams():
    qmm, dev = _gpu.lib(), _gpu.dev()
    p = problem(6, 4, 2, 128, 64, F32, F16, 16, seed=7)
    want, cs = check(p, 8, 64)
    d = {n: t.to(dev) for n, t in p.items()}
    k, v = qmm.qmm_quant_cache_read(*cs, 8, 64, d["slots"])
    mine = caches(p, 8, 64)
    out, ko, vo = torch.empty_like(want), torch.empty_like(k), torch.empty_like(v)

    def call():
        qmm.qmm_qk_norm_rope_quant(d["q"], d["k"], d["v"], d["q_weight"], d["k_weight"], d["positions"], d["inv_freq"],
                                   d["slots"], *mine, 8, 64, out=out)
        qmm.qmm_quant_cache_read(*mine, 8, 64, d["slots"], k_out=ko, v_out=vo)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(ko, k) and torch.equal(vo, v)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(4):
        for t in (out, ko, vo):
            t.fill_(float("nan"))
        for t in mine:
            t.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(ko, k) and torch.equal(vo, v)


def test_offsets_past_32_bits():
    """Rows whose byte offsets pass 2^32."""
    dev, qmm = _gpu.dev(), _gpu.lib()
    pages, Hkv, ps, D = 3 * 4096 * 2, 8, 128, 256
    words = [torch.zeros(pages, Hkv, ps, D // 4, dtype=torch.int32, device=dev) for _ in range(2)]
    pairs = [torch.zeros(pages, Hkv, ps, D // 64, dtype=torch.int32, device=dev) for _ in range(2)]
    assert words[0].numel() * 4 > 1 << 32
    p = problem(3, 8, Hkv, D, 64, F32, F16, 128, seed=8)
    d = {n: t.to(dev) for n, t in p.items()}
    d["slots"] = torch.tensor([pages * ps - 1, 5, (pages - 7) * ps + 77], dtype=torch.int32, device=dev)
    qmm.qmm_qk_norm_rope_quant(d["q"], d["k"], d["v"], d["q_weight"], d["k_weight"], d["positions"], d["inv_freq"],
                               d["slots"], words[0], pairs[0], words[1], pairs[1], 8, 64)
    got = qmm.qmm_quant_cache_read(words[0], pairs[0], words[1], pairs[1], 8, 64, d["slots"])
    small = caches(p, 8, 64)
    qmm.qmm_qk_norm_rope_quant(d["q"], d["k"], d["v"], d["q_weight"], d["k_weight"], d["positions"], d["inv_freq"],
                               d["slots"] * 0 + torch.arange(3, dtype=torch.int32, device=dev), *small, 8, 64)
    want = qmm.qmm_quant_cache_read(*small, 8, 64, torch.arange(3, dtype=torch.int32, device=dev))
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and got[0].abs().sum() > 0
