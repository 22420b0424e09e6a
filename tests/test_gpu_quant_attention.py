"""qmm_paged_attention_quant against the plain 64-bit form over the numbers that
the codes stand for: head layouts, row counts, pages, lengths, windows, splits of
the length, and everything that lies in places no row sees."""
import numpy as np
import pytest
import torch

from tests import _gpu, _quant, _step
from tests._quant import Problem

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D,G", [(64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (192, 32), (192, 64),
                                 (256, 32), (256, 64), (256, 128)])
@pytest.mark.parametrize("rows,group", [(1, 1), (3, 7), (16, 6)])
def test_head_layouts(dtype, bits, D, G, rows, group):
    Problem([rows, 65, 130], [rows, 1, rows], 2, group, D, 16, dtype, bits, G, seed=D + rows).check()


@pytest.mark.parametrize("page", [1, 8, 16, 17, 32, 48, 100, 256])
@pytest.mark.parametrize("lens", [[1], [31], [32], [33], [0, 1, 2], [63, 64, 65, 257]])
def test_lengths_and_pages(page, lens):
    Problem(lens, [1] * len(lens), 1, 4, 64, page, BF16, 4, 32, seed=page).check()


@pytest.mark.parametrize("bits,D,page", [(8, 96, 17), (4, 96, 16), (8, 128, 5), (4, 256, 33), (8, 256, 128), (4, 192, 1)])
def test_pages_of_wide_heads(bits, D, page):
    Problem([127, 128, 129, 300], [2, 1, 3, 1], 2, 3, D, page, F16, bits, 32, seed=page).check()


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 0), (32, 0), (33, 4), (64, 33), (7, 400), (1000, 4),
                                          ((1 << 31) - 1, 2)])
@pytest.mark.parametrize("rows", [1, 5])
def test_windows_and_sinks(window, sinks, rows):
    Problem([rows, 50, 200, 333], [rows] * 4, 2, 3, 128, 24, F16, 8, 64, seed=window % 97).check(window, sinks)


def test_window_pages_that_are_gone():
    """Pages behind the window may have been given away."""
    p = Problem([300, 290], [2, 1], 2, 4, 64, 16, BF16, 4, 64, seed=5)
    want, _ = p.check(64, 20)
    for b in range(2):
        for i in range(2, 13):  # tokens 32 .. 207: past the sinks, before the window
            pg = int(p.table[b, i])
            p.caches[1][pg] = 0x7E007E00
            p.caches[3][pg] = 0x7C007C00
            p.table[b, i] = [-1, 1 << 30, -(1 << 31)][i % 3]
    got, _ = p.run(64, 20)
    assert torch.equal(got, want)


@pytest.mark.parametrize("D,page,dtype,bits,G", [(128, 16, BF16, 8, 64), (256, 33, F16, 4, 32), (96, 16, BF16, 4, 32)])
@pytest.mark.parametrize("max_context", [0, 700, 5000, 100000])
def test_split_length(D, page, dtype, bits, G, max_context):
    """Many splits; the estimate of the longest context sets their number but not
    what is computed."""
    Problem([2500, 31, 1030], [2, 2, 1], 2, 2, D, page, dtype, bits, G, seed=3).check(max_context=max_context)


def test_many_sequences():
    """More sequences than a wave's lanes, some without rows: runs that hold the
    end of one item and the beginning of the next."""
    g = np.random.default_rng(1)
    lens = g.integers(1, 400, 70).tolist()
    rows = [int(min(n, r)) for n, r in zip(lens, g.integers(0, 4, 70))]
    Problem(lens, rows, 1, 3, 64, 16, F16, 8, 32, seed=4).check(max_context=5000)


def test_rows_that_see_nothing():
    """Length 0, more rows than tokens, a sequence without rows, and pages that
    are all out of range."""
    p = Problem([0, 3, 40, 20], [2, 5, 0, 1], 2, 2, 64, 8, BF16, 8, 32, seed=6)
    p.table[3, :3] = torch.tensor([-1, 1 << 20, -7], dtype=torch.int32)
    out, lse = p.check()
    assert (out[:4] == 0).all() and torch.isinf(lse[:4]).all()
    assert (out[7] == 0).all() and torch.isinf(lse[7]).all()


def test_bad_page_in_the_middle():
    p = Problem([100], [1], 2, 2, 128, 16, F16, 4, 64, seed=8)
    p.table[0, 2] = p.caches[0].shape[0]
    p.check()


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("window", [0, 3])
def test_non_finite_values_reach_only_rows_that_see_them(value, window, bits):
    """A verify row's own group has a bias that is not finite: earlier rows (and
    later ones past a window) do not change, rows that see it follow the formula."""
    p = Problem([40], [6], 2, 3, 64, 16, BF16, bits, 32, seed=9, q_scale=1.0)
    clean, clean_lse = p.check(window)
    pg, off = int(p.table[0, 37 // 16]), 37 % 16  # the token of row 3
    word = int(_quant.pack(np.zeros((1, 32), int), np.array([0.5]), np.array([value]), 8)[1][0])
    p.caches[3][pg, 1, off, 0] = word
    p.caches[3][pg, 0, off, 1] = word
    out, lse = p.run(window)
    sees, rest = [3, 4, 5], [0, 1, 2]
    assert torch.equal(out[rest], clean[rest]) and torch.equal(lse, clean_lse)
    want = clean[sees].float().cpu().clone()
    want[:, :3, 32:] = value
    want[:, 3:, :32] = value
    got = out[sees].float().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    keep = ~torch.isnan(want)
    assert torch.equal(got[keep], want[keep])
    p.caches[1][pg, 0, off] = 0x7E007E00  # a key that is not finite
    out, _ = p.run(window)
    assert torch.equal(out[rest], clean[rest])
    assert torch.isnan(out[sees][:, :3]).all() and not torch.isnan(out[sees][:, 4:, 32:]).any()


def test_infinities_in_fully_visible_tiles():
    """As for 16-bit rows: infinity for the rows that see it, not NaN."""
    p = Problem([700], [2], 1, 2, 128, 16, F16, 8, 64, seed=10, q_scale=1.0)
    clean, lse0 = p.check()
    pg = int(p.table[0, 3])
    p.caches[3][pg, 0, 5, 1] = 0x7C00 << 16 | 0x3800
    out, lse = p.run()
    assert torch.equal(lse, lse0) and torch.equal(out[..., :64], clean[..., :64])
    assert (out[..., 64:] == float("inf")).all()


@pytest.mark.parametrize("bits,D,G,page", [(8, 192, 64, 16), (4, 192, 32, 7), (8, 256, 128, 5), (4, 256, 64, 32), (8, 256, 32, 48),
                                           (4, 96, 32, 16)])
def test_infinities_in_any_group_of_wide_heads(bits, D, G, page):
    """One group of one token each, in every part of the head: infinity there, and
    everywhere else what it was."""
    p = Problem([400], [2], 1, 3, D, page, F16, bits, G, seed=D + bits, q_scale=1.0)
    clean, lse0 = p.check()
    # (the places that hold no token stand for NaN)
    largest = np.nan_to_num(np.abs(_quant.numbers(p.caches[2], p.caches[3], bits, G))).max()
    assert largest < 10
    for group in range(D // G):
        for token in (0, 77 + 37 * group):
            at = (int(p.table[0, token // page]), 0, token % page, group)
            before = int(p.caches[3][at])
            p.caches[3][at] = 0x7C00 << 16 | 0x3800
            out, lse = p.run()
            p.caches[3][at] = before
            rest = torch.ones(D, dtype=torch.bool)
            rest[group * G:(group + 1) * G] = False
            # The token's finite groups are added apart from its tile: at most 400 terms of up to
            # max |v| times a weight, the weights adding up to 1, in another order, 2^-24 of that
            # an addition on either side, then one step of fp16 where that crosses a rounding.
            away = (out[..., rest].double() - clean[..., rest].double()).abs()
            steps = clean[..., rest].double().abs() * 2.0 ** -10 + 2.0 ** -24
            assert torch.equal(lse, lse0) and (away <= 2 * 400 * 2.0 ** -24 * largest + steps).all(), (group, token)
            assert (out[..., ~rest] == float("inf")).all(), (group, token)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_lowest_and_large_scores(dtype):
    """Scores of hundreds: the running maximum moves far, weights underflow."""
    p = Problem([300], [2], 1, 4, 64, 16, dtype, 8, 64, seed=10, q_scale=40.0)
    p.check()
    p.check(scale=-0.5)
    p.check(scale=0.0)


@pytest.mark.parametrize("rows", [1, 24])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -20, 1.0, 2.0 ** 30, 2.0 ** 110])
def test_queries_of_any_size(size, D, rows):
    """bf16 queries past fp16's range on both sides, with a scale that brings the
    scores back, rows of zeros, and rows of other sizes beside them."""
    p = Problem([rows + 40], [rows], 1, 4, D, 16, BF16, 8, 64, seed=11, q_scale=2.0)
    p.q[0, 1] = 0
    q = p.q.double()
    q[:, 2] *= 2.0 ** -10
    p.q = (q * size).to(BF16)
    p.check(scale=D ** -0.5 / size)


def test_queries_that_are_not_finite():
    p = Problem([50], [3], 1, 2, 64, 16, BF16, 8, 64, seed=12)
    clean, _ = p.check()
    p.q[1, 0, 5] = float("nan")
    p.q[2, 1, 6] = float("inf")
    out, _ = p.run()
    assert torch.isnan(out[1, 0]).all() and torch.equal(out[0], clean[0]) and torch.equal(out[1, 1], clean[1, 1])
    assert torch.isnan(out[2, 1]).all() and torch.equal(out[2, 0], clean[2, 0])


def test_strided_queries_and_unheld_rows():
    p = Problem([70, 33], [3, 2], 2, 2, 128, 16, BF16, 4, 32, seed=11)
    want, want_lse = p.check()
    dev = _gpu.dev()
    wide = torch.full((5, 4 * 128 + 64), float("nan"), dtype=BF16, device=dev)
    view = wide[:, 32:32 + 512].unflatten(1, (4, 128))
    view.copy_(p.q.to(dev))
    got, lse = p.run(q=view)
    assert torch.equal(got, want) and torch.equal(lse, want_lse)
    more = torch.cat((p.q, p.q[:2])).to(dev)  # two rows that no sequence holds
    got, lse = p.run(q=more)
    assert torch.equal(got[:5], want) and torch.isnan(got[5:]).all() and torch.isnan(lse[5:]).all()


@pytest.mark.parametrize("bits", [8, 4])
def test_many_rows_and_reruns(bits):
    """A prompt's rows (many column chunks); reruns are bitwise equal, on another
    stream too."""
    p = Problem([150, 77], [150, 40], 1, 4, 64, 16, F16, bits, 32, seed=13)
    want, _ = p.check()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        again, _ = p.run()
    side.synchronize()
    assert torch.equal(again, want)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_equals_attention_over_rows_read_back(D, bits):
    """The same numbers read back to an fp16 cache give the same output, up to its
    rounding and the order of the sums."""
    p = Problem([200, 900], [2, 3], 2, 4, D, 16, F16, bits, 32, seed=14)
    got, lse = p.run()
    dev, qmm = _gpu.dev(), _gpu.lib()
    pages, Hkv, ps, _ = p.caches[0].shape
    slots = torch.arange(pages * ps, dtype=torch.int32, device=dev)
    k, v = (t.reshape(pages, ps, Hkv, D).transpose(1, 2).contiguous() for t in
            qmm.qmm_quant_cache_read(*(t.to(dev) for t in p.caches), bits, 32, slots))
    lse2 = torch.empty_like(lse)
    want = qmm.qmm_paged_attention(p.q.to(dev), k, v, p.table.to(dev), torch.tensor(p.lens, dtype=torch.int32, device=dev),
                                   p.starts.to(dev), 3, 900, lse=lse2)
    # Both outputs are rounded (2^-11 each), and the weights here are single fp16 numbers (2^-11 of a
    # weighted mean of magnitudes, which is below the largest); 2^-18 for the sums' order.
    tol = want.float().abs() * 2.0 ** -10 + 2.0 ** -11 * v.nan_to_num().abs().max().item() + 2.0 ** -18
    off = (got.float() - want.float()).abs()
    assert bool((off <= tol).all()), float((off / tol).max())
    assert float((lse - lse2).abs().max()) <= 2.0 ** -18


@pytest.mark.parametrize("ctx", [90, 4000])
def test_graph_replays(ctx):
    """Captured with and without splits; every replay equals the eager call, and a
    replay follows lengths changed in place."""
    qmm, dev = _gpu.lib(), _gpu.dev()
    p = Problem([ctx, ctx // 2], [2, 1], 2, 3, 128, 16, BF16, 8, 64, seed=15)
    q, table, starts = (t.to(dev) for t in (p.q, p.table, p.starts))
    cs = [t.to(dev) for t in p.caches]
    lens = torch.tensor(p.lens, dtype=torch.int32, device=dev)
    need = qmm.qmm_paged_attention_quant_workspace_bytes(3, 2, 6, 2, 128, 2, ctx, 0, 0, 8, 64)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    out = torch.empty_like(q)

    def call():
        qmm.qmm_paged_attention_quant(q, *cs, 8, 64, table, lens, starts, 2, ctx, out=out, workspace=ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for rep in range(4):
        lens.copy_(torch.tensor([ctx - 3 * rep, ctx // 2 - rep], dtype=torch.int32))
        call()
        torch.cuda.synchronize()
        eager = out.clone()
        out.fill_(float("nan"))
        ws.random_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), f"replay {rep}"


def test_offsets_past_32_bits():
    """Pages whose byte offsets pass 2^32, 4-bit codes."""
    dev, qmm = _gpu.dev(), _gpu.lib()
    pages, Hkv, ps, D = 6 * 4096, 8, 256, 256
    big = [torch.zeros(pages, Hkv, ps, D // 8 if i % 2 == 0 else D // 32, dtype=torch.int32, device=dev) for i in range(4)]
    assert big[0].numel() * 4 > 1 << 32
    p = Problem([600], [1], Hkv, 2, D, ps, BF16, 4, 32, seed=16)
    want, _ = p.run()
    far = [pages - 1, pages - 4000, 1]
    for i, pg in enumerate(far):
        for b, c in zip(big, p.caches):
            b[pg] = c[int(p.table[0, i])].to(dev)
    starts, lens = (torch.tensor(x, dtype=torch.int32, device=dev) for x in ([0, 1], [600]))
    got = qmm.qmm_paged_attention_quant(p.q.to(dev), *big, 4, 32, torch.tensor([far], dtype=torch.int32, device=dev), lens,
                                        starts, 1, 600)
    assert torch.equal(got, want) and got.abs().sum() > 0
