"""qmm_paged_attention against the plain 64-bit form: head layouts, row counts,
page sizes and lengths around the tile of 32 tokens, windows with sinks, splits
of the length, and everything that lies in places no row sees."""
import numpy as np
import pytest
import torch

from tests import _gpu, _step

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


class Problem:
    """Sequences of given lengths and row counts over a shuffled pool. Every
    place of the cache that holds no token is NaN, and table entries past a
    sequence's pages are out of range."""

    def __init__(self, lens, rows, Hkv, G, D, page, dtype, seed=0, q_scale=2.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.rows = lens, rows
        need = [-(-L // page) for L in lens]
        total = sum(need) + 2
        perm = torch.randperm(total, generator=g).tolist()
        width = max(1, max(need) + 1)
        self.table = torch.full((len(lens), width), -1, dtype=torch.int32)
        self.table[:, -1] = total + 5
        kc = torch.full((total, Hkv, page, D), float("nan"), dtype=dtype)
        vc = kc.clone()
        for b, L in enumerate(lens):
            for i in range(need[b]):
                pg = perm.pop()
                self.table[b, i] = pg
                n = min(page, L - i * page)
                kc[pg, :, :n] = torch.randn(Hkv, n, D, generator=g).to(dtype)
                vc[pg, :, :n] = torch.randn(Hkv, n, D, generator=g).to(dtype)
        self.starts = torch.tensor([0] + list(np.cumsum(rows)), dtype=torch.int32)
        T = int(self.starts[-1])
        self.q = (torch.randn(T, Hkv * G, D, generator=g) * q_scale).to(dtype)
        self.kc, self.vc, self.dtype, self.D = kc, vc, dtype, D

    def run(self, window=0, sinks=0, scale=None, max_context=None, max_rows=None, q=None):
        qmm, dev = _gpu.lib(), _gpu.dev()
        q = self.q.to(dev) if q is None else q
        T, Hq, _ = q.shape
        out = torch.full((T, Hq, self.D), float("nan"), dtype=self.dtype, device=dev)
        lse = torch.full((T, Hq), float("nan"), device=dev)
        qmm.qmm_paged_attention(q, self.kc.to(dev), self.vc.to(dev), self.table.to(dev),
                                torch.tensor(self.lens, dtype=torch.int32, device=dev), self.starts.to(dev),
                                max_rows or max(1, max(self.rows)),
                                max(self.lens) if max_context is None else max_context, scale=scale, window=window,
                                sinks=sinks, out=out, lse=lse)
        torch.cuda.synchronize()
        return out, lse

    def check(self, window=0, sinks=0, scale=None, **kw):
        out, lse = self.run(window, sinks, scale, **kw)
        (ro, ob), (rl, lb), held = _step.attention_reference(
            _step.f64(self.q), _step.f64(self.kc), _step.f64(self.vc), self.table.numpy(), self.lens,
            self.starts.tolist(), self.D ** -0.5 if scale is None else scale, window, sinks, self.dtype)
        assert held.all()
        _step.assert_rounded(out, ro, ob, "out")
        _step.assert_rounded(lse, rl, lb, "lse")
        return out, lse


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("rows,G", [(1, 1), (1, 6), (3, 7), (16, 6)])
def test_head_layouts(dtype, D, rows, G):
    Problem([rows, 65, 130], [rows, 1, rows], 2, G, D, 16, dtype, seed=D + rows).check()


@pytest.mark.parametrize("page", [1, 8, 16, 17, 32, 48, 100, 256])
@pytest.mark.parametrize("lens", [[1], [31], [32], [33], [0, 1, 2], [63, 64, 65, 257]])
def test_lengths_and_pages(page, lens):
    Problem(lens, [1] * len(lens), 1, 4, 64, page, BF16, seed=page).check()


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 0), (32, 0), (33, 4), (40, 1), (64, 33), (7, 400), (1000, 4),
                                          ((1 << 31) - 1, 2)])
@pytest.mark.parametrize("rows", [1, 5])
def test_windows_and_sinks(window, sinks, rows):
    Problem([rows, 50, 200, 333], [rows] * 4, 2, 3, 128, 24, F16, seed=window % 97).check(window, sinks)


def test_window_pages_that_are_gone():
    """Pages behind the window may have been given away: their table entries are
    anything, their contents NaN."""
    p = Problem([300, 290], [2, 1], 2, 4, 64, 16, BF16, seed=5)
    want, _ = p.check(64, 20)
    for b in range(2):
        for i in range(2, 13):  # tokens 32 .. 207: past the sinks, before the window
            pg = int(p.table[b, i])
            p.kc[pg] = float("nan")
            p.vc[pg] = float("inf")
            p.table[b, i] = [-1, 1 << 30, -(1 << 31)][i % 3]
    got, _ = p.run(64, 20)
    assert torch.equal(got, want)


@pytest.mark.parametrize("D,page,dtype", [(128, 16, BF16), (256, 33, F16)])
@pytest.mark.parametrize("max_context", [0, 700, 5000, 100000])
def test_split_length(D, page, dtype, max_context):
    """Many splits; the estimate of the longest context sets their number but
    not what is computed."""
    p = Problem([2500, 31, 1030], [2, 2, 1], 2, 2, D, page, dtype, seed=3)
    p.check(max_context=max_context)


def test_window_split():
    Problem([3000, 900], [4, 1], 1, 2, 64, 16, BF16, seed=4).check(1500, 4)


def test_rows_that_see_nothing():
    """Length 0, more rows than tokens, a sequence without rows, and pages that
    are all out of range."""
    p = Problem([0, 3, 40, 20], [2, 5, 0, 1], 2, 2, 64, 8, BF16, seed=6)
    p.table[3, :3] = torch.tensor([-1, 1 << 20, -7], dtype=torch.int32)
    out, lse = p.check()
    assert (out[:4] == 0).all() and torch.isinf(lse[:4]).all()
    assert (out[7] == 0).all() and torch.isinf(lse[7]).all()


def test_bad_page_in_the_middle():
    p = Problem([100], [1], 2, 2, 128, 16, F16, seed=8)
    p.table[0, 2] = p.kc.shape[0]
    p.check()


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("window", [0, 3])
def test_non_finite_values_reach_only_rows_that_see_them(value, window):
    """A verify row's own value is not finite: earlier rows (and later ones past
    a window) do not change, rows that see it follow the formula."""
    p = Problem([40], [6], 2, 3, 64, 16, BF16, seed=9, q_scale=1.0)
    clean, clean_lse = p.check(window)
    pg, off = int(p.table[0, 37 // 16]), 37 % 16  # the token of row 3
    p.vc[pg, 1, off, 5] = value
    p.vc[pg, 0, off, 63] = value
    out, lse = p.run(window)
    sees = [3, 4, 5]
    rest = [0, 1, 2]
    assert torch.equal(out[rest], clean[rest]) and torch.equal(lse, clean_lse)
    got = out[sees].float().cpu()
    want = clean[sees].float().cpu().clone()
    want[:, :3, 63] = value
    want[:, 3:, 5] = value
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    keep = ~torch.isnan(want)
    assert torch.equal(got[keep], want[keep])
    # a key that is not finite
    p.kc[pg, 0, off] = float("nan")
    out, _ = p.run(window)
    assert torch.equal(out[rest], clean[rest])
    assert torch.isnan(out[sees][:, :3]).all() and not torch.isnan(out[sees][:, 4:, :5]).any()


def test_lowest_and_large_scores():
    """Scores of hundreds: the running maximum moves far, weights underflow."""
    p = Problem([300], [2], 1, 4, 64, 16, F16, seed=10, q_scale=40.0)
    p.check()
    p.check(scale=-0.5)
    p.check(scale=0.0)


def test_strided_queries_and_unheld_rows():
    """Queries as a view of wider rows; rows of q outside row_starts stay."""
    p = Problem([70, 33], [3, 2], 2, 2, 128, 16, BF16, seed=11)
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


def test_unsound_row_starts_compute_nothing():
    p = Problem([70, 33], [3, 2], 2, 2, 64, 16, BF16, seed=12)
    for starts in ([0, 3, 9], [4, 2, 1], [-3, -1, 0]):
        p.starts = torch.tensor(starts, dtype=torch.int32)
        out, _ = p.run()
        if starts[2] == 9:
            assert torch.isnan(out[3:]).all()
        else:
            assert torch.isnan(out).all()


def test_many_rows_and_reruns():
    """A prompt's rows (many column chunks); reruns are bitwise equal, on
    another stream too."""
    p = Problem([150, 77], [150, 40], 1, 4, 64, 16, F16, seed=13)
    want, _ = p.check()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        again, _ = p.run()
    side.synchronize()
    assert torch.equal(again, want)


def test_offsets_past_32_bits():
    """Pages whose byte offsets pass 2^32 (a 6 GiB cache)."""
    dev, qmm = _gpu.dev(), _gpu.lib()
    pages, Hkv, ps, D = 6 * 4096, 8, 64, 256
    shape = (pages, Hkv, ps, D)
    kc = torch.zeros(shape, dtype=BF16, device=dev)
    vc = torch.zeros(shape, dtype=BF16, device=dev)
    assert kc.numel() * 2 > 1 << 32
    g = torch.Generator().manual_seed(14)
    small_k = torch.randn(3, Hkv, ps, D, generator=g).to(BF16)
    small_v = torch.randn(3, Hkv, ps, D, generator=g).to(BF16)
    far = [pages - 1, pages - 4000, 1]
    for i, pg in enumerate(far):
        kc[pg], vc[pg] = small_k[i].to(dev), small_v[i].to(dev)
    q = torch.randn(1, 16, D, generator=g).to(BF16).to(dev)
    starts, lens = (torch.tensor(x, dtype=torch.int32, device=dev) for x in ([0, 1], [150]))
    got = qmm.qmm_paged_attention(q, kc, vc, torch.tensor([far], dtype=torch.int32, device=dev), lens, starts, 1, 150)
    want = qmm.qmm_paged_attention(q, small_k.to(dev), small_v.to(dev),
                                   torch.tensor([[0, 1, 2]], dtype=torch.int32, device=dev), lens, starts, 1, 150)
    assert torch.equal(got, want) and got.abs().sum() > 0


@pytest.mark.parametrize("ctx", [90, 4000])
def test_graph_replays(ctx):
    """Captured with and without splits; every replay equals the eager call, and
    a replay follows lengths changed in place."""
    qmm, dev = _gpu.lib(), _gpu.dev()
    p = Problem([ctx, ctx // 2], [2, 1], 2, 3, 128, 16, BF16, seed=15)
    q, kc, vc, table, starts = (t.to(dev) for t in (p.q, p.kc, p.vc, p.table, p.starts))
    lens = torch.tensor(p.lens, dtype=torch.int32, device=dev)
    need = qmm.qmm_paged_attention_workspace_bytes(3, 2, 6, 2, 128, 2, ctx)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    out = torch.empty_like(q)

    def call():
        qmm.qmm_paged_attention(q, kc, vc, table, lens, starts, 2, ctx, out=out, workspace=ws)
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
