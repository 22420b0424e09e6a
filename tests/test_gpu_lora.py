"""qmm_lora against the plain 64-bit form: ranks, sizes, rows of many adapters in
any order, rows without one, fused projections, and values that are not finite."""
import numpy as np
import pytest
import torch

from tests import _gpu, _step

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


class Problem:
    def __init__(self, M, K, Ns, r, adapters, dtype, ids=None, seed=0, scaled=True):
        g = torch.Generator().manual_seed(seed)
        self.x = torch.randn(M, K, generator=g).to(dtype)
        self.pairs = [((torch.randn(adapters, r, K, generator=g) * K ** -0.5).to(dtype),
                       (torch.randn(adapters, n, r, generator=g) * r ** -0.5).to(dtype)) for n in Ns]
        self.ids = torch.randint(-1, adapters, (M,), generator=g) if ids is None else torch.tensor(ids)
        self.ids = self.ids.to(torch.int32)
        self.scales = torch.rand(adapters, generator=g) + 0.5 if scaled else None
        self.ys = [torch.randn(M, n, generator=g) for n in Ns]

    def run(self, **kw):
        dev = _gpu.dev()
        ys = [y.to(dev) for y in self.ys]
        got = _gpu.lib().qmm_lora(self.x.to(dev), [(a.to(dev), b.to(dev)) for a, b in self.pairs], self.ids.to(dev), ys,
                                  scales=None if self.scales is None else self.scales.to(dev), **kw)
        torch.cuda.synchronize()
        assert got is ys
        return ys

    def reference(self):
        """[(y, bound)] in 64 bits. The first product: K roundings of 2^-24 of the sum of its
        magnitudes, a few more for the parts; the split: 2^-22 of h and 2^-39 of the row's
        largest; the second: r roundings; three of y's or the result's size."""
        out = []
        x, ids = _step.f64(self.x), self.ids.tolist()
        K = x.shape[1]
        for y0, (a, b) in zip(self.ys, self.pairs):
            a, b, y = _step.f64(a), _step.f64(b), _step.f64(y0)
            r = a.shape[1]
            bound = np.zeros_like(y)
            for m, i in enumerate(ids):
                if not 0 <= i < a.shape[0]:
                    continue
                s = 1.0 if self.scales is None else float(self.scales[i])
                h = s * (a[i] @ x[m])
                eh = (K + 8) * 2.0 ** -24 * abs(s) * (np.abs(a[i]) @ np.abs(x[m])) + np.abs(h) * 2.0 ** -22
                eh += 2.0 ** -39 * np.abs(h).max()
                d = b[i] @ h
                mag = np.abs(b[i]) @ np.abs(h)
                bound[m] = np.abs(b[i]) @ eh + mag * (3 * r + 4) * 2.0 ** -24 + 2 * (np.abs(y[m]) + np.abs(d)) * 2.0 ** -24
                y[m] += d
            out.append((y, bound))
        return out

    def check(self, **kw):
        got = self.run(**kw)
        for g, y0, (want, bound) in zip(got, self.ys, self.reference()):
            g = _step.f64(g)
            assert (np.abs(g - want) <= bound).all(), np.max(np.abs(g - want) / np.maximum(bound, 1e-30))
            n = len(self.pairs[0][0])
            off = [m for m, i in enumerate(self.ids.tolist()) if not 0 <= i < n]
            assert np.array_equal(g[off], _step.f64(y0)[off])
        return got


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("M", [1, 5, 33])
def test_ranks(dtype, r, M):
    Problem(M, 512, [100], r, 4, dtype, seed=r + M).check()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("K", [32, 64, 96, 256, 288, 1024, 1056, 2080, 5120])
@pytest.mark.parametrize("N", [1, 3, 16, 63, 64, 65, 257, 1000])
def test_sizes(dtype, K, N):
    Problem(18, K, [N], 16, 3, dtype, seed=K + N).check()


@pytest.mark.parametrize("M,adapters,ids", [
    (16, 16, list(range(16))), (17, 40, [(7 * i) % 40 for i in range(17)]), (1, 1, [0]), (1, 5, [4]), (3, 2, [-1, -1, -1]),
    (40, 3, [0] * 13 + [2] * 20 + [-1] * 3 + [1] * 4), (35, 2, [i % 2 for i in range(35)]),
    (20, 4, [3, -7, 4, 1 << 30, -(1 << 31), 3, 0, 99] * 2 + [0, 1, 2, 3]), (64, 64, list(range(63, -1, -1)))])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_rows_of_adapters(dtype, M, adapters, ids):
    Problem(M, 320, [130, 64], 16, adapters, dtype, ids=ids, seed=M).check()


@pytest.mark.parametrize("Ns", [[192, 32, 32], [33, 300, 1, 257], [64, 63]])
def test_fused_projections(Ns):
    p = Problem(21, 640, Ns, 32, 5, F16, seed=1)
    got = p.check()
    for i, n in enumerate(Ns):  # each equal to a call of its own up to how K is cut
        one = Problem(21, 640, [n], 32, 5, F16)
        one.x, one.ids, one.scales, one.pairs, one.ys = p.x, p.ids, p.scales, [p.pairs[i]], [p.ys[i]]
        (y,), ((_, bound),) = one.run(), one.reference()
        assert (np.abs(_step.f64(y) - _step.f64(got[i])) <= 2 * bound).all()


@pytest.mark.parametrize("M,run", [(700, 1), (700, 90), (2100, 2100)])
def test_many_rows(M, run):
    """Workgroups that take several adapters of a block, and prompts."""
    p = Problem(M, 256, [96], 16, 9, BF16, ids=[(i // run) % 10 - (i // run) % 11 // 10 for i in range(M)], seed=2)
    p.check()


def test_without_scales_and_tiny_or_large_values():
    Problem(20, 256, [50], 8, 3, F16, scaled=False).check()
    for size in (1e-4, 300.0):
        p = Problem(20, 256, [50], 24, 3, F16, seed=3)
        p.x = (p.x * size).half()
        p.check()
    p = Problem(20, 256, [50], 16, 3, BF16, seed=4)
    p.x = (p.x.double() * 2.0 ** 60).to(BF16)
    p.pairs = [(a, (b.double() * 2.0 ** -60).to(BF16)) for a, b in p.pairs]
    p.check()
    p = Problem(20, 512, [50], 16, 3, F16, seed=5)  # A x past fp16's largest
    p.x = torch.full_like(p.x, 60000.0)
    p.pairs = [(torch.full_like(a, 2.0), b) for a, b in p.pairs]
    p.check()


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_non_finite_values_stay_in_their_rows(dtype):
    p = Problem(20, 256, [70], 16, 3, dtype, ids=[0, 1, 2, -1] * 5, seed=6)
    clean = p.check()[0]
    p.x[4, 7] = float("nan")
    p.x[6, 3] = float("inf")
    p.x[7, 3] = float("inf")        # a row without an adapter
    p.pairs[0][0][1, 2, 5] = float("nan")
    p.pairs[0][1][1, 33, 4] = float("inf")
    got = p.run()[0]
    ids = p.ids.numpy()
    plain = [m for m in range(20) if ids[m] != 1 and m not in (4, 6)]
    assert torch.equal(got[plain], clean[plain])
    assert torch.isnan(got[4]).all() and torch.isnan(got[[m for m in range(20) if ids[m] == 1]]).all()
    assert not torch.isfinite(got[6]).any()


def test_infinite_results():
    """h of +infinity times rows of B of one sign: infinities, not NaN."""
    p = Problem(3, 64, [20], 8, 1, F16, ids=[0, 0, 0], seed=7)
    p.pairs[0][0][:] = p.pairs[0][0].abs() + 0.1
    p.pairs[0][1][:] = p.pairs[0][1].abs() + 0.1
    p.x[:] = p.x.abs()
    p.x[1, 9] = float("inf")
    got = p.run()[0]
    assert (got[1] == float("inf")).all() and torch.isfinite(got[[0, 2]]).all()


def test_reruns_streams_workspace():
    qmm, dev = _gpu.lib(), _gpu.dev()
    p = Problem(50, 2048, [300, 20], 16, 6, F16, seed=8)
    want = p.check()
    need = qmm.qmm_lora_workspace_bytes([300, 20], 50, 2048, 16, 6)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=dev)  # NaN in every place
    got = p.run(workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = p.run()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(qmm.QmmError):
        p.run(workspace=ws[:need - 16])


def test_refusals_on_the_gpu():
    qmm, dev = _gpu.lib(), _gpu.dev()
    p = Problem(4, 64, [20], 8, 2, F16)
    x, (a, b), ids, y = p.x.to(dev), (t.to(dev) for t in p.pairs[0]), p.ids.to(dev), p.ys[0].to(dev)
    for bad, kind in (([(a, b[:, :, :4])], ValueError), ([(a.bfloat16(), b)], TypeError), ([(a, b)] * 2, ValueError),
                      ([(a, b, b)], TypeError), ([], ValueError), ([a], TypeError)):
        with pytest.raises(kind):
            qmm.qmm_lora(x, bad, ids, [y])
    with pytest.raises(ValueError):
        qmm.qmm_lora(x, [(a, b)], ids, [y[:, :19]])
    with pytest.raises(TypeError):
        qmm.qmm_lora(x, [(a, b)], ids.long(), [y])
    with pytest.raises(qmm.QmmError):
        qmm.qmm_lora(x, [(a[:, :4].contiguous(), b[:, :, :4].contiguous())], ids, [y])


def test_graph_replays():
    """Replays follow ids and x changed in place, and add to y as it is."""
    qmm, dev = _gpu.lib(), _gpu.dev()
    p = Problem(30, 1024, [200, 64], 16, 5, F16, seed=9)
    x, ids, scales = p.x.to(dev), p.ids.to(dev), p.scales.to(dev)
    pairs = [(a.to(dev), b.to(dev)) for a, b in p.pairs]
    ys = [y.to(dev) for y in p.ys]
    ws = torch.empty(qmm.qmm_lora_workspace_bytes([200, 64], 30, 1024, 16, 5), dtype=torch.uint8, device=dev)
    qmm.qmm_lora(x, pairs, ids, ys, scales=scales, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qmm.qmm_lora(x, pairs, ids, ys, scales=scales, workspace=ws)
    for rep in range(4):
        x.copy_(torch.randn(30, 1024, generator=torch.Generator().manual_seed(rep)).half())
        ids.copy_(torch.randint(-1, 5, (30,), generator=torch.Generator().manual_seed(rep)).to(torch.int32))
        for y, y0 in zip(ys, p.ys):
            y.copy_(y0)
        eager = [y.clone() for y in ys]
        qmm.qmm_lora(x, pairs, ids, eager, scales=scales)
        ws.random_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ys, eager)), f"replay {rep}"


def test_offsets_past_32_bits():
    """Adapters and y past 2^32 bytes."""
    qmm, dev = _gpu.lib(), _gpu.dev()
    n, r, K, N = 700, 128, 16384, 16384
    a = torch.zeros(n, r, K, dtype=F16, device=dev)
    b = torch.zeros(n, N, r, dtype=F16, device=dev)
    assert a.numel() * 2 > 1 << 31 and b.numel() * 2 > 1 << 31
    p = Problem(3, K, [N], r, 1, F16, ids=[0, 0, -1], scaled=False, seed=10)
    (want,) = p.check()
    a[n - 1], b[n - 1] = p.pairs[0][0][0].to(dev), p.pairs[0][1][0].to(dev)
    M = 70000
    x = torch.zeros(M, K, dtype=F16, device=dev)
    x[-3:] = p.x.to(dev)
    y = torch.zeros(M, N, device=dev)
    assert y.numel() * 4 > 1 << 32 and x.numel() * 2 > 1 << 31
    y[-3:] = p.ys[0].to(dev)
    ids = torch.full((M,), -1, dtype=torch.int32, device=dev)
    ids[-3:-1] = n - 1
    qmm.qmm_lora(x, [(a, b)], ids, [y])
    ((_, bound),) = p.reference()
    assert (np.abs(_step.f64(y[-3:]) - _step.f64(want)) <= 2 * bound).all() and not y[:-3].any()
