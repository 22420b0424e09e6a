"""qmm_logprobs against the plain 64-bit form: types, sizes around slices and 16
bytes, ties, infinities and NaN, rows that are flat, strides and graphs."""
import numpy as np
import pytest
import torch

from tests import _gpu, _logprobs, _step

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def run(x, tokens, n):
    out = _gpu.lib().qmm_logprobs(x, tokens, n)
    torch.cuda.synchronize()
    return out


def check(x, tokens, n):
    """x [M, V] on the CPU or GPU, maybe strided."""
    dev = _gpu.dev()
    got = run(x.to(dev) if x.device.type == "cpu" else x, torch.as_tensor(tokens, dtype=torch.int32, device=dev), n)
    lp, rank, ent, top, tlp = (t.cpu().numpy() for t in got)
    rows = _step.f64(x)
    for m, row in enumerate(rows):
        r_lp, r_rank, r_ent, r_top, r_tlp = _logprobs.reference(row, int(tokens[m]), n)
        b_lp, b_ent = _logprobs.bounds(np.where(np.isnan(row), -np.inf, row), len(row))
        assert rank[m] == r_rank, (m, rank[m], r_rank)
        assert np.array_equal(top[m], r_top), (m, top[m], r_top)
        for g, w, b in [(lp[m], r_lp, b_lp), (ent[m], r_ent, b_ent)] + [(a, c, b_lp) for a, c in zip(tlp[m], r_tlp)]:
            with np.errstate(over="ignore"):
                w32 = np.float32(w)  # the results' type: -6.8e38 (logits at both ends of fp32) rounds to -infinity
            if np.isinf(w32):
                assert g == w32
            else:
                assert abs(float(g) - w) <= b + abs(w) * 2.0 ** -24, (m, g, w, b)
    return got


def normal(M, V, dtype, spread, seed=0):
    return (torch.randn(M, V, generator=torch.Generator().manual_seed(seed)) * spread).to(dtype)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("V", [1, 2, 7, 63, 64, 65, 1000, 2047, 2048, 2049, 16384, 16391, 32003, 50257])
@pytest.mark.parametrize("n", [0, 1, 20, 64])
def test_sizes(dtype, V, n):
    M = 3
    check(normal(M, V, dtype, 3.0, seed=V), [0, V - 1, V // 2], n)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,V,n", [(1, 131072, 20), (300, 17001, 5), (300, 16384, 64), (40, 151001, 0)])
def test_batches(dtype, M, V, n):
    """Long and short slices, one and several."""
    check(normal(M, V, dtype, 2.5, seed=M), np.random.default_rng(M).integers(0, V, M), n)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_ranks_of_every_kind(dtype):
    """Tokens that are the largest, among many equal ones, at both ends of a slice
    and of 16 bytes, -infinity, NaN and outside."""
    V = 5003
    x = torch.round(normal(1, V, F32, 3.0, seed=1)).to(dtype)
    x[0, [5, 17, 4999]] = float("-inf")
    x[0, [6, 2048]] = float("nan")
    tokens = [int(x[0].nan_to_num(-9e9).argmax()), 0, 1, 5, 6, 7, 8, 17, 2047, 2048, 2049, 4095, 4096, 4999, 5002, -1, V,
              -(1 << 31), (1 << 31) - 1]
    check(x.expand(len(tokens), V).contiguous(), tokens, 30)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("V", [9, 3001, 40000])
def test_rows_of_special_values(dtype, V):
    rows = torch.zeros(8, V)
    rows[1] = float("-inf")
    rows[2] = float("nan")
    rows[3] = float("inf")
    rows[4, 3] = float("inf")
    rows[5] = float("-inf")
    rows[5, [1, 7]] = torch.tensor([-1000.0, -1001.0])  # all but two masked
    rows[6] = float(torch.finfo(dtype).min)             # masked by the lowest value
    rows[6, 8] = 1.0
    rows[7] = float(torch.finfo(dtype).max)
    rows[7, 2] = float(torch.finfo(dtype).min)
    check(rows.to(dtype), [0, 3, 4, 5, 3, 7, 8, 2], 5)
    check(rows.to(dtype), [V - 1, V - 1, 0, V - 1, 4, 0, 0, 3], 0)


@pytest.mark.parametrize("n", [1, 20, 64])
@pytest.mark.parametrize("M,V", [(2, 40000), (300, 20000)])
def test_flat_and_sorted_rows(M, V, n):
    """More equal logits than a list holds, a few steps, rising and falling rows."""
    x = torch.zeros(M, V)
    x[1] = torch.arange(V) % 7
    if M > 4:
        x[2] = torch.arange(V)
        x[3] = -torch.arange(V).float()
        x[4] = (torch.arange(V) // 128) % 5
        x[5:] = normal(M - 5, V, F32, 1.0)
    check(x, np.random.default_rng(n).integers(0, V, M), n)


def test_peaked_and_wide_rows():
    """All but one at a distance of 100, and logits of 1e4 apart."""
    x = normal(3, 30000, F32, 1.0, seed=3)
    x[0, 77] = 100.0
    x[1] *= 1e4
    x[2] = x[2] * 1e-6 + 1e4
    check(x, [77, 5, 6], 10)


def test_strides_and_alignments():
    """Rows that begin at every place within 16 bytes; what lies beside them is not used."""
    dev = _gpu.dev()
    for dtype, places in ((F32, 4), (BF16, 8), (F16, 8)):
        wide = torch.full((places + 3, 3001 + 16), float("inf"), dtype=dtype, device=dev)
        for at in range(places):
            view = wide[:, at:at + 3001]
            view.copy_(normal(places + 3, 3001, dtype, 3.0, seed=at))
            if at % 2:
                view[:, 0] = 30.0
                view[:, -1] = 30.0
            tokens = [0, 3000, 1, 2999, 5, 7, 8, 100, 2048, 11, 12][:places + 3]
            check(view, tokens, 7)
            wide.fill_(float("inf"))


def test_reruns_streams_and_given_outputs():
    dev, qmm = _gpu.dev(), _gpu.lib()
    x = normal(5, 70000, BF16, 2.0, seed=4).to(dev)
    t = torch.tensor([1, 2, 3, 69999, 0], dtype=torch.int32, device=dev)
    want = check(x, t.tolist(), 20)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        again = qmm.qmm_logprobs(x, t, 20)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, want))
    need = qmm.qmm_logprobs_workspace_bytes(5, 70000, 20)
    out = [torch.empty_like(w) for w in want]
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    got = qmm.qmm_logprobs(x, t, 20, logprobs=out[0], ranks=out[1], entropy=out[2], top_tokens=out[3], top_logprobs=out[4],
                           workspace=ws)
    assert all(a is b for a, b in zip(got, out)) and all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(qmm.QmmError):
        qmm.qmm_logprobs(x, t, 20, workspace=ws[:need - 16])
    with pytest.raises(qmm.QmmError):
        qmm.qmm_logprobs(x, t, 65)


@pytest.mark.parametrize("V", [1500, 60000])
def test_graph_replays(V):
    dev, qmm = _gpu.dev(), _gpu.lib()
    x = normal(4, V, F32, 2.0, seed=5).to(dev)
    t = torch.tensor([1, 2, 3, 4], dtype=torch.int32, device=dev)
    ws = torch.empty(max(16, qmm.qmm_logprobs_workspace_bytes(4, V, 9)), dtype=torch.uint8, device=dev)
    out = [o.clone() for o in qmm.qmm_logprobs(x, t, 9, workspace=ws)]
    kw = dict(zip(("logprobs", "ranks", "entropy", "top_tokens", "top_logprobs"), out))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qmm.qmm_logprobs(x, t, 9, workspace=ws, **kw)
    for rep in range(4):
        x.copy_(normal(4, V, F32, 2.0, seed=6 + rep))
        t.add_(7)
        eager = [o.clone() for o in qmm.qmm_logprobs(x, t, 9)]
        for o in out:
            o.fill_(-5)
        ws.random_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), f"replay {rep}"
