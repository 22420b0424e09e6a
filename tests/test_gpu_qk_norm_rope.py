"""qmm_qk_norm_rope against the plain 64-bit form: head sizes, rotated parts,
both pair orders, types, far positions, strided rows and padding slots."""
import numpy as np
import pytest
import torch

from tests import _gpu, _step

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def problem(M, Hq, Hkv, D, R, din, dout, page, seed=0, far=262143, pages=None):
    g = torch.Generator().manual_seed(seed)
    pool = pages or (M + page) // page + 2
    slots = torch.randperm(pool * page, generator=g)[:M].to(torch.int32)
    return dict(
        q=(torch.randn(M, Hq, D, generator=g) * 2).to(din), k=(torch.randn(M, Hkv, D, generator=g) * 0.3).to(din),
        v=torch.randn(M, Hkv, D, generator=g).to(din), q_weight=torch.randn(D, generator=g) * 0.3 + 1,
        k_weight=torch.randn(D, generator=g) * 0.3 + 1,
        positions=torch.randint(0, far + 1, (M,), generator=g).to(torch.int32),
        inv_freq=(1e7 ** (-torch.arange(0, R, 2).double() / max(R, 1))).float(), slots=slots,
        k_cache=torch.randn(pool, Hkv, page, D, generator=g).to(dout),
        v_cache=torch.randn(pool, Hkv, page, D, generator=g).to(dout))


def run(p, **kw):
    qmm, dev = _gpu.lib(), _gpu.dev()
    d = {n: t.to(dev) if t is not None else None for n, t in p.items()}
    out = qmm.qmm_qk_norm_rope(d["q"], d["k"], d["v"], d["q_weight"], d["k_weight"], d["positions"], d["inv_freq"],
                               d["slots"], d["k_cache"], d["v_cache"], **kw)
    torch.cuda.synchronize()
    return out, d["k_cache"], d["v_cache"]


def check(p, eps=1e-6, weight_offset=0.0, interleaved=False):
    got = run(p, eps=eps, weight_offset=weight_offset, interleaved=interleaved)
    want = _step.rope_reference(*(_step.f64(p[n]) for n in ("q", "k", "v", "q_weight", "k_weight")),
                                p["positions"].numpy(), p["inv_freq"].double().numpy(), p["slots"].numpy(),
                                _step.f64(p["k_cache"]), _step.f64(p["v_cache"]), eps, weight_offset, interleaved)
    for name, g, (r, b) in zip(("q", "k_cache", "v_cache"), got, want):
        _step.assert_rounded(g, r, b, name)
    return got


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("din,dout", [(F32, BF16), (F32, F16), (BF16, BF16), (F16, F16), (BF16, F16)])
@pytest.mark.parametrize("D,R", [(8, 8), (64, 64), (64, 0), (80, 32), (96, 96), (128, 128), (128, 16), (192, 64),
                                 (256, 64), (256, 256), (248, 120)])
def test_heads_and_types(D, R, din, dout, interleaved):
    check(problem(5, 3, 2, D, R, din, dout, 16, seed=D + R), interleaved=interleaved)


@pytest.mark.parametrize("M,Hq,Hkv,page", [(1, 24, 4, 16), (1, 1, 1, 1), (2, 48, 8, 17), (37, 7, 1, 100)])
def test_rows_and_pages(M, Hq, Hkv, page):
    check(problem(M, Hq, Hkv, 128, 64, F32, BF16, page, seed=M), weight_offset=1.0, eps=1e-5)


def test_many_rows():
    """Enough rows that a workgroup walks over the heads of a whole row."""
    check(problem(2100, 3, 1, 64, 32, F32, F16, 32, seed=1))


def test_padding_and_slots_past_the_cache():
    """Rows with a negative slot or one past the cache write nothing; their
    queries are computed all the same."""
    p = problem(9, 2, 2, 64, 64, F32, BF16, 5, seed=2)
    total = p["k_cache"].shape[0] * 5
    p["slots"][[1, 4, 6, 8]] = torch.tensor([-1, total, (1 << 31) - 1, -(1 << 31)], dtype=torch.int32)
    check(p)


def test_extreme_positions():
    p = problem(6, 2, 1, 128, 128, F32, F16, 16, seed=3)
    p["positions"] = torch.tensor([0, 1, 1 << 20, (1 << 31) - 1, -1, 262143], dtype=torch.int32)
    check(p)


def test_rows_of_zeros_tiny_and_large_values():
    p = problem(4, 2, 2, 64, 32, F32, BF16, 16, seed=4)
    p["q"][0] = 0
    p["k"][1] *= 1e-12
    p["q"][2] *= 1e12
    check(p)


def same_bits(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_non_finite_values_stay_in_their_head():
    p = problem(3, 2, 2, 64, 32, F32, BF16, 16, seed=5)
    clean = check(p)
    p["q"][1, 0, 3] = float("nan")
    p["k"][2, 1, 60] = float("inf")
    p["v"][0, 0, 7] = float("nan")
    out, kc, vc = run(p)
    out2, kc2, vc2 = (t.clone() for t in clean)
    out2[1, 0] = out[1, 0]
    page, off = divmod(int(p["slots"][2]), 16)
    kc2[page, 1, off] = kc[page, 1, off]
    assert same_bits(out, out2) and same_bits(kc, kc2)
    assert torch.isnan(out[1, 0]).all()
    # x = inf: the norm's factor is 0, every finite value gives 0
    assert torch.isnan(kc[page, 1, off, 60]) and (kc[page, 1, off, 32:60] == 0).all()
    page, off = divmod(int(p["slots"][0]), 16)
    assert torch.isnan(vc[page, 0, off, 7])
    vc2[page, 0, off, 7] = vc[page, 0, off, 7]
    assert same_bits(vc, vc2)


def test_views_of_a_fused_projection():
    """q, k and v as column ranges of one fused output."""
    p = problem(7, 4, 2, 64, 64, F32, BF16, 16, seed=6)
    want = check(p)
    fused = torch.full((7, 8 * 64 + 16), float("nan"))
    views = {}
    at = 8
    for n, h in (("q", 4), ("k", 2), ("v", 2)):
        fused[:, at:at + h * 64] = p[n].flatten(1)
        views[n] = (at, h)
        at += h * 64
    dev, qmm = _gpu.dev(), _gpu.lib()
    f = fused.to(dev)
    d = {n: t.to(dev) for n, t in p.items()}
    q, k, v = (f[:, a:a + h * 64].unflatten(1, (h, 64)) for a, h in views.values())
    out = qmm.qmm_qk_norm_rope(q, k, v, d["q_weight"], d["k_weight"], d["positions"], d["inv_freq"], d["slots"],
                               d["k_cache"], d["v_cache"])
    for a, b in zip((out, d["k_cache"], d["v_cache"]), want):
        assert torch.equal(a, b)


def test_graph_replays_and_streams():
    qmm, dev = _gpu.lib(), _gpu.dev()
    p = problem(6, 4, 2, 128, 64, F32, BF16, 16, seed=7)
    want = check(p)
    d = {n: t.to(dev) for n, t in p.items()}
    out = torch.empty_like(want[0])

    def call():
        qmm.qmm_qk_norm_rope(d["q"], d["k"], d["v"], d["q_weight"], d["k_weight"], d["positions"], d["inv_freq"],
                             d["slots"], d["k_cache"], d["v_cache"], out=out)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(out, want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(4):
        out.fill_(float("nan"))
        d["k_cache"].copy_(p["k_cache"])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(d["k_cache"], want[1])
