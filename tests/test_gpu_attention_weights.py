"""qmm_paged_attention where small weights make up the output: one token with a
large score and a small value (as first tokens often are) before a long tail,
whose weights lie far below the largest. The bounds count roundings of single
weights; nothing in them grows with a type's smallest number."""
import math

import numpy as np
import pytest
import torch

from tests import _gpu, _step

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
FLOOR = {F16: 2.0 ** -40, BF16: 0.0}  # of the largest weight: what a weight's second part leaves in fp16


def run(q, k, v, page, max_context=None):
    """One sequence of k, v [n, Hkv, D] in pages in reverse order, q [rows, Hq, D] its newest rows."""
    qmm, dev = _gpu.lib(), _gpu.dev()
    n, Hkv, D = k.shape
    pages = -(-n // page)
    table = torch.arange(pages - 1, -1, -1, dtype=torch.int32)
    caches = []
    for x in (k, v):
        c = torch.zeros(pages * page, Hkv, D, dtype=x.dtype)
        c[:n] = x
        caches.append(c.unflatten(0, (pages, page)).transpose(1, 2)[table.long()].contiguous().to(dev))
    rows = q.shape[0]
    ints = [torch.tensor(x, dtype=torch.int32, device=dev) for x in ([n], [0, rows])]
    lse = torch.full((rows, q.shape[1]), float("nan"), device=dev)
    out = qmm.qmm_paged_attention(q.to(dev), *caches, table[None].to(dev), *ints, rows, max_context or n, scale=1.0,
                                  lse=lse)
    torch.cuda.synchronize()
    return out, lse


def check(q, k, v, out, lse):
    rows, Hq, D = q.shape
    n, G = k.shape[0], Hq // k.shape[1]
    qd, kd, vd = _step.f64(q), _step.f64(k), _step.f64(v)
    ref, bound = np.zeros(q.shape), np.zeros(q.shape)
    rl, lb = np.zeros((rows, Hq)), np.zeros((rows, Hq))
    dtype = q.dtype
    for r in range(rows):
        see = n - rows + r + 1
        for h in range(Hq):
            kk, vv = kd[:see, h // G], vd[:see, h // G]
            s = kk @ qd[r, h]
            m = s.max()
            w = np.exp(s - m)
            total = w.sum()
            ref[r, h] = w @ vv / total
            rl[r, h] = m + math.log(total)
            # Of a weight: the score's products, the scale and the maximum, the
            # exponential. Of the sums: a lane adds 4 of 64 tokens, the matrix
            # unit 32 at a time; 64 for their joins.
            e = ((D + 2) * 2.0 ** -24 * (np.abs(kk) @ np.abs(qd[r, h])).max() * 1.01
                 + 4 * 2.0 ** -24 * 1.45 * np.abs(s).max() + 2.0 ** -21 + (see / 16 + 64) * 2.0 ** -24)
            bound[r, h] = (w @ np.abs(vv) / total * (2 * e + _step.HALF_STEP[dtype] ** 2)
                           + see * FLOOR[dtype] * np.abs(vv).max(0) / total)
            lb[r, h] = e + abs(rl[r, h]) * 2.0 ** -22 + 2.0 ** -22
    _step.assert_rounded(out, ref, bound, "out")
    _step.assert_rounded(lse, rl, lb, "lse")


def sink(n, at, gap, D, dtype, rows=1, G=2, seed=0):
    """Scores of 0 but for token `at`, whose score is `gap` and whose value is
    small; every fourth value is 1 (nothing cancels in the tail's sum)."""
    g = torch.Generator().manual_seed(seed)
    q, k = torch.zeros(rows, G, D), torch.zeros(n, 1, D)
    q[..., 0], k[at, 0, 0] = 1.0, gap
    v = torch.randn(n, 1, D, generator=g)
    v[:, 0, ::4] = 1.0
    v[at] = 0.0
    v[at, 0, 1] = 2.0 ** -12
    return q.to(dtype), k.to(dtype), v.to(dtype)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("gap", [10.0, 12.0, 14.0, 16.0, 17.0, 18.0])
@pytest.mark.parametrize("n,D,page", [(4096, 64, 16), (4096, 128, 24), (4096, 256, 64), (200, 128, 16)])
def test_small_weights_after_a_large_one(n, D, page, gap, dtype):
    q, k, v = sink(n, 0, gap, D, dtype)
    check(q, k, v, *run(q, k, v, page))
    check(q, k, v, *run(q, k, v, page, max_context=1))  # whole, in one workgroup


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("gap", [14.0, 16.0, 18.0])
@pytest.mark.parametrize("D", [128, 256])
def test_small_weights_of_a_long_context(D, gap, dtype):
    q, k, v = sink(131072, 5, gap, D, dtype, rows=2, G=6)
    check(q, k, v, *run(q, k, v, 64))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rise", [0.25, 0.4, 3.0])
@pytest.mark.parametrize("max_context", [1, 1500])
def test_rising_scores(rise, max_context, dtype):
    """Every tile's largest score is above the ones before: by less and by more
    than what the running maximum lets pass."""
    n, D = 1500, 128
    g = torch.Generator().manual_seed(3)
    q, k = torch.zeros(3, 4, D), torch.zeros(n, 2, D)
    q[..., 0], q[..., 1] = 1.0, 0.25
    steps = torch.arange(n) // 64 * rise
    k[..., 0] = steps.round()[:, None]
    k[..., 1] = ((steps - steps.round()) * 4)[:, None] + torch.rand(n, 2, generator=g)
    v = torch.randn(n, 2, D, generator=g)
    q, k, v = (x.to(dtype) for x in (q, k, v))
    check(q, k, v, *run(q, k, v, 32, max_context))
