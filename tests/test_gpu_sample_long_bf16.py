"""qmm_sample of many bf16 rows of 131073 to 196608 logits: vocabularies between,
logits that fill a row once, twice or nearly three times over what a count of 16
bits holds, in both signs, and the first length past the limit."""
import numpy as np
import pytest
import torch

from tests import _step
from tests.test_gpu_sample import MARGIN, check, logits, sample, uniform

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
MOST = 3 * 65536 - 1


@pytest.mark.parametrize("V", [131073, 152064, 151936, MOST - 5, MOST, MOST + 1])
def test_filters(V):
    M = 64
    check(logits(M, V, BF16, V), uniform(M, V), T=np.resize([1.0, 0.7, 1.4], M), k=np.resize([0, 50, 1000, 0], M),
          p=np.resize([1.0, 0.9, 0.95, 0.5, 1.0], M), mp=np.resize([0.0, 0.0, 0.02], M))


@pytest.mark.parametrize("first,second", [(1.5, -2.0), (-0.0, 0.0), (-3.0, -3.25), (2.0, 2.0), (0.5, "-inf"), (-7.0, "nan")],
                         ids=str)
def test_two_logits_fill_the_row(first, second):
    """Two logits of 65536 elements each and a third of 65535, and more uneven parts."""
    M, V = 66, MOST
    x = torch.full((M, V), -1.0).to(BF16)
    g = torch.Generator().manual_seed(3)
    for i in range(M):
        order = torch.randperm(V, generator=g)
        n, m = [(65536, 65536), (130000, 66000), (65535, 65537), (100, V - 100), (V, 0), (65536, 131071)][i % 6]
        x[i, order[:n]] = float(first)
        x[i, order[n:n + m]] = float(second)
    u = uniform(M, 4)
    tok, lp = sample(x, u, k=np.resize([0, 70000, 0, 150], M), p=np.resize([1.0, 0.75, 0.4], M))
    for i in range(M):
        want, want_lp, margin = _step.sample_reference(_step.f64(x[i]), float(u[i]), 1.0, [0, 70000, 0, 150][i % 4],
                                                       float(np.float32([1.0, 0.75, 0.4][i % 3])), 0.0)
        if margin >= MARGIN or want == -1:
            assert tok[i] == want, f"row {i}: {tok[i]}, want {want} (margin {margin:.1e})"
            assert want == -1 or abs(float(lp[i]) - want_lp) <= 2.0 ** -27 + abs(want_lp) * 2.0 ** -24
        else:
            assert 0 <= tok[i] < V


@pytest.mark.parametrize("value", [0.0, -0.0, -5.0, 11.0])
def test_equal_logits(value):
    """One logit for the whole row: sums of ones are exact."""
    M = 64
    u = uniform(M, 5)
    tok, lp = sample(torch.full((M, MOST), value).to(BF16), u)
    assert np.array_equal(tok, np.floor(u.astype(np.float64) * MOST).astype(int))
    assert np.abs(lp + np.log(MOST)).max() <= 2.0 ** -20
