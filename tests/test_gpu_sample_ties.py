"""qmm_sample where the element looked for lies among many equal or nearly equal
logits: more than are ranked by pairs (1024), while the list of the wanted bins
still holds them (11264), so that a search starts on the list and goes on over
the row; and around both limits."""
import numpy as np
import pytest
import torch

from tests.test_gpu_sample import check, uniform

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def rows(M, V, equal, dtype, seed, spread=0.0):
    """`equal` logits of (about) 3 at random places among others far below, and
    two larger ones."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, V, generator=g) - 12.0
    for i in range(M):
        order = torch.randperm(V, generator=g)
        x[i, order[:equal]] = 3.0 + spread * torch.rand(equal, generator=g)
        x[i, order[equal:equal + 2]] = torch.tensor([4.5, 6.0])
    return x.to(dtype)


# 20000 and 60000 logits are gathered by the workgroup that finishes them, 100000
# and more by a launch of their own; V // 20 as a slice's list has 1024 places.
@pytest.mark.parametrize("V,dtype", [(20000, F32), (20000, F16), (60000, F32), (100000, F32), (151001, F16), (7000, BF16)])
@pytest.mark.parametrize("equal", [1020, 1024, 1025, 1026, 1500, 4000, 5500])
def test_more_ties_than_are_ranked(V, dtype, equal):
    M = 12
    x = rows(M, V, equal, dtype, equal)
    u = uniform(M, equal)
    check(x, u)
    check(x, u, k=np.resize([0, 700, 1025, equal, equal + 2], M), p=np.resize([1.0, 0.5, 0.93], M),
          mp=np.resize([0.0, 0.01, 0.04], M))


@pytest.mark.parametrize("V", [30000, 120000])
def test_more_near_ties_than_are_ranked(V):
    """Within 2^-12 of one another: one part of a bin, many different values."""
    x = rows(10, V, 3000, F32, 5, 2.0 ** -12)
    check(x, uniform(10, 6), k=np.resize([0, 1500, 3000], 10), p=np.resize([0.4, 0.9], 10))


def test_many_rows_of_ties_repeat():
    x = rows(64, 40000, 2500, F32, 7)
    first = check(x, uniform(64, 8), p=0.8)
    for _ in range(5):
        again = check(x, uniform(64, 8), p=0.8)
        assert all(np.array_equal(a, b) for a, b in zip(first, again))
