"""The step operators at the largest sizes that the host admits."""
import pytest
import torch

from tests import _gpu

pytestmark = pytest.mark.gpu


def test_most_rows_of_the_norm():
    """2^24 - 1 rows: the first, the last and some between are bitwise those of small calls."""
    qmm, dev = _gpu.lib(), _gpu.dev()
    M, D, page = (1 << 24) - 1, 8, 64
    g = torch.Generator(device=dev).manual_seed(1)
    q, k, v = (torch.randn(M, 1, D, generator=g, device=dev).half() for _ in range(3))
    w = torch.ones(D, device=dev)
    positions = torch.arange(M, dtype=torch.int32, device=dev)
    freq = torch.tensor([1.0, 0.1, 0.01, 0.001], device=dev)
    kc = torch.zeros(M // page + 1, 1, page, D, dtype=torch.float16, device=dev)
    vc = torch.zeros_like(kc)
    out = qmm.qmm_qk_norm_rope(q, k, v, w, w, positions, freq, positions, kc, vc)
    for at in (0, M // 2, M - 37):
        rows = slice(at, at + 37)
        kc2, vc2 = torch.zeros(1, 1, page, D, dtype=torch.float16, device=dev), torch.zeros(1, 1, page, D, dtype=torch.float16, device=dev)
        slots = torch.arange(37, dtype=torch.int32, device=dev)
        want = qmm.qmm_qk_norm_rope(q[rows], k[rows], v[rows], w, w, positions[rows].clone(), freq, slots, kc2, vc2)
        assert torch.equal(out[rows], want)
        assert torch.equal(kc.view(-1, D)[rows], kc2.view(-1, D)[:37])
        assert torch.equal(vc.view(-1, D)[rows], vc2.view(-1, D)[:37])
