"""qmm_sample with u close to the border between two heavy tokens: within 1e-9 to
4e-9 of the kept mass, where weights to 2^-28 are not enough. Two logits and
their copies carry the mass, so that an error of a weight is that of all."""
import numpy as np
import pytest
import torch

from tests import _gpu

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
NEAR, FAR = 1e-9, 4e-9  # the documented distance, and the search's


def pairs(dtype, rows, seed, copies):
    """(logits [M, 2 copies], temperatures, u, tokens): of random pairs those whose
    border lies between NEAR and FAR from a 32-bit u."""
    rng = np.random.default_rng(seed)
    n = rows * 40
    top = torch.tensor(rng.uniform(-6, 6, n)).to(dtype)
    low = (top.double() - torch.tensor(rng.uniform(0.02, 1.5, n))).to(dtype)
    T = np.float32(rng.uniform(0.4, 1.6, n))
    hi, lo = top.double().numpy(), low.double().numpy()
    border = 1 / (1 + np.exp((lo - hi) / T.astype(np.float64)))
    u = np.float32(border)
    off = u.astype(np.float64) - border
    take = np.nonzero((np.abs(off) >= NEAR) & (np.abs(off) <= FAR) & (hi > lo))[0][:rows]
    x = torch.full((len(take), 2 * copies), float("-inf"), dtype=dtype)
    x[:, :copies] = low[take, None]      # the larger ones behind, in index order
    x[:, copies:] = top[take, None]
    # past the border: the first of the smaller ones; before it: the last of the larger ones
    return x, T[take], u[take], np.where(off[take] > 0, 0, 2 * copies - 1)


@pytest.mark.parametrize("copies", [1, 3, 50])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_near_a_border(dtype, copies):
    x, T, u, want = pairs(dtype, 3000, copies, copies)
    assert len(want) > 1500
    dev, qmm = _gpu.dev(), _gpu.lib()
    got = qmm.qmm_sample(x.to(dev), torch.tensor(u, device=dev), torch.tensor(T, device=dev)).cpu().numpy()
    wrong = got != want
    assert not wrong.any(), f"{int(wrong.sum())} of {len(want)} rows"


@pytest.mark.parametrize("V", [70000, 151001])
def test_near_a_border_in_long_rows(V):
    """The same pairs far apart in a row of logits without weight."""
    x, T, u, want = pairs(F32, 200, V, 1)
    wide = torch.full((len(want), V), -1e4)
    wide[:, 1000], wide[:, V - 7] = x[:, 0], x[:, 1]
    dev, qmm = _gpu.dev(), _gpu.lib()
    got = qmm.qmm_sample(wide.to(dev), torch.tensor(u, device=dev), torch.tensor(T, device=dev)).cpu().numpy()
    assert np.array_equal(got, np.where(want == 0, 1000, V - 7))


def test_log_probabilities():
    """The logarithm of a share, to its rounding and 2^-29."""
    x, T, u, _ = pairs(F32, 1500, 9, 1)
    dev, qmm = _gpu.dev(), _gpu.lib()
    lp = torch.empty(len(T), device=dev)
    # away from the border, either token
    u = np.float32(np.where(np.arange(len(u)) % 2, 0.01, 0.999))
    got = qmm.qmm_sample(x.to(dev), torch.tensor(u, device=dev), torch.tensor(T, device=dev), logprobs=lp).cpu().numpy()
    d = (x[:, 0].double() - x[:, 1].double()).numpy() / T.astype(np.float64)
    share = np.where(got == 1, 1 / (1 + np.exp(d)), np.exp(d) / (1 + np.exp(d)))
    want = np.log(share)
    assert (np.abs(lp.double().cpu().numpy() - want) <= np.abs(want) * 2.0 ** -24 + 2.0 ** -29).all()


@pytest.mark.parametrize("V", [131072, 250000, 250001])
@pytest.mark.parametrize("z", [0.4999, -0.4999])
def test_bins_full_of_their_heaviest_and_lightest_weights(V, z):
    """A whole row at the upper or lower end of one bin, up to where counts and
    sums of weights fill the fields that they share."""
    dev, qmm = _gpu.dev(), _gpu.lib()
    u = np.float32(np.random.default_rng(V).random(12, dtype=np.float32))
    x = torch.full((12, V), z / 8, device=dev)
    lp = torch.empty(12, device=dev)
    got = qmm.qmm_sample(x, torch.tensor(u, device=dev), logprobs=lp).cpu().numpy()
    assert np.array_equal(got, np.floor(u.astype(np.float64) * V).astype(int))
    assert np.abs(lp.double().cpu().numpy() + np.log(V)).max() <= 2.0 ** -28 + np.log(V) * 2.0 ** -24
