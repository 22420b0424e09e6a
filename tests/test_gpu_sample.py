"""qmm_sample against the plain 64-bit form: vocabulary sizes, types, filters and
their combinations, ties, masks, extreme temperatures and logits, lists that
overflow. Tokens are compared for equality."""
import math

import numpy as np
import pytest
import torch

from tests import _gpu, _step

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
# Weights are good to 2^-28 of themselves: where u or top_p comes nearer than
# this to a border (as a share of the mass), the 64-bit form's token is not asked for.
MARGIN = 2.0 ** -27


def sample(x, u, T=None, k=None, p=None, mp=None):
    qmm, dev = _gpu.lib(), _gpu.dev()
    M = x.shape[0]

    def col(v, dtype):
        if v is None:
            return None
        return torch.as_tensor(np.broadcast_to(np.asarray(v, dtype=np.float64), (M,)).copy()).to(dtype).to(dev)
    lp = torch.full((M,), float("nan"), device=dev)
    tok = qmm.qmm_sample(x.to(dev), col(u, F32), col(T, F32), col(k, torch.int32), col(p, F32), col(mp, F32),
                         logprobs=lp)
    torch.cuda.synchronize()
    return tok.cpu().numpy(), lp.cpu().numpy()


def check(x, u, T=None, k=None, p=None, mp=None, borders=False, most_near=None):
    """`borders`: the inputs put u or p exactly on borders, and the answer there
    is exact in both forms. `most_near`: how many rows the inputs put near one."""
    got, lp = sample(x, u, T, k, p, mp)
    M = x.shape[0]

    def at(v, i, default):
        return default if v is None else float(np.float32(np.broadcast_to(np.asarray(v, dtype=np.float64), (M,))[i]))
    near = 0
    for i in range(M):
        tok, want_lp, margin = _step.sample_reference(
            _step.f64(x[i]), at(u, i, 0), at(T, i, 1.0), int(at(k, i, 0)), at(p, i, 1.0), at(mp, i, 0.0))
        if margin < MARGIN and not borders:
            near += 1
            continue
        assert got[i] == tok, f"row {i}: token {got[i]}, want {tok} (margin {margin:.2e})"
        if math.isinf(want_lp):
            assert lp[i] == want_lp
        else:
            # weights and their sum to 2^-28 each, one rounding
            assert abs(float(lp[i]) - want_lp) <= 2.0 ** -27 + abs(want_lp) * 2.0 ** -24, f"row {i}: {lp[i]} {want_lp}"
    assert near <= max(1, M // 20 if most_near is None else most_near), f"{near} of {M} rows near a border"
    return got, lp


def logits(M, V, dtype, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, V, generator=g) * spread).to(dtype)


def uniform(M, seed):
    return np.float32(np.random.default_rng(seed).random(M, dtype=np.float32))


FILTERS = [dict(), dict(k=1), dict(k=50), dict(p=0.9), dict(mp=0.05), dict(k=40, p=0.8), dict(k=1000, p=0.95, mp=0.01),
           dict(p=0.3, mp=0.2), dict(T=0.3, p=0.99), dict(T=2.5, k=300), dict(T=1.7, p=0.5)]


@pytest.mark.parametrize("f", FILTERS, ids=str)
@pytest.mark.parametrize("V,dtype", [(1, F32), (2, F16), (63, BF16), (1000, F32), (4097, F16), (20011, BF16),
                                     (32768, F32), (151001, F32), (151001, BF16)])
def test_sizes_types_and_filters(V, dtype, f):
    M = 9
    check(logits(M, V, dtype, V), uniform(M, V + 1), **f)


@pytest.mark.parametrize("M", [1, 2, 100, 300, 600])
def test_row_counts(M):
    """Rows cut into many slices down to one workgroup a row."""
    check(logits(M, 20000, F32, M), uniform(M, M), T=np.linspace(0.2, 1.5, M), k=(np.arange(M) % 4) * 30,
          p=0.5 + (np.arange(M) % 3) * 0.25, mp=(np.arange(M) % 5) * 0.01)


def test_large_vocabulary():
    check(logits(2, 300007, F16, 5), uniform(2, 5), p=0.97)
    check(logits(300, 140000, BF16, 6), uniform(300, 6), p=0.9)


@pytest.mark.parametrize("spread", [0.01, 0.5, 20.0, 60.0])
def test_flat_and_peaked(spread):
    check(logits(64, 8000, F32, 7, spread), uniform(64, 7), p=0.9)
    check(logits(64, 8000, F32, 8, spread), uniform(64, 8))


@pytest.mark.parametrize("V", [4, 1000, 4096, 131072])
@pytest.mark.parametrize("value", [0.0, -7.25, 900.0, -3.0e38])
def test_equal_logits(V, value):
    """Every logit the same (the type's lowest among them): borders at exact
    multiples of 1/V (exact in 64 bits), lists that overflow, ties by index."""
    M = 8
    x = torch.full((M, V), value)
    u = np.array([0, 0.25, 0.5, 0.75, 0.125, 1 - 2.0 ** -24, 0.5 - 2.0 ** -12, 0.3125])
    for f in (dict(), dict(k=3), dict(p=0.5), dict(p=0.25, k=V // 2), dict(mp=1.0), dict(T=0.1, p=0.75)):
        check(x, u, borders=True, **f)


def test_few_distinct_values():
    """Thousands of ties on the borders (an 8-bit grid of logits)."""
    x = (logits(40, 60000, F32, 9) * 2).round() / 2
    for f in (dict(), dict(p=0.9), dict(k=700), dict(k=5000, p=0.7, mp=0.002)):
        check(x, uniform(40, 9), **f)


def test_signed_zeros_are_equal():
    x = torch.zeros(4, 16)
    x[:, ::2] = -0.0
    got, _ = sample(x, [0.0, 0.3, 0.6, 0.99])
    assert got.tolist() == [0, 4, 9, 15]


def test_masked_logits():
    """-inf, the type's lowest value and NaN are never chosen; rows with nothing else."""
    for dtype in (F32, F16, BF16):
        x = logits(6, 3000, dtype, 10)
        x[0, 5:] = float("-inf")
        x[1, ::2] = float("nan")
        x[2, 100:] = torch.finfo(dtype).min
        x[3] = float("-inf")
        x[4] = float("nan")
        x[5] = float("-inf")
        x[5, 2999] = -50.0
        check(x, uniform(6, 10), p=0.95)
        got, lp = sample(x, uniform(6, 11), T=0.0)
        assert got[3] == got[4] == -1 and np.isneginf(lp[3:5]).all() and got[5] == 2999 and lp[5] == 0
        assert got[0] == int(x[0, :5].float().argmax()) and got[2] == int(x[2].float().argmax())


def test_infinite_logits():
    x = logits(5, 2000, F32, 11)
    x[:, 700] = float("inf")
    x[1:, 30] = float("inf")
    x[2, 31] = float("-inf")
    u = np.array([0.7, 0.2, 0.7, 0.5, 0.5])
    got, lp = sample(x, u, T=[1, 1, 1, 0, 0.5], p=0.9, k=[0, 0, 0, 0, 1])
    assert got.tolist() == [700, 30, 700, 30, 30]
    assert np.allclose(lp, [0, -math.log(2), -math.log(2), 0, 0], atol=1e-6)


@pytest.mark.parametrize("T", [1e-30, 1e-6, 0.004, 0.02, 50.0, 1e6, float("inf")])
def test_extreme_temperatures(T):
    if math.isinf(T):
        got, lp = sample(logits(3, 512, F32, 12), [0.0, 0.5, 0.999], T=T)
        assert np.allclose(lp, -math.log(512), atol=1e-6)
        return
    check(logits(20, 5000, F32, 12), uniform(20, 12), T=T)
    check(logits(20, 5000, F32, 13), uniform(20, 13), T=T, p=0.6, mp=0.001)


@pytest.mark.parametrize("offset,scale", [(400.0, 1.0), (520.0, 2.0), (-470.0, 1.0), (-463.0, 3.0), (1e6, 1.0),
                                          (-1e30, 1e27), (1e38, 1e37)])
def test_logits_far_from_zero(offset, scale):
    """Around and past the ends of the histogram's range."""
    x = logits(20, 5000, F32, 14) * scale + offset
    check(x, uniform(20, 14), p=0.9)
    check(x, uniform(20, 15), k=20)
    check(x, uniform(20, 16), T=scale)


def test_greedy():
    """Temperature 0, below 0 and NaN: the largest, of equal ones the lowest index."""
    x = logits(6, 40000, BF16, 15)
    x[0, 39000] = x[0, 123] = 60.0
    got, lp = sample(x, uniform(6, 17), T=[0.0, -1.0, float("nan"), 0.0, -0.0, 0.0], p=0.5, mp=0.5, k=5)
    top = x.float().max(1, keepdim=True).values
    want = [int((x[i].float() == top[i]).nonzero()[0]) for i in range(6)]
    assert got.tolist() == want and (lp == 0).all() and got[0] == 123


def test_numbers_outside():
    """u, top_p, top_k and min_p outside their ranges are taken as the nearest inside."""
    x = logits(1, 3000, F32, 16).repeat(7, 1)
    got, _ = sample(x, [float("nan"), -1.0, 0.0, 1.0, 2.0, float("inf"), 1 - 2.0 ** -24])
    assert got[0] == got[1] == got[2] and len(set(got[3:])) == 1
    inside, _ = sample(x, uniform(7, 18))
    for kw in (dict(p=7.0), dict(p=float("nan")), dict(k=-5), dict(k=1 << 30), dict(mp=-1.0), dict(mp=float("nan"))):
        got, _ = sample(x, uniform(7, 18), **kw)
        assert np.array_equal(got, inside), kw
    best = int(x[0].argmax())
    for kw in (dict(p=0.0), dict(p=-3.0), dict(mp=1.0), dict(mp=9.0)):
        got, lp = sample(x, uniform(7, 19), **kw)
        assert (got == best).all() and (lp == 0).all(), kw


def test_strided_and_unaligned_rows():
    for dtype in (F32, F16):
        x = logits(5, 5000, dtype, 17)
        want, want_lp = sample(x, uniform(5, 20), p=0.9)
        wide = torch.full((5, 5011), 99.0, dtype=dtype, device=_gpu.dev())
        for at in (1, 3, 8):
            view = wide[:, at:at + 5000]
            view.copy_(x)
            got, lp = sample(view, uniform(5, 20), p=0.9)
            assert np.array_equal(got, want) and np.array_equal(lp, want_lp)
            view.fill_(99.0)


@pytest.mark.parametrize("M,V,dtype", [(1, 90000, F32), (3, 5000, F32), (280, 30000, F32), (3, 30000, BF16),
                                       (70, 131072, BF16), (70, 131072, F16)])
def test_graph_replays_reruns_and_streams(M, V, dtype):
    qmm, dev = _gpu.lib(), _gpu.dev()
    x = logits(M, V, dtype, 18).to(dev)
    u = torch.as_tensor(uniform(M, 21)).to(dev)
    p = torch.full((M,), 0.9, device=dev)
    ws = torch.empty(qmm.qmm_sample_workspace_bytes(M, V), dtype=torch.uint8, device=dev)
    tok, lp = torch.empty(M, dtype=torch.int32, device=dev), torch.empty(M, device=dev)

    def call():
        qmm.qmm_sample(x, u, top_p=p, tokens=tok, logprobs=lp, workspace=ws)
    call()
    torch.cuda.synchronize()
    eager, eager_lp = tok.clone(), lp.clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(tok, eager) and torch.equal(lp, eager_lp)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for rep in range(4):
        ws.random_()
        tok.fill_(-7)
        lp.fill_(float("nan"))
        if rep == 2:
            u.copy_(torch.as_tensor(uniform(M, 22)))
            call()
            torch.cuda.synchronize()
            eager, eager_lp = tok.clone(), lp.clone()
            tok.fill_(-7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(tok, eager) and torch.equal(lp, eager_lp), f"replay {rep}"


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("heavy", [(0.0,), (-3.0,), (0.0, -0.0), (1.5, 1.25), ("lowest",), (2.0, "-inf")], ids=str)
def test_logits_of_more_than_65535_elements(heavy, dtype):
    """One or two logits fill most of a row, as the largest, among the others or far below."""
    M, V = 66, 131072
    x = logits(M, V, dtype, 1)
    x[::2] = logits(M // 2, V, dtype, 2, 1.0)
    g = torch.Generator().manual_seed(10)
    for i in range(M):
        order, at = torch.randperm(V, generator=g), 0
        for h in heavy:
            value = torch.finfo(dtype).min if h == "lowest" else float(h)
            n = [65536, 100000, V][i % 3] if len(heavy) == 1 else [65536, 65535, 66000][i % 3]
            x[i, order[at:at + n]] = value
            at += n
    u, T, k = uniform(M, 3), np.tile([1.0, 0.7, 1.3, 1.0, 1.0, 0.7], 11), np.tile([0, 0, 60000, 70000, 100, 0], 11)
    p, mp = np.tile([1.0, 0.9, 0.95, 1.0, 1.0, 0.5], 11), np.tile([0.0, 0.0, 0.0, 0.1, 0.0, 0.0], 11)
    tok, lp = check(x, u, T, k, p, mp, most_near=M // 6)  # half of equal logits is a border: every sixth row
    if len(heavy) == 1:
        for i in range(5, M, 6):  # the first half by index, and u takes its place in it
            assert tok[i] == int(np.floor(np.float64(u[i]) * (V // 2)))


@pytest.mark.parametrize("n", [65534, 65535, 65536])
@pytest.mark.parametrize("value", [0.0, -0.0, -7.0, 5.0])
def test_row_of_65536_bf16_logits_that_are_nearly_all_equal(value, n):
    M, V = 5, 65536
    x = torch.full((M, V), value).to(BF16)
    x[:, n:] = -1.0
    u = uniform(M, 23)
    tok, lp = sample(x, u)
    assert (tok >= 0).all()
    for i in range(M):
        if n == V:  # sums of ones are exact
            assert tok[i] == int(np.floor(np.float64(u[i]) * n)) and abs(lp[i] + math.log(n)) <= 2.0 ** -20
        want, want_lp, margin = _step.sample_reference(_step.f64(x[i]), float(u[i]), 1.0, 0, 1.0, 0.0)
        if margin >= MARGIN:
            assert tok[i] == want and abs(float(lp[i]) - want_lp) <= 2.0 ** -27 + abs(want_lp) * 2.0 ** -24


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,V", [(24, 1), (24, 17), (24, 9001), (24, 131073), (400, 16384), (100, 65001), (65, 131071),
                                 (64, 131072)])
def test_16_bit_rows_of_every_alignment(M, V, dtype):
    """Rows whose first elements lie at every distance from 16 bytes; tokens among equal logits by their index."""
    x = torch.empty(M, V + 3, dtype=dtype)[:, :V]
    x.copy_(logits(M, V, dtype, V, 2.0))
    g = torch.Generator().manual_seed(V)
    x[::3] = torch.randint(0, 3, x[::3].shape, generator=g).to(dtype)
    check(x, uniform(M, V), k=np.resize([0, 3, 700], M), p=np.resize([1.0, 0.9, 1.0, 0.6], M),
          mp=np.resize([0.0] * 20 + [0.3] * 4, M))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_many_16_bit_rows_of_all_kinds(dtype):
    """Masks, infinities, NaN, zeros of both signs, extreme temperatures and parameters, in one call of many rows."""
    M, V = 400, 16389
    x = logits(M, V, dtype, 5)
    inf, low = float("inf"), torch.finfo(dtype).min
    g = torch.Generator().manual_seed(6)
    some = torch.rand(M, V, generator=g) < 0.9
    T = np.ones(M)
    k, p, mp = np.zeros(M, int), np.ones(M), np.zeros(M)
    for i in range(M):
        kind = i % 20
        if kind in (1, 2, 3):
            x[i, some[i]] = [-inf, low, float("nan")][kind - 1]
        elif kind == 4:
            x[i] = -inf
        elif kind == 5:
            x[i], x[i, 77] = -inf, -5.0
        elif kind == 6:
            x[i, 5::1000] = inf
        elif kind == 7:
            x[i], x[i, ::2] = -1.0, -0.0
            x[i, 1::4] = 0.0
        elif kind == 8:
            x[i] = float("nan")
        elif kind == 9:
            x[i] = low
        elif kind == 10:
            x[i] = x[i] * 1000
        elif kind == 11:
            x[i] = x[i] * 2.0 ** -12
        T[i] = {12: 1e-30, 13: 0.004, 14: 50.0, 15: 1e6, 16: inf, 17: 0.0, 18: -1.0}.get(kind, 1.0)
        j = i // 20
        k[i] = [0, 1, 50, V, 2 * V][j % 5]
        p[i] = [1.0, 0.9, 0.5, 0.0][j % 4]
        mp[i] = [0.0, 0.05, 1.0][j % 3]
    check(x, uniform(M, 7), T=T, k=k, p=p, mp=mp)
