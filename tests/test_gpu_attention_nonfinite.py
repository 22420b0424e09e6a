"""qmm_paged_attention with infinities and NaN in values and keys anywhere in a
context, in tiles that every row sees whole above all: rows that see the token
give what the formula gives, rows that do not are bitwise what they were."""
import pytest
import torch

from tests import _gpu
from tests.test_gpu_paged_attention import Problem

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
INF, NAN = float("inf"), float("nan")


def place(p, b, j, page):
    return int(p.table[b, j // page]), j % page


def same(got, want):
    """Bitwise where finite, the same infinities, NaN where NaN."""
    g, w = got.float().cpu(), want.float().cpu()
    assert torch.equal(torch.isnan(g), torch.isnan(w)), "NaN in other places"
    keep = ~torch.isnan(w)
    assert torch.equal(g[keep], w[keep])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("D,G,page", [(64, 1, 16), (64, 12, 24), (96, 3, 16), (128, 6, 16), (192, 2, 33), (256, 6, 64)])
@pytest.mark.parametrize("max_context", [1, 300])  # one workgroup an item, and in pieces
def test_infinities_in_any_tile(D, G, page, dtype, max_context):
    p = Problem([300, 40], [3, 2], 2, G, D, page, dtype, seed=D + G, q_scale=1.0)
    clean, clean_lse = p.check(max_context=max_context)
    want = clean.clone()
    # token, dimension and value of kv head 1 of the first sequence
    for j, d, value in ((0, 0, INF), (20, 1, -INF), (63, 2, INF), (64, D - 1, INF), (128, 17, NAN), (200, 33, -INF),
                        (5, 40, INF), (250, 40, INF), (7, 41, INF), (130, 41, -INF)):
        pg, at = place(p, 0, j, page)
        p.vc[pg, 1, at, d] = value
        want[:3, G:, d] = NAN if d == 41 else value
    out, lse = p.run(max_context=max_context)
    assert torch.equal(lse, clean_lse)
    same(out, want)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_infinities_inside_and_behind_a_window(value, dtype):
    """Only the rows whose window or sinks hold the token change."""
    page, G = 16, 2
    p = Problem([400], [4], 2, G, 64, page, dtype, seed=2, q_scale=1.0)
    window, sinks = 150, 3  # row r stands at 396 + r and sees from 247 + r on
    clean, clean_lse = p.check(window, sinks)
    want = clean.clone()
    for j, h, d in ((1, 0, 3), (100, 0, 4), (246, 1, 5), (248, 1, 6), (249, 0, 7), (300, 1, 8)):
        pg, at = place(p, 0, j, page)
        p.vc[pg, h, at, d] = value
        for r in range(4):
            if j < sinks or j >= 247 + r:
                want[r, h * G:(h + 1) * G, d] = value
    out, lse = p.run(window, sinks)
    assert torch.equal(lse, clean_lse)
    same(out, want)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("max_context", [1, 2000])
def test_weights_near_zero_of_an_infinite_value(dtype, max_context):
    """An infinity whose weight is far below the type's smallest number is still one."""
    p = Problem([2000], [1], 1, 4, 128, 16, dtype, seed=3, q_scale=0.0)
    p.q[..., 0] = 1.0
    p.kc[..., 0] = 0.0
    pg, at = place(p, 0, 1500, 16)
    p.kc[pg, 0, at, 0] = 40.0   # weights of the others: e^-40
    clean, _ = p.check(scale=1.0, max_context=max_context)
    pg, at = place(p, 0, 70, 16)
    p.vc[pg, 0, at, 9] = INF
    want = clean.clone()
    want[..., 9] = INF
    out, _ = p.run(scale=1.0, max_context=max_context)
    same(out, want)


@pytest.mark.parametrize("max_context", [1, 300])
def test_keys_that_are_not_finite(max_context):
    """NaN in a key of an early token: all of the head's rows, and no other head's."""
    p = Problem([300, 200], [2, 1], 2, 3, 128, 16, BF16, seed=4)
    clean, clean_lse = p.check(max_context=max_context)
    pg, at = place(p, 0, 30, 16)
    p.kc[pg, 1, at, 11] = NAN
    out, lse = p.run(max_context=max_context)
    want, want_lse = clean.clone(), clean_lse.clone()
    want[:2, 3:], want_lse[:2, 3:] = NAN, NAN
    same(out, want)
    same(lse, want_lse)


def test_infinities_in_runs_of_many_items():
    """Workgroups that go on to further items after one with an infinity; the
    others' outputs are bitwise what they were."""
    g = torch.Generator().manual_seed(6)
    lens = torch.randint(200, 400, (70,), generator=g).tolist()
    p = Problem(lens, [1] * 70, 4, 2, 128, 16, BF16, seed=5, q_scale=1.0)
    clean, clean_lse = p.run(max_context=400)
    want = clean.clone()
    for b in range(0, 70, 3):
        h, d = b % 4, (7 * b) % 128
        pg, at = place(p, b, (11 * b) % 190, 16)
        p.vc[pg, h, at, d] = -INF if b % 2 else INF
        want[b, 2 * h:2 * h + 2, d] = -INF if b % 2 else INF
    out, lse = p.run(max_context=400)
    assert torch.equal(lse, clean_lse)
    same(out, want)


@pytest.mark.parametrize("max_context", [1, 300])
def test_scores_that_are_all_minus_infinity(max_context):
    """A row whose every score is -infinity is as one that sees nothing; one finite score is enough."""
    p = Problem([300, 200], [1, 1], 2, 2, 128, 16, BF16, seed=8)
    p.q[:] = p.q.abs() + 0.5
    p.kc[torch.isfinite(p.kc)] = 1.0
    clean, clean_lse = p.run(max_context=max_context)
    for j in range(300):
        pg, at = place(p, 0, j, 16)
        p.kc[pg, 0, at, 3] = -INF
    out, lse = p.run(max_context=max_context)
    want, want_lse = clean.clone(), clean_lse.clone()
    want[0, :2], want_lse[0, :2] = 0.0, -INF
    same(out, want)
    same(lse, want_lse)
    pg, at = place(p, 0, 77, 16)
    p.kc[pg, 0, at, 3] = 1.0
    out, lse = p.run(max_context=max_context)
    v = p.vc[pg, 0, at].to(out.device)
    assert torch.equal(out[0, 0], v) and torch.equal(out[0, 1], v) and torch.isfinite(lse[0]).all()
