"""Plain 64-bit forms of the operators between the products (numpy, loops over
rows and tokens, nothing shared with the kernels), and the tolerances of the
tests that use them."""
from __future__ import annotations

import math

import numpy as np
import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
# half a step among the subnormals (absolute)
HALF_STEP_LOW = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


# ---------------------------------------------------------------------------
# q/k norm, rotation, append
# ---------------------------------------------------------------------------
def rope_head(x, w, pos, inv_freq, eps, offset, interleaved):
    """One head's D values: (result, bound of what 32-bit arithmetic may add)."""
    D, R = x.shape[0], 2 * len(inv_freq)
    n = x / math.sqrt(np.mean(x * x) + eps) * (offset + w)
    y, mag = n.copy(), np.abs(n)
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, R // 2 + i)
        angle = float(pos) * float(inv_freq[i])
        co, si = math.cos(angle), math.sin(angle)
        y[a], y[b] = n[a] * co - n[b] * si, n[b] * co + n[a] * si
        mag[a] = mag[b] = abs(n[a]) + abs(n[b])
    # Norm: D additions in lanes and a tree (D/8 + 8 roundings at most, halved by
    # the root), the root, two products, 1/D: D/16 + 12 half steps. Rotation: the
    # angle to within 2^-26 of a turn plus sine and cosine to 4 half steps and
    # three roundings: under 2^-21 of the pair's size.
    return y, mag * ((D / 16 + 12) * 2.0 ** -24 + 2.0 ** -21)


def rope_reference(q, k, v, qw, kw, positions, inv_freq, slots, k_cache, v_cache, eps, offset, interleaved):
    """(q_out, k_cache, v_cache) in 64 bits and their 32-bit bounds, from numpy arrays."""
    M = q.shape[0]
    qo, qb = np.zeros_like(q), np.zeros_like(q)
    kc, vc = k_cache.copy(), v_cache.copy()
    kb, vb = np.zeros_like(kc), np.zeros_like(vc)
    pages, _, ps, _ = kc.shape
    for m in range(M):
        for h in range(q.shape[1]):
            qo[m, h], qb[m, h] = rope_head(q[m, h], qw, positions[m], inv_freq, eps, offset, interleaved)
        if 0 <= slots[m] < pages * ps:
            p, o = divmod(int(slots[m]), ps)
            for h in range(k.shape[1]):
                kc[p, h, o], kb[p, h, o] = rope_head(k[m, h], kw, positions[m], inv_freq, eps, offset, interleaved)
                vc[p, h, o] = v[m, h]
    return (qo, qb), (kc, kb), (vc, vb)


def assert_rounded(got: torch.Tensor, ref: np.ndarray, bound: np.ndarray, what: str):
    """|got - ref| <= bound + half a step of got's type (relative, or absolute
    among its subnormals); equal where the reference is not finite."""
    g = f64(got)
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(g), np.isnan(ref)), f"{what}: NaN in other places"
    assert np.array_equal(g[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)]), f"{what}: infinities differ"
    step = HALF_STEP[got.dtype]
    tol = bound * (1 + step) + np.maximum(np.abs(ref) * step, HALF_STEP_LOW[got.dtype])
    with np.errstate(invalid="ignore"):
        bad = fine & ~(np.abs(g - ref) <= tol)
    if bad.any():
        i = np.unravel_index(int(np.argmax(np.where(bad, np.abs(g - ref) / tol, 0))), bad.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; worst at {i}: got {g[i]!r} "
                             f"want {ref[i]!r} tolerance {tol[i]:.3g}")


# ---------------------------------------------------------------------------
# attention over the paged cache
# ---------------------------------------------------------------------------
def visible_tokens(p, window, sinks):
    return [j for j in range(p + 1) if window == 0 or j > p - window or j < sinks]


def attention_reference(q, k_cache, v_cache, table, lens, starts, scale, window, sinks, dtype):
    """(out, bound), (lse, bound), rows that a sequence holds."""
    T, Hq, D = q.shape
    pages, Hkv, ps, _ = k_cache.shape
    G = Hq // Hkv
    out, ob = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, lb = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    held = np.zeros(T, bool)
    split = HALF_STEP[dtype] ** 2  # e^s as a rounding and the rounded rest
    low = HALF_STEP_LOW[dtype]
    for b, L in enumerate(lens):
        n = starts[b + 1] - starts[b]
        for r in range(n):
            t = starts[b] + r
            held[t] = True
            rows = []
            for j in visible_tokens(L - n + r, window, sinks):
                if j // ps < table.shape[1] and 0 <= table[b, j // ps] < pages:
                    rows.append((table[b, j // ps], j % ps))
            if not rows:
                continue
            pg, of = np.array([x[0] for x in rows]), np.array([x[1] for x in rows])
            for h in range(Hq):
                k, v = k_cache[pg, h // G, of], v_cache[pg, h // G, of]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = (k @ q[t, h]) * scale
                    m = s.max()
                    p = np.exp(s - m)
                    w = p / p.sum()
                    out[t, h] = w @ v
                    lse[t, h] = m + math.log(p.sum()) if np.isfinite(m) else m
                    # Relative error of an e^s: D additions of the score's
                    # products, the scale and the maximum (three roundings of
                    # numbers up to |s|), the exponential (two steps). Sums over
                    # the tokens: n additions. Both for numerator and sum.
                    ds = (D + 2) * 2.0 ** -24 * (np.abs(k) @ np.abs(q[t, h])).max() * abs(scale) * 1.01
                    e = ds + 4 * 2.0 ** -24 * 1.45 * np.abs(s).max() + 2.0 ** -21 + len(rows) * 2.0 ** -24
                    mass = w @ np.abs(v)
                    ob[t, h] = mass * (2 * e + split) + len(rows) * low * np.abs(v).max() / 1.0
                    lb[t, h] = e + abs(lse[t, h]) * 2.0 ** -22 + 2.0 ** -22
    return (out, ob), (lse, lb), held


# ---------------------------------------------------------------------------
# sampling
# ---------------------------------------------------------------------------
def sample_reference(x, u, T, k, p, min_p):
    """(token, log probability, distance of u to the nearest border as a share of
    the kept mass) of one row in 64 bits."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    order = np.argsort(-x, kind="stable")
    best = x[order[0]]
    if best == -np.inf:
        return -1, -math.inf, 1.0
    if T <= 0:
        return int(order[0]), 0.0, 1.0
    with np.errstate(invalid="ignore"):
        d = np.where(x[order] == best, 0.0, x[order] - best) / T
    w = np.exp(d)
    if k > 0:
        w = w[:k]
    cum = np.cumsum(w)
    margin = 1.0
    if p < 1:
        before = cum - w
        margin = min(margin, float(np.abs(before[1:] - p * cum[-1]).min() / cum[-1]) if len(w) > 1 else 1.0)
        n = max(1, int((before < p * cum[-1]).sum()))
        w = w[:n]
    n = max(1, int((w >= min_p).sum()))
    w = w[:n]
    cum = np.cumsum(w)
    r = u * cum[-1]
    at = min(int((cum <= r).sum()), len(w) - 1)
    while w[at] == 0:
        at -= 1
    inner = cum[:-1][w[1:] > 0] if len(w) > 1 else cum[:0]
    margin = min(margin, float(np.abs(inner - r).min() / cum[-1]) if inner.size else 1.0)
    return int(order[at]), math.log(w[at] / cum[-1]), margin
