"""The plain 64-bit form of qmm_logprobs, one row at a time."""
import math

import numpy as np


def reference(x, token, n):
    """(logprob, rank, entropy, top tokens, top logprobs) of the row x."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    V, m = len(x), x.max()
    order = np.argsort(-x, kind="stable")
    if m == -np.inf:
        logp, entropy = np.full(V, -np.inf), 0.0
    elif m == np.inf:
        count = int((x == np.inf).sum())
        logp, entropy = np.where(x == np.inf, -math.log(count), -np.inf), math.log(count)
    else:
        logp = x - m - math.log(np.exp(x - m).sum())
        p = np.exp(logp)
        entropy = float(-(p[p > 0] * logp[p > 0]).sum())
    known = 0 <= token < V
    best = [int(j) for j in order[:n] if x[j] > -np.inf]
    fill = n - len(best)
    return (logp[token] if known else -np.inf, int(np.nonzero(order == token)[0][0]) if known else -1, entropy,
            np.array(best + [-1] * fill), np.array([logp[j] for j in best] + [-np.inf] * fill))


def bounds(x, V):
    """What fp32 may add to (a log probability, the entropy) of the row x.

    A term e^d: d is rounded once (relative 2^-24), d log2(e) once more, the
    exponential to 2^-23: 2 |d| 2^-24 + 2^-23 of the term. A thread adds up to 32 of
    them: 32 * 2^-24. Terms weigh by e^d, under which |d| e^d <= e^-1. The rest is in
    64 bits. A logarithm takes S's relative error absolutely; the entropy those of S
    and T, and T / S. Results are rounded to fp32 once, besides."""
    finite = x[np.isfinite(x)].astype(np.float64)
    if not len(finite):
        return 2.0 ** -40, 2.0 ** -40
    d = finite - finite.max()
    e = np.exp(d)
    S = e.sum()
    term = 2 * np.abs(d) * 2.0 ** -24 + 2.0 ** -23 + 32 * 2.0 ** -24
    rel_s = float((e * term).sum() / S)
    err_t = float((e * np.abs(d) * (term + 2.0 ** -23)).sum() / S)
    return rel_s + 2.0 ** -40, rel_s + err_t + rel_s * float((e * np.abs(d)).sum() / S) + 2.0 ** -40
