"""Plain forms of the quantized cache (numpy, nothing shared with the kernels),
and problems for the tests that use it."""
from __future__ import annotations

import numpy as np
import torch

from tests import _gpu, _step

MOST = 65280.0
# every finite fp16 number in rising order
HALVES = np.sort(np.unique(np.arange(65536, dtype=np.uint16).view(np.float16)[
    np.isfinite(np.arange(65536, dtype=np.uint16).view(np.float16))].astype(np.float64)))


def quantize(y, bits, G):
    """(codes, scales, biases, place of y between the levels) of y [..., D] in 64 bits."""
    g = np.clip(y, -MOST, MOST).reshape(*y.shape[:-1], -1, G)
    lo, hi = g.min(-1), g.max(-1)
    levels = 2 ** bits - 1
    with np.errstate(invalid="ignore"):
        b = HALVES[np.clip(np.searchsorted(HALVES, lo, side="right") - 1, 0, None)]
        s = HALVES[np.clip(np.searchsorted(HALVES, (hi - b) / levels), 0, len(HALVES) - 1)]
        place = np.where(s[..., None] > 0, (g - b[..., None]) / np.where(s > 0, s, 1)[..., None], 0.0)
        codes = np.clip(np.rint(np.nan_to_num(place)), 0, levels).astype(np.uint32)
    odd = np.isnan(g).any(-1)
    s, b = np.where(odd, np.nan, s), np.where(odd, 0, b)
    codes[odd] = 0
    return codes.reshape(y.shape), s, b, place.reshape(y.shape)


def pack(codes, s, b, bits):
    """int32 words of codes [..., D] and of (scale, bias) pairs."""
    per = 32 // bits
    c = codes.reshape(*codes.shape[:-1], -1, per).astype(np.uint32)
    words = np.zeros(c.shape[:-1], np.uint32)
    for i in range(per):
        words |= c[..., i] << np.uint32(i * bits)
    with np.errstate(over="ignore"):
        sb = (np.asarray(s, np.float16).view(np.uint16).astype(np.uint32)
              | np.asarray(b, np.float16).view(np.uint16).astype(np.uint32) << np.uint32(16))
    return torch.from_numpy(words.view(np.int32)), torch.from_numpy(sb.view(np.int32))


def unpack(words, sb, bits, G):
    """(codes, scales, biases) of int32 words."""
    w, p = words.cpu().numpy().view(np.uint32), sb.cpu().numpy().view(np.uint32)
    codes = np.stack([w >> np.uint32(i * bits) & np.uint32(2 ** bits - 1) for i in range(32 // bits)], -1)
    s = (p & np.uint32(0xFFFF)).astype(np.uint16).view(np.float16).astype(np.float64)
    b = (p >> np.uint32(16)).astype(np.uint16).view(np.float16).astype(np.float64)
    return codes.reshape(*w.shape[:-1], -1), s, b


def numbers(words, sb, bits, G):
    """What the codes stand for, in 64 bits: scale * code + bias has at most 11 + 8
    bits beside the bias's 11, exact in 64, and is rounded to fp16 once."""
    codes, s, b = unpack(words, sb, bits, G)
    with np.errstate(over="ignore", invalid="ignore"):
        return (codes * np.repeat(s, G, -1) + np.repeat(b, G, -1)).astype(np.float16).astype(np.float64)


class Problem:
    """Sequences of given lengths and row counts over a shuffled quantized pool.
    Every place of the cache that holds no token stands for NaN, and table entries
    past a sequence's pages are out of range."""

    def __init__(self, lens, rows, Hkv, group, D, page, dtype, bits, G, seed=0, q_scale=2.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.rows, self.bits, self.G = lens, rows, bits, G
        need = [-(-L // page) for L in lens]
        total = sum(need) + 2
        perm = torch.randperm(total, generator=g).tolist()
        width = max(1, max(need) + 1)
        self.table = torch.full((len(lens), width), -1, dtype=torch.int32)
        self.table[:, -1] = total + 5
        y = np.full((2, total, Hkv, page, D), np.nan)
        for b, L in enumerate(lens):
            for i in range(need[b]):
                pg = perm.pop()
                self.table[b, i] = pg
                n = min(page, L - i * page)
                y[:, pg, :, :n] = torch.randn(2, Hkv, n, D, generator=g).numpy()
        self.caches = [t for c in y for t in pack(*quantize(c, bits, G)[:3], bits)]
        self.starts = torch.tensor([0] + list(np.cumsum(rows)), dtype=torch.int32)
        T = int(self.starts[-1])
        self.q = (torch.randn(T, Hkv * group, D, generator=g) * q_scale).to(dtype)
        self.dtype, self.D = dtype, D

    def values(self):
        k, kw, v, vw = self.caches
        return numbers(k, kw, self.bits, self.G), numbers(v, vw, self.bits, self.G)

    def run(self, window=0, sinks=0, scale=None, max_context=None, max_rows=None, q=None):
        qmm, dev = _gpu.lib(), _gpu.dev()
        q = self.q.to(dev) if q is None else q
        T, Hq, _ = q.shape
        out = torch.full((T, Hq, self.D), float("nan"), dtype=self.dtype, device=dev)
        lse = torch.full((T, Hq), float("nan"), device=dev)
        qmm.qmm_paged_attention_quant(q, *(t.to(dev) for t in self.caches), self.bits, self.G, self.table.to(dev),
                                      torch.tensor(self.lens, dtype=torch.int32, device=dev), self.starts.to(dev),
                                      max_rows or max(1, max(self.rows)),
                                      max(self.lens) if max_context is None else max_context, scale=scale,
                                      window=window, sinks=sinks, out=out, lse=lse)
        torch.cuda.synchronize()
        return out, lse

    def check(self, window=0, sinks=0, scale=None, **kw):
        """Against the 64-bit form over the codes' numbers. A weight is one fp16
        number, off by at most half a step of 2^-11 of itself: that moves the output by
        at most 2^-11 of the weighted mean of the magnitudes, in the place of the 2^-22
        of a weight in two parts (which the reference's bound has)."""
        out, lse = self.run(window, sinks, scale, **kw)
        args = (_step.f64(self.q), *self.values(), self.table.numpy(), self.lens, self.starts.tolist(),
                self.D ** -0.5 if scale is None else scale, window, sinks, torch.float16)
        (ro, ob), (rl, lb), held = _step.attention_reference(*args)
        k, v = args[1:3]
        with np.errstate(invalid="ignore"):
            (mass, _), _, _ = _step.attention_reference(args[0], k, np.abs(v), *args[3:])
        ob = ob + mass * 2.0 ** -11
        assert held.all()
        _step.assert_rounded(out, ro, ob, "out")
        _step.assert_rounded(lse, rl, lb, "lse")
        return out, lse
