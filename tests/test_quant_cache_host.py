"""Host-side checks of the quantized cache's operators: refusals with the
documented codes before any launch (no GPU needed), the binding's own, and the
plain forms that the GPU tests compare with."""
import numpy as np
import pytest
import torch

import affine_group_quantized_qmm_amd as qmm
from tests import _quant

A = 0x10000  # a fake, 16-byte aligned address: checks never dereference it
LIB = qmm._lib


def rope(**kw):
    a = dict(q=A, k=A, v=A, qs=512, ks=128, vs=128, tin=2, qw=A, kw=A, eps=1e-6, off=0.0, pos=A, f=A, R=64, inter=0,
             slots=A, out=A, kc=A, ksb=A, vc=A, vsb=A, tout=1, M=3, Hq=4, Hkv=1, D=128, bits=8, G=64, pages=4, ps=16)
    a.update(kw)
    return LIB.qmm_qk_norm_rope_quant(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(kc=None), -1), (dict(ksb=None), -1), (dict(vc=None), -1), (dict(vsb=None), -1),
    (dict(f=None), -1), (dict(slots=None), -1), (dict(out=None), -1),
    (dict(M=0), -2), (dict(M=1 << 24), -2), (dict(Hq=0), -2), (dict(pages=0), -2), (dict(ps=0), -2),
    (dict(pages=1 << 20, ps=1 << 11), -2), (dict(qs=504), -2), (dict(ks=120), -2),
    (dict(tin=3), -11), (dict(tout=2), -11),
    (dict(bits=0), -3), (dict(bits=6), -3), (dict(bits=16), -3), (dict(G=0), -4), (dict(G=16), -4), (dict(G=256), -4),
    (dict(D=96), -12), (dict(D=264), -12), (dict(D=0), -12), (dict(R=136), -12), (dict(G=128, D=64, R=32), -12),
    (dict(q=A + 8), -7), (dict(kc=A + 8), -7), (dict(vc=A + 4), -7), (dict(ksb=A + 2), -7), (dict(vsb=A + 1), -7),
    (dict(qs=516), -7),
])
def test_rope_refuses(kw, code):
    assert rope(**kw) == code


def read(**kw):
    a = dict(kc=A, ksb=A, vc=A, vsb=A, slots=A, ko=A, vo=A, tout=0, M=3, Hkv=2, D=128, bits=4, G=32, pages=4, ps=16)
    a.update(kw)
    return LIB.qmm_quant_cache_read(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(kc=None), -1), (dict(ksb=None), -1), (dict(vc=None), -1), (dict(vsb=None), -1), (dict(slots=None), -1),
    (dict(ko=None), -1), (dict(vo=None), -1), (dict(tout=2), -11), (dict(tout=-1), -11),
    (dict(M=0), -2), (dict(M=-1), -2), (dict(Hkv=0), -2), (dict(Hkv=1 << 17), -2), (dict(ps=0), -2),
    (dict(pages=1 << 20, ps=1 << 11), -2), (dict(M=1 << 24), -2), (dict(M=1 << 20, Hkv=128, D=256), -2),
    (dict(bits=2), -3), (dict(G=48), -4), (dict(D=80), -12), (dict(D=512), -12), (dict(D=0), -12),
    (dict(kc=A + 8), -7), (dict(vo=A + 8), -7), (dict(ksb=A + 2), -7), (dict(slots=A + 2), -7),
])
def test_read_refuses(kw, code):
    assert read(**kw) == code


def attn(**kw):
    a = dict(q=A, qs=512, kc=A, ksb=A, vc=A, vsb=A, type=1, table=A, lens=A, starts=A, out=A, lse=None, T=4, B=2, Hq=4,
             Hkv=2, D=128, bits=8, G=64, pages=100, ps=16, max_pages=50, max_rows=2, max_ctx=800, scale=0.1, window=0,
             sinks=0, ws=A, wsb=1 << 40)
    a.update(kw)
    return LIB.qmm_paged_attention_quant(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(kc=None), -1), (dict(ksb=None), -1), (dict(vc=None), -1), (dict(vsb=None), -1),
    (dict(table=None), -1), (dict(lens=None), -1), (dict(starts=None), -1), (dict(out=None), -1),
    (dict(ws=None, max_ctx=100000), -1),
    (dict(T=0), -2), (dict(B=0), -2), (dict(max_rows=5), -2), (dict(max_ctx=-1), -2), (dict(window=-1), -2),
    (dict(pages=0), -2), (dict(max_pages=0), -2), (dict(qs=504), -2), (dict(scale=float("nan")), -2),
    (dict(max_pages=1 << 28), -2), (dict(ps=1, max_pages=(1 << 31) - 512), -2), (dict(pages=1 << 27), -2),
    (dict(type=2), -11), (dict(Hq=5, qs=640), -12), (dict(D=160, qs=640, G=32), -12), (dict(D=32, qs=128, G=32), -12),
    (dict(D=96, qs=384), -12), (dict(bits=5), -3), (dict(G=16), -4),
    (dict(wsb=16, max_ctx=100000), -6),
    (dict(q=A + 2), -7), (dict(kc=A + 8), -7), (dict(vsb=A + 2), -7), (dict(ws=A + 4, max_ctx=100000), -7),
    (dict(lse=A + 1), -7), (dict(qs=516), -7),
])
def test_attention_refuses(kw, code):
    assert attn(**kw) == code


def test_attention_workspace():
    f = qmm.qmm_paged_attention_quant_workspace_bytes
    assert f(4, 2, 4, 2, 128, 2, 64, 0, 0, 8, 64) == 0
    big = f(4, 2, 4, 2, 128, 2, 100000, 0, 0, 8, 64)
    assert big > 0 and f(4, 2, 4, 2, 128, 2, 10 ** 7, 0, 0, 8, 64) == big
    assert f(4, 2, 4, 2, 128, 2, 100000, 0, 0, 5, 64) == 0 and f(4, 2, 4, 2, 128, 2, 100000, 0, 0, 8, 48) == 0
    assert f(4, 2, 4, 2, 96, 2, 100000, 0, 0, 8, 64) == 0


def test_binding_refuses():
    """Shapes, types and devices, before the library is called."""
    c = torch.zeros(4, 2, 16, 16, dtype=torch.int32)
    w = torch.zeros(4, 2, 16, 1, dtype=torch.int32)
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):  # not on the GPU
        qmm.qmm_quant_cache_read(c, w, c, w, 8, 64, i)
    with pytest.raises(ValueError):
        qmm.qmm_qk_norm_rope_quant(q, q[:, :2], q[:, :2], torch.ones(64), torch.ones(64), i, None, i, c, w, c, w, 8, 64)
    with pytest.raises(ValueError):
        qmm.qmm_paged_attention_quant(q, c, w, c, w, 8, 64, torch.zeros(1, 4, dtype=torch.int32), i[:1], i[:2], 3, 10)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("scale", [1.0, 1e-6, 3e4])
def test_plain_form(bits, scale):
    """Every value lies between two levels, within half a step of the nearest, and
    words go back to the codes that they were made of."""
    y = np.random.default_rng(bits).standard_normal((5, 128)) * scale
    y[1] = 0
    y[2] = y[2, 0]
    y[3] = np.abs(y[3]) + 1
    codes, s, b, place = _quant.quantize(y, bits, 32)
    levels = 2 ** bits - 1
    assert (place >= 0).all() and (place <= levels).all()
    step = np.repeat(s, 32, -1)
    got = codes * step + np.repeat(b, 32, -1)
    assert (np.abs(got - np.clip(y, -_quant.MOST, _quant.MOST)) <= step / 2 * (1 + 1e-12)).all()
    words, sb = _quant.pack(codes, s, b, bits)
    c2, s2, b2 = _quant.unpack(words, sb, bits, 32)
    assert (c2 == codes).all() and (s2 == s).all() and (b2 == b).all()
    assert np.isfinite(_quant.numbers(words, sb, bits, 32)).all()
