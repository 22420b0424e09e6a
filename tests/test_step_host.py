"""Host-side checks of the operators between the products: refusals with the
documented codes before any launch (no GPU needed), and the binding's own."""
import pytest
import torch

import affine_group_quantized_qmm_amd as qmm

A = 0x10000  # a fake, 16-byte aligned address: checks never dereference it
LIB = qmm._lib


def rope(**kw):
    a = dict(q=A, k=A, v=A, qs=512, ks=128, vs=128, tin=2, qw=A, kw=A, eps=1e-6, off=0.0, pos=A, f=A, R=64, inter=0,
             slots=A, out=A, kc=A, vc=A, tout=1, M=3, Hq=4, Hkv=1, D=128, pages=4, ps=16)
    a.update(kw)
    return LIB.qmm_qk_norm_rope(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(qw=None), -1), (dict(kw=None), -1),
    (dict(pos=None), -1), (dict(f=None), -1), (dict(slots=None), -1), (dict(out=None), -1), (dict(kc=None), -1),
    (dict(vc=None), -1),
    (dict(M=0), -2), (dict(Hq=0), -2), (dict(Hkv=0), -2), (dict(pages=0), -2), (dict(ps=0), -2),
    (dict(pages=1 << 20, ps=1 << 11), -2), (dict(qs=504), -2), (dict(ks=120), -2), (dict(vs=0), -2),
    (dict(pages=1 << 19, ps=1 << 11, Hkv=8, ks=1024, vs=1024), -2),
    (dict(tin=3), -11), (dict(tin=-1), -11), (dict(tout=2), -11),
    (dict(D=0), -12), (dict(D=132), -12), (dict(D=264), -12), (dict(R=136), -12), (dict(R=12), -12), (dict(R=-8), -12),
    (dict(q=A + 8), -7), (dict(kc=A + 2), -7), (dict(out=A + 4), -7), (dict(f=A + 4), -7), (dict(pos=A + 2), -7),
    (dict(qs=516), -7), (dict(vs=130), -7),
])
def test_rope_refuses(kw, code):
    assert rope(**kw) == code


def attn(**kw):
    a = dict(q=A, qs=512, kc=A, vc=A, type=1, table=A, lens=A, starts=A, out=A, lse=None, T=4, B=2, Hq=4, Hkv=2, D=128,
             pages=100, ps=16, max_pages=50, max_rows=2, max_ctx=800, scale=0.1, window=0, sinks=0, ws=A, wsb=1 << 40)
    a.update(kw)
    return LIB.qmm_paged_attention(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(kc=None), -1), (dict(vc=None), -1), (dict(table=None), -1), (dict(lens=None), -1),
    (dict(starts=None), -1), (dict(out=None), -1), (dict(ws=None, max_ctx=100000), -1),
    (dict(T=0), -2), (dict(B=0), -2), (dict(Hq=0), -2), (dict(Hkv=0), -2), (dict(max_rows=0), -2),
    (dict(max_rows=5), -2), (dict(max_ctx=-1), -2), (dict(window=-1), -2), (dict(sinks=-1), -2), (dict(pages=0), -2),
    (dict(ps=0), -2), (dict(max_pages=0), -2), (dict(qs=504), -2), (dict(scale=float("nan")), -2),
    (dict(scale=float("inf")), -2), (dict(max_pages=1 << 28), -2), (dict(B=1 << 17), -2),
    (dict(pages=1 << 27), -2), (dict(pages=1 << 26, ps=31, Hkv=4), -2),
    (dict(type=2), -11), (dict(type=7), -11),
    (dict(Hq=5, qs=640), -12), (dict(D=80), -12), (dict(D=512, qs=2048), -12),
    (dict(wsb=16, max_ctx=100000), -6),
    (dict(q=A + 2), -7), (dict(kc=A + 8), -7), (dict(out=A + 8), -7), (dict(ws=A + 4, max_ctx=100000), -7),
    (dict(table=A + 2), -7), (dict(lse=A + 1), -7), (dict(qs=516), -7),
])
def test_attention_refuses(kw, code):
    assert attn(**kw) == code


def test_attention_workspace():
    f = qmm.qmm_paged_attention_workspace_bytes
    assert f(4, 2, 4, 2, 128, 2, 64) == 0          # one workgroup for each sequence and head
    big = f(4, 2, 4, 2, 128, 2, 100000)
    assert big > 0 and f(4, 2, 4, 2, 128, 2, 10 ** 7) == big  # a full GPU, however long the context
    assert f(4, 2, 4, 2, 128, 2, 100000, 256, 4) < big  # a window is short whatever the context
    assert f(4, 2, 4, 3, 128, 2, 100000) == 0 and f(0, 2, 4, 2, 128, 2, 100000) == 0


def sample(**kw):
    a = dict(x=A, stride=1000, type=2, u=A, T=None, k=None, p=None, mp=None, tok=A, lp=None, M=3, V=1000, ws=A,
             wsb=1 << 30)
    a.update(kw)
    return LIB.qmm_sample(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(u=None), -1), (dict(tok=None), -1), (dict(ws=None), -1),
    (dict(M=0), -2), (dict(M=1 << 16), -2), (dict(V=0), -2), (dict(V=(1 << 23) + 1, stride=1 << 24), -2),
    (dict(stride=999), -2), (dict(type=3), -11), (dict(wsb=100), -6),
    (dict(x=A + 2), -7), (dict(x=A + 1, type=0), -7), (dict(u=A + 2), -7), (dict(T=A + 1), -7), (dict(k=A + 2), -7),
    (dict(p=A + 3), -7), (dict(mp=A + 2), -7), (dict(tok=A + 2), -7), (dict(lp=A + 2), -7), (dict(ws=A + 8), -7),
])
def test_sample_refuses(kw, code):
    assert sample(**kw) == code


def test_sample_workspace():
    f = qmm.qmm_sample_workspace_bytes
    assert f(1, 1000) > 0 and f(2, 1000) == 2 * f(1, 1000)
    assert f(0, 1000) == 0 and f(1, 0) == 0 and f(1, (1 << 23) + 1) == 0 and f(1 << 16, 10) == 0


def test_messages():
    for code in (-11, -12):
        assert "unknown" not in qmm.qmm_strerror(code)


def test_binding_refuses():
    """Shapes, types and devices, before the library is called."""
    c = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    i = torch.zeros(3, dtype=torch.int32)
    t = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError):  # not on the GPU
        qmm.qmm_paged_attention(q, c, c, t, i[:1], i[:2], 3, 10)
    with pytest.raises(ValueError):
        qmm.qmm_paged_attention(q[0], c, c, t, i[:1], i[:2], 3, 10)
    with pytest.raises(ValueError):
        qmm.qmm_qk_norm_rope(q, q[:, :2], q[:, :2], torch.ones(64), torch.ones(64), i, None, i, c, c)
    with pytest.raises(ValueError):
        qmm.qmm_sample(torch.zeros(2, 10), torch.zeros(2))
    with pytest.raises(ValueError):
        qmm.qmm_sample(torch.zeros(10), torch.zeros(1))
    with pytest.raises(ValueError):
        qmm.qmm_qk_norm_rope(q[0], q, q, torch.ones(64), torch.ones(64), i, None, i, c, c)
