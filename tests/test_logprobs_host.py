"""Host-side checks of qmm_logprobs: refusals with the documented codes before any
launch (no GPU needed), the binding's own, and the plain form."""
import numpy as np
import pytest
import torch

import affine_group_quantized_qmm_amd as qmm
from tests import _logprobs

A = 0x10000
LIB = qmm._lib


def call(**kw):
    a = dict(x=A, stride=100000, type=2, tok=A, lp=A, rank=None, ent=None, n=5, tt=A, tl=A, M=3, V=100000, ws=A, wsb=1 << 40)
    a.update(kw)
    return LIB.qmm_logprobs(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(tok=None), -1), (dict(lp=None), -1), (dict(tt=None), -1), (dict(tl=None), -1),
    (dict(ws=None), -1), (dict(type=3), -11), (dict(type=-1), -11),
    (dict(M=0), -2), (dict(V=0), -2), (dict(V=(1 << 23) + 1, stride=1 << 24), -2), (dict(n=-1), -2), (dict(n=65), -2),
    (dict(stride=99999), -2), (dict(M=1 << 24, V=10, stride=10), -2), (dict(M=(1 << 31) - 1, V=10, stride=10), -2),
    (dict(M=1 << 20, V=1 << 22, stride=1 << 22), -2),
    (dict(wsb=100), -6),
    (dict(x=A + 2), -7), (dict(x=A + 1, type=0), -7), (dict(tok=A + 2), -7), (dict(lp=A + 1), -7), (dict(rank=A + 2), -7),
    (dict(ent=A + 2), -7), (dict(tt=A + 2), -7), (dict(tl=A + 3), -7), (dict(ws=A + 8), -7),
])
def test_refuses(kw, code):
    assert call(**kw) == code


def test_workspace():
    f = qmm.qmm_logprobs_workspace_bytes
    assert f(1, 1000, 5) == 0  # one slice
    assert f(1, 100000, 5) > f(1, 100000, 0) > 0
    assert f(0, 100, 5) == 0 and f(1, 0, 5) == 0 and f(1, 100000, 65) == 0 and f(1, (1 << 23) + 1, 1) == 0


def test_binding_refuses():
    with pytest.raises(ValueError):  # not on the GPU
        qmm.qmm_logprobs(torch.zeros(2, 10), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        qmm.qmm_logprobs(torch.zeros(10), torch.zeros(1, dtype=torch.int32))


def test_plain_form():
    x = np.array([1.0, 3.0, 3.0, -np.inf, np.nan, 2.0])
    lp, rank, ent, top, tlp = _logprobs.reference(x, 2, 6)
    p = np.exp([1, 3, 3, 2.0]) / np.exp([1, 3, 3, 2.0]).sum()
    assert rank == 1 and abs(lp - np.log(p[2])) < 1e-14 and abs(ent + (p * np.log(p)).sum()) < 1e-14
    assert top.tolist() == [1, 2, 5, 0, -1, -1] and np.isinf(tlp[4:]).all() and abs(np.exp(tlp).sum() - 1) < 1e-14
    assert _logprobs.reference(x, 4, 0)[:2] == (-np.inf, 5) and _logprobs.reference(x, 6, 0)[1] == -1
