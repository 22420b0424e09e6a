"""Host-side checks of qmm_lora: refusals with the documented codes before any
launch (no GPU needed), and the binding's own."""
import ctypes

import pytest
import torch

import affine_group_quantized_qmm_amd as qmm

A = 0x10000
LIB = qmm._lib


def call(count=2, a=(A, A), b=(A, A), y=(A, A), N=(64, 33), arrays=True, **kw):
    k = dict(x=A, type=0, ids=A, scales=None, M=20, K=512, r=16, adapters=3, ws=A, wsb=1 << 40)
    k.update(kw)

    def ptrs(v):
        return (ctypes.c_void_p * len(v))(*v) if arrays else None
    return LIB.qmm_lora(k["x"], k["type"], count, ptrs(a), ptrs(b), ptrs(y), (ctypes.c_int * len(N))(*N), k["ids"],
                        k["scales"], k["M"], k["K"], k["r"], k["adapters"], k["ws"], k["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(arrays=False), -1), (dict(a=(A, None)), -1), (dict(b=(None, A)), -1), (dict(y=(A, None)), -1),
    (dict(ids=None), -1), (dict(ws=None), -1), (dict(type=2), -11), (dict(type=-1), -11),
    (dict(count=0), -2), (dict(count=5, a=(A,) * 5, b=(A,) * 5, y=(A,) * 5, N=(8,) * 5), -2), (dict(count=-1), -2),
    (dict(M=0), -2), (dict(M=65535 * 16 + 1), -2), (dict(K=0), -2), (dict(K=48), -2), (dict(K=(1 << 28) + 32), -2),
    (dict(r=0), -2), (dict(r=4), -2), (dict(r=12), -2), (dict(r=136), -2), (dict(adapters=0), -2), (dict(N=(64, 0)), -2),
    (dict(N=(-1, 64)), -2), (dict(N=(64, (1 << 28) + 1)), -2), (dict(M=65535 * 16, N=(1 << 27, 64)), -2),
    (dict(wsb=100), -6),
    (dict(x=A + 8), -7), (dict(a=(A, A + 8)), -7), (dict(b=(A + 2, A)), -7), (dict(y=(A, A + 4)), -7), (dict(ids=A + 2), -7),
    (dict(scales=A + 2), -7), (dict(ws=A + 8), -7),
    # outputs that overlap: the same one twice, the second's first value in the first's last row
    (dict(), -2), (dict(y=(A, A + 20 * 64 * 4 - 16)), -2), (dict(y=(A + 20 * 33 * 4 - 16, A)), -2),
])
def test_refuses(kw, code):
    assert call(**kw) == code


def test_workspace():
    f = qmm.qmm_lora_workspace_bytes
    assert f([64], 1, 512, 16, 3) == 16 * 4
    assert f([64, 64], 1, 512, 16, 3) == 2 * 16 * 4
    assert f([64], 20, 5120, 16, 3) % (20 * 16 * 4) == 0
    assert f([64], 0, 512, 16, 3) == 0 and f([64], 1, 512, 12, 3) == 0 and f([0], 1, 512, 16, 3) == 0


def test_binding_refuses():
    x = torch.zeros(2, 64, dtype=torch.float16)
    a, b, y = torch.zeros(3, 8, 64).half(), torch.zeros(3, 5, 8).half(), torch.zeros(2, 5)
    ids = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):  # not on the GPU
        qmm.qmm_lora(x, [(a, b)], ids, [y])
    with pytest.raises(ValueError):
        qmm.qmm_lora(x[0], [(a, b)], ids, [y])
