"""Error texts name what a caller has to look at, for the products and for the
operators between them."""
import pytest

import affine_group_quantized_qmm_amd as qmm


@pytest.mark.parametrize("code,names", [
    (-2, ["M, K, N", "multiple of G", "between the products"]),
    (-6, ["qmm_splitk_workspace_bytes(M, N, split_k)", "*_workspace_bytes"]),
    (-7, ["x, wq, scales, biases, y and workspace", "16-byte", "per-row parameters 4", "multiples of 8"]),
    (-11, ["type"]), (-12, ["Hq", "Hkv"]),
])
def test_texts(code, names):
    text = qmm.qmm_strerror(code)
    for name in names:
        assert name in text, text
