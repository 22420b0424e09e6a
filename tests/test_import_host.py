"""The package without the step operators' compiled part: the products load and
work as before, the step operators say what is missing (no GPU needed)."""
import shutil
import subprocess
import sys
from pathlib import Path

import pytest

import affine_group_quantized_qmm_amd as qmm

PROGRAM = """
import torch
import affine_group_quantized_qmm_amd as qmm
assert qmm.__file__.startswith({root!r}), qmm.__file__
assert qmm.qmm_kernel_name(1, 512, 512, 4, 32) and qmm.qmm_strerror(0) == "success"
assert qmm.qmm_sample_workspace_bytes(1, 1000) > 0  # the C library has them all
try:
    qmm.qmm_forward(torch.zeros(1, 64).half(), torch.zeros(8, 8, dtype=torch.int32), torch.zeros(8, 2).half(),
                    torch.zeros(8, 2).half(), 4, 32)
except ValueError as e:
    assert "GPU" in str(e), e
c, i = torch.zeros(4, 2, 16, 64).half(), torch.zeros(3, dtype=torch.int32)
q = torch.zeros(3, 4, 64).half()
for call in (lambda: qmm.qmm_sample(torch.zeros(2, 10), torch.zeros(2)),
             lambda: qmm.qmm_paged_attention(q, c, c, i[None], i[:1], i[:2], 3, 10),
             lambda: qmm.qmm_qk_norm_rope(q, q[:, :2], q[:, :2], torch.ones(64), torch.ones(64), i, None, i, c, c)):
    try:
        call()
    except ImportError as e:
        assert "_qmm_torch.so" in str(e) and e.__cause__ is not None, e
    else:
        raise AssertionError("no error")
print("as wanted")
"""


@pytest.mark.parametrize("broken", [False, True])
def test_products_without_the_compiled_binding(tmp_path, broken):
    source = Path(qmm.__file__).resolve().parent
    package = tmp_path / source.name
    package.mkdir()
    shutil.copy(source / "__init__.py", package)
    (package / "libqmm.so").symlink_to(source / "libqmm.so")
    if broken:  # as one that was built against another torch does not load
        (package / "_qmm_torch.so").write_text("not a library")
    r = subprocess.run([sys.executable, "-c", PROGRAM.format(root=str(tmp_path))], cwd=tmp_path, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "as wanted" in r.stdout, r.stderr[-2000:]
