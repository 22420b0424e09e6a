"""qmm_sample where u times the kept mass is, to the last bit of 64, the rounded
sum of the mass of several bins of the histogram, and that sum is rounded up by
one step at a later bin that has no elements. (Rows found by searching for such
coincidences, one in 2^29 of random ones.) The tokens on either side of the
border are right, another is not."""
import numpy as np
import pytest
import torch

from tests.test_gpu_sample import sample

pytestmark = pytest.mark.gpu

# twelve logits, one that 100 elements have, u, and the place before the border
ROWS = [
    ("0x1.0be2ep+2 0x1.fc2328p+1 0x1.b96c2ap+1 0x1.9b65cep+1 0x1.51783ep+1 0x1.2f9b14p+1 0x1.ee02c4p+0 0x1.7de83p+0 "
     "0x1.2a2a5cp+0 0x1.05806ep+0 0x1.92b6ccp-1 0x1.a72b7ap-2", "-0x1.bae148p-1", "0x1.72a67ep-1", 3),
    ("0x1.06117p+2 0x1.f96668p+1 0x1.de86e4p+1 0x1.b6a72cp+1 0x1.84e84p+1 0x1.5ec92ep+1 0x1.3081e4p+1 0x1.e6558cp+0 "
     "0x1.a52984p+0 0x1.4f558ap+0 0x1.b953ecp-1 0x1.6694f6p-1", "-0x1.bae148p-1", "0x1.9ecd8cp-1", 5),
    ("0x1.081cdp+2 0x1.e4e61cp+1 0x1.9b6fcap+1 0x1.7d45a8p+1 0x1.3d05cap+1 0x1.f1a34ep+0 0x1.5fbfbap+0 0x1.fd43b2p-1 "
     "0x1.2bdb88p-1 0x1.03a718p-3 -0x1.9e24c4p-2 -0x1.4a21a4p-1", "-0x1.bae148p-1", "0x1.4d1938p-1", 2),
]


@pytest.mark.parametrize("row", range(len(ROWS)))
@pytest.mark.parametrize("padding", [0, 5000, 66000])
def test_crossing_at_a_bin_without_elements(row, padding):
    few, many, u, before = ROWS[row]
    x = [float.fromhex(v) for v in few.split()]
    x = torch.tensor(x + [float.fromhex(many)] * 100 + [-1e4] * padding)
    order = torch.randperm(len(x), generator=torch.Generator().manual_seed(row))
    got, _ = sample(x[order][None], [float.fromhex(u)], k=62)  # 50 of the hundred
    assert int(order[got[0]]) in (before, before + 1)
