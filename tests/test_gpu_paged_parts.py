"""Items of one head of the cache that are cut over nearly every block: few rows over many keys."""
import pytest
import torch

from test_gpu_paged import Case

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,G", [(20, 1), (4, 8), (1, 33), (9, 7)])
def test_one_item_in_every_block(kda, new, G, d, dtype):
    # 20 to 63 rows over 40000 keys: 150 to 300 parts, joined one after the other
    c = Case([new], [40000], G, 1, d, 64, dtype, packed=False)
    out, lse = c.check(kda)
    again = c.attend(kda, want_lse=True)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
