"""Values are copied into the cache as they are, whatever their bits mean."""
import pytest
import torch

import _paged_ref as R
from test_gpu_paged import Case, DEV, bits, freqs, rand

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,rot,layout", [(16, 16, "half"), (32, 8, "interleaved"), (64, 64, "interleaved"), (128, 64, "half"),
                                          (128, 0, "half")])
def test_values_keep_their_bits(kda, d, rot, layout, dtype):
    new, lens = [3, 1, 20], [40, 9, 20]
    c = Case(new, lens, 4, 2, d, 16, dtype)
    whole, top = (torch.int16, 1 << 15) if dtype is BF else (torch.int32, 1 << 31)
    v = torch.randint(-top, top, (c.T, 2, d), generator=c.gen, device=DEV).to(whole)
    # NaNs of either sign with payloads, signalling ones among them, infinities, the smallest subnormal, -0
    odd = [0x7f81, 0x7fc1, -0x7f, -1, 0x7f80, -0x80, 1, -0x8000]
    v[:, 1, :8] = torch.tensor([x if dtype is BF else x << 16 for x in odd], device=DEV).to(whole)
    v = v.view(dtype)
    k = rand(c.gen, c.T, 2, d, dtype=dtype)
    kda.kda_kv_append(k, v, c.kc, c.vc, c.table, c.lens, c.cu, inv_freq=freqs(rot) if rot else None, layout=layout)
    for n, (a, b) in enumerate(zip(c.cu_list, c.cu_list[1:])):
        page, slot = R.slots(c.table.cpu(), n, 16, range(lens[n] - new[n], lens[n]))
        assert torch.equal(bits(c.vc[page.to(DEV), :, slot.to(DEV)]), bits(v[a:b])), f"sequence {n}"
