"""dA_log as a sum over very many tokens that all add alike, where an fp32
running sum would round the same way at every one of them."""
import numpy as np
import pytest
import torch

import _block_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
G_MIN = -5.0


@pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.mem_get_info()[1] < 60 << 30, reason="needs 60 GB")
@pytest.mark.parametrize("T,H,d", [(131072, 152, 64), (262144, 20, 64), (100000, 7, 33)])
def test_dA_log_of_equal_tokens(kda, T, H, d):
    """152 heads: blocks of 64 channels, whose lanes hold an eighth of all tokens; 20: blocks of 16; 7 x 33: elementwise."""
    xs = torch.tensor([1.0 + h / 64.0 for h in range(H)], device=DEV).bfloat16()  # a value of its own for every head
    x = xs[None, :, None].expand(T, H, d).contiguous()
    z = torch.full_like(x, 0.5)
    A = torch.zeros(H, device=DEV)
    got = kda.kda_scan_bwd(x, z, x, A, G_MIN)["dA_log"].double().cpu().numpy()
    v = xs.double().cpu().numpy()
    s = 1.0 / (1.0 + np.exp(-0.5))
    a, slope = np.exp(G_MIN * s), G_MIN * s * (1.0 - s)
    h = v * (1.0 - a ** np.arange(T)[:, None]) / (1.0 - a)              # h_{t-1}
    D = v * (1.0 - a ** np.arange(T, 0, -1)[:, None]) / (1.0 - a)
    want = d * np.sum(a * D * h, 0) * slope * 0.5
    # alpha = 0.045, so h and D hold little more than a token each: 64 half steps of its update and 64 / 20 of what
    # came before; the power, the slope (12 + 8 s z) and five products; a tile's 16 additions: all below 256
    off = np.abs(got - want) / np.abs(want)
    assert (off <= 256 * ref.U).all(), float(off.max() / ref.U)
