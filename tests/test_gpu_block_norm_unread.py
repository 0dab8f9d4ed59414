"""What the norms' backward does not read: pre_weight without d_normed."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width", [33, 64, 264, 4096])
def test_pre_weight_without_d_normed(kda, width, dtype, res):
    """NaN and infinities in pre_weight reach no gradient when there is no d_normed, and its alignment does not matter."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    y, gate, r, do = n(9, width).to(dtype), n(9, width).to(dtype), n(9, width).to(res), n(9, width).to(res)
    p = dict(residual=r, gate=gate, post_weight=1 + 0.2 * n(width), scale=n(width))
    want = kda.kda_block_norm_bwd(y, do, **p)
    for bad in (float("nan"), float("inf")):
        for shift in (0, 1):
            w2 = torch.full((width + 1,), bad, device=DEV)[shift:shift + width]
            got = kda.kda_block_norm_bwd(y, do, pre_weight=w2, **p)
            assert got["d_pre_weight"] is None and want["d_pre_weight"] is None
            for name, t in want.items():
                if t is not None:
                    assert t.isfinite().all() and torch.equal(got[name], t), name
