"""Block norms: every pair of types in the shapes for many narrow rows, and a
backward whose tensors are larger than 2^31 elements."""
import pytest
import torch

import _block_ref as ref
import test_gpu_block_norm as norm
from _block_ref import assert_within, np64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width", [8, 16, 24, 32, 64, 128, 200, 256])
@pytest.mark.parametrize("dtype,res", [(norm.BF, norm.F32), (norm.F32, norm.BF), (norm.F32, norm.F32), (norm.BF, None)])
def test_many_narrow_rows(kda, width, dtype, res):
    norm.check_all(kda, norm.make(16385, width, dtype, res, seed=21))


@pytest.mark.parametrize("rows,width", [(700, 320), (700, 512), (700, 1024), (640, 2048), (330, 4096), (160, 8192)])
@pytest.mark.parametrize("dtype,res", norm.TYPES)
def test_wide_rows(kda, rows, width, dtype, res):
    """More rows than the grid of the backward takes at once."""
    norm.check_all(kda, norm.make(rows, width, dtype, res, seed=22))


@pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.mem_get_info()[1] < 80 << 30, reason="needs 80 GB")
def test_backward_past_32_bits(kda):
    rows, width = 600000, 4096  # 2.46e9 elements
    gen = torch.Generator(device=norm.DEV)
    gen.manual_seed(23)
    y, gate, res, do, dn = (torch.randn(rows, width, generator=gen, device=norm.DEV, dtype=norm.BF) for _ in range(5))
    w1, sc, w2 = (torch.rand(width, generator=gen, device=norm.DEV) + 0.5 for _ in range(3))
    gr = kda.kda_block_norm_bwd(y, do, dn, residual=res, gate=gate, post_weight=w1, scale=sc, pre_weight=w2,
                                post_eps=norm.E1, pre_eps=norm.E2)
    for r in (0, rows // 2, (1 << 31) // width - 1, (1 << 31) // width, rows - 1):
        c = slice(r, r + 1)
        want = ref.block_norm(np64(y[c]), np64(res[c]), np64(gate[c]), True, np64(w1), np64(sc), np64(w2), norm.E1, norm.E2,
                              True, np64(do[c]), np64(dn[c]))
        for name in ("d_y", "d_gate", "d_residual"):
            assert_within(gr[name][c], *want[name], norm.BF, f"{name} of row {r}")
