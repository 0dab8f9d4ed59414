"""The rotation's sines and cosines by themselves, against fp64."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("top", [1 << 7, 1 << 20])
def test_sines_and_cosines(kda, top, layout):
    # Rows of (1, 0) turn into (cos, sin), products with 1 and 0 being exact.  position * inv_freq has 20 + 24 bits, so
    # that fp64 holds it whole.
    #
    # Bound: the reduced angle is off by 2^-30 of a turn (2 pi 2^-30 = 0.10 U).  What is left of it after whole
    # quarters are taken out, at most 1/4 of a half turn, rounds to fp32 by 2^-27 of a half turn at most (pi / 8 U =
    # 0.40 U).  sincospif is documented to 1 ulp, which is U for results from 1/2 to 1.  In all 1.5 U; an angle that is
    # rounded with all of its half turn before is off by pi / 2 U by that alone.
    T, d = 8192, 16
    gen = torch.Generator(device=DEV).manual_seed(top)
    pos = torch.randint(-top, top, (T,), generator=gen, device=DEV).to(torch.int32)
    f = torch.tensor([1.0, 0.7, 0.31622776, 0.1, 0.0316, -0.9, 0.01, 1e-3], device=DEV)
    x = torch.zeros(T, 1, d, device=DEV)
    a, b = (range(8), range(8, 16)) if layout == "half" else (range(0, 16, 2), range(1, 16, 2))
    x[..., list(a)] = 1.0
    y, _ = kda.kda_qk_rope_fwd(x, positions=pos, inv_freq=f, layout=layout, norm=False)
    want = pos.double()[:, None] * f.double()
    for name, at, ref in (("cos", a, torch.cos(want)), ("sin", b, torch.sin(want))):
        err = float((y[:, 0, list(at)].double() - ref).abs().max())
        assert err <= 1.5 * U, f"{name}: {err / U:.2f} U"
