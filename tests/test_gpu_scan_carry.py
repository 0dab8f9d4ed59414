"""How a state (and, backwards, a gradient) is carried over thousands of tokens
in which it decays alone, against fp64: the error is at most half a step of
fp32 a token."""
import pytest
import torch

import _block_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
G_MIN = -5.0

# A tile of 16 tokens may shift the carried value by, in half steps (g about -0.0075, so its log-sum S is about -0.12):
# the sum of its logs 16 |S| < 2.3; expm1 below 6 of 1 - alpha < 0.13, or the power 4 (two of its steps) and its
# argument |S| < 0.2; one joining 3; applying it 2: below 16, that is one a token.  With logits the log itself is off
# by 30 of |S|, 4 more at the most, over the 3.7 that are left.  Outputs within a tile come from products of up to 16
# powers: 16 x (4 of the power, 1 of its argument, 1 of the product).
PER_TOKEN, IN_TILE = 1.25, 96.0

# heads, channels: blocks of 16 channels (8 with rows off 16 bytes) on a cluster, whose CTAs join up to 64 tiles (32 with
# fp32 decays on 16 bytes) into one span; on one CTA
SHAPES = {"cluster": (1, 32), "cluster_elementwise": (1, 33), "ring": (25, 64), "ring_elementwise": (21, 33)}
T = 9000


def gates(kind, steady, H, d, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    # a decay of its own for every channel, so that roundings fall every way; a tile's log-sum is just above -1/8
    g = torch.linspace(-0.0070, -0.0077, H * d, device=DEV).view(1, H, d).expand(T, H, d).contiguous()
    if not steady:
        g *= 0.99 + 0.02 * torch.rand(T, H, d, generator=gen, device=DEV)
    if kind.startswith("given"):
        g = g.to(torch.bfloat16 if kind == "given_bf16" else torch.float32)
        return g, None, g.double()
    s = g.double() / G_MIN
    z = torch.log(s / (1 - s)).float()  # (alpha follows from the rounded z)
    return z, torch.zeros(H, device=DEV), G_MIN * torch.sigmoid(z.double())


@pytest.mark.parametrize("steady", [False, True])
@pytest.mark.parametrize("kind", ["given", "given_bf16", "logit"])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_a_state_that_decays_alone(kda, shape, kind, steady):
    H, d = SHAPES[shape]
    decay, A, g = gates(kind, steady, H, d, seed=1)
    big = torch.full((1, H, d), 1e30, device=DEV)
    zero = torch.zeros(T, H, d, device=DEV)
    out, fs, states = kda.kda_scan_fwd(zero, decay, A, G_MIN, big, want_states=True)
    h = big[0].double() * torch.exp(torch.cumsum(g, 0))  # 1e30 .. about 1e1
    n = torch.arange(1, T + 1, device=DEV, dtype=torch.float64)[:, None, None]
    off = (out.double() - h).abs() / h
    assert (off <= (PER_TOKEN * n + IN_TILE) * ref.U).all(), float((off / ref.U).max())
    off = (fs[0].double() - h[-1]).abs() / h[-1]
    assert (off <= (PER_TOKEN * T + 16) * ref.U).all(), float((off / ref.U).max())
    gr = kda.kda_scan_bwd(zero, decay, zero, A, G_MIN, big, big, states=states)
    off = (gr["d_initial_state"][0].double() - h[-1]).abs() / h[-1]
    assert (off <= (PER_TOKEN * T + 16) * ref.U).all(), float((off / ref.U).max())
    back = big[0].double() * torch.exp(torch.flip(torch.cumsum(torch.flip(g, [0]), 0), [0]) - g)  # after the token
    off = (gr["dx"].double() - back).abs() / back
    assert (off <= (PER_TOKEN * torch.flip(n, [0]) + IN_TILE) * ref.U).all(), float((off / ref.U).max())
