"""Paged attention at the ends of fp32's range: sums that are in range where every
probability is at most 1, whichever kernel has the rows."""
import pytest
import torch

from test_gpu_paged import Case

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,score", [(3, 5.1875), (150, 5.1875), (150, 5.5), (150, 6.0)])
def test_large_values_of_keys_that_outweigh_the_first_ones(kda, new, score, d, dtype):
    # Key 130 (behind the first tile of 128) has a score of 7.5 to 8.7 powers of two above all the others and a value of
    # 3e36: times 2^7.5 this is past fp32's 3.4e38, the weighted mean is about 1e36.  256 items, more than
    # blocks, so that a block has the tile of the first keys and the one of key 130 of the same rows.
    N, kv = 64, 300
    c = Case([new] * N, [kv] * N, 4, 4, d, 64, dtype)
    c.q.zero_()
    c.q[:, :, 0] = 1.0
    c.kc[..., 0] = 0.0
    for n in range(N):
        p, s = c.at(n, 130)
        c.kc[p, :, s, 0] = score
        c.vc[p, :, s] = 3e36
    c.check(kda, scale=1.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("new", [1, 150])
def test_infinite_values_of_probabilities_that_underflow(kda, new, d, dtype):
    # an infinity that stands 300 powers of two below the largest key shows in its channel, as itself or as NaN, and nowhere else
    N, kv = 40, 300
    c = Case([new] * N, [kv] * N, 4, 4, d, 64, dtype)
    c.q.zero_()
    c.q[:, :, 0] = 1.0
    c.kc[..., 0] = 0.0
    for n in range(N):
        p, s = c.at(n, 140)
        c.kc[p, :, s, 0] = 208.0
    clean, lse = c.check(kda, scale=1.0)
    for n in range(N):
        p, s = c.at(n, 10 + n)
        c.vc[p, :, s, 5] = float("inf")
    out, got = c.attend(kda, scale=1.0, want_lse=True)
    assert not bool(torch.isfinite(out[..., 5]).any()) and not bool((out[..., 5] == -float("inf")).any())
    rest = [i for i in range(d) if i != 5]
    assert torch.equal(out[..., rest], clean[..., rest]) and torch.equal(got, lse)
