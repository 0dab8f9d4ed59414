"""The fp64 definitions that the rotation and the paged attention are compared
with, pinned to closed forms and differences (CPU)."""
import math

import torch

import _paged_ref as R


def rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def test_rotation_by_quarter_turns():
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0, 5.0, 6.0]]], dtype=torch.float64)
    f = torch.tensor([math.pi / 2, 0.0], dtype=torch.float64)
    y, _ = R.turn(x, None, torch.tensor([1]), f, "half", norm=False)      # pairs (0, 2), (1, 3)
    assert torch.allclose(y, torch.tensor([[[-3.0, 2.0, 1.0, 4.0, 5.0, 6.0]]], dtype=torch.float64))
    y, _ = R.turn(x, None, torch.tensor([1]), f, "interleaved", norm=False)  # pairs (0, 1), (2, 3)
    assert torch.allclose(y, torch.tensor([[[-2.0, 1.0, 3.0, 4.0, 5.0, 6.0]]], dtype=torch.float64))
    y, _ = R.turn(x, None, torch.tensor([1]), f, "interleaved", rot_scale=2.0, norm=False)
    assert torch.allclose(y, torch.tensor([[[-4.0, 2.0, 6.0, 8.0, 5.0, 6.0]]], dtype=torch.float64))


def test_scores_depend_on_distances_alone():
    q, k, f = rand(1, 1, 16), rand(1, 1, 16, seed=1), torch.tensor([1.0, 0.3, 0.1, 0.03], dtype=torch.float64)
    for layout in ("half", "interleaved"):
        dots = [float((R.turn(q, None, torch.tensor([p + 7]), f, layout)[0]
                       * R.turn(k, None, torch.tensor([p]), f, layout)[0]).sum()) for p in (0, 5, 1000)]
        assert max(dots) - min(dots) < 1e-9


def test_norm_of_a_worked_row():
    x = torch.tensor([[[3.0, 4.0]]], dtype=torch.float64)
    y, _ = R.turn(x, torch.tensor([1.0, 2.0], dtype=torch.float64), None, None, eps=0.0)
    r = math.sqrt(12.5)
    assert torch.allclose(y, torch.tensor([[[3 / r, 8 / r]]], dtype=torch.float64))
    # weights of d^-1/2 make it the L2 norm
    y, _ = R.turn(rand(3, 2, 16), torch.full((16,), 0.25, dtype=torch.float64), None, None, eps=0.0)
    assert torch.allclose(y.pow(2).sum(-1), torch.ones(3, 2, dtype=torch.float64))


def test_gradients_are_differences():
    x, dy, w = rand(3, 2, 16), rand(3, 2, 16, seed=1), rand(16, seed=2)
    pos, f = torch.tensor([0, 5, -3]), torch.tensor([1.0, 0.5], dtype=torch.float64)
    for layout in ("half", "interleaved"):
        for norm in (True, False):
            def loss(a, b):
                return float((R.turn(a, b, pos, f, layout, 1.3, norm)[0] * dy).sum())
            _, (dx, _), dw = R.turn(x, w, pos, f, layout, 1.3, norm, dy=dy)
            for i in (0, 2, 9, 15):
                h = torch.zeros_like(x)
                h[1, 1, i] = 1e-6
                assert abs((loss(x + h, w) - loss(x - h, w)) / 2e-6 - float(dx[1, 1, i])) < 1e-6
                if norm:
                    h = torch.zeros_like(w)
                    h[i] = 1e-6
                    assert abs((loss(x, w + h) - loss(x, w - h)) / 2e-6 - float(dw[0][i])) < 1e-6


def cache(lens, page, Hk, d, seed=3):
    N, most = len(lens), max(1, max((n + page - 1) // page for n in lens))
    kc, vc = rand(N * most, Hk, page, d, seed=seed), rand(N * most, Hk, page, d, seed=seed + 1)
    perm = torch.randperm(N * most, generator=torch.Generator().manual_seed(seed))
    return kc, vc, perm.view(N, most)


def test_attention_closed_forms():
    lens = [7, 3]
    kc, vc, table = cache(lens, 4, 2, 16)
    # queries of zero: means of the values that are seen
    out, _, lse, _ = R.attention(torch.zeros(6, 4, 16, dtype=torch.float64), kc, vc, table, lens)
    for n, kv in enumerate(lens):
        at = R.slots(table, n, 4, range(kv))
        for i in range(3):
            seen = kv - 3 + i + 1
            for g in range(4):
                assert torch.allclose(out[3 * n + i, g], vc[at[0], g // 2, at[1]][:seen].mean(0))
            assert torch.allclose(lse[3 * n + i], torch.full((4,), math.log(seen), dtype=torch.float64))
    # a query along one key, far longer than the others: that key's value
    at = R.slots(table, 0, 4, range(7))
    k = kc[at[0], 0, at[1]]
    out, _, _, _ = R.attention((k[2] * 1e4).expand(1, 2, 16), kc, vc, table[:1], lens[:1])
    best = int((k @ k[2]).argmax())
    assert torch.allclose(out[0, 0], vc[at[0], 0, at[1]][best])


def test_attention_rows_without_keys():
    kc, vc, table = cache([2, 0], 4, 1, 16)
    out, _, lse, _ = R.attention(rand(8, 1, 16, seed=9), kc, vc, table, [2, 0])
    assert bool((out[:2] == 0).all()) and bool((lse[:2] == -math.inf).all())      # positions -2 and -1
    assert bool(torch.isfinite(lse[2:4]).all())
    assert bool((out[4:] == 0).all()) and bool((lse[4:] == -math.inf).all())      # length 0


def test_attention_joins_by_its_log_sums():
    kc, vc, table = cache([12], 4, 1, 16)
    q = rand(1, 3, 16, seed=5)
    whole, _, lse, _ = R.attention(q, kc, vc, table, [12], causal=False)
    a, _, la, _ = R.attention(q, kc, vc, table, [8], causal=False)
    b, _, lb, _ = R.attention(q, kc, vc, table[:, 2:], [4], causal=False)
    assert torch.allclose(torch.logaddexp(la, lb), lse)
    assert torch.allclose(torch.exp(la - lse)[..., None] * a + torch.exp(lb - lse)[..., None] * b, whole)


def test_attention_hidden_values_stay_hidden():
    kc, vc, table = cache([5], 4, 1, 16)
    clean, _, _, _ = R.attention(rand(3, 1, 16), kc, vc, table, [5])
    at = R.slots(table, 0, 4, [4])
    vc[at[0], 0, at[1], 3] = math.inf
    out, _, _, _ = R.attention(rand(3, 1, 16), kc, vc, table, [5])
    assert torch.equal(out[:2], clean[:2]) and float(out[2, 0, 3]) == math.inf
    assert torch.equal(out[2, 0, :3], clean[2, 0, :3])
