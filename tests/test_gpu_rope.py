"""Norm and rotation of queries and keys against the fp64 definition."""
import math

import pytest
import torch

import _paged_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def rand(gen, *shape, dtype=F32, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * std + mean).to(dtype)


def gen_of(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def freqs(rot):
    return (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().to(DEV)


def check(kda, T, Hq, Hk, d, rot, dtype, layout="half", norm=True, weights=True, rot_scale=1.0, far=0, fused=False,
          eps=1e-6, seed=0):
    gen = gen_of(seed)
    if fused:
        qkv, dqkv = rand(gen, T, Hq + 2 * Hk, d, dtype=dtype), rand(gen, T, Hq + 2 * Hk, d, dtype=dtype)
        q, k, dy, dyk = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], dqkv[:, :Hq], dqkv[:, Hq:Hq + Hk]
    else:
        q, k, dy, dyk = (rand(gen, T, H, d, dtype=dtype) for H in (Hq, Hk, Hq, Hk))
    pos = (torch.arange(T, device=DEV, dtype=torch.int32) * 3 - 5) + far
    f = freqs(rot) if rot else None
    w = {n: rand(gen, d, std=0.3, mean=1.0) if weights and norm else None for n in ("q", "k")}
    how = dict(layout=layout, rot_scale=rot_scale, norm=norm, eps=eps)
    args = (q, k if Hk else None, pos if rot else None, f, w["q"], w["k"] if Hk else None)
    yq, yk = kda.kda_qk_rope_fwd(*args, **how)
    gr = kda.kda_qk_rope_bwd(dy, dyk if Hk else None, *args, **how)
    for n, x, y, g in (("q", q, yq, dy), ("k", k, yk, dyk))[:2 if Hk else 1]:
        ref = R.turn(R.f64(x), R.f64(w[n]), pos.cpu(), None if f is None else f.cpu(), dy=R.f64(g), **how)
        R.assert_within(y, *ref[0], dtype, f"{n}_out")
        R.assert_within(gr["d_" + n], *ref[1], dtype, f"d_{n}")
        if w[n] is not None:
            R.assert_within(gr[f"d_{n}_weight"], *ref[2], F32, f"d_{n}_weight")
        else:
            assert gr[f"d_{n}_weight"] is None
    if not Hk:
        assert yk is None and gr["d_k"] is None


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(16, 16), (16, 8), (32, 24), (32, 0), (64, 64), (64, 40), (128, 128), (128, 64),
                                   (128, 8)])
def test_forward_and_gradients(kda, d, rot, layout, dtype):
    check(kda, 37, 5, 3, d, rot, dtype, layout)
    check(kda, 37, 5, 3, d, rot, dtype, layout, norm=rot == 0, weights=rot == 0, rot_scale=1.3)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (1, 32, 8), (2, 1, 0), (257, 40, 1), (1300, 7, 7), (5000, 4, 2)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_counts_of_tokens_and_heads(kda, T, Hq, Hk, dtype):
    check(kda, T, Hq, Hk, 64, 32, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_parts_of_a_projection(kda, dtype):
    check(kda, 301, 6, 2, 128, 128, dtype, fused=True)
    check(kda, 64, 6, 2, 32, 16, dtype, "interleaved", fused=True)


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 200, -(1 << 31) + 5, -12345])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions(kda, far, layout):
    check(kda, 60, 2, 1, 64, 64, F32, layout, norm=False, far=far)


def test_odd_frequencies(kda):
    f = torch.tensor([1.0, -0.25, 0.0, 1e-30, 3.0e4, 6.2831855, 1e-9, -7e3], device=DEV)
    gen = gen_of(3)
    q = rand(gen, 50, 2, 16)
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (50,), generator=gen, device=DEV).to(torch.int32)
    y, _ = kda.kda_qk_rope_fwd(q, positions=pos, inv_freq=f, norm=False)
    R.assert_within(y, *R.turn(R.f64(q), None, pos.cpu(), f.cpu(), norm=False), F32, "q_out")


def test_is_the_l2_norm_of_the_recurrence(kda):
    gen = gen_of(4)
    q, k = rand(gen, 100, 4, 128, dtype=BF), rand(gen, 100, 4, 128, dtype=BF)
    w = torch.full((128,), 128 ** -0.5, device=DEV)
    yq, yk = kda.kda_qk_rope_fwd(q, k, q_weight=w, k_weight=w, eps=0.0)
    for x, y in ((q, yq), (k, yk)):
        ref = R.f64(x) / R.f64(x).norm(dim=-1, keepdim=True)
        R.assert_within(y, ref, 20 * R.U * ref.abs(), BF, "unit rows")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place(kda, dtype):
    gen = gen_of(5)
    q, k, dq, dk = (rand(gen, 90, H, 64, dtype=dtype) for H in (4, 2, 4, 2))
    w, f, pos = rand(gen, 64), freqs(32), torch.arange(90, device=DEV, dtype=torch.int32)
    want = kda.kda_qk_rope_fwd(q, k, pos, f, w, w)
    gr = kda.kda_qk_rope_bwd(dq, dk, q, k, pos, f, w, w)
    q2, k2 = q.clone(), k.clone()
    kda.kda_qk_rope_fwd(q2, k2, pos, f, w, w, q_out=q2, k_out=k2)
    assert torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    out = dict(d_q=dq, d_k=dk, d_q_weight=torch.empty_like(w), d_k_weight=torch.empty_like(w))
    kda.kda_qk_rope_bwd(dq, dk, q, k, pos, f, w, w, grads=out)
    for n in gr:
        assert torch.equal(out[n], gr[n]), n
    # both parts of one buffer, beside a part that stays
    qkv = torch.cat([q, k, k], 1)
    a, b = qkv[:, :4], qkv[:, 4:6]
    kda.kda_qk_rope_fwd(a, b, pos, f, w, w, q_out=a, k_out=b)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(qkv[:, 6:], k)


def test_batched_shapes(kda):
    gen = gen_of(6)
    q, k = rand(gen, 3, 11, 4, 32, dtype=BF), rand(gen, 3, 11, 2, 32, dtype=BF)
    pos = torch.arange(11, device=DEV, dtype=torch.int32).repeat(3, 1)
    yq, yk = kda.kda_qk_rope_fwd(q, k, pos, freqs(32))
    fq, fk = kda.kda_qk_rope_fwd(q.view(33, 4, 32), k.view(33, 2, 32), pos.view(33), freqs(32))
    assert yq.shape == q.shape and torch.equal(yq.view_as(fq), fq) and torch.equal(yk.view_as(fk), fk)


def test_zeros_and_bad_rows(kda):
    q = rand(gen_of(7), 8, 4, 64, dtype=BF)
    clean, _ = kda.kda_qk_rope_fwd(q)
    q[2, 1] = 0
    q[5, 3, 7] = math.inf
    q[6, 0, 1] = math.nan
    y, _ = kda.kda_qk_rope_fwd(q)
    assert bool((y[2, 1] == 0).all()) and bool(torch.isnan(y[5, 3, 7])) and bool(torch.isnan(y[6, 0]).all())
    for t, h in ((2, 1), (5, 3), (6, 0)):
        y[t, h] = clean[t, h]
    assert torch.equal(y, clean)
    assert float(kda.kda_qk_rope_fwd(torch.zeros(1, 1, 16, device=DEV), eps=0.0)[0].isnan().sum()) == 16


def test_no_tokens(kda):
    q, k = torch.empty(0, 4, 64, device=DEV), torch.empty(0, 2, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    yq, yk = kda.kda_qk_rope_fwd(q, k, torch.empty(0, dtype=torch.int32, device=DEV), freqs(64), w, w)
    assert yq.shape == q.shape and yk.shape == k.shape
    gr = kda.kda_qk_rope_bwd(q, k, q, k, torch.empty(0, dtype=torch.int32, device=DEV), freqs(64), w, w)
    assert float(gr["d_q_weight"].abs().sum()) == 0 and float(gr["d_k_weight"].abs().sum()) == 0


def test_results_repeat_bitwise(kda):
    gen = gen_of(8)
    q, k, w = rand(gen, 3001, 8, 128, dtype=BF), rand(gen, 3001, 2, 128, dtype=BF), rand(gen, 128)
    pos = torch.arange(3001, device=DEV, dtype=torch.int32)
    runs = [kda.kda_qk_rope_bwd(q, k, q, k, pos, freqs(128), w, w) for _ in range(3)]
    for r in runs[1:]:
        for n in r:
            assert torch.equal(r[n], runs[0][n]), n


def test_directional_difference(kda):
    gen = gen_of(9)
    q, k, d, dy, dyk = (rand(gen, 40, H, 64) for H in (3, 2, 3, 3, 2))
    w, dw, f = rand(gen, 64, mean=1.0, std=0.2), rand(gen, 64), freqs(48)
    pos = torch.arange(40, device=DEV, dtype=torch.int32)
    gr = kda.kda_qk_rope_bwd(dy, dyk, q, k, pos, f, w, w, layout="interleaved")
    h = 2.0 ** -7

    def loss(s):
        y, _ = kda.kda_qk_rope_fwd(q + s * h * d, k, pos, f, w + s * h * dw, w, layout="interleaved")
        return float((y.double() * dy.double()).sum())
    want = float((gr["d_q"].double() * d.double()).sum() + (gr["d_q_weight"].double() * dw.double()).sum())
    # a central difference is off by h^2 / 6 of a third derivative (rows of norm 8 moved by 8 h: below 0.01 of the
    # sum's scale) and by the losses' own roundings, 2^-24 of sum |y dy| each over 2 h
    scale = float(dy.double().norm() * d.double().norm())
    assert abs((loss(1) - loss(-1)) / (2 * h) - want) < 20 * h * h * scale ** 0.5 + 1e-3 * scale ** 0.5


def test_captured_and_replayed(kda):
    gen = gen_of(10)
    q, k, w, f = rand(gen, 64, 4, 64, dtype=BF), rand(gen, 64, 2, 64, dtype=BF), rand(gen, 64), freqs(64)
    pos = torch.arange(64, device=DEV, dtype=torch.int32)
    yq, yk = torch.empty_like(q), torch.empty_like(k)
    out = dict(d_q=torch.empty_like(q), d_k=torch.empty_like(k), d_q_weight=torch.empty_like(w), d_k_weight=torch.empty_like(w))
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)

    def both():
        kda.kda_qk_rope_fwd(q, k, pos, f, w, w, q_out=yq, k_out=yk)
        kda.kda_qk_rope_bwd(yq, yk, q, k, pos, f, w, w, grads=out, workspace=ws)
    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    q.copy_(rand(gen, 64, 4, 64, dtype=BF))
    pos.add_(1000)
    graph.replay()
    got = [t.clone() for t in (yq, yk, *out.values())]
    both()
    for a, b in zip(got, (yq, yk, *out.values())):
        assert torch.equal(a, b)


def test_side_stream(kda):
    gen = gen_of(11)
    q, k, f = rand(gen, 2000, 8, 128, dtype=BF), rand(gen, 2000, 8, 128, dtype=BF), freqs(128)
    pos, w = torch.arange(2000, device=DEV, dtype=torch.int32), rand(gen, 128)
    want = kda.kda_qk_rope_fwd(q, k, pos, f, w, w)
    wg = kda.kda_qk_rope_bwd(q, k, q, k, pos, f, w, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream(device=DEV)
    got = kda.kda_qk_rope_fwd(q, k, pos, f, w, w, stream=s)
    gg = kda.kda_qk_rope_bwd(q, k, q, k, pos, f, w, w, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(torch.equal(gg[n], wg[n]) for n in wg)


def test_offsets_past_32_bits(kda):
    # rows 1.2 M elements apart: the last ones lie behind 2^31 elements
    T, stride = 2000, 1_200_000
    buf = torch.empty(T * stride, dtype=BF, device=DEV)
    q = buf.as_strided((T, 2, 32), (stride, 32, 1))
    q.copy_(rand(gen_of(12), T, 2, 32, dtype=BF))
    pos = torch.arange(T, device=DEV, dtype=torch.int32)
    dense = q.contiguous()
    want, _ = kda.kda_qk_rope_fwd(dense, positions=pos, inv_freq=freqs(32))
    wg = kda.kda_qk_rope_bwd(dense, None, dense, positions=pos, inv_freq=freqs(32))
    gr = kda.kda_qk_rope_bwd(q, None, q, positions=pos, inv_freq=freqs(32))
    assert torch.equal(gr["d_q"], wg["d_q"])
    kda.kda_qk_rope_fwd(q, positions=pos, inv_freq=freqs(32), q_out=q)
    assert torch.equal(q.contiguous(), want)


def test_refusals(kda):
    q, k = torch.zeros(4, 2, 64, device=DEV), torch.zeros(4, 1, 64, device=DEV)
    pos, f = torch.zeros(4, dtype=torch.int32, device=DEV), freqs(64)
    for bad in (lambda: kda.kda_qk_rope_fwd(q, k.bfloat16()), lambda: kda.kda_qk_rope_fwd(q, k, pos.long(), f),
                lambda: kda.kda_qk_rope_fwd(q, k, pos, f.double()), lambda: kda.kda_qk_rope_fwd(q.half())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: kda.kda_qk_rope_fwd(q, k[:3]), lambda: kda.kda_qk_rope_fwd(q, k, None, f),
                lambda: kda.kda_qk_rope_fwd(q, k, pos[:3], f), lambda: kda.kda_qk_rope_fwd(q, layout="other"),
                lambda: kda.kda_qk_rope_fwd(q.transpose(0, 1)), lambda: kda.kda_qk_rope_fwd(q.cpu()),
                lambda: kda.kda_qk_rope_fwd(q, q_weight=torch.ones(64)), lambda: kda.kda_qk_rope_fwd(q[0])):
        with pytest.raises(ValueError):
            bad()
    for bad, status in ((lambda: kda.kda_qk_rope_fwd(torch.zeros(4, 2, 48, device=DEV)), -2),
                        (lambda: kda.kda_qk_rope_fwd(q, k, pos, freqs(12)), -2),
                        (lambda: kda.kda_qk_rope_fwd(q, norm=False, q_weight=torch.ones(64, device=DEV)), -7),
                        (lambda: kda.kda_qk_rope_fwd(q, eps=-1.0), -5),
                        (lambda: kda.kda_qk_rope_fwd(q, rot_scale=math.inf), -5),
                        (lambda: kda.kda_qk_rope_fwd(q, k, q_out=q[:, :1].expand(4, 2, 64).contiguous(), k_out=q[:, :1]), -8)):
        with pytest.raises(kda.KdaError) as e:
            bad()
        assert e.value.status == status
