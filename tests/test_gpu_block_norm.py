"""Norms around a block (kda_block_norm_fwd, kda_block_norm_bwd) against their
fp64 definition, with error bounds (see _block_ref)."""
import itertools

import numpy as np
import pytest
import torch

import _block_ref as ref
from _block_ref import assert_within, np64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
E1, E2 = 1e-6, 1e-5
TYPES = [(BF, None), (BF, BF), (BF, F32), (F32, None), (F32, F32), (F32, BF)]


def make(rows, width, dtype, res, gate=True, post=True, weights=True, seed=0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    rdt = dtype if res is None else res
    return dict(y=n(rows, width).to(dtype), residual=None if res is None else (2 * n(rows, width)).to(res),
                gate=(2 * n(rows, width)).to(dtype) if gate else None,
                post_weight=1 + 0.2 * n(width) if post and weights else None,
                scale=0.5 + 0.2 * n(width) if weights else None, pre_weight=1 + 0.2 * n(width) if weights else None,
                d_out=n(rows, width).to(rdt), d_normed=n(rows, width).to(dtype), post=post)


def definition(a, d_out=True, d_normed=True, normed=True):
    return ref.block_norm(np64(a["y"]), np64(a["residual"]), np64(a["gate"]), a["post"], np64(a["post_weight"]),
                          np64(a["scale"]), np64(a["pre_weight"]), E1, E2, normed,
                          np64(a["d_out"]) if d_out else None, np64(a["d_normed"]) if d_normed else None)


def parts(a):
    return dict(residual=a["residual"], gate=a["gate"], post_norm=a["post"], post_weight=a["post_weight"],
                scale=a["scale"], pre_weight=a["pre_weight"], post_eps=E1, pre_eps=E2)


def check_all(kda, a):
    want = definition(a)
    rows = a["y"].shape[0]
    out, normed = kda.kda_block_norm_fwd(a["y"], want_normed=True, **parts(a))
    gr = kda.kda_block_norm_bwd(a["y"], a["d_out"], a["d_normed"], **parts(a))
    for name, t in dict(out=out, normed=normed, **gr).items():
        if t is not None:
            assert_within(t, *want[name], t.dtype, f"{name} of {rows} rows")
    assert (gr["d_gate"] is None) == (a["gate"] is None) and (gr["d_residual"] is None) == (a["residual"] is None)


@pytest.mark.parametrize("dtype,res", TYPES)
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 7), (5, 128), (2, 1001), (700, 40), (9, 2048), (4, 4096), (3, 8192),
                                        (2, 8191), (40, 256), (33, 520)])
def test_every_part(kda, rows, width, dtype, res):
    check_all(kda, make(rows, width, dtype, res))


@pytest.mark.parametrize("width", [24, 1000])
@pytest.mark.parametrize("gate,post,weights,res", list(itertools.product([False, True], [False, True], [False, True],
                                                                        [None, F32])))
def test_each_part_left_out(kda, width, gate, post, weights, res):
    check_all(kda, make(6, width, BF, res, gate, post, weights, seed=1))


@pytest.mark.parametrize("width", [96, 4096])
def test_one_output_or_gradient_alone(kda, width):
    a = make(10, width, BF, F32, seed=2)
    p = parts(a)
    both = kda.kda_block_norm_fwd(a["y"], want_normed=True, **p)
    out, none = kda.kda_block_norm_fwd(a["y"], **{**p, "pre_weight": None})
    assert none is None and torch.equal(out, both[0])
    none, normed = kda.kda_block_norm_fwd(a["y"], want_out=False, want_normed=True, **p)
    assert none is None and torch.equal(normed, both[1])
    want = definition(a, d_normed=False)
    gr = kda.kda_block_norm_bwd(a["y"], a["d_out"], None, **p)
    assert gr["d_pre_weight"] is None
    for name in ("d_y", "d_residual", "d_gate", "d_post_weight", "d_scale"):
        assert_within(gr[name], *want[name], gr[name].dtype, name)
    want = definition(a, d_out=False)
    gr = kda.kda_block_norm_bwd(a["y"], None, a["d_normed"], **p)
    for name, t in gr.items():
        assert_within(t, *want[name], t.dtype, name)
    # gradients of weights that are ones, without the tensors
    b = dict(a, post_weight=None, scale=None, pre_weight=None)
    want = definition(b)
    gr = dict(d_y=torch.empty_like(a["y"]), d_gate=torch.empty_like(a["y"]),
              **{n: torch.empty(width, device=DEV) for n in ("d_post_weight", "d_scale", "d_pre_weight")})
    kda.kda_block_norm_bwd(b["y"], b["d_out"], b["d_normed"], grads=gr, **parts(b))
    for name, t in gr.items():
        assert_within(t, *want[name], t.dtype, name)


@pytest.mark.parametrize("width", [128, 333])
def test_in_place(kda, width):
    a = make(20, width, BF, BF, seed=3)
    p = parts(a)
    out, normed = kda.kda_block_norm_fwd(a["y"], want_normed=True, **p)
    gr = kda.kda_block_norm_bwd(a["y"], a["d_out"], a["d_normed"], **p)
    res = a["residual"].clone()
    o2, n2 = kda.kda_block_norm_fwd(a["y"], want_normed=True, out=res, **{**p, "residual": res})
    assert o2 is res and torch.equal(res, out) and torch.equal(n2, normed)
    d = a["d_out"].clone()
    g2 = dict(d_y=torch.empty_like(d), d_gate=torch.empty_like(d), d_residual=d)
    kda.kda_block_norm_bwd(a["y"], d, a["d_normed"], grads=g2, **p)
    for n in g2:
        assert torch.equal(g2[n], gr[n]), n


def test_is_the_output_equation_of_the_recurrence(kda):
    """Rows of one head each: the norm and gate that kda_layer_fwd applies, on [tokens, H, dv]."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(4)
    o, g = (torch.randn(50, 4, 128, generator=gen, device=DEV).to(BF) for _ in range(2))
    w = torch.rand(128, generator=gen, device=DEV) + 0.5
    y, _ = kda.kda_block_norm_fwd(o, gate=g, post_weight=w, post_eps=E1)
    want = ref.block_norm(np64(o).reshape(200, 128), None, np64(g).reshape(200, 128), True, np64(w), e1=E1,
                          normed=False)["out"]
    assert y.shape == o.shape
    assert_within(y.reshape(200, 128), *want, BF, "y")


@pytest.mark.parametrize("width", [8, 16, 24, 32, 64, 128, 200, 256])
@pytest.mark.parametrize("dtype,res", [(BF, BF), (F32, None)])
def test_many_narrow_rows(kda, width, dtype, res):
    """Row counts past the rule that takes two at once, odd ones, and every narrow shape."""
    check_all(kda, make(16385, width, dtype, res, seed=19))


def test_zero_rows_and_rows_of_zeros(kda):
    y = torch.zeros(3, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    out, normed = kda.kda_block_norm_fwd(y, want_normed=True, post_weight=w)
    assert torch.equal(out, y) and torch.equal(normed, y)
    gr = kda.kda_block_norm_bwd(y, y + 1, y + 1, post_weight=w, pre_weight=w, pre_eps=1e-6)
    assert all(t.isfinite().all() for t in gr.values() if t is not None)
    e = torch.empty(0, 64, device=DEV)
    out, normed = kda.kda_block_norm_fwd(e, want_normed=True, post_weight=w)
    assert out.shape == normed.shape == (0, 64)
    gr = kda.kda_block_norm_bwd(e, e, e, post_weight=w, scale=w, pre_weight=w)
    for n in ("d_post_weight", "d_scale", "d_pre_weight"):
        assert torch.equal(gr[n], torch.zeros_like(w))


def test_bad_rows_stay_alone(kda):
    """NaN and infinities of one row reach its own outputs and the weight gradients, no other row."""
    a = make(30, 264, BF, BF, seed=5)
    p = parts(a)
    o0, n0 = kda.kda_block_norm_fwd(a["y"], want_normed=True, **p)
    g0 = kda.kda_block_norm_bwd(a["y"], a["d_out"], a["d_normed"], **p)
    y = a["y"].clone()
    y[7, 3] = float("nan")
    y[20, 263] = float("inf")
    o1, n1 = kda.kda_block_norm_fwd(y, want_normed=True, **p)
    g1 = kda.kda_block_norm_bwd(y, a["d_out"], a["d_normed"], **p)
    ok = [r for r in range(30) if r not in (7, 20)]
    for q0, q1 in ((o0, o1), (n0, n1), (g0["d_y"], g1["d_y"]), (g0["d_gate"], g1["d_gate"]),
                   (g0["d_residual"], g1["d_residual"])):
        assert torch.equal(q0[ok], q1[ok])
    assert n1[7].isnan().all() and o1[20, 263].isnan()


@pytest.mark.parametrize("rows,width", [(5001, 1), (5001, 30), (5001, 33), (5001, 63), (5001, 130), (2500, 257), (1300, 511),
                                        (650, 1001), (330, 1070), (7, 2047), (160, 3001), (3, 4095), (160, 8001)])
@pytest.mark.parametrize("dtype,res", [(BF, BF), (BF, F32), (F32, F32)])
def test_rows_off_16_bytes(kda, rows, width, dtype, res):
    """Widths that no 16-byte piece divides, with more rows than the grid takes at once."""
    check_all(kda, make(rows, width, dtype, res, seed=20))


@pytest.mark.parametrize("width", [264, 33])
def test_infinite_residual_without_normed(kda, width):
    """Without d_normed no gradient depends on the residual's values, infinite or NaN as they may be."""
    a = make(9, width, BF, BF, seed=18)
    p = {**parts(a), "pre_weight": None}
    want = kda.kda_block_norm_bwd(a["y"], a["d_out"], None, **p)
    res = a["residual"].clone()
    res[2, 5], res[4, 0], res[7] = float("inf"), -float("inf"), float("nan")
    got = kda.kda_block_norm_bwd(a["y"], a["d_out"], None, **{**p, "residual": res})
    assert torch.equal(got["d_residual"], a["d_out"])
    for n in want:
        if want[n] is not None:
            assert torch.equal(got[n], want[n]), n


def test_extreme_gates(kda):
    """Closed and open gates: sigmoid and its slope at +-200 and +-inf."""
    a = make(4, 48, F32, F32, seed=6)
    a["gate"][0], a["gate"][1], a["gate"][2], a["gate"][3] = 200.0, -200.0, float("inf"), -float("inf")
    out, _ = kda.kda_block_norm_fwd(a["y"], **{**parts(a), "pre_weight": None})
    gr = kda.kda_block_norm_bwd(a["y"], a["d_out"], a["d_normed"], **parts(a))
    assert torch.equal(out[1], a["residual"][1]) and torch.equal(out[3], a["residual"][3])
    assert all(t.isfinite().all() for t in gr.values())
    assert (gr["d_gate"].abs() < 1e-30).all() and (gr["d_y"][1].abs() < 1e-30).all()


def test_unaligned_tensors(kda):
    a = make(6, 64, BF, F32, seed=7)

    def shifted(t):
        return None if t is None else torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].view(t.shape).copy_(t)

    b = {n: shifted(t) if torch.is_tensor(t) else t for n, t in a.items()}
    check_all(kda, b)


def test_results_repeat_bitwise(kda):
    a = make(3000, 320, BF, F32, seed=8)
    runs = [list(kda.kda_block_norm_bwd(a["y"], a["d_out"], a["d_normed"], **parts(a)).values()) for _ in range(2)]
    for p, q in zip(*runs):
        assert torch.equal(p, q)


def test_many_rows(kda):
    """More rows than one launch's resident blocks, rows past 2^31 elements apart are addressed in 64 bits."""
    a = make(20011, 16, F32, None, seed=9)
    check_all(kda, a)


@pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.mem_get_info()[1] < 60 << 30, reason="needs 60 GB")
def test_offsets_past_32_bits(kda):
    rows, width = 600000, 4096  # 2.46e9 elements
    gen = torch.Generator(device=DEV)
    gen.manual_seed(10)
    y = torch.randn(rows, width, generator=gen, device=DEV, dtype=BF)
    w = torch.rand(width, generator=gen, device=DEV) + 0.5
    out, _ = kda.kda_block_norm_fwd(y, post_weight=w, post_eps=E1)
    for r in (0, rows // 2, rows - 1):
        want = ref.block_norm(np64(y[r:r + 1]), w1=np64(w), e1=E1, normed=False)["out"]
        assert_within(out[r:r + 1], *want, BF, f"row {r}")


def test_captured_and_replayed(kda):
    def step(a):
        out, normed = kda.kda_block_norm_fwd(a["y"], want_normed=True, **parts(a))
        return [out, normed] + list(kda.kda_block_norm_bwd(a["y"], a["d_out"], a["d_normed"], **parts(a)).values())

    bufs = [make(300, 136, BF, F32, seed=11), make(300, 136, BF, F32, seed=12)]
    step(bufs[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for b in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(b))
        graphs.append(g)
    fresh = [make(300, 136, BF, F32, seed=13), make(300, 136, BF, F32, seed=14)]
    for b, f in zip(bufs, fresh):
        for n, t in b.items():
            if torch.is_tensor(t):
                t.copy_(f[n])
    for g in graphs:
        g.replay()
    want = [step(f) for f in fresh]
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        for p, q in zip(got, w):
            assert torch.equal(p, q)


def test_side_stream(kda):
    a = make(500, 256, BF, BF, seed=15)
    want = kda.kda_block_norm_bwd(a["y"], a["d_out"], a["d_normed"], **parts(a))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = kda.kda_block_norm_bwd(a["y"], a["d_out"], a["d_normed"], stream=side, **parts(a))
    side.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n])


def test_directional_difference(kda):
    a = make(12, 40, F32, F32, seed=16)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(17)
    gr = kda.kda_block_norm_bwd(a["y"], a["d_out"], a["d_normed"], **parts(a))

    def loss(b):
        out, normed = kda.kda_block_norm_fwd(b["y"], want_normed=True, **parts(b))
        return float((out.double() * a["d_out"].double()).sum() + (normed.double() * a["d_normed"].double()).sum())

    for name in ("y", "residual", "gate", "post_weight", "scale", "pre_weight"):
        v = torch.randn(a[name].shape, generator=gen, device=DEV)
        e = 3e-3
        diff = (loss(dict(a, **{name: a[name] + e * v})) - loss(dict(a, **{name: a[name] - e * v}))) / (2 * e)
        got = float((gr["d_" + name].double() * v.double()).sum())
        # fp32 outputs' 1e-7 of each of n = 960 terms of order one, random, over 2e: 5e-4; third derivatives times
        # e^2 / 6 = 1.5e-6 per element
        assert abs(diff - got) <= 2e-2 + 2e-3 * abs(got), name
