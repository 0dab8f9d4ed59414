"""Gated linear recurrence (kda_scan_fwd, kda_scan_bwd, kda_scan_step) against
its fp64 definition, with running error bounds (see _block_ref)."""
import numpy as np
import pytest
import torch

import _block_ref as ref
from _block_ref import assert_within, np64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
KINDS = [("bf16", "fp32"), ("bf16", "bf16"), ("bf16", "logit"), ("fp32", "fp32"), ("fp32", "bf16"), ("fp32", "logit")]
# lengths, rows behind the last sequence, H, d
SHAPES = {
    "one_token": ([1], 0, 2, 128),
    "tile_edges": ([15, 16, 17, 1, 0, 32, 33], 0, 3, 20),
    "empty_ends": ([0, 5, 0, 0, 70, 0], 9, 5, 33),
    "narrow": ([40, 3], 1, 1, 1),
    "batch": (None, 0, 4, 64),          # B x T without cu_seqlens
    "long": ([2049], 0, 1, 36),
    "many": ([3] * 70 + [130], 2, 2, 16),
}
G_MIN = -5.0


def make(shape, dtype, gate, seed=0):
    lens, tail, H, d = SHAPES[shape] if isinstance(shape, str) else shape
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    batch = lens is None
    lens = [97] * 3 if batch else lens
    T, N = sum(lens) + tail, len(lens)
    n = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    a = dict(x=n(T, H, d).to(DT[dtype]), initial_state=n(N, H, d), d_out=n(T, H, d).to(DT[dtype]), dST=n(N, H, d))
    if gate == "logit":
        a["decay"] = (2 * n(T, H, d) - 3).to(DT[dtype])
        a["A_log"] = 0.3 * n(H)
    else:
        a["decay"] = (-torch.exp(n(T, H, d) * 2 - 3)).to(DT[gate])
        a["A_log"] = None
    cu = np.concatenate([[0], np.cumsum(lens)])
    a["cu"] = [int(c) for c in cu]
    a["cu_seqlens"] = None if batch else torch.tensor(cu, dtype=torch.int32, device=DEV)
    a["B"] = 3 if batch else None
    return a


def definition(a, write, bwd=False, use_state=True):
    return ref.scan(np64(a["x"]), np64(a["decay"]), np64(a["A_log"]), G_MIN, np64(a["initial_state"]) if use_state
                    else None, a["cu"], write, np64(a["d_out"]) if bwd else None,
                    np64(a["dST"]) if bwd and use_state else None)


def live_rows(a):
    return a["cu"][-1]


def check(got, want, dtype, rows, what):
    v, e = want
    if rows is not None:
        got, v, e = got[:rows], v[:rows], e[:rows]
    assert_within(got, v, e, dtype, what)


@pytest.mark.parametrize("write", ["one", "complement"])
@pytest.mark.parametrize("dtype,gate", KINDS)
@pytest.mark.parametrize("shape", list(SHAPES))
def test_forward_and_gradients(kda, shape, dtype, gate, write):
    a = make(shape, dtype, gate)
    rows = live_rows(a)
    want = definition(a, write, bwd=True)
    mark = 7.0  # rows behind the last sequence keep it
    out = torch.full_like(a["x"], mark)
    o, fs, states = kda.kda_scan_fwd(a["x"], a["decay"], a["A_log"], G_MIN, a["initial_state"], a["cu_seqlens"],
                                     out, write=write, want_states=True, B=a["B"], validate=True)
    assert o is out
    check(o, want["out"], a["x"].dtype, rows, "out")
    check(fs, want["final_state"], torch.float32, None, "final_state")
    assert (out[rows:] == mark).all()
    for st in (states, None):
        gr = dict(dx=torch.full_like(a["x"], mark), d_decay=torch.full_like(a["decay"], mark),
                  dA_log=None if a["A_log"] is None else torch.empty_like(a["A_log"]),
                  d_initial_state=torch.empty_like(fs))
        kda.kda_scan_bwd(a["x"], a["decay"], a["d_out"], a["A_log"], G_MIN, a["initial_state"], a["dST"],
                         a["cu_seqlens"], st, write=write, B=a["B"], grads=gr)
        check(gr["dx"], want["dx"], a["x"].dtype, rows, "dx")
        check(gr["d_decay"], want["d_decay"], a["decay"].dtype, rows, "d_decay")
        check(gr["d_initial_state"], want["d_initial_state"], torch.float32, None, "d_initial_state")
        if a["A_log"] is not None:
            check(gr["dA_log"], want["dA_log"], torch.float32, None, "dA_log")
        assert (gr["dx"][rows:] == mark).all() and (gr["d_decay"][rows:] == mark).all()


LAYOUTS = {
    # few chains, long: a cluster of CTAs along the sequence; and the same elementwise
    "cluster": ([5000, 90], 1, 1, 32),
    "cluster_elementwise": ([1500, 90], 1, 1, 33),
    # up to one block of 16 channels for an SM: rings of 16 (8 in fp32) warps, several rounds
    "ring16": ([1500], 2, 25, 64),
    # more of them: rings of 8 warps
    "ring8": ([700, 40], 3, 24, 64),
    # enough blocks of 64 channels
    "wide": ([300, 129, 128, 15], 5, 48, 64),
}


@pytest.mark.parametrize("dtype,gate", KINDS)
@pytest.mark.parametrize("shape", list(LAYOUTS))
def test_every_layout(kda, shape, dtype, gate):
    """Shapes on both sides of each rule that lays chains over the GPU."""
    write = "complement" if gate != "fp32" else "one"
    a = make(LAYOUTS[shape], dtype, gate, seed=40)
    rows = live_rows(a)
    want = definition(a, write, bwd=True)
    o, fs, states = kda.kda_scan_fwd(a["x"], a["decay"], a["A_log"], G_MIN, a["initial_state"], a["cu_seqlens"],
                                     write=write, want_states=True)
    check(o, want["out"], a["x"].dtype, rows, "out")
    check(fs, want["final_state"], torch.float32, None, "final_state")
    gr = kda.kda_scan_bwd(a["x"], a["decay"], a["d_out"], a["A_log"], G_MIN, a["initial_state"], a["dST"],
                          a["cu_seqlens"], states, write=write)
    check(gr["dx"], want["dx"], a["x"].dtype, rows, "dx")
    check(gr["d_decay"], want["d_decay"], a["decay"].dtype, rows, "d_decay")
    check(gr["d_initial_state"], want["d_initial_state"], torch.float32, None, "d_initial_state")
    if a["A_log"] is not None:
        check(gr["dA_log"], want["dA_log"], torch.float32, None, "dA_log")


@pytest.mark.parametrize("dtype,gate", KINDS)
def test_without_states(kda, dtype, gate):
    """No initial state, no final state wanted, no final-state gradient."""
    a = make("tile_edges", dtype, gate, seed=1)
    want = definition(a, "one", bwd=True, use_state=False)
    o, fs = kda.kda_scan_fwd(a["x"], a["decay"], a["A_log"], G_MIN, None, a["cu_seqlens"], want_final_state=False)
    assert fs is None
    check(o, want["out"], a["x"].dtype, None, "out")
    gr = kda.kda_scan_bwd(a["x"], a["decay"], a["d_out"], a["A_log"], G_MIN, None, None, a["cu_seqlens"],
                          want_d_initial_state=False)
    assert gr["d_initial_state"] is None
    check(gr["dx"], want["dx"], a["x"].dtype, None, "dx")
    check(gr["d_decay"], want["d_decay"], a["decay"].dtype, None, "d_decay")


@pytest.mark.parametrize("write", ["one", "complement"])
@pytest.mark.parametrize("dtype,gate", KINDS)
@pytest.mark.parametrize("N,H,d", [(1, 32, 128), (5, 3, 33), (64, 2, 20)])
def test_step(kda, N, H, d, dtype, gate, write):
    a = make(([1] * N, 0, H, d), dtype, gate, seed=2)
    want = definition(a, write)
    before = a["initial_state"].clone()
    out, st = kda.kda_scan_step(a["x"], a["decay"], a["initial_state"], a["A_log"], G_MIN,
                                state_out=torch.empty_like(before), write=write, validate=True)
    check(out, want["out"], a["x"].dtype, None, "out")
    check(st, want["final_state"], torch.float32, None, "state")
    assert torch.equal(before, a["initial_state"])
    out2, st2 = kda.kda_scan_step(a["x"], a["decay"], a["initial_state"], a["A_log"], G_MIN, write=write)
    assert st2 is a["initial_state"] and torch.equal(st2, st) and torch.equal(out2, out)


def test_steps_are_the_prefill(kda):
    """Token by token through the step, and in one call: same states within the bounds."""
    a = make(([50] * 4, 0, 2, 64), "bf16", "logit", seed=3)
    want = definition(a, "complement")
    x = a["x"].view(4, 50, 2, 64)
    z = a["decay"].view(4, 50, 2, 64)
    st = a["initial_state"].clone()
    for t in range(50):
        o, _ = kda.kda_scan_step(x[:, t].contiguous(), z[:, t].contiguous(), st, a["A_log"], G_MIN, write="complement")
        v, e = (w.reshape(4, 50, 2, 64)[:, t] for w in want["out"])
        assert_within(o, v, e, torch.bfloat16, f"token {t}")
    check(st, want["final_state"], torch.float32, None, "final state")
    o4, fs4 = kda.kda_scan_fwd(x, z, a["A_log"], G_MIN, a["initial_state"], write="complement")
    assert o4.shape == x.shape
    check(fs4, want["final_state"], torch.float32, None, "final state of the prefill")


def test_slow_decay_over_a_long_sequence(kda):
    """alpha = exp(-2e-5) constant: a memory of 50,000 tokens.  Rounding alpha
    itself to fp32 would shift it by up to 3e-8, that is the state by up to
    1.5e-3; the bound of the definition test (64 half steps a token of the
    state's running sum) stands below."""
    T, D = 60000, 24
    gen = torch.Generator(device=DEV)
    gen.manual_seed(4)
    x = torch.randn(T, 1, D, generator=gen, device=DEV) + 1.0
    g = torch.full_like(x, -2e-5)
    out, fs = kda.kda_scan_fwd(x, g)
    h = torch.zeros(1, D, dtype=torch.float64)
    xs, a = x.double().cpu(), torch.exp(g.double().cpu()[0])
    for t in range(T):
        h = a * h + xs[t]
    # every token rounds the state once (2^-24 of it, unbiased: 50,000 of them reach sqrt(50000) = 224 half
    # steps at one sigma); 1500 half steps is over 6 sigma and still 16 times under the loss of a rounded alpha
    assert ((fs.double().cpu()[0] - h).abs() <= 1500 * ref.U * h.abs()).all()


def test_full_and_no_decay(kda):
    """alpha = 0 drops a large state exactly; alpha = 1 keeps it exactly."""
    x = torch.randn(40, 2, 12, device=DEV)
    g = torch.zeros_like(x)
    g[17] = -float("inf")
    s0 = torch.full((1, 2, 12), 1e30, device=DEV)
    out, _ = kda.kda_scan_fwd(x, g, None, initial_state=s0, cu_seqlens=torch.tensor([0, 40], dtype=torch.int32, device=DEV),
                              validate=True)
    assert torch.equal(out[17], x[17])
    assert torch.equal(out[:17], torch.full_like(out[:17], 1e30))
    keep, _ = kda.kda_scan_fwd(torch.zeros_like(x), torch.zeros_like(x), initial_state=s0)
    assert torch.equal(keep, torch.full_like(keep, 1e30))
    big = torch.full_like(x, -200.0)  # far below the gate's floor: alpha underflows to 0
    o, _ = kda.kda_scan_fwd(x, big, initial_state=s0)
    assert torch.equal(o, x)


def test_infinite_logits(kda):
    """z = -inf keeps the state, z = +inf decays by exp(g_min); gradients by z are 0 there, and dA_log is finite."""
    a = make(([30, 30], 0, 2, 8), "fp32", "logit", seed=5)
    a["decay"][3:9] = -float("inf")
    a["decay"][40:44] = float("inf")
    want = definition(a, "one", bwd=True)
    out, fs = kda.kda_scan_fwd(a["x"], a["decay"], a["A_log"], G_MIN, a["initial_state"], a["cu_seqlens"], validate=True)
    check(out, want["out"], torch.float32, None, "out")
    gr = kda.kda_scan_bwd(a["x"], a["decay"], a["d_out"], a["A_log"], G_MIN, a["initial_state"], a["dST"], a["cu_seqlens"])
    check(gr["dx"], want["dx"], torch.float32, None, "dx")
    assert (gr["d_decay"][3:9].abs() < 1e-30).all() and (gr["d_decay"][40:44].abs() < 1e-30).all()
    check(gr["dA_log"], want["dA_log"], torch.float32, None, "dA_log")


def test_nan_and_inf_stay_in_their_chain(kda):
    """A NaN input reaches the later tokens of its own channel and sequence, and nothing else."""
    a = make(([60, 60], 0, 2, 40), "bf16", "fp32", seed=6)
    clean, _ = kda.kda_scan_fwd(a["x"], a["decay"], None, G_MIN, a["initial_state"], a["cu_seqlens"])
    x = a["x"].clone()
    x[20, 1, 7] = float("nan")
    x[70, 0, 3] = float("inf")
    out, fs = kda.kda_scan_fwd(x, a["decay"], None, G_MIN, a["initial_state"], a["cu_seqlens"])
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[20:60, 1, 7] = True
    hit[70:120, 0, 3] = True
    assert torch.equal(out[~hit], clean[~hit])
    assert out[20:60, 1, 7].isnan().all() and not out[70:, 0, 3].isfinite().any()


def test_in_place_resume(kda):
    """A sequence in two calls through one state buffer, final_state = initial_state."""
    a = make(([90], 0, 3, 20), "fp32", "fp32", seed=7)
    want = definition(a, "one")
    st = a["initial_state"]
    for lo, hi in ((0, 37), (37, 90)):
        o, fs = kda.kda_scan_fwd(a["x"][lo:hi], a["decay"][lo:hi], initial_state=st, final_state=st)
        assert fs is st
        v, e = (w[lo:hi] for w in want["out"])
        assert_within(o, v, e, torch.float32, "out")
    check(st, want["final_state"], torch.float32, None, "final_state")


def test_unaligned_tensors(kda):
    """Views that start off a 16-byte boundary give the results of aligned ones."""
    a = make(([70], 0, 2, 32), "bf16", "fp32", seed=8)

    def shifted(t):
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].view(t.shape)
        return b.copy_(t)

    want = definition(a, "one", bwd=True)
    b = {n: shifted(a[n]) for n in ("x", "decay", "initial_state", "d_out", "dST")}
    o, fs = kda.kda_scan_fwd(b["x"], b["decay"], initial_state=b["initial_state"], out=shifted(a["x"]))
    check(o, want["out"], torch.bfloat16, None, "out")
    gr = kda.kda_scan_bwd(b["x"], b["decay"], b["d_out"], initial_state=b["initial_state"], d_final_state=b["dST"])
    for n in ("dx", "d_decay", "d_initial_state"):
        check(gr[n], want[n], gr[n].dtype, None, n)


def test_no_tokens(kda):
    s0 = torch.randn(2, 3, 8, device=DEV)
    x = torch.empty(0, 3, 8, device=DEV)
    cu = torch.zeros(3, dtype=torch.int32, device=DEV)
    o, fs = kda.kda_scan_fwd(x, x, initial_state=s0, cu_seqlens=cu, validate=True)
    assert o.numel() == 0 and torch.equal(fs, s0)
    A = torch.zeros(3, device=DEV)
    gr = kda.kda_scan_bwd(x, x, x, A, initial_state=s0, d_final_state=s0, cu_seqlens=cu)
    assert torch.equal(gr["d_initial_state"], s0) and torch.equal(gr["dA_log"], torch.zeros_like(A))
    o, fs = kda.kda_scan_fwd(x, x, B=2)
    assert torch.equal(fs, torch.zeros_like(s0))


def test_results_repeat_bitwise(kda):
    a = make(([700, 1, 300], 0, 3, 72), "bf16", "logit", seed=9)
    runs = []
    for _ in range(2):
        o, fs, st = kda.kda_scan_fwd(a["x"], a["decay"], a["A_log"], G_MIN, a["initial_state"], a["cu_seqlens"],
                                     want_states=True)
        gr = kda.kda_scan_bwd(a["x"], a["decay"], a["d_out"], a["A_log"], G_MIN, a["initial_state"], a["dST"],
                              a["cu_seqlens"], st)
        runs.append([o, fs] + list(gr.values()))
    for p, q in zip(*runs):
        assert torch.equal(p, q)


def test_directional_difference(kda):
    """The gradients against central differences of the library's own forward (fp32)."""
    a = make(([33, 47], 0, 2, 16), "fp32", "logit", seed=10)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(11)

    def loss(x, z, A, s0):
        o, fs = kda.kda_scan_fwd(x, z, A, G_MIN, s0, a["cu_seqlens"], write="complement")
        return (o.double() * a["d_out"].double()).sum() + (fs.double() * a["dST"].double()).sum()

    gr = kda.kda_scan_bwd(a["x"], a["decay"], a["d_out"], a["A_log"], G_MIN, a["initial_state"], a["dST"],
                          a["cu_seqlens"], write="complement")
    args = [a["x"], a["decay"], a["A_log"], a["initial_state"]]
    for i, name in enumerate(("dx", "d_decay", "dA_log", "d_initial_state")):
        v = torch.randn(args[i].shape, generator=gen, device=DEV)
        e = 1e-2
        plus, minus = ([t + s * e * v if j == i else t for j, t in enumerate(args)] for s in (1, -1))
        diff = float(loss(*plus) - loss(*minus)) / (2 * e)
        got = float((gr[name].double() * v.double()).sum())
        # e^2 / 6 of the third derivative (of order one per element, random signs over sqrt(n)) and the fp32
        # forward's 1e-6 of a sum of sqrt(n) terms over 2e: below 2e-3 of sqrt(n)
        assert abs(diff - got) <= 2e-3 * np.sqrt(a["x"].numel()) + 2e-3 * abs(got), name


def test_side_stream(kda):
    """A call on a stream of its own, its tensors dropped at once."""
    a = make(([500, 300], 0, 4, 64), "bf16", "fp32", seed=12)
    o0, fs0 = kda.kda_scan_fwd(a["x"], a["decay"], None, G_MIN, a["initial_state"], a["cu_seqlens"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, fs = kda.kda_scan_fwd(a["x"].clone(), a["decay"], None, G_MIN, a["initial_state"], a["cu_seqlens"], stream=side)
    side.synchronize()
    # the clone was made on the current stream without an order to the side stream: only its lifetime is at stake
    torch.cuda.synchronize()
    o, fs = kda.kda_scan_fwd(a["x"], a["decay"], None, G_MIN, a["initial_state"], a["cu_seqlens"], stream=side)
    gr = kda.kda_scan_bwd(a["x"], a["decay"], a["d_out"], None, G_MIN, a["initial_state"], a["dST"], a["cu_seqlens"],
                          stream=side)
    side.synchronize()
    assert torch.equal(o, o0) and torch.equal(fs, fs0)
    ref_gr = kda.kda_scan_bwd(a["x"], a["decay"], a["d_out"], None, G_MIN, a["initial_state"], a["dST"], a["cu_seqlens"])
    assert torch.equal(gr["dx"], ref_gr["dx"])


def test_captured_and_replayed(kda):
    """Two captured graphs (forward + backward each) replayed in turn on new
    inputs, next to eager calls: each has a workspace of its own."""
    def static(seed):
        return make(([260, 64, 1], 0, 3, 40), "fp32", "logit", seed=seed)

    def step(a):
        o, fs, st = kda.kda_scan_fwd(a["x"], a["decay"], a["A_log"], G_MIN, a["initial_state"], a["cu_seqlens"],
                                     want_states=True)
        gr = kda.kda_scan_bwd(a["x"], a["decay"], a["d_out"], a["A_log"], G_MIN, a["initial_state"], a["dST"],
                              a["cu_seqlens"], st)
        gr2 = kda.kda_scan_bwd(a["x"], a["decay"], a["d_out"], a["A_log"], G_MIN, a["initial_state"], a["dST"],
                               a["cu_seqlens"])
        return [o, fs] + list(gr.values()) + list(gr2.values())

    bufs, graphs, outs = [static(20), static(21)], [], []
    step(bufs[0])
    torch.cuda.synchronize()
    for b in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(b))
        graphs.append(g)
    for rnd in range(2):
        fresh = [static(30 + 2 * rnd), static(31 + 2 * rnd)]
        for b, f in zip(bufs, fresh):
            for n in ("x", "decay", "A_log", "initial_state", "d_out", "dST"):
                b[n].copy_(f[n])
        for g in graphs:
            g.replay()
        want = [step(f) for f in fresh]
        torch.cuda.synchronize()
        for got, w in zip(outs, want):
            for p, q in zip(got, w):
                assert torch.equal(p, q)


def test_malformed_cu_seqlens(kda):
    """Refused in validate mode; without it no memory outside the tensors is touched."""
    x = torch.randn(64, 2, 16, device=DEV)
    g = -torch.rand_like(x)
    for bad in ([1, 30, 64], [0, 40, 30], [0, 30, 65], [0, -3, 64]):
        cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
        with pytest.raises(kda.KdaError, match="KDA_ERR_RANGE"):
            kda.kda_scan_fwd(x, g, cu_seqlens=cu, validate=True)
    buf = torch.full((64 + 128, 2, 16), 5.0, device=DEV)
    cu = torch.tensor([-50, 40, 1000], dtype=torch.int32, device=DEV)
    kda.kda_scan_fwd(x, g, cu_seqlens=cu, out=buf[64:128])
    torch.cuda.synchronize()
    assert (buf[:64] == 5).all() and (buf[128:] == 5).all()


def test_rows_behind_the_last_sequence_are_not_read(kda):
    """NaN there passes validate mode and reaches nothing."""
    a = make(([40, 23], 9, 2, 24), "fp32", "logit", seed=41)
    clean = kda.kda_scan_bwd(a["x"], a["decay"], a["d_out"], a["A_log"], G_MIN, a["initial_state"], a["dST"], a["cu_seqlens"])
    o0, fs0 = kda.kda_scan_fwd(a["x"], a["decay"], a["A_log"], G_MIN, a["initial_state"], a["cu_seqlens"])
    for n in ("x", "decay", "d_out"):
        a[n][63:] = float("nan")
    o, fs = kda.kda_scan_fwd(a["x"], a["decay"], a["A_log"], G_MIN, a["initial_state"], a["cu_seqlens"], validate=True)
    gr = kda.kda_scan_bwd(a["x"], a["decay"], a["d_out"], a["A_log"], G_MIN, a["initial_state"], a["dST"], a["cu_seqlens"],
                          validate=True)
    assert torch.equal(o[:63], o0[:63]) and torch.equal(fs, fs0)
    assert torch.equal(gr["dA_log"], clean["dA_log"]) and torch.equal(gr["d_initial_state"], clean["d_initial_state"])
    assert torch.equal(gr["dx"][:63], clean["dx"][:63])


def test_lowest_values_as_masks(kda):
    """The type's lowest value in place of -inf: as a log-decay it forgets, as a logit it keeps."""
    for dt in (torch.float32, torch.bfloat16):
        low = torch.finfo(dt).min
        x = torch.randn(50, 1, 16, device=DEV).to(dt)
        g = torch.full_like(x, -0.01)
        g[20:23] = low
        g2 = g.clone()
        g2[20:23] = -float("inf")
        s0 = torch.full((1, 1, 16), 1e20, device=DEV)
        for write in ("one", "complement"):
            p, q = (kda.kda_scan_fwd(x, v, initial_state=s0, write=write) for v in (g, g2))
            assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])
            assert torch.equal(p[0][20:23], x[20:23])
            A = torch.zeros(1, device=DEV)
            r = kda.kda_scan_bwd(x, g, x, A, d_final_state=s0, write=write)
            r2 = kda.kda_scan_bwd(x, g2, x, A, d_final_state=s0, write=write)
            for n in r:
                assert r[n].isfinite().all() and torch.equal(r[n], r2[n]), n


@pytest.mark.skipif(torch.cuda.is_available() and torch.cuda.mem_get_info()[1] < 80 << 30, reason="needs 80 GB")
def test_offsets_past_32_bits(kda):
    """2.3e9 elements: the tail behind a token that forgets, against a call on the tail alone."""
    T, H, d, cut = 70010, 256, 128, 69950
    gen = torch.Generator(device=DEV)
    gen.manual_seed(42)
    x = torch.randn(T, H, d, generator=gen, device=DEV, dtype=torch.bfloat16)
    g = torch.full_like(x, -0.125)
    g[cut] = -float("inf")
    o, fs, st = kda.kda_scan_fwd(x, g, want_states=True)
    o2, fs2 = kda.kda_scan_fwd(x[cut:], g[cut:])
    # the two calls cut the tail into tiles at other tokens: fp32 roundings, then one of bf16
    assert float((o[cut:].float() - o2.float()).norm() / o2.float().norm()) <= 2.0 ** -8
    assert float((fs - fs2).norm() / fs2.norm()) <= 1e-5
    gr = kda.kda_scan_bwd(x, g, x, states=st)
    g2 = kda.kda_scan_bwd(x[cut:], g[cut:], x[cut:])
    for n in ("dx", "d_decay"):
        assert float((gr[n][cut:].float() - g2[n].float()).norm() / g2[n].float().norm()) <= 2.0 ** -8, n


def test_value_checks(kda):
    x = torch.randn(8, 1, 4, device=DEV)
    for bad in (0.5, float("nan")):
        g = torch.zeros_like(x)
        g[3, 0, 2] = bad
        with pytest.raises(kda.KdaError, match="KDA_ERR_RANGE"):
            kda.kda_scan_fwd(x, g, validate=True)
    A = torch.zeros(1, device=DEV)
    z = torch.zeros_like(x)
    z[0, 0, 0] = float("nan")
    with pytest.raises(kda.KdaError, match="KDA_ERR_RANGE"):
        kda.kda_scan_fwd(x, z, A, validate=True)
    with pytest.raises(kda.KdaError, match="KDA_ERR_RANGE"):
        kda.kda_scan_fwd(x, torch.zeros_like(x), torch.full_like(A, float("inf")), validate=True)
    with pytest.raises(kda.KdaError, match="KDA_ERR_RANGE"):
        kda.kda_scan_fwd(x, torch.zeros_like(x), A, 0.0)
