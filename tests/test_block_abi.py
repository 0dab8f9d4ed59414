"""Refusals of the recurrence's and the norms' entry points, on the CPU: each is
reported before any CUDA call."""
import ctypes

import pytest
import torch

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    from hybrid_linear_attention_chunk_gb300 import _lib
    return _lib.load()


def scan_desc(**kw):
    from hybrid_linear_attention_chunk_gb300 import KdaScanDesc
    return KdaScanDesc(**dict(dict(B=1, T=64, H=2, d=16, num_seqs=0, dtype=1, gate_dtype=0, write=0, validate=0), **kw))


def norm_desc(**kw):
    from hybrid_linear_attention_chunk_gb300 import KdaNormDesc
    return KdaNormDesc(**dict(dict(rows=8, width=64, dtype=1, res_dtype=1, post_norm=1, post_eps=1e-6, pre_eps=1e-6), **kw))


def fwd(lib, d, **kw):
    p = dict(x=FAKE, g=2 * FAKE, A=None, g_min=-5.0, s0=None, cu=None, o=3 * FAKE, sT=None, states=None)
    p.update(kw)
    return lib.kda_scan_fwd(ctypes.byref(d), p["x"], p["g"], p["A"], p["g_min"], p["s0"], p["cu"], p["o"], p["sT"],
                            p["states"], None)


def bwd(lib, d, **kw):
    p = dict(x=FAKE, g=2 * FAKE, A=None, g_min=-5.0, s0=None, cu=None, states=None, do=3 * FAKE, dST=None, dx=4 * FAKE,
             dg=5 * FAKE, dA=None, ds0=None, ws=6 * FAKE, n=1 << 19)
    p.update(kw)
    return lib.kda_scan_bwd(ctypes.byref(d), p["x"], p["g"], p["A"], p["g_min"], p["s0"], p["cu"], p["states"],
                            p["do"], p["dST"], p["dx"], p["dg"], p["dA"], p["ds0"], p["ws"], p["n"], None)


def step(lib, d, **kw):
    p = dict(x=FAKE, g=2 * FAKE, A=None, g_min=-5.0, si=3 * FAKE, so=3 * FAKE, o=4 * FAKE)
    p.update(kw)
    return lib.kda_scan_step(ctypes.byref(d), p["x"], p["g"], p["A"], p["g_min"], p["si"], p["so"], p["o"], None)


def test_scan_refusals(lib):
    d = scan_desc
    assert lib.kda_scan_fwd(None, FAKE, FAKE, None, -5.0, None, None, FAKE, None, None, None) == -1
    for n in ("x", "g", "o"):
        assert fwd(lib, d(), **{n: None}) == -1
    for kw in (dict(B=0), dict(T=-1), dict(H=0), dict(d=0), dict(num_seqs=2), dict(write=2), dict(write=-1),
               dict(num_seqs=-1), dict(B=1 << 20, T=1 << 20), dict(H=1 << 16, d=1 << 16)):
        assert fwd(lib, d(**kw)) == -2, kw
    assert fwd(lib, d(B=2, num_seqs=2), cu=9 * FAKE) == -2
    assert fwd(lib, d(), cu=9 * FAKE) == -2                       # cu_seqlens without num_seqs
    assert fwd(lib, d(dtype=2)) == -3 and fwd(lib, d(gate_dtype=5)) == -3
    assert fwd(lib, d(), x=FAKE + 1) == -4 and fwd(lib, d(), g=2 * FAKE + 2) == -4
    assert fwd(lib, d(), sT=7 * FAKE + 2) == -4 and fwd(lib, d(), states=7 * FAKE + 2) == -4
    for g_min in (0.0, -5.5, float("nan"), 1.0):
        assert fwd(lib, d(), A=8 * FAKE, g_min=g_min) == -5, g_min
    assert fwd(lib, d(), o=FAKE) == -8 and fwd(lib, d(), o=2 * FAKE + 64) == -8
    assert fwd(lib, d(), s0=7 * FAKE, sT=7 * FAKE + 4) == -8      # neither equal nor apart
    assert fwd(lib, d(), sT=3 * FAKE) == -8 and fwd(lib, d(), states=FAKE) == -8
    assert fwd(lib, d(), sT=7 * FAKE, states=7 * FAKE) == -8


def test_scan_bwd_refusals(lib):
    d = scan_desc
    for n in ("x", "g", "do", "dx", "dg"):
        assert bwd(lib, d(), **{n: None}) == -1
    assert bwd(lib, d(), A=8 * FAKE) == -1                        # dA_log is due
    assert bwd(lib, d(), dA=8 * FAKE) == -7                       # dA_log without A_log
    assert bwd(lib, d(), dx=4 * FAKE + 1) == -4 and bwd(lib, d(), ds0=9 * FAKE + 1) == -4
    assert bwd(lib, d(), ws=6 * FAKE + 8) == -4
    assert bwd(lib, d(), n=16) == -2                              # workspace too small
    assert bwd(lib, d(), dx=FAKE) == -8 and bwd(lib, d(), dx=3 * FAKE) == -8 and bwd(lib, d(), dg=4 * FAKE) == -8
    assert bwd(lib, d(), ws=FAKE) == -8 and bwd(lib, d(), states=4 * FAKE) == -8
    assert bwd(lib, d(), dST=9 * FAKE, ds0=9 * FAKE) == -8


def test_scan_step_refusals(lib):
    d = lambda **kw: scan_desc(**dict(dict(B=4, T=1), **kw))  # noqa: E731
    for n in ("x", "g", "si", "so", "o"):
        assert step(lib, d(), **{n: None}) == -1
    assert step(lib, d(T=2)) == -2 and step(lib, d(num_seqs=1)) == -2 and step(lib, d(B=0)) == -2
    assert step(lib, d(), so=3 * FAKE + 16) == -8 and step(lib, d(), o=3 * FAKE) == -8
    assert step(lib, d(), so=FAKE) == -8 and step(lib, d(), si=3 * FAKE + 2, so=7 * FAKE) == -4


def test_scan_sizes(lib):
    n = ctypes.c_size_t()
    assert lib.kda_scan_states_size(ctypes.byref(scan_desc(T=100, H=3, d=5)), ctypes.byref(n)) == 0
    assert n.value == (100 // 16 + 1) * 15 * 4
    # the slots of packed sequences never meet, whatever their lengths
    import random
    r = random.Random(0)
    for _ in range(300):
        lens = [r.choice([0, 1, 15, 16, 17, 31, 32, 33, r.randrange(200)]) for _ in range(r.randrange(1, 12))]
        used, bos = set(), 0
        for i, ln in enumerate(lens):
            mine = {bos // 16 + i + j for j in range((ln + 15) // 16)}
            assert not used & mine
            used |= mine
            bos += ln
        assert not used or max(used) < bos // 16 + len(lens)
    assert lib.kda_scan_states_size(None, ctypes.byref(n)) == -1
    assert lib.kda_scan_states_size(ctypes.byref(scan_desc(H=-1)), ctypes.byref(n)) == -2
    sizes = []
    for logits in (0, 1):
        for have in (0, 1):
            assert lib.kda_scan_bwd_workspace_size(ctypes.byref(scan_desc()), logits, have, ctypes.byref(n)) == 0
            sizes.append(n.value)
    assert sizes[1] == 0 and sizes[2] - sizes[3] == sizes[0] > 0 and sizes[3] > 0


def nfwd(lib, d, **kw):
    p = dict(y=FAKE, res=2 * FAKE, gate=3 * FAKE, w1=None, sc=None, w2=None, out=4 * FAKE, normed=5 * FAKE)
    p.update(kw)
    return lib.kda_block_norm_fwd(ctypes.byref(d), p["y"], p["res"], p["gate"], p["w1"], p["sc"], p["w2"], p["out"],
                                  p["normed"], None)


def nbwd(lib, d, **kw):
    p = dict(y=FAKE, res=2 * FAKE, gate=3 * FAKE, w1=None, sc=None, w2=None, do=4 * FAKE, dn=5 * FAKE, dy=6 * FAKE,
             dres=7 * FAKE, dgate=8 * FAKE, dw1=None, dsc=None, dw2=None, ws=16 * FAKE, n=1 << 24)
    p.update(kw)
    return lib.kda_block_norm_bwd(ctypes.byref(d), p["y"], p["res"], p["gate"], p["w1"], p["sc"], p["w2"], p["do"],
                                  p["dn"], p["dy"], p["dres"], p["dgate"], p["dw1"], p["dsc"], p["dw2"], p["ws"],
                                  p["n"], None)


def test_norm_refusals(lib):
    d = norm_desc
    assert nfwd(lib, d(), y=None) == -1 and nfwd(lib, d(), out=None, normed=None) == -1
    for kw in (dict(rows=-1), dict(width=0), dict(width=8193), dict(rows=1 << 31)):
        assert nfwd(lib, d(**kw)) == -2, kw
    assert nfwd(lib, d(dtype=2)) == -3 and nfwd(lib, d(res_dtype=-1)) == -3
    assert nfwd(lib, d(res_dtype=0), res=None) == -3              # out's dtype without a residual
    assert nfwd(lib, d(post_eps=-1.0)) == -5 and nfwd(lib, d(pre_eps=float("nan"))) == -5
    assert nfwd(lib, d(post_norm=0), w1=9 * FAKE) == -7 and nfwd(lib, d(), normed=None, w2=9 * FAKE) == -7
    assert nfwd(lib, d(), gate=3 * FAKE + 1) == -4 and nfwd(lib, d(), w1=9 * FAKE + 2) == -4
    assert nfwd(lib, d(), out=2 * FAKE + 16) == -8 and nfwd(lib, d(), out=FAKE) == -8
    assert nfwd(lib, d(), normed=2 * FAKE) == -8 and nfwd(lib, d(), normed=4 * FAKE) == -8


def test_norm_bwd_refusals(lib):
    d = norm_desc
    assert nbwd(lib, d(), dy=None) == -1 and nbwd(lib, d(), do=None, dn=None) == -1
    assert nbwd(lib, d(), dgate=None) == -1 and nbwd(lib, d(), gate=None) == -7
    assert nbwd(lib, d(), res=None) == -7                         # d_residual without a residual
    assert nbwd(lib, d(post_norm=0), dw1=9 * FAKE) == -1 and nbwd(lib, d(), dn=None, dw2=9 * FAKE) == -1
    assert nbwd(lib, d(), n=64) == -2 and nbwd(lib, d(), ws=16 * FAKE + 4) == -4
    assert nbwd(lib, d(), dres=4 * FAKE + 2) == -8 and nbwd(lib, d(), dy=FAKE) == -8
    assert nbwd(lib, d(), dsc=9 * FAKE, dw1=9 * FAKE) == -8 and nbwd(lib, d(), dy=4 * FAKE) == -8


def test_sizes_past_32_bits_are_refused():
    from hybrid_linear_attention_chunk_gb300 import _lib
    with pytest.raises(ValueError):
        _lib._scan_sized(1, (1 << 31) + 5, 1, 1, 0, 1, 0, 0, 0)
    with pytest.raises(ValueError):
        _lib._norm_sized(1 << 31, 8, 1, 1, 1, 1e-6, 1e-6)


def test_binding_refusals():
    import hybrid_linear_attention_chunk_gb300 as kda
    x = torch.randn(8, 2, 4)
    g = -torch.rand(8, 2, 4)
    s = torch.zeros(1, 2, 4)
    bad = [
        (ValueError, lambda: kda.kda_scan_fwd(x, g)),                                  # not on a GPU
        (ValueError, lambda: kda.kda_scan_fwd(x[0], g[0])),
        (ValueError, lambda: kda.kda_scan_fwd(x, g[:4])),
        (TypeError, lambda: kda.kda_scan_fwd(x.half(), g)),
        (TypeError, lambda: kda.kda_scan_fwd(x, g.bfloat16(), torch.zeros(2))),        # logits in another dtype
        (ValueError, lambda: kda.kda_scan_fwd(x, g, torch.zeros(3))),
        (ValueError, lambda: kda.kda_scan_fwd(x, g, initial_state=s[:, :1])),
        (TypeError, lambda: kda.kda_scan_fwd(x, g, initial_state=s.double())),
        (ValueError, lambda: kda.kda_scan_fwd(x, g, write="half")),
        (ValueError, lambda: kda.kda_scan_fwd(x, g, B=3)),
        (ValueError, lambda: kda.kda_scan_fwd(x, g, B=2, cu_seqlens=torch.tensor([0, 8], dtype=torch.int32))),
        (TypeError, lambda: kda.kda_scan_fwd(x, g, cu_seqlens=torch.tensor([0, 8]))),
        (ValueError, lambda: kda.kda_scan_fwd(x, g, out=x[:4])),
        (ValueError, lambda: kda.kda_scan_bwd(x, g, x[:4])),
        (TypeError, lambda: kda.kda_scan_bwd(x, g, x.bfloat16())),
        (ValueError, lambda: kda.kda_scan_step(x, g, s)),
        (TypeError, lambda: kda.kda_block_norm_fwd(x.half())),
        (ValueError, lambda: kda.kda_block_norm_fwd(x, residual=x[:4])),
        (TypeError, lambda: kda.kda_block_norm_fwd(x, gate=x.bfloat16())),
        (ValueError, lambda: kda.kda_block_norm_fwd(x, scale=torch.ones(3))),
        (TypeError, lambda: kda.kda_block_norm_fwd(x, post_weight=torch.ones(4).bfloat16())),
        (ValueError, lambda: kda.kda_block_norm_fwd(x)),
        (ValueError, lambda: kda.kda_block_norm_bwd(x, x[:4])),
    ]
    for i, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
