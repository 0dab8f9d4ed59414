"""Refusals of the rotation's, the append's and the paged attention's entry
points, on the CPU: each is reported before any CUDA call."""
import ctypes

import pytest
import torch

M = 1 << 24  # fake addresses, far enough apart for every tensor below


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    from hybrid_linear_attention_chunk_gb300 import _lib
    return _lib.load()


def rope_desc(**kw):
    from hybrid_linear_attention_chunk_gb300 import KdaRopeDesc
    return KdaRopeDesc(**dict(dict(tokens=8, Hq=4, Hk=2, d=64, dtype=1, rot=64, layout=0, rot_scale=1.0, norm=1, eps=1e-6), **kw))


def paged_desc(**kw):
    from hybrid_linear_attention_chunk_gb300 import KdaPagedDesc
    return KdaPagedDesc(**dict(dict(B=2, T=4, Hq=4, Hk=2, d=64, num_seqs=0, page_size=16, num_pages=10, max_pages=5,
                                    dtype=1, rot=64, layout=0, rot_scale=1.0, norm=1, eps=1e-6, causal=1, scale=0.125), **kw))


def fwd(lib, d, **kw):
    p = dict(q=M, k=2 * M, pos=3 * M, f=4 * M, wq=5 * M, wk=6 * M, qo=7 * M, ko=8 * M)
    p.update(kw)
    return lib.kda_qk_rope_fwd(ctypes.byref(d), *(p[n] for n in ("q", "k", "pos", "f", "wq", "wk", "qo", "ko")), None)


def bwd(lib, d, **kw):
    p = dict(q=M, k=2 * M, pos=3 * M, f=4 * M, wq=5 * M, wk=6 * M, dqo=7 * M, dko=8 * M, dq=9 * M, dk=10 * M, dwq=11 * M,
             dwk=12 * M, ws=13 * M, n=1 << 20)
    p.update(kw)
    return lib.kda_qk_rope_bwd(ctypes.byref(d), *(p[n] for n in ("q", "k", "pos", "f", "wq", "wk", "dqo", "dko", "dq", "dk",
                                                                 "dwq", "dwk", "ws", "n")), None)


def append(lib, d, **kw):
    p = dict(q=M, k=2 * M, v=3 * M, lens=4 * M, cu=None, table=5 * M, f=6 * M, wq=7 * M, wk=8 * M, qo=9 * M, kc=10 * M, vc=11 * M)
    p.update(kw)
    return lib.kda_kv_append(ctypes.byref(d), *(p[n] for n in ("q", "k", "v", "lens", "cu", "table", "f", "wq", "wk", "qo",
                                                               "kc", "vc")), None)


def attn(lib, d, **kw):
    p = dict(q=M, kc=2 * M, vc=3 * M, lens=4 * M, cu=None, table=5 * M, out=6 * M, lse=7 * M, ws=8 * M, n=256 << 20)
    p.update(kw)
    return lib.kda_paged_attn(ctypes.byref(d), *(p[n] for n in ("q", "kc", "vc", "lens", "cu", "table", "out", "lse", "ws", "n")), None)


NAN, INF = float("nan"), float("inf")


def test_rope_refusals(lib):
    d = rope_desc
    assert lib.kda_qk_rope_fwd(None, *[M] * 8, None) == -1
    for n in ("q", "k", "qo", "ko", "f", "pos"):
        assert fwd(lib, d(), **{n: None}) == -1, n
    for kw in (dict(tokens=-1), dict(Hq=0), dict(Hk=-1), dict(d=48), dict(d=256), dict(rot=12), dict(rot=72), dict(rot=-8),
               dict(layout=2), dict(q_stride=100), dict(q_stride=260), dict(k_stride=-8), dict(q_out_stride=8),
               dict(tokens=(1 << 31) - 1), dict(Hq=1 << 22), dict(q_stride=1 << 33), dict(tokens=1 << 30, q_stride=1 << 20)):
        assert fwd(lib, d(**kw)) == -2, kw
    assert fwd(lib, d(dtype=2)) == -3
    for n in ("q", "k", "qo", "ko"):
        assert fwd(lib, d(), **{n: 20 * M + 8}) == -4, n
    for n in ("pos", "f", "wq", "wk"):
        assert fwd(lib, d(), **{n: 20 * M + 2}) == -4, n
    for kw in (dict(eps=-1.0), dict(eps=NAN), dict(rot_scale=INF), dict(rot_scale=NAN)):
        assert fwd(lib, d(**kw)) == -5, kw
    assert fwd(lib, d(norm=0)) == -7 and fwd(lib, d(norm=0), wq=None) == -7
    assert fwd(lib, d(), qo=2 * M) == -8 and fwd(lib, d(), ko=M) == -8 and fwd(lib, d(), ko=7 * M) == -8
    assert fwd(lib, d(), qo=M + 256) == -8 and fwd(lib, d(q_out_stride=264), qo=M) == -8
    assert fwd(lib, d(), qo=5 * M) == -8 and fwd(lib, d(), ko=3 * M) == -8


def test_rope_bwd_refusals(lib):
    d = rope_desc
    for n in ("q", "k", "dqo", "dko", "dq", "dk"):
        assert bwd(lib, d(), **{n: None}) == -1, n
    assert bwd(lib, d(norm=0), wq=None, wk=None) == -7                # weights' gradients without weights
    assert bwd(lib, d(), n=16) == -2 and bwd(lib, d(), ws=13 * M + 8) == -4 and bwd(lib, d(), dwq=11 * M + 1) == -4
    assert bwd(lib, d(dq_stride=8)) == -2
    assert bwd(lib, d(), dq=M) == -8 and bwd(lib, d(), dk=9 * M) == -8 and bwd(lib, d(), dwk=11 * M) == -8
    assert bwd(lib, d(), ws=M) == -8 and bwd(lib, d(), dwq=7 * M) == -8 and bwd(lib, d(), dq=8 * M) == -8
    n = ctypes.c_size_t()
    assert lib.kda_qk_rope_bwd_workspace_size(ctypes.byref(d()), ctypes.byref(n)) == 0 and n.value > 0
    assert lib.kda_qk_rope_bwd_workspace_size(ctypes.byref(d(d=40)), ctypes.byref(n)) == -2 and n.value == 0
    assert lib.kda_qk_rope_bwd_workspace_size(None, ctypes.byref(n)) == -1


def test_parts_of_a_buffer_are_no_aliases(lib):
    # rows beside each other in one buffer: nothing is launched for 0 tokens, but two rows are checked
    s = 8 * 64
    d = rope_desc(tokens=2, q_stride=s, k_stride=s, q_out_stride=s, k_out_stride=s)
    assert fwd(lib, d, q=M, k=M + 4 * 128, qo=M + 128, ko=8 * M) == -8       # shifted by a head
    assert fwd(lib, d, q=M, k=M + 4 * 128, qo=M + 5 * 128, ko=8 * M) == -8   # past the row's end, into the next
    d0 = rope_desc(tokens=0, q_stride=s, k_stride=s, q_out_stride=s, k_out_stride=s)
    assert fwd(lib, d0, q=M, k=M + 4 * 128, qo=M, ko=M + 4 * 128) == 0


def test_append_refusals(lib):
    d = paged_desc
    assert lib.kda_kv_append(None, *[M * (i + 1) for i in range(4)], None, *[M * (i + 5) for i in range(7)], None) == -1
    for n in ("q", "k", "v", "lens", "table", "f", "qo", "kc", "vc"):
        assert append(lib, d(), **{n: None}) == -1, n
    bad = (dict(B=0), dict(T=-1), dict(Hq=0), dict(Hk=0), dict(Hq=3), dict(d=20), dict(num_seqs=2), dict(num_seqs=-1),
           dict(page_size=0), dict(num_pages=0), dict(max_pages=0), dict(page_size=1 << 20, max_pages=1 << 12), dict(q_stride=7),
           dict(cache_stride=16), dict(cache_stride=2052), dict(cache_stride=-8), dict(num_pages=(1 << 31) - 1, cache_stride=1 << 20),
           dict(B=1 << 16, T=1 << 16), dict(B=1 << 30, T=1, Hq=8))
    for kw in bad + (dict(rot=4), dict(v_stride=64), dict(layout=3), dict(out_stride=100)):
        assert append(lib, d(**kw)) == -2, kw
    assert append(lib, d(B=2, num_seqs=2), cu=12 * M) == -2 and append(lib, d(), cu=12 * M) == -2
    assert append(lib, d(dtype=5)) == -3
    for n in ("q", "k", "v", "qo", "kc", "vc"):
        assert append(lib, d(), **{n: 20 * M + 8}) == -4, n
    for n in ("lens", "table", "f", "wq", "wk"):
        assert append(lib, d(), **{n: 20 * M + 2}) == -4, n
    assert append(lib, d(B=1, num_seqs=2), cu=20 * M + 2) == -4
    assert append(lib, d(eps=-1.0)) == -5 and append(lib, d(rot_scale=NAN)) == -5
    assert append(lib, d(norm=0)) == -7 and append(lib, d(), q=None, qo=None) == -7
    assert append(lib, d(), vc=10 * M) == -8 and append(lib, d(), kc=2 * M) == -8 and append(lib, d(), qo=2 * M) == -8
    assert append(lib, d(), kc=4 * M) == -8 and append(lib, d(), qo=10 * M) == -8
    for kw in bad:
        assert attn(lib, d(**kw)) == -2, kw


def test_attn_refusals(lib):
    d = paged_desc
    for n in ("q", "kc", "vc", "lens", "table", "out"):
        assert attn(lib, d(), **{n: None}) == -1, n
    for s in (0.0, -1.0, NAN, INF):
        assert attn(lib, d(scale=s)) == -5, s
    assert attn(lib, d(dtype=2)) == -3
    for n in ("q", "kc", "vc", "out", "ws"):
        assert attn(lib, d(), **{n: 40 * M + 8}) == -4, n
    assert attn(lib, d(), lse=20 * M + 2) == -4 and attn(lib, d(), table=20 * M + 1) == -4
    assert attn(lib, d(), n=64) == -2
    assert attn(lib, d(), out=M) == -8 and attn(lib, d(), out=2 * M) == -8 and attn(lib, d(), lse=6 * M) == -8
    assert attn(lib, d(), ws=M) == -8 and attn(lib, d(), lse=4 * M) == -8
    n = ctypes.c_size_t()
    for dt in (0, 1):
        for T in (1, 400):
            assert lib.kda_paged_attn_workspace_size(ctypes.byref(d(T=T, dtype=dt)), ctypes.byref(n)) == 0
            assert 0 < n.value < 256 << 20 and n.value % 16 == 0
    assert lib.kda_paged_attn_workspace_size(None, ctypes.byref(n)) == -1
    assert lib.kda_paged_attn_workspace_size(ctypes.byref(d(d=8)), ctypes.byref(n)) == -2 and n.value == 0


def test_binding_refuses_before_the_library():
    import hybrid_linear_attention_chunk_gb300 as kda
    q = torch.zeros(4, 2, 64)
    for call in (lambda: kda.kda_qk_rope_fwd(q), lambda: kda.kda_qk_rope_bwd(q, None, q),
                 lambda: kda.kda_kv_append(q, q, q[None], q[None], q, q),
                 lambda: kda.kda_paged_attn(q, q[None], q[None], q, q)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


def test_rows_and_pages_that_share_their_memory_are_refused():
    # (a stride of 0 is dense to the library: one row that stands for all tokens is not)
    from hybrid_linear_attention_chunk_gb300 import _lib
    rows = torch.zeros(12, 3, 16)
    for t, stride in ((rows, 48), (rows[:1].expand(1, 3, 16), 0), (rows[::2], 96), (rows.view(3, 4, 3, 16), 48),
                      (rows.view(3, 4, 3, 16)[:, :1], 192), (rows.view(1, 12, 3, 16), 48), (rows[:0], 0)):
        assert _lib._token_stride("t", t) == stride
    for t in (rows[:1].expand(12, 3, 16), rows[:1, None].expand(3, 4, 3, 16), rows[:3, None].expand(3, 4, 3, 16),
              rows[:4].expand(3, 4, 3, 16), rows[:1, None].expand(3, 1, 3, 16), rows[:, :1].expand(12, 3, 16),
              rows[..., :1].expand(12, 3, 16)):
        with pytest.raises(ValueError):
            _lib._token_stride("t", t)
    pages, one = torch.zeros(5, 2, 8, 16), torch.zeros(1, 2, 8, 16)
    lens, table = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 4, dtype=torch.int32)

    def call(k, v):
        return _lib._paged_call((6, 4, 16), 4, torch.float32, k, v, table, lens, None, -1)
    call(pages, pages)
    call(one.expand(1, 2, 8, 16), one)
    for k, v in ((one.expand(5, 2, 8, 16), one.expand(5, 2, 8, 16)), (pages, one.expand(5, 2, 8, 16)),
                 (one.expand(5, 2, 8, 16), pages), (pages[:, :1].expand(5, 2, 8, 16),) * 2):
        with pytest.raises(ValueError):
            call(k, v)
