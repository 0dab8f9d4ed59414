"""Append to a paged cache and attention over it, against the fp64 definitions."""
import math
import random

import pytest
import torch

import _paged_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def gen_of(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rand(gen, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def bits(t):
    """A tensor's bits: equal ones are equal, NaN included."""
    return t.contiguous().view(torch.int16 if t.dtype is BF else torch.int32)


class Case:
    """Sequences with `new` tokens each and `lens` tokens in the cache after them.  What no
    sequence owns in the cache is NaN, table entries behind a sequence's pages are far off, and `behind`
    token rows lie behind the last sequence."""

    def __init__(self, new, lens, Hq, Hk, d, page, dtype, seed=0, packed=True, behind=0, spare=3, halves=False,
                 std=1.0):
        self.new, self.lens_list, self.page, self.d, self.Hq, self.Hk = new, lens, page, d, Hq, Hk
        self.dtype, self.N, self.T = dtype, len(new), sum(new) + behind
        gen = self.gen = gen_of(seed)
        r = random.Random(seed)
        pages = [(n + page - 1) // page for n in lens]
        total = sum(pages) + spare
        ids = list(range(total))
        r.shuffle(ids)
        most = max(1, max(pages)) + 1
        self.table_list = [[ids.pop() for _ in range(p)] + [-(1 << 31) + i for i in range(most - p)] for p in pages]
        if halves:
            both = torch.full((total, 2, Hk, page, d), math.nan, dtype=dtype, device=DEV)
            self.kc, self.vc = both[:, 0], both[:, 1]
        else:
            self.kc, self.vc = (torch.full((total, Hk, page, d), math.nan, dtype=dtype, device=DEV) for _ in range(2))
        for n, kv in enumerate(lens):
            for c in (self.kc, self.vc):
                for i in range(pages[n]):
                    m = min(page, kv - i * page)
                    c[self.table_list[n][i], :, :m] = rand(gen, Hk, m, d, dtype=dtype, std=std)
        self.table, self.lens = i32(self.table_list), i32(lens)
        self.cu_list = [0]
        for n in new:
            self.cu_list.append(self.cu_list[-1] + n)
        self.cu = i32(self.cu_list) if packed else None
        self.q = rand(gen, self.T, Hq, d, dtype=dtype, std=std)
        if behind:
            self.q[sum(new):] = math.nan

    def at(self, n, j):
        """Page and slot of key j of sequence n."""
        return self.table_list[n][j // self.page], j % self.page

    def attend(self, kda, **how):
        return kda.kda_paged_attn(self.q, self.kc, self.vc, self.table, self.lens, self.cu, **how)

    def check(self, kda, causal=True, scale=None, **how):
        out, lse = torch.full_like(self.q, 7.0), torch.full(self.q.shape[:2], 7.0, device=DEV)
        got = self.attend(kda, causal=causal, scale=scale, out=out, lse=lse, **how)
        assert got[0] is out and got[1] is lse
        ref = R.attention(R.f64(self.q), R.f64(self.kc), R.f64(self.vc), self.table.cpu(), self.lens_list, self.cu_list,
                          causal, scale, self.dtype is BF)
        rows = slice(0, self.cu_list[-1])
        R.assert_within(out[rows], ref[0][rows], ref[1][rows], self.dtype, "out")
        R.assert_within(lse[rows], ref[2][rows], ref[3][rows], F32, "lse")
        assert bool((out[self.cu_list[-1]:] == 7.0).all()) and bool((lse[self.cu_list[-1]:] == 7.0).all())
        alone, none = self.attend(kda, causal=causal, scale=scale, **how)
        assert none is None and torch.equal(bits(alone[rows]), bits(out[rows]))
        return out, lse


HEADS = [(1, 1), (6, 2), (8, 1), (5, 5), (21, 3)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hk", HEADS)
def test_packed_sequences(kda, d, Hq, Hk, dtype):
    new, lens = [3, 0, 1, 70, 17, 1, 5], [40, 9, 200, 70, 130, 1, 5]
    Case(new, lens, Hq, Hk, d, 16, dtype).check(kda)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 64, 100, 128, 256, 1000])
def test_page_sizes(kda, page, dtype):
    Case([5, 1, 33, 140], [300, 257, 33, 500], 4, 2, 64, page, dtype, seed=page).check(kda)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_one_token_each(kda, d, dtype):
    lens = [1, 2, 63, 64, 65, 127, 128, 129, 1000, 0, 3, 500]
    for Hq, Hk in ((8, 2), (3, 3), (16, 1), (40, 1)):
        Case([1] * len(lens), lens, Hq, Hk, d, 32, dtype, packed=False, behind=0).check(kda)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("new,kv,Hq,Hk", [(1, 5000, 4, 1), (1, 5000, 5, 5), (7, 3000, 2, 2), (300, 1500, 8, 4),
                                          (129, 129, 1, 1), (128, 256, 2, 1), (513, 600, 3, 1)])
def test_one_sequence_over_many_blocks(kda, new, kv, Hq, Hk, dtype):
    Case([new], [kv], Hq, Hk, 128, 64, dtype, packed=False).check(kda)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_not_causal(kda, dtype):
    new, lens = [3, 0, 1, 70, 200], [40, 9, 200, 70, 130]
    for d, page in ((64, 16), (128, 48)):
        Case(new, lens, 6, 2, d, page, dtype).check(kda, causal=False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [32, 128])
def test_rows_without_keys(kda, d, dtype):
    # fewer tokens in the cache than new ones: the first rows stand before it; a length of 0 leaves none
    for causal in (True, False):
        Case([5, 4, 200, 3, 1], [2, 0, 150, 3, 0], 4, 2, d, 16, dtype).check(kda, causal=causal)
    Case([1, 1], [0, 0], 4, 2, d, 16, dtype, packed=False).check(kda)
    Case([300], [0], 2, 2, d, 16, dtype).check(kda)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (32, 16)])
def test_rows_behind_the_last_sequence(kda, d, page, dtype):
    Case([30, 1, 200], [30, 100, 300], 4, 2, d, page, dtype, behind=9).check(kda)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [1e-3, 0.3, 3.0])
def test_scales(kda, scale, dtype):
    Case([40, 1], [90, 77], 2, 1, 64, 16, dtype, std=2.0).check(kda, scale=scale)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rising_scores(kda, dtype):
    # every key outweighs those before it by far, so that the running maximum moves at every tile
    for new, kv, d in ((1, 700, 64), (300, 700, 128), (260, 300, 64)):
        c = Case([new], [kv], 2, 1, d, 16, dtype, std=0.1)
        u = torch.ones(d, device=DEV) / math.sqrt(d)
        c.q.copy_((c.q.float() + 4.0 * u).to(dtype))
        for j in range(kv):
            p, s = c.at(0, j)
            c.kc[p, :, s] = (c.kc[p, :, s].float() + 0.5 * j * u).to(dtype)
        c.check(kda, scale=1.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (16, 16), (64, 24)])
@pytest.mark.parametrize("new,kv", [(6, 40), (150, 300), (300, 300)])
def test_values_that_are_not_finite(kda, new, kv, d, page, dtype):
    c = Case([new, 3], [kv, 50], 4, 2, d, page, dtype)
    for j, ch, h, x in ((kv - 1, 1, 0, math.inf), (kv - 2, 5, 1, math.nan), (kv - new // 2, 7, 0, -math.inf),
                        (kv - new // 2, 8, 0, math.inf), (kv - new, 9, 0, math.nan), (kv - 3, 15, 1, math.inf)):
        p, s = c.at(0, j)
        c.vc[p, h, s, ch] = x
    c.check(kda)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("new", [6, 200])
def test_keys_that_are_not_finite(kda, new, dtype):
    c = Case([new, 3], [250, 50], 2, 1, 64, 16, dtype)
    clean, _ = c.check(kda)
    p, s = c.at(0, 250 - 3)
    c.kc[p, 0, s, 4] = math.nan
    out, lse = c.attend(kda, want_lse=True)
    seen = new - 3
    assert torch.equal(out[:seen], clean[:seen]) and torch.equal(out[new:], clean[new:])
    assert bool(torch.isnan(out[seen:new]).all()) and bool(torch.isnan(lse[seen:new]).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_lowest_values(kda, dtype):
    # keys and values at the ends of the type's range
    big = torch.finfo(dtype).max
    c = Case([4], [70], 1, 1, 64, 16, dtype)
    p, s = c.at(0, 10)
    c.vc[p, 0, s, 3] = -big
    p, s = c.at(0, 30)
    c.kc[p, 0, s] = 0
    c.kc[p, 0, s, 0] = 1e30
    c.q[:, :, 0] = -1.0
    c.check(kda)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_sequences(kda, dtype):
    r = random.Random(1)
    new = [r.choice([0, 1, 1, 2, 5, 40]) for _ in range(700)]
    lens = [n + r.choice([0, 0, 3, 30]) for n in new]
    Case(new, lens, 2, 1, 32, 8, dtype).check(kda)


def test_shared_pages(kda):
    # two sequences over the same prefix
    c = Case([2, 2], [64, 64], 4, 2, 64, 16, BF)
    c.table_list[1][:3] = c.table_list[0][:3]
    c.table = i32(c.table_list)
    c.check(kda)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides(kda, dtype):
    c = Case([30, 1, 3], [30, 100, 300], 6, 2, 64, 16, dtype, halves=True)
    want, _ = c.check(kda)
    wide = torch.full((c.T, 10, 64), 3.0, dtype=dtype, device=DEV)
    wide[:, 2:8] = c.q
    out = torch.full((c.T, 7, 64), 3.0, dtype=dtype, device=DEV)
    kda.kda_paged_attn(wide[:, 2:8], c.kc, c.vc, c.table, c.lens, c.cu, out=out[:, 1:])
    assert torch.equal(out[:, 1:], want) and bool((out[:, 0] == 3.0).all())


def test_batched_shapes(kda):
    c = Case([5, 5, 5], [30, 100, 5], 6, 2, 64, 16, BF, packed=False)
    want, lse = c.check(kda)
    out, l4 = kda.kda_paged_attn(c.q.view(3, 5, 6, 64), c.kc, c.vc, c.table, c.lens, want_lse=True)
    assert out.shape == (3, 5, 6, 64) and torch.equal(out.view_as(want), want) and torch.equal(l4.view_as(lse), lse)


def test_no_tokens(kda):
    c = Case([2], [5], 2, 1, 64, 16, BF)
    out, lse = kda.kda_paged_attn(c.q[:0], c.kc, c.vc, c.table, c.lens, i32([0, 0]), want_lse=True)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    out, _ = kda.kda_paged_attn(torch.empty(1, 0, 2, 64, dtype=BF, device=DEV), c.kc, c.vc, c.table, c.lens)
    assert out.shape == (1, 0, 2, 64)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_results_repeat_bitwise(kda, dtype):
    c = Case([300, 1, 40], [700, 2000, 41], 8, 2, 128, 64, dtype)
    runs = [c.attend(kda, want_lse=True) for _ in range(4)]
    assert all(torch.equal(r[0], runs[0][0]) and torch.equal(r[1], runs[0][1]) for r in runs)


def test_joins_with_another_call_by_log_sums(kda):
    # keys in two calls, the later ones causal: the log-sums join them to the one call
    c = Case([40], [240], 4, 2, 64, 8, F32)
    want, wl = c.check(kda)
    a, la = kda.kda_paged_attn(c.q, c.kc, c.vc, c.table, i32([200]), c.cu, causal=False, want_lse=True)
    b, lb = kda.kda_paged_attn(c.q, c.kc, c.vc, c.table[:, 25:].contiguous(), i32([40]), c.cu, want_lse=True)
    l = torch.logaddexp(la, lb)
    got = torch.exp(la - l)[..., None] * a + torch.exp(lb - l)[..., None] * b
    # each part has fp32's error of its own call, below 3e-6 here, and the join adds a few roundings
    assert float((got - want).abs().max()) < 2e-5 and float((l - wl).abs().max()) < 2e-5


@pytest.mark.parametrize("dtype,d,page", [(BF, 128, 64), (BF, 64, 24), (F32, 64, 16)])
def test_captured_and_replayed(kda, dtype, d, page):
    # lengths, tables and sequences are read on the device: a replay sees new ones
    c = Case([200, 1, 3], [300, 500, 3], 4, 2, d, page, dtype)
    size = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(c.q), torch.empty(c.T, 4, device=DEV)

    def call(ws):
        return c.attend(kda, out=out, lse=lse, workspace=ws)
    call(size)
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    for g in (one, two):  # two graphs that share a workspace and run in order
        with torch.cuda.graph(g):
            call(size)
    for lens, cu in (([250, 500, 9], [0, 100, 150, 204]), ([300, 8, 0], [0, 204, 204, 204])):
        c.lens.copy_(i32(lens))
        c.cu.copy_(i32(cu))
        c.q.copy_(rand(c.gen, c.T, 4, d, dtype=dtype))
        for g in (one, two):
            out.fill_(5.0)
            g.replay()
            got, gl = out.clone(), lse.clone()
            call(size)
            assert torch.equal(bits(got), bits(out)) and torch.equal(bits(gl), bits(lse))


def test_two_calls_at_once(kda):
    # two streams, each call with a workspace of its own
    cases = [Case([300, 1, 40], [1700, 2000, 41], 8, 2, 128, 64, BF, seed=1), Case([1] * 9, [3000] * 9, 8, 2, 128, 64, BF, seed=2),
             Case([500], [900], 6, 3, 64, 16, BF, seed=3), Case([70, 3], [400, 300], 4, 2, 32, 16, F32, seed=4)]
    want = [c.attend(kda)[0] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(device=DEV) for _ in cases]
    got = [[c.attend(kda, stream=s)[0] for c, s in zip(cases, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for turn in got:
        for g, w in zip(turn, want):
            assert torch.equal(g, w)


def test_groups_of_one_sequence_in_every_kernel(kda):
    # rows that fill 1, 16, 17, 32, 33, 128, 129, 256 and 257 of a head of the cache, by tokens and by shared heads
    for G, new in ((1, 1), (16, 1), (17, 1), (4, 8), (3, 11), (1, 128), (43, 3), (2, 128), (1, 257)):
        for d in (64, 128):
            Case([new, new], [new + 130, new + 1], 2 * G, 2, d, 16, BF, packed=False).check(kda)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("G", [1, 3, 8, 12])
def test_a_chunk_among_single_tokens(kda, G, d, dtype):
    # few rows to a head on average, one chunk of many items; sequences that see nothing, values that are not finite
    new = [1] * 40 + [97] + [1] * 23
    lens = [(37 * n) % 300 for n in range(40)] + [530] + [(91 * n) % 170 for n in range(23)]
    c = Case(new, lens, 2 * G, 2, d, 16, dtype, seed=G)
    c.check(kda)
    c.check(kda, causal=False)
    for j, x in ((450, math.inf), (500, math.nan), (529, -math.inf)):
        page, slot = c.at(40, j)
        c.vc[page, :, slot, d // 2] = x
    c.check(kda)


def test_side_stream(kda):
    c = Case([300, 1, 40], [700, 2000, 41], 8, 2, 128, 64, BF)
    want, _ = c.attend(kda)
    torch.cuda.synchronize()
    s = torch.cuda.Stream(device=DEV)
    got, _ = c.attend(kda, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("new", [1, 140])
def test_offsets_past_32_bits(kda, new, dtype):
    # a pool of more than 2^31 elements, of which the sequences own the last pages
    page, Hk, d = 64, 8, 128
    pages = (1 << 31) // (page * Hk * d) + 40
    kc, vc = (torch.empty(pages, Hk, page, d, dtype=dtype, device=DEV) for _ in range(2))
    c = Case([new, new], [300, 200], 16, Hk, d, page, dtype)
    own = sorted({p for row in c.table_list for p in row if p >= 0})
    to = {p: pages - 1 - i for i, p in enumerate(own)}
    for p in own:
        kc[to[p]], vc[to[p]] = c.kc[p], c.vc[p]
    table = i32([[to.get(p, -1) for p in row] for row in c.table_list])
    want, _ = c.attend(kda)
    got, _ = kda.kda_paged_attn(c.q, kc, vc, table, c.lens, c.cu)
    assert torch.equal(got, want)
    k, v = rand(c.gen, c.T, Hk, d, dtype=dtype), rand(c.gen, c.T, Hk, d, dtype=dtype)
    kda.kda_kv_append(k, v, kc, vc, table, c.lens, c.cu)
    at = R.slots(table.cpu(), 1, page, range(200 - new, 200))
    assert torch.equal(kc[at[0].to(DEV), :, at[1].to(DEV)], k[new:])
    assert torch.equal(vc[at[0].to(DEV), :, at[1].to(DEV)], v[new:])


# --------------------------------------------------------------------- append

def freqs(rot):
    return (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().to(DEV)


def check_append(kda, c, rot, layout="half", norm=True, with_q=True, rot_scale=1.0, fused=False, **how):
    T, Hq, Hk, d, dtype, gen = c.T, c.Hq, c.Hk, c.d, c.dtype, c.gen
    if fused:
        qkv = rand(gen, T, Hq + 2 * Hk, d, dtype=dtype)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    else:
        q, k, v = (rand(gen, T, H, d, dtype=dtype) for H in (Hq, Hk, Hk))
    wq, wk = ((rand(gen, d), rand(gen, d)) if norm else (None, None))
    f = freqs(rot) if rot else None
    q_out = torch.full((T, Hq, d), 7.0, dtype=dtype, device=DEV) if with_q else None
    kc0, vc0 = c.kc.clone(), c.vc.clone()
    got = kda.kda_kv_append(k, v, c.kc, c.vc, c.table, c.lens, c.cu, q=q if with_q else None, inv_freq=f,
                            q_weight=wq if with_q else None, k_weight=wk, layout=layout, rot_scale=rot_scale, norm=norm,
                            q_out=q_out, **how)
    assert got is q_out
    pos = R.token_positions(T, c.N, c.lens_list, c.cu_list)
    mine = [t for t in range(T) if pos[t] is not None]
    p = torch.tensor([pos[t] for t in mine])
    turn = dict(layout=layout, rot_scale=rot_scale, norm=norm)
    fc = None if f is None else f.cpu()
    if with_q:
        R.assert_within(q_out[mine], *R.turn(R.f64(q)[mine], R.f64(wq), p, fc, **turn), dtype, "q_out")
        rest = [t for t in range(T) if pos[t] is None]
        assert bool((q_out[rest] == 7.0).all())
    yk, ek = R.turn(R.f64(k)[mine], R.f64(wk), p, fc, **turn)
    want_v = vc0.clone()
    seen = torch.zeros(c.kc.shape[0], c.page, dtype=torch.bool)
    for i, t in enumerate(mine):
        if pos[t] < 0:
            continue
        n = next(n for n in range(c.N) if c.cu_list[n] <= t < c.cu_list[n + 1])
        a, s = c.at(n, pos[t])
        seen[a, s] = True
        want_v[a, :, s] = v[t]
        R.assert_within(c.kc[a, :, s], yk[i], ek[i], dtype, f"key of token {t}")
    assert torch.equal(bits(c.vc), bits(want_v))
    rest = (~seen)[:, None, :, None].expand_as(c.kc).to(DEV)
    assert torch.equal(bits(c.kc)[rest], bits(kc0)[rest])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,rot,layout", [(16, 16, "half"), (32, 8, "interleaved"), (64, 64, "half"), (128, 64, "half"),
                                          (128, 128, "interleaved"), (64, 0, "half")])
@pytest.mark.parametrize("page", [1, 16, 24])
def test_append(kda, page, d, rot, layout, dtype):
    new, lens = [3, 0, 1, 20, 5, 1], [40, 9, 50, 20, 3, 0]  # position -2 and -1 of a sequence, and one of length 0
    check_append(kda, Case(new, lens, 6, 2, d, page, dtype, behind=3), rot, layout)
    check_append(kda, Case(new, lens, 6, 2, d, page, dtype, behind=3, halves=True), rot, layout, norm=False,
                 rot_scale=1.5, fused=True)


def test_append_without_queries_and_one_token_each(kda):
    check_append(kda, Case([1] * 9, list(range(9)), 4, 4, 64, 4, BF, packed=False), 64, with_q=False)
    check_append(kda, Case([1] * 9, list(range(9)), 8, 4, 64, 4, BF, packed=False), 64)


def test_append_many_sequences(kda):
    r = random.Random(2)
    new = [r.choice([0, 0, 1, 1, 2, 7]) for _ in range(600)]
    lens = [n + r.choice([0, 3, 30]) for n in new]
    check_append(kda, Case(new, lens, 2, 1, 16, 8, BF), 16)
    check_append(kda, Case([1500, 0, 2, 1000], [1500, 4, 9, 1200], 3, 1, 16, 64, BF), 16)


def test_append_is_the_rotation(kda):
    # the same arithmetic as kda_qk_rope_fwd, bit for bit
    c = Case([50], [50], 4, 2, 128, 16, BF)
    q, k, v = (rand(c.gen, 50, H, 128, dtype=BF) for H in (4, 2, 2))
    w, f = rand(c.gen, 128), freqs(64)
    got = kda.kda_kv_append(k, v, c.kc, c.vc, c.table, c.lens, c.cu, q=q, inv_freq=f, q_weight=w, k_weight=w, norm=True)
    yq, yk = kda.kda_qk_rope_fwd(q, k, torch.arange(50, device=DEV, dtype=torch.int32), f, w, w)
    at = R.slots(c.table.cpu(), 0, 16, range(50))
    assert torch.equal(got, yq) and torch.equal(c.kc[at[0].to(DEV), :, at[1].to(DEV)], yk)
    q2 = q.clone()
    assert kda.kda_kv_append(k, v, c.kc, c.vc, c.table, c.lens, c.cu, q=q2, inv_freq=f, q_weight=w, k_weight=w,
                             norm=True, q_out=q2) is q2
    assert torch.equal(q2, yq)


def test_append_on_a_side_stream_and_captured(kda):
    c = Case([3, 1], [40, 9], 4, 2, 64, 16, BF)
    q, k, v = (rand(c.gen, 4, H, 64, dtype=BF) for H in (4, 2, 2))
    f = freqs(64)
    kc, vc = c.kc.clone(), c.vc.clone()
    want = kda.kda_kv_append(k, v, kc, vc, c.table, c.lens, c.cu, q=q, inv_freq=f)
    s = torch.cuda.Stream(device=DEV)
    s.wait_stream(torch.cuda.current_stream())
    got = kda.kda_kv_append(k, v, c.kc, c.vc, c.table, c.lens, c.cu, q=q, inv_freq=f, stream=s)
    s.synchronize()
    own = ~torch.isnan(vc)
    assert torch.equal(got, want) and torch.equal(c.vc[own], vc[own]) and torch.equal(c.kc[own], kc[own])
    # a captured decode step: append, then attend; its lengths move on by themselves
    c = Case([1, 1], [5, 9], 4, 2, 64, 16, BF, packed=False)
    q, k, v = (rand(c.gen, 2, H, 64, dtype=BF) for H in (4, 2, 2))
    out, qo = torch.empty_like(q), torch.empty_like(q)

    def step():
        c.lens.add_(1)
        kda.kda_kv_append(k, v, c.kc, c.vc, c.table, c.lens, q=q, inv_freq=f, q_out=qo)
        kda.kda_paged_attn(qo, c.kc, c.vc, c.table, c.lens, out=out)
    eager = []
    kc, vc = c.kc.clone(), c.vc.clone()
    for _ in range(4):
        step()
        eager.append(out.clone())
    c.kc.copy_(kc)
    c.vc.copy_(vc)
    c.lens.copy_(i32([5, 9]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        g.replay()
        assert torch.equal(out, eager[i]), i


# ----------------------------------------------------- values that are out of range

def test_value_checks(kda):
    c = Case([3, 1], [40, 9], 4, 2, 64, 16, BF)
    k, v = rand(c.gen, 4, 2, 64, dtype=BF), rand(c.gen, 4, 2, 64, dtype=BF)
    far = c.table.clone()
    far[0, 2] = c.kc.shape[0]
    low = c.table.clone()
    low[1, 0] = -1
    for table, lens, cu in ((c.table, i32([-1, 9]), c.cu), (c.table, i32([40, 65]), c.cu), (c.table, c.lens, i32([1, 3, 4])),
                            (c.table, c.lens, i32([0, 5, 4])), (c.table, c.lens, i32([0, 3, 5])), (far, c.lens, c.cu),
                            (low, c.lens, c.cu)):
        for call in (lambda: kda.kda_paged_attn(c.q, c.kc, c.vc, table, lens, cu, validate=True),
                     lambda: kda.kda_kv_append(k, v, c.kc, c.vc, table, lens, cu, validate=True)):
            with pytest.raises(kda.KdaError) as e:
                call()
            assert e.value.status == -5
    c.check(kda, validate=True)
    check_append(kda, c, 64, validate=True)


def test_clamped_values(kda):
    # without the check: lengths and sequences are cut to their ranges, tokens on pages that do not
    # exist are not stored, and their keys are read from the nearest page
    c = Case([3, 1], [40, 9], 4, 2, 64, 16, BF)
    k, v = rand(c.gen, 4, 2, 64, dtype=BF), rand(c.gen, 4, 2, 64, dtype=BF)
    pages = c.kc.shape[0]
    c.kc.copy_(rand(c.gen, *c.kc.shape, dtype=BF))
    c.vc.copy_(rand(c.gen, *c.vc.shape, dtype=BF))
    bad, good = c.table.clone(), c.table.clone()
    bad[0, 2], good[0, 2] = pages + 5, pages - 1
    bad[1], good[1] = -7, 0
    good.clamp_(0, pages - 1)
    kc, vc = c.kc.clone(), c.vc.clone()
    for lens, cut in (([40, 9], [40, 9]), ([-5, 1 << 30], [0, 64])):
        want, _ = kda.kda_paged_attn(c.q, kc, vc, good, i32(cut), c.cu)
        got, _ = kda.kda_paged_attn(c.q, kc, vc, bad, i32(lens), c.cu)
        assert torch.equal(got, want)
    kda.kda_kv_append(k, v, kc, vc, bad, c.lens, c.cu)
    assert torch.equal(kc, c.kc) and torch.equal(vc, c.vc)
    want, _ = kda.kda_paged_attn(c.q, kc, vc, good, c.lens, i32([0, 4, 4]))
    got, _ = kda.kda_paged_attn(c.q, kc, vc, good, c.lens, i32([-3, 100, 7]))
    assert torch.equal(got, want)


def test_refusals(kda):
    c = Case([3, 1], [40, 9], 4, 2, 64, 16, BF)
    a = (c.kc, c.vc, c.table, c.lens, c.cu)
    for bad in (lambda: kda.kda_paged_attn(c.q.float(), *a), lambda: kda.kda_paged_attn(c.q, c.kc, c.vc.float(), *a[2:]),
                lambda: kda.kda_paged_attn(c.q, *a[:2], c.table.long(), c.lens, c.cu),
                lambda: kda.kda_paged_attn(c.q.half(), c.kc.half(), c.vc.half(), *a[2:])):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: kda.kda_paged_attn(c.q[..., :32].contiguous(), *a), lambda: kda.kda_paged_attn(c.q, c.kc, c.vc[:1], *a[2:]),
                lambda: kda.kda_paged_attn(c.q, *a[:3], c.lens[:1], c.cu), lambda: kda.kda_paged_attn(c.q, *a[:4], c.cu[:2]),
                lambda: kda.kda_paged_attn(c.q[:3], *a[:4]), lambda: kda.kda_paged_attn(c.q.transpose(0, 1), *a),
                lambda: kda.kda_paged_attn(c.q, c.kc.transpose(1, 2), c.vc.transpose(1, 2), *a[2:]),
                lambda: kda.kda_paged_attn(c.q.cpu(), *a), lambda: kda.kda_paged_attn(c.q, *a[:3], c.lens.cpu(), c.cu),
                lambda: kda.kda_kv_append(c.q, c.q, *a), lambda: kda.kda_kv_append(c.q[:, :2], c.q[:, 2:], *a, q_out=c.q)):
        with pytest.raises(ValueError):
            bad()
    k = c.q[:, :2].contiguous()
    for bad, status in ((lambda: kda.kda_paged_attn(c.q[:, :3], *a), -2), (lambda: kda.kda_paged_attn(c.q, *a, scale=0.0), -5),
                        (lambda: kda.kda_paged_attn(c.q, *a, scale=math.nan), -5),
                        (lambda: kda.kda_paged_attn(c.q, *a, out=c.q), -8),
                        (lambda: kda.kda_paged_attn(c.q, *a, workspace=torch.empty(16, dtype=torch.uint8, device=DEV)), -2),
                        (lambda: kda.kda_kv_append(k, k, c.kc, c.kc, *a[2:]), -8),
                        (lambda: kda.kda_kv_append(k, k, *a, inv_freq=freqs(12)), -2),
                        (lambda: kda.kda_kv_append(k, k, *a, k_weight=torch.ones(64, device=DEV)), -7)):
        with pytest.raises(kda.KdaError) as e:
            bad()
        assert e.value.status == status
