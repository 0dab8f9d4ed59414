"""A recurrent and a softmax-attention layer of a hybrid model together, as it is
served and trained, against the same layers in fp64 on the CPU."""
import math

import pytest
import torch

import _paged_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-6


def params(M, Hq, Hk, d, seed):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    p = {"pre1": 1 + 0.1 * n(M), "pre2": 1 + 0.1 * n(M), "post": 1 + 0.1 * n(d), "qw": 1 + 0.1 * n(d), "kw": 1 + 0.1 * n(d)}
    for name, cols in (("qkv1", 3 * M), ("g1", M), ("o1", M), ("qkv2", (Hq + 2 * Hk) * d), ("g2", Hq * d)):
        p[name] = n(M, cols) / math.sqrt(M)
    p["o2"] = n(Hq * d, M) / math.sqrt(Hq * d)
    return {k: v.float().double() for k, v in p.items()}


def rms(v, w):
    return v * w / torch.sqrt(v.pow(2).mean(-1, keepdim=True) + EPS)


def layers_fp64(p, x, la, beta, Hq, Hk, d, f):
    """One sequence x [T, M]: a delta-rule block and an attention block, token by token."""
    T, M = x.shape
    n = rms(x, p["pre1"])
    q, k, v = (n @ p["qkv1"]).view(T, 3, -1, d).unbind(1)
    q, k = (t / torch.sqrt(t.pow(2).sum(-1, keepdim=True) + d * EPS) for t in (q, k))
    S, rows = torch.zeros(M // d, d, d, dtype=torch.float64), []
    for t in range(T):
        S = torch.exp(la[t])[:, :, None] * S
        u = beta[t][:, None] * (v[t] - torch.einsum("hkv,hk->hv", S, k[t]))
        S = S + k[t][:, :, None] * u[:, None, :]
        rows.append(torch.einsum("hkv,hk->hv", S, q[t]))
    x = x + (torch.sigmoid((n @ p["g1"]).view(T, -1, d)) * rms(torch.stack(rows), p["post"])).reshape(T, M) @ p["o1"]
    n = rms(x, p["pre2"])
    qkv = (n @ p["qkv2"]).view(T, Hq + 2 * Hk, d)
    pos = torch.arange(T)
    q, _ = R.turn(qkv[:, :Hq], p["qw"], pos, f)
    k, _ = R.turn(qkv[:, Hq:Hq + Hk], p["kw"], pos, f)
    out = torch.empty(T, Hq, d, dtype=torch.float64)
    hidden = torch.ones(T, T, dtype=torch.bool).triu(1)
    for h in range(Hq):
        s = (q[:, h] @ k[:, h // (Hq // Hk)].T / math.sqrt(d)).masked_fill(hidden, -math.inf)
        out[:, h] = torch.softmax(s, -1) @ qkv[:, Hq + Hk + h // (Hq // Hk)]
    return x + (torch.sigmoid(n @ p["g2"]) * out.reshape(T, -1)) @ p["o2"]


class Hybrid:
    """The two layers through the library in fp32, over a paged cache and a recurrent state for each sequence."""

    def __init__(self, kda, p, N, Hq, Hk, d, page, f):
        self.kda, self.Hq, self.Hk, self.d, self.f = kda, Hq, Hk, d, f.to(DEV)
        self.p = {k: v.float().to(DEV) for k, v in p.items()}
        M = p["pre1"].shape[0]
        self.state = torch.zeros(N, M // d, d, d, device=DEV)
        self.cache = torch.full((N * 8, 2, Hk, page, d), math.nan, device=DEV)
        self.table = torch.randperm(N * 8, generator=torch.Generator().manual_seed(1)).view(N, 8).int().to(DEV)
        self.lens = torch.zeros(N, dtype=torch.int32, device=DEV)
        self.l2 = torch.full((d,), d ** -0.5, device=DEV)

    def step(self, x, la, beta, new, cu=None):
        """x [tokens, M] of sequences with `new` [N] more tokens each (cu_seqlens cu, or one each)."""
        kda, p, d = self.kda, self.p, self.d
        T, M = x.shape
        self.lens += new
        _, n = kda.kda_block_norm_fwd(x, post_norm=False, pre_weight=p["pre1"], pre_eps=EPS, want_out=False, want_normed=True)
        qkv = (n @ p["qkv1"]).view(T, 3 * M // d, d)
        H = M // d
        q, k = kda.kda_qk_rope_fwd(qkv[:, :H], qkv[:, H:2 * H], q_weight=self.l2, k_weight=self.l2, eps=EPS)
        v = qkv[:, 2 * H:].contiguous()
        if cu is None:
            o = kda.kda_decode_step(q, k, v, la, beta, self.state)
        else:
            o, self.state = kda.kda_chunk_fwd(q, k, v, la, beta, self.state, cu)
        y, _ = kda.kda_block_norm_fwd(o, gate=(n @ p["g1"]).view(T, H, d), post_weight=p["post"], post_eps=EPS)
        x = x + y.view(T, M) @ p["o1"]
        _, n = kda.kda_block_norm_fwd(x, post_norm=False, pre_weight=p["pre2"], pre_eps=EPS, want_out=False, want_normed=True)
        qkv = (n @ p["qkv2"]).view(T, self.Hq + 2 * self.Hk, d)
        kc, vc = self.cache[:, 0], self.cache[:, 1]
        q = kda.kda_kv_append(qkv[:, self.Hq:self.Hq + self.Hk], qkv[:, self.Hq + self.Hk:], kc, vc, self.table, self.lens, cu,
                              q=qkv[:, :self.Hq], inv_freq=self.f, q_weight=p["qw"], k_weight=p["kw"], norm=True, eps=EPS)
        o, _ = kda.kda_paged_attn(q, kc, vc, self.table, self.lens, cu)
        y, _ = kda.kda_block_norm_fwd(o.view(T, -1), gate=n @ p["g2"], post_norm=False)
        return x + y @ p["o2"]


def test_prefill_in_chunks_then_generation(kda):
    Hq, Hk, d, page, lens = 6, 2, 32, 16, [100, 37, 64]
    M, N = 64, len(lens)
    p = params(M, Hq, Hk, d, 0)
    f = 10000.0 ** (-torch.arange(0, 16, 2, dtype=torch.float64) / 16)
    f = f.float()
    gen = torch.Generator().manual_seed(2)
    xs = [torch.randn(n, M, generator=gen).double() for n in lens]
    las = [-torch.rand(n, M // d, d, generator=gen).double() for n in lens]
    betas = [torch.rand(n, M // d, generator=gen).double() for n in lens]
    want = [layers_fp64(p, x, la, b, Hq, Hk, d, f) for x, la, b in zip(xs, las, betas)]
    net = Hybrid(kda, p, N, Hq, Hk, d, page, f)
    at = [0] * N
    got = [[] for _ in lens]
    last = [n - 5 for n in lens]  # the last five tokens are generated one by one
    for chunk in ([40, 0, 33], [1, 20, 7], [9999] * 3):
        new = [min(c, e - a) for c, e, a in zip(chunk, last, at)]
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        rows = [torch.cat([t[a:a + n] for t, a, n in zip(ts, at, new)]).float().to(DEV) for ts in (xs, las, betas)]
        y = net.step(*rows, torch.tensor(new, dtype=torch.int32, device=DEV), torch.tensor(cu, dtype=torch.int32, device=DEV))
        for n in range(N):
            got[n].append(y[cu[n]:cu[n + 1]])
            at[n] += new[n]
    one = torch.ones(N, dtype=torch.int32, device=DEV)
    for _ in range(5):
        rows = [torch.stack([t[a] for t, a in zip(ts, at)]).float().to(DEV) for ts in (xs, las, betas)]
        y = net.step(*rows, one)
        for n in range(N):
            got[n].append(y[n:n + 1])
            at[n] += 1
    for n in range(N):
        g = torch.cat(got[n]).double().cpu()
        # every operator here is fp32 on values of order 1 (the library's own fp32 tolerance, 1e-4 of a tensor's
        # norm, for each of two layers)
        err = float((g - want[n]).norm() / want[n].norm())
        assert err <= 2e-4, f"sequence {n}: {err:.2e}"
    flags = kda.load()
    import ctypes
    word = ctypes.c_uint(7)
    assert flags.kda_device_watchdog(ctypes.byref(word), 0) == 0 and word.value == 0


def test_unit_queries_and_keys_of_the_recurrence_trained(kda):
    """q and k divided by their L2 norms in front of the delta rule: forward and backward of both."""
    T, H, d, cu = 90, 2, 64, [0, 57, 90]
    gen = torch.Generator().manual_seed(3)
    q, k, v, do = (torch.randn(T, H, d, generator=gen).double() for _ in range(4))
    la, beta = -torch.rand(T, H, d, generator=gen).double(), torch.rand(T, H, generator=gen).double()
    leaf = [t.clone().requires_grad_() for t in (q, k, v)]
    u, w = (t / torch.sqrt(t.pow(2).sum(-1, keepdim=True) + d * EPS) for t in leaf[:2])
    rows = []
    for a, b in zip(cu, cu[1:]):
        S = torch.zeros(H, d, d, dtype=torch.float64)
        for t in range(a, b):
            S = torch.exp(la[t])[:, :, None] * S
            x = beta[t][:, None] * (leaf[2][t] - torch.einsum("hkv,hk->hv", S, w[t]))
            S = S + w[t][:, :, None] * x[:, None, :]
            rows.append(torch.einsum("hkv,hk->hv", S, u[t]))
    o = torch.stack(rows)
    want = torch.autograd.grad((o * do).sum(), leaf)
    g = lambda t: t.float().to(DEV).contiguous()  # noqa: E731
    l2, icu = torch.full((d,), d ** -0.5, device=DEV), torch.tensor(cu, dtype=torch.int32, device=DEV)
    uq, uk = kda.kda_qk_rope_fwd(g(q), g(k), q_weight=l2, k_weight=l2, eps=EPS)
    out, _ = kda.kda_chunk_fwd(uq, uk, g(v), g(la), g(beta), cu_seqlens=icu)
    gr = kda.kda_chunk_bwd(uq, uk, g(v), g(la), g(beta), g(do), cu_seqlens=icu)
    gx = kda.kda_qk_rope_bwd(gr["dq"], gr["dk"], g(q), g(k), q_weight=l2, k_weight=l2, eps=EPS)
    # the library's fp32 tolerance of the delta rule's outputs and gradients
    for name, got, ref in (("out", out, o.detach()), ("dq", gx["d_q"], want[0]), ("dk", gx["d_k"], want[1]), ("dv", gr["dv"], want[2])):
        err = float((got.double().cpu() - ref).norm() / ref.norm())
        assert err <= 1e-4, f"{name}: {err:.2e}"
