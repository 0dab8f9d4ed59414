"""The recurrence-block operators together, as a model uses them: a block of
KDA and a block of the gated linear recurrence on one residual stream, forward
and backward, against the same two blocks in fp64 under torch's autograd (CPU);
and generation token by token against the prefill."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
G_MIN, EPS = -5.0, 1e-6


def params(H, d, seed):
    gen = torch.Generator().manual_seed(seed)
    M = H * d
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    p = {"pre1": 1 + 0.1 * n(M), "pre2": 1 + 0.1 * n(M), "post": 1 + 0.1 * n(d), "post2": 1 + 0.1 * n(M),
         "scale1": 0.7 + 0.1 * n(M), "scale2": 0.5 + 0.1 * n(M), "A": 0.2 * n(H)}
    for name in ("wq", "wk", "wv", "wg", "wo", "wx", "wz", "wg2"):
        p[name] = n(M, M) / np.sqrt(M)
    return {k: v.float().double() for k, v in p.items()}  # fp32 values, so that both sides start alike


def rms(v, w, eps=EPS):
    return v * w / torch.sqrt(v.pow(2).mean(-1, keepdim=True) + eps)


def blocks_fp64(p, x, la, beta, s0, h0):
    """x [T, M]; la [T, H, d]; beta [T, H]; s0 [1, H, d, d]; h0 [1, H, d]."""
    T, M = x.shape
    H, d = la.shape[1:]
    n = rms(x, p["pre1"])
    q, k, v, gate = ((n @ p[w]).view(T, H, d) for w in ("wq", "wk", "wv", "wg"))
    k = k / k.norm(dim=-1, keepdim=True)
    S, rows = s0[0], []
    for t in range(T):
        S = torch.exp(la[t])[:, :, None] * S
        u = beta[t][:, None] * (v[t] - torch.einsum("hkv,hk->hv", S, k[t]))
        S = S + k[t][:, :, None] * u[:, None, :]
        rows.append(torch.einsum("hkv,hk->hv", S, q[t]))
    o = torch.stack(rows)
    y = torch.sigmoid(gate) * rms(o, p["post"])
    x = x + p["scale1"] * (y.reshape(T, M) @ p["wo"])
    n = rms(x, p["pre2"])
    xs, z, gate2 = (n @ p[w] for w in ("wx", "wz", "wg2"))
    g = G_MIN * torch.sigmoid(torch.exp(p["A"])[:, None] * z.view(T, H, d))
    h, rows = h0[0], []
    for t in range(T):
        h = torch.exp(g[t]) * h - torch.expm1(g[t]) * xs.view(T, H, d)[t]
        rows.append(h)
    hs = torch.stack(rows).reshape(T, M)
    return x + p["scale2"] * torch.sigmoid(gate2) * rms(hs, p["post2"]), S, h


def test_two_blocks_forward_and_backward(kda):
    T, H, d = 75, 2, 64
    M = H * d
    p64 = params(H, d, 0)
    gen = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=gen).double()  # noqa: E731
    x64, la64 = n(T, M), -torch.exp(n(T, H, d) - 2).float().double()
    beta64 = torch.sigmoid(n(T, H)).float().double()
    s064, h064 = 0.1 * n(1, H, d, d), n(1, H, d)
    s064 = s064.float().double()
    dy = n(T, M)

    leaf = {k: v.clone().requires_grad_() for k, v in {**p64, "x": x64, "s0": s064, "h0": h064}.items()}
    y64, _, _ = blocks_fp64({k: leaf[k] for k in p64}, leaf["x"], la64, beta64, leaf["s0"], leaf["h0"])
    want = dict(zip(leaf, torch.autograd.grad((y64 * dy).sum(), list(leaf.values()))))

    # the library's way, fp32; the projections and the key's normalisation are the model's own
    p = {k: v.float().to(DEV) for k, v in p64.items()}
    x, la, beta, s0, h0 = (t.float().to(DEV).contiguous() for t in (x64, la64, beta64, s064, h064))
    _, n1 = kda.kda_block_norm_fwd(x, post_norm=False, pre_weight=p["pre1"], want_out=False, want_normed=True, pre_eps=EPS)
    q, kraw, v, gate = ((n1 @ p[w]).view(T, H, d) for w in ("wq", "wk", "wv", "wg"))
    knorm = kraw.norm(dim=-1, keepdim=True)
    k = kraw / knorm
    o, _ = kda.kda_chunk_fwd(q, k, v, la, beta, s0)
    y1, _ = kda.kda_block_norm_fwd(o, gate=gate, post_weight=p["post"], post_eps=EPS)
    br = y1.view(T, M) @ p["wo"]
    x1, n2 = kda.kda_block_norm_fwd(br, residual=x, post_norm=False, scale=p["scale1"], pre_weight=p["pre2"],
                                    want_normed=True, pre_eps=EPS)
    xs, z, gate2 = (n2 @ p["wx"]).view(T, H, d), (n2 @ p["wz"]).view(T, H, d), n2 @ p["wg2"]
    hs, _, states = kda.kda_scan_fwd(xs, z, p["A"], G_MIN, h0, write="complement", want_states=True)
    tail = dict(residual=x1, gate=gate2, post_weight=p["post2"], scale=p["scale2"], post_eps=EPS)
    y, _ = kda.kda_block_norm_fwd(hs.view(T, M), **tail)

    got = {}
    dyd = dy.float().to(DEV)
    g5 = kda.kda_block_norm_bwd(hs.view(T, M), dyd, **tail)
    got["post2"], got["scale2"] = g5["d_post_weight"], g5["d_scale"]
    g4 = kda.kda_scan_bwd(xs, z, g5["d_y"].view(T, H, d), p["A"], G_MIN, h0, states=states, write="complement")
    got["A"], got["h0"] = g4["dA_log"], g4["d_initial_state"]
    dxs, dz, dg2 = g4["dx"].view(T, M), g4["d_decay"].view(T, M), g5["d_gate"]
    dn2 = dxs @ p["wx"].T + dz @ p["wz"].T + dg2 @ p["wg2"].T
    got["wx"], got["wz"], got["wg2"] = (n2.T @ t for t in (dxs, dz, dg2))
    g3 = kda.kda_block_norm_bwd(br, g5["d_residual"], dn2, residual=x, post_norm=False, scale=p["scale1"],
                                pre_weight=p["pre2"], pre_eps=EPS)
    got["scale1"], got["pre2"] = g3["d_scale"], g3["d_pre_weight"]
    got["wo"] = y1.view(T, M).T @ g3["d_y"]
    g2 = kda.kda_block_norm_bwd(o, (g3["d_y"] @ p["wo"].T).view(T, H, d), gate=gate, post_weight=p["post"], post_eps=EPS)
    got["post"] = g2["d_post_weight"]
    g1 = kda.kda_chunk_bwd(q, k, v, la, beta, g2["d_y"], s0)
    got["s0"] = g1["d_initial_state"]
    dk = (g1["dk"] - k * (k * g1["dk"]).sum(-1, keepdim=True)) / knorm
    heads = {"wq": g1["dq"], "wk": dk, "wv": g1["dv"], "wg": g2["d_gate"]}
    dn1 = 0
    for w, t in heads.items():
        t = t.reshape(T, M)
        got[w] = n1.T @ t
        dn1 = dn1 + t @ p[w].T
    g0 = kda.kda_block_norm_bwd(x, None, dn1, post_norm=False, pre_weight=p["pre1"], pre_eps=EPS)
    got["pre1"] = g0["d_pre_weight"]
    got["x"] = g0["d_y"] + g3["d_residual"]

    def off(a, b):
        return float((a.double().cpu() - b).norm() / b.norm())

    # the delta rule's fp32 forward and backward are held to 1e-4 each by their own tests; the norms, the scan and
    # the fp32 products (128 terms, 2^-24 each) are below 1e-5; two blocks pass errors on through norms and gates of
    # slope up to about 2
    assert off(y, y64.detach()) <= 5e-4
    assert set(got) == set(want)
    for name in want:
        assert got[name].shape == want[name].shape, name
        assert off(got[name], want[name].detach()) <= 1e-3, (name, off(got[name], want[name].detach()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_generation_after_a_prefill(kda, dtype):
    """Packed prompts, then steps in one captured graph, against one prefill of
    the whole sequences: states and the gated, residual output."""
    H, d, new = 3, 40, 6
    M, lens = H * d, [17, 1, 50]
    gen = torch.Generator(device=DEV).manual_seed(2)
    n = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    whole = [m + new for m in lens]
    N, T = len(lens), sum(whole)
    x, z, gate, res = n(T, H, d).to(dtype), (n(T, H, d) - 2).to(dtype), n(T, M).to(dtype), n(T, M)
    A, w, w2 = 0.2 * n(H), 1 + 0.1 * n(M), 1 + 0.1 * n(M)
    cu = np.concatenate([[0], np.cumsum(whole)])
    icu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    h_all, s_all = kda.kda_scan_fwd(x, z, A, G_MIN, cu_seqlens=icu, write="complement")
    want, want_n = kda.kda_block_norm_fwd(h_all.view(T, M), residual=res, gate=gate, post_weight=w, pre_weight=w2,
                                          want_normed=True)
    at = [torch.arange(cu[i], cu[i] + lens[i], device=DEV) for i in range(N)]
    prompt = torch.cat(at)
    pcu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    _, state = kda.kda_scan_fwd(x[prompt], z[prompt], A, G_MIN, cu_seqlens=pcu, write="complement")
    rows = lambda t: torch.tensor([cu[i] + lens[i] + t for i in range(N)], device=DEV)  # noqa: E731
    bx, bz, bg, br = x[rows(0)].clone(), z[rows(0)].clone(), gate[rows(0)].clone(), res[rows(0)].clone()

    def one():
        h, _ = kda.kda_scan_step(bx, bz, state, A, G_MIN, write="complement")
        return kda.kda_block_norm_fwd(h.view(N, M), residual=br, gate=bg, post_weight=w, pre_weight=w2, want_normed=True)

    keep = state.clone()
    one()
    state.copy_(keep)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, normed = one()
    state.copy_(keep)
    for t in range(new):
        r = rows(t)
        for buf, src in ((bx, x), (bz, z), (bg, gate), (br, res)):
            buf.copy_(src[r])
        graph.replay()
        torch.cuda.synchronize()
        # the prefill and the steps round fp32 states differently (1e-5 covers their bounds many times), and in bf16
        # both round h once, to neighbours at most (2 half steps of 2^-8), which the norm passes on to `out` and
        # once more, rounded, to `normed`
        tol = 1e-5 if dtype == torch.float32 else 3 * 2.0 ** -8
        for a, b in ((out, want[r]), (normed, want_n[r])):
            assert float((a.double() - b.double()).norm() / b.double().norm()) <= tol
    assert float((state - s_all).norm() / s_all.norm()) <= 1e-5


def test_calls_from_two_threads(kda):
    """Two threads, a stream each, the same calls over and over on data of their own."""
    import threading
    gen = torch.Generator(device=DEV).manual_seed(3)
    sets = []
    for T in (400, 130):
        x, z, do = (torch.randn(T, 3, 40, generator=gen, device=DEV) for _ in range(3))
        sets.append((x, z, do, torch.randn(3, generator=gen, device=DEV) * 0.2))

    def calls(x, z, do, A):
        h, fs, st = kda.kda_scan_fwd(x, z, A, G_MIN, want_states=True)
        g = kda.kda_scan_bwd(x, z, do, A, G_MIN, states=st)
        w = torch.ones(40, device=DEV)
        n = kda.kda_block_norm_bwd(h, do, do, post_weight=w, scale=w, pre_weight=w)
        return [h, fs, *(v for v in g.values() if v is not None), *(v for v in n.values() if v is not None)]

    want = [calls(*s) for s in sets]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(60):
                got = calls(*sets[i])
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
