"""Workloads of the softmax-attention layers that stand between the recurrent
layers of a hybrid model: the norms of queries and keys with the position
rotation (kda_qk_rope_fwd, kda_qk_rope_bwd), the append of keys and values to
a paged cache (kda_kv_append) and the attention of new tokens over that cache
(kda_paged_attn).

With ``own`` false the operators run in their plain form, elementary torch
operations in fp32 (angles in fp64), rounded once at the end; with ``own``
true they run through the library.  ``exact`` is the definition in fp64.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _lib():
    import hybrid_linear_attention_chunk_gb300 as kda
    return kda


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a training step's query and key norms with the rotation, forward and backward: 4 x 8192 tokens
        dict(name="rope_train", kind="rope_train", T=32768, Hq=32, Hk=8, d=128, rot=128, layout="half", norm=True,
             dtype="bf16", far=0, packed=True),
        # training in fp32 of a small model with a partial, interleaved rotation and a token count of no round size
        dict(name="rope_train_odd", kind="rope_train", T=777, Hq=5, Hk=5, d=64, rot=32, layout="interleaved",
             norm=True, dtype="fp32", far=0, packed=False),
        # prefill at far positions of a long document, frequencies stretched for it, rotation without norms
        dict(name="rope_far", kind="rope", T=8192, Hq=32, Hk=32, d=128, rot=64, layout="interleaved", norm=False,
             dtype="bf16", far=1 << 20, packed=False),
        # one decode step of 256 requests: the new token's query and key normed and rotated, key and value stored
        dict(name="append_decode", kind="append", N=256, T=256, ctx=4096, ragged=True, Hq=32, Hk=8, d=128, rot=128,
             layout="half", norm=True, dtype="bf16", page=64),
        # a batch of prefill chunks of very different lengths appended to their requests' pages
        dict(name="append_chunks", kind="append", N=12, T=16384, ctx=8192, ragged=True, Hq=32, Hk=8, d=128, rot=64,
             layout="half", norm=True, dtype="bf16", page=64),
        # one request generating its next token: a single call's latency
        dict(name="attn_1seq", kind="attn", N=1, T=1, ctx=4096, ragged=False, Hq=32, Hk=8, d=128, dtype="bf16",
             page=64, lse=False),
        # a full decode batch over contexts of very different lengths
        dict(name="attn_decode", kind="attn", N=128, T=128, ctx=8192, ragged=True, Hq=32, Hk=8, d=128, dtype="bf16",
             page=64, lse=False),
        # one token of one request over a very long document
        dict(name="attn_decode_long", kind="attn", N=1, T=1, ctx=262144, ragged=False, Hq=16, Hk=4, d=128,
             dtype="bf16", page=128, lse=True),
        # prefill of one request of 8192 tokens from an empty cache
        dict(name="attn_prefill", kind="attn", N=1, T=8192, ctx=0, ragged=False, Hq=32, Hk=8, d=128, dtype="bf16",
             page=64, lse=False),
        # a chunk of 2048 new tokens over a prefix of 65536 cached ones
        dict(name="attn_chunk_long", kind="attn", N=1, T=2048, ctx=65536, ragged=False, Hq=32, Hk=8, d=128,
             dtype="bf16", page=128, lse=False),
        # a mixed step: 40 requests, most with a few new tokens and some in the middle of their prefill
        dict(name="attn_mixed", kind="attn", N=40, T=5001, ctx=3000, ragged=True, Hq=12, Hk=4, d=64, dtype="bf16",
             page=16, lse=True),
        # a small fp32 model with heads of 32 channels and pages of no round size
        dict(name="attn_fp32", kind="attn", N=5, T=1203, ctx=700, ragged=True, Hq=6, Hk=3, d=32, dtype="fp32",
             page=24, lse=False),
    ]


def _log_int(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


MOST_SCORES = 1 << 32       # pairs of a query head and a key that it may attend to
MOST_CACHE = 1 << 31        # bytes of the keys


def draw(rng):
    kind = rng.choice(["rope_train", "rope", "append", "append", "attn", "attn", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    d = rng.choice([16, 32, 64, 64, 128, 128, 128])
    Hk = _log_int(rng, 1, 16)
    Hq = Hk * rng.choice([1, 1, 2, 3, 4, 5, 7, 8])
    if kind.startswith("rope"):
        rot = rng.choice([0, d // 2, d, d, 8 * rng.randint(0, d // 8)])
        T = _log_int(rng, 1, min(1 << 16, (1 << 27) // (Hq + Hk) // d))
        return dict(kind=kind, T=T, Hq=Hq, Hk=Hk, d=d, rot=rot, layout=rng.choice(["half", "interleaved"]),
                    norm=rng.random() < 0.7 or rot == 0, dtype=dtype, far=rng.choice([0, 0, 1 << 20]),
                    packed=rng.random() < 0.5)
    N = _log_int(rng, 1, 192)
    case = dict(kind=kind, N=N, T=N, ctx=0, ragged=rng.random() < 0.7, Hq=Hq, Hk=Hk, d=d, dtype=dtype,
                page=rng.choice([1, 16, 16, 24, 32, 64, 64, 100, 128, 256, 512]))
    if rng.random() < 0.6:  # a chunk of tokens for each sequence, else one
        case["T"] = N * _log_int(rng, 1, max(1, 32768 // N))
        if case["ragged"]:
            case["T"] += rng.randint(0, N)
    if kind == "append":
        case.update(rot=rng.choice([0, d // 2, d, d]), layout=rng.choice(["half", "interleaved"]),
                    norm=rng.random() < 0.7, ctx=rng.choice([0, _log_int(rng, 1, 8192)]))
        most = (1 << 27) // (Hk * d)
        case["T"] = min(case["T"], most - most % N)
        case["ctx"] = min(case["ctx"], (most - case["T"]) // N)
        return case
    # an average sequence has T / N new tokens over ctx cached ones, a long one several times as many
    spread = 6 if case["ragged"] else 1
    new = case["T"] // N + 1
    rows = MOST_CACHE // (N * Hk * d * (2 if dtype == "bf16" else 4))
    most = min(rows, MOST_SCORES // (case["T"] * Hq * spread)) - spread * new
    if most < 1:
        case["T"] = N
        most = min(rows, MOST_SCORES // (N * Hq * spread)) - spread
    if dtype == "fp32":  # the CUDA cores' rate
        most = min(most, MOST_SCORES // 16 // (case["T"] * Hq * spread))
    case["ctx"] = rng.choice([0, _log_int(rng, 1, max(1, min(most, 1 << 18)))]) if most > 0 else 0
    case["lse"] = rng.random() < 0.4
    return case


def _shares(total, N, seed, spread=24.0, least=0):
    """N whole numbers of the given sum, log-uniform shares of what lies above `least`."""
    r = random.Random(seed)
    share = [math.exp(r.uniform(0.0, math.log(spread))) for _ in range(N)]
    part = [least + int((total - N * least) * s / sum(share)) for s in share]
    part[r.randrange(N)] += total - sum(part)
    return part


def _lengths(case):
    """New tokens of each sequence, and tokens that its cache held before them."""
    N, T = case["N"], case["T"]
    if not case["ragged"]:
        return [T // N] * N, [case["ctx"]] * N
    new = [1] * N if T == N else _shares(T, N, 31 * T + N, spread=400.0, least=1)
    return new, _shares(case["ctx"] * N, N, 17 * T + N + 1)


# ----------------------------------------------------------------- the inputs

def _freqs(rot, far):
    """Inverse frequencies of rot channels; for far positions the slow ones are stretched eightfold."""
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    f = 10000.0 ** (-i / max(rot, 1))
    if far:
        f = torch.where(f * 8192 < 2 * math.pi, f / 8, f)
    return f.float().to(DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=torch.float32, mean=0.0, std=1.0):
        if math.prod(shape) > 1 << 28:
            return torch.empty(*shape, device=DEV, dtype=dtype).normal_(mean, std, generator=gen)
        return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).mul_(std).add_(mean).to(dtype)

    T, Hq, Hk, d = case["T"], case["Hq"], case["Hk"], case["d"]
    s = {"case": dict(case)}
    if case["kind"] != "attn":
        s["inv_freq"] = _freqs(case["rot"], case.get("far", 0))
        s["rot_scale"] = 1.2 if case.get("far", 0) else 1.0
        s["q_weight"] = normal(d, mean=1.0, std=0.2) if case["norm"] else None
        s["k_weight"] = normal(d, mean=1.0, std=0.2) if case["norm"] else None
    if case["kind"].startswith("rope"):
        if case["packed"]:  # what one projection makes of a token: its query, key and value heads in a row
            qkv = normal(T, Hq + 2 * Hk, d, dtype=dt, std=1.5)
            s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        else:
            s["q"], s["k"] = normal(T, Hq, d, dtype=dt, std=1.5), normal(T, Hk, d, dtype=dt, std=1.5)
        # sequences of 4096 tokens, the far ones at the end of a long document
        s["positions"] = (torch.arange(T, device=DEV, dtype=torch.int32) % 4096) + case["far"]
        if case["kind"] == "rope_train":
            s["d_q_out"], s["d_k_out"] = normal(T, Hq, d, dtype=dt), normal(T, Hk, d, dtype=dt)
        return s
    new, past = _lengths(case)
    N, page = case["N"], case["page"]
    lens = [a + b for a, b in zip(new, past)]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    pages = [(n + page - 1) // page for n in lens]
    total = sum(pages) + 1  # a pool with a page to spare, handed out in no order
    order = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros(N, max(pages), dtype=torch.int32, device=DEV)
    at = 0
    for n, p in enumerate(pages):
        table[n, :p] = order[at:at + p]
        at += p
    s.update(new=new, lens_list=lens, cu_list=cu, page_table=table,
             lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
             cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV) if case["ragged"] else None,
             q=normal(T, Hq, d, dtype=dt, std=1.5),
             k_cache=normal(total, Hk, page, d, dtype=dt), v_cache=normal(total, Hk, page, d, dtype=dt))
    if case["kind"] == "append":
        s["k"], s["v"] = normal(T, Hk, d, dtype=dt, std=1.5), normal(T, Hk, d, dtype=dt)
    return s


# ------------------------------------------------------------- the plain forms

def _angles(positions, inv_freq, scale):
    f = positions.double()[:, None] * inv_freq.double()
    return (torch.cos(f) * scale).float()[:, None], (torch.sin(f) * scale).float()[:, None]


def _pairs(x, rot, layout):
    if layout == "half":
        return x[..., :rot // 2], x[..., rot // 2:rot]
    return x[..., 0:rot:2], x[..., 1:rot:2]


def _joined(a, b, rest, layout):
    turned = torch.cat([a, b], -1) if layout == "half" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([turned, rest], -1)


def _plain_turn(x, w, cos, sin, case):
    """Norm and rotation in fp32: the result, the normed row and the inverse root."""
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) if case["norm"] else None
    u = x if r is None else x * r * w
    rot = case["rot"]
    if rot == 0:
        return u, r
    a, b = _pairs(u, rot, case["layout"])
    return _joined(a * cos - b * sin, b * cos + a * sin, u[..., rot:], case["layout"]), r


def _plain_turn_back(dy, x, w, r, cos, sin, case):
    g, rot = dy.float(), case["rot"]
    if rot:
        a, b = _pairs(g, rot, case["layout"])
        g = _joined(a * cos + b * sin, b * cos - a * sin, g[..., rot:], case["layout"])
    if r is None:
        return g, None
    xh = x.float() * r
    gw = g * w
    return r * (gw - xh * (gw * xh).mean(-1, keepdim=True)), (g * xh).sum((0, 1), dtype=torch.float64).float()


def _plain_rope(s, train):
    c, dt = s["case"], s["q"].dtype
    cos, sin = _angles(s["positions"], s["inv_freq"], s["rot_scale"])
    ans = {}
    for n in ("q", "k"):
        y, r = _plain_turn(s[n], s[n + "_weight"], cos, sin, c)
        ans[n] = y.to(dt)
        if train:
            dx, dw = _plain_turn_back(s[f"d_{n}_out"], s[n], s[n + "_weight"], r, cos, sin, c)
            ans["d_" + n] = dx.to(dt)
            if dw is not None:
                ans[f"d_{n}_weight"] = dw
    return ans


def _plain_append(s):
    c, dt = s["case"], s["q"].dtype
    N, page = c["N"], c["page"]
    new = torch.tensor(s["new"], device=DEV)
    seq = torch.repeat_interleave(torch.arange(N, device=DEV), new, output_size=c["T"])
    first = torch.tensor(s["cu_list"][1:], device=DEV)
    pos = s["lens"].long()[seq] - first[seq] + torch.arange(c["T"], device=DEV)
    cos, sin = _angles(pos, s["inv_freq"], s["rot_scale"])
    q, _ = _plain_turn(s["q"], s["q_weight"], cos, sin, c)
    k, _ = _plain_turn(s["k"], s["k_weight"], cos, sin, c)
    at = s["page_table"].long()[seq, pos // page]
    s["k_cache"][at, :, pos % page] = k.to(dt)
    s["v_cache"][at, :, pos % page] = s["v"]
    return {"q": q.to(dt), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attn(s):
    c = s["case"]
    Hq, Hk, d, page = c["Hq"], c["Hk"], c["d"], c["page"]
    G, scale = Hq // Hk, d ** -0.5
    out = torch.empty_like(s["q"])
    lse = torch.empty(c["T"], Hq, device=DEV)
    for n in range(c["N"]):
        a, b, L = s["cu_list"][n], s["cu_list"][n + 1], s["lens_list"][n]
        table = s["page_table"][n, :(L + page - 1) // page].long()
        k, v = (s[name][table].permute(1, 0, 2, 3).reshape(Hk, -1, d)[:, :L].float() for name in ("k_cache", "v_cache"))
        rows = min(b - a, max(1, (1 << 29) // (Hq * L)))  # queries whose scores are held at a time
        for i in range(a, b, rows):
            e = min(i + rows, b)
            qs = s["q"][i:e].float().view(e - i, Hk, G, d).transpose(0, 1).reshape(Hk, -1, d)
            sc = (qs @ k.transpose(1, 2)).view(Hk, e - i, G, L) * scale
            pos = torch.arange(L - b + i, L - b + e, device=DEV)
            sc.masked_fill_(torch.arange(L, device=DEV) > pos[:, None, None], -math.inf)
            m = sc.amax(-1, keepdim=True)
            p = sc.sub_(m).exp_()
            z = p.sum(-1, keepdim=True)
            o = (p.view(Hk, -1, L) @ v).view(Hk, e - i, G, d) / z
            out[i:e] = o.transpose(0, 1).reshape(e - i, Hq, d).to(out.dtype)
            lse[i:e] = (m + torch.log(z))[..., 0].transpose(0, 1).reshape(e - i, Hq)
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}


# ------------------------------------------------------------ the library's way

def _own_rope(s, train):
    kda, c = _lib(), s["case"]
    how = dict(layout=c["layout"], rot_scale=s["rot_scale"], norm=c["norm"], eps=EPS)
    args = s["q"], s["k"], s["positions"], s["inv_freq"], s["q_weight"], s["k_weight"]
    q, k = kda.kda_qk_rope_fwd(*args, **how)
    ans = {"q": q, "k": k}
    if train:
        gr = kda.kda_qk_rope_bwd(s["d_q_out"], s["d_k_out"], *args, **how)
        ans.update({n: t for n, t in gr.items() if t is not None})
    return ans


def _own_append(s):
    c = s["case"]
    q = _lib().kda_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["lens"], s["cu_seqlens"],
                             q=s["q"], inv_freq=s["inv_freq"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                             layout=c["layout"], rot_scale=s["rot_scale"], norm=c["norm"], eps=EPS)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attn(s):
    out, lse = _lib().kda_paged_attn(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lens"], s["cu_seqlens"],
                                     want_lse=s["case"]["lse"])
    return {"out": out, "lse": lse} if s["case"]["lse"] else {"out": out}


def run(state):
    kind = state["case"]["kind"]
    if kind == "append":
        return _own_append(state) if own else _plain_append(state)
    if kind == "attn":
        return _own_attn(state) if own else _plain_attn(state)
    return (_own_rope if own else _plain_rope)(state, kind == "rope_train")


# -------------------------------------------------------------------- the work

def work(case):
    e = {"bf16": 2, "fp32": 4}[case["dtype"]]
    T, Hq, Hk, d = case["T"], case["Hq"], case["Hk"], case["d"]
    if case["kind"].startswith("rope"):
        n = T * (Hq + Hk) * d
        small = 4 * T + 2 * case["rot"] + (8 * d if case["norm"] else 0)
        if case["kind"] == "rope":
            return {"bytes": 2 * n * e + small, "flops": 8 * n}
        return {"bytes": 4 * n * e + small + (8 * d if case["norm"] else 0), "flops": 24 * n}
    new, past = _lengths(case)
    lens = [a + b for a, b in zip(new, past)]
    table = 4 * sum((n + case["page"] - 1) // case["page"] for n in lens) + 8 * case["N"]
    if case["kind"] == "append":
        small = 2 * case["rot"] + (8 * d if case["norm"] else 0) + 4 * T + 8 * case["N"]
        return {"bytes": 2 * T * (Hq + 2 * Hk) * d * e + small, "flops": 8 * T * (Hq + Hk) * d}
    scores = Hq * sum(n * p + n * (n + 1) // 2 for n, p in zip(new, past))
    nbytes = 2 * T * Hq * d * e + 2 * sum(lens) * Hk * d * e + table + (4 * T * Hq if case["lse"] else 0)
    return {"bytes": nbytes, "flops": scores * (4 * d + 4)}


# ---------------------------------------------------------- the definition, fp64

def _exact_turn(x, w, f, scale, case):
    """Norm and rotation of leaf x, pairs taken as complex numbers."""
    u = x
    if case["norm"]:
        u = w * x / torch.sqrt(x.pow(2).mean(2, keepdim=True) + EPS)
    rot = case["rot"]
    if rot == 0:
        return u
    head, tail = u[:, :, :rot], u[:, :, rot:]
    if case["layout"] == "half":
        head = head.unflatten(2, (2, rot // 2)).transpose(2, 3)
    else:
        head = head.unflatten(2, (rot // 2, 2))
    z = torch.view_as_complex(head.contiguous()) * torch.polar(torch.full_like(f, scale), f)[:, None]
    z = torch.view_as_real(z)
    z = z.transpose(2, 3) if case["layout"] == "half" else z
    return torch.cat([z.flatten(2), tail], 2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "attn":
        return _exact_attn(case, s)
    if case["kind"] == "append":
        new, past = _lengths(case)
        pos = torch.cat([torch.arange(p, p + n) for n, p in zip(new, past)]).to(DEV)
        f = torch.outer(pos.double(), s["inv_freq"].double())
        w = {n: None if s[n] is None else s[n].double() for n in ("q_weight", "k_weight")}
        k = _exact_turn(s["k"].double(), w["k_weight"], f, s["rot_scale"], case)
        ans = {"q": _exact_turn(s["q"].double(), w["q_weight"], f, s["rot_scale"], case)}
        for name, rows in (("k_cache", k), ("v_cache", s["v"].double())):
            ans[name] = s[name].double().transpose(1, 2).contiguous()
            t = 0
            for i in range(case["N"]):
                slots = torch.arange(past[i], past[i] + new[i], device=DEV)
                where = s["page_table"][i].long()[slots // case["page"]] * case["page"] + slots % case["page"]
                ans[name].flatten(0, 1)[where] = rows[t:t + new[i]]
                t += new[i]
            ans[name] = ans[name].transpose(1, 2).contiguous()
        return ans
    with torch.enable_grad():
        f = torch.outer(s["positions"].double(), s["inv_freq"].double())
        ans, loss, leaves = {}, 0.0, {}
        for n in ("q", "k"):
            x = leaves[n] = s[n].double().requires_grad_()
            w = None
            if case["norm"]:
                w = leaves[n + "_weight"] = s[n + "_weight"].double().requires_grad_()
            ans[n] = _exact_turn(x, w, f, s["rot_scale"], case)
            if case["kind"] == "rope_train":
                loss = loss + (ans[n] * s[f"d_{n}_out"].double()).sum()
        if case["kind"] == "rope_train":
            for n, g in zip(leaves, torch.autograd.grad(loss, list(leaves.values()))):
                ans["d_" + n] = g
    return {n: t.detach() for n, t in ans.items()}


def _exact_attn(case, s):
    new, past = _lengths(case)
    Hq, Hk, d, page = case["Hq"], case["Hk"], case["d"], case["page"]
    if 4 * d * Hq * sum(n * (n + p) for n, p in zip(new, past)) > 6e12:
        return None
    out = torch.empty(case["T"], Hq, d, dtype=torch.float64, device=DEV)
    lse = torch.empty(case["T"], Hq, dtype=torch.float64, device=DEV)
    t = 0
    for n, (count, p) in enumerate(zip(new, past)):
        L = count + p
        keys = torch.arange(L, device=DEV)
        where = s["page_table"][n].long()[keys // page], keys % page
        for h in range(Hk):
            k = s["k_cache"][:, h][where].double()
            v = s["v_cache"][:, h][where].double()
            for g in range(h * (Hq // Hk), (h + 1) * (Hq // Hk)):
                step = max(1, (1 << 28) // L)
                for i in range(0, count, step):
                    j = min(i + step, count)
                    x = torch.einsum("id,jd->ij", s["q"][t + i:t + j, g].double(), k) / math.sqrt(d)
                    hidden = torch.ones(j - i, L, dtype=torch.bool, device=DEV).triu(p + i + 1)
                    x = torch.where(hidden, -torch.inf, x)
                    z = torch.logsumexp(x, 1)
                    out[t + i:t + j, g] = torch.exp(x - z[:, None]) @ v
                    lse[t + i:t + j, g] = z
        t += count
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
