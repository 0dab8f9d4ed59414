"""Workloads of the library's recurrence-block operators: the gated linear
recurrence (kda_scan_fwd, kda_scan_bwd, kda_scan_step) and the norms around a
block with its gate and residual scale (kda_block_norm_fwd,
kda_block_norm_bwd).

With ``own`` false the operators run in their plain form, elementary torch
operations in fp32 (fp64 where a long sum needs it), rounded once at the end;
with ``own`` true they run through the library.  ``exact`` is the definition
in fp64, token by token for the recurrence.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
G_MIN = -5.0  # the log-decay floor of the decay gate
EPS_POST, EPS_PRE = 1e-6, 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _lib():
    import hybrid_linear_attention_chunk_gb300 as kda
    return kda


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one sequence generating its next token: a single call's latency
        dict(name="step_1seq", kind="step", N=1, H=32, d=128, dtype="bf16", gate="logit", write="complement"),
        # a full decode batch, one token for each of 256 sequences
        dict(name="step_256seq", kind="step", N=256, H=32, d=128, dtype="bf16", gate="fp32", write="one"),
        # prefill of a packed batch of 24 requests of very different lengths
        dict(name="scan_packed", kind="scan", N=24, T=49152, H=32, d=128, ragged=True, dtype="bf16", gate="fp32",
             write="one"),
        # prefill of one very long document
        dict(name="scan_long", kind="scan", N=1, T=262144, H=16, d=128, ragged=False, dtype="bf16", gate="logit",
             write="complement"),
        # a small fp32 model with a channel count that is no multiple of a vector, ragged batch with short sequences
        dict(name="scan_odd", kind="scan", N=7, T=3001, H=5, d=33, ragged=True, dtype="fp32", gate="bf16",
             write="one"),
        # a training step's recurrence layer: forward and backward of a batch of 4 x 8192 tokens
        dict(name="scan_train", kind="scan_train", N=4, T=32768, H=32, d=128, ragged=False, dtype="bf16",
             gate="logit", write="complement"),
        # training in fp32 on packed sequences, with a given log-decay
        dict(name="scan_train_fp32", kind="scan_train", N=9, T=10007, H=6, d=72, ragged=True, dtype="fp32",
             gate="fp32", write="one"),
        # the boundary between two blocks for a decode batch of 8 tokens
        dict(name="norm_decode", kind="norm", rows=8, width=4096, dtype="bf16", res="bf16", gate=False, post=True,
             scale=True, normed=True),
        # the boundary between two blocks in a prefill of 32768 tokens, with an fp32 residual stream
        dict(name="norm_prefill", kind="norm", rows=32768, width=4096, dtype="bf16", res="fp32", gate=True, post=True,
             scale=True, normed=True),
        # the per-head norm and gate after the recurrence: 8192 tokens x 32 heads of 128 channels
        dict(name="norm_heads", kind="norm", rows=262144, width=128, dtype="bf16", res="", gate=True, post=True,
             scale=False, normed=False),
        # a training step's block boundary
        dict(name="norm_train", kind="norm_train", rows=16384, width=4096, dtype="bf16", res="bf16", gate=True,
             post=True, scale=True, normed=True),
        # training in fp32 at a width that is no multiple of a vector
        dict(name="norm_train_odd", kind="norm_train", rows=777, width=1001, dtype="fp32", res="fp32", gate=True,
             post=True, scale=True, normed=True),
    ]


def _log_int(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


MOST_ELEMENTS = {"scan": 1 << 28, "scan_train": 1 << 26, "norm": 1 << 26, "norm_train": 1 << 25}


def draw(rng):
    kind = rng.choice(["step", "scan", "scan", "scan_train", "norm", "norm", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if kind.startswith("norm"):
        width = rng.choice([_log_int(rng, 16, 8192), 8 * _log_int(rng, 2, 1024), 128])
        rows = _log_int(rng, 1, min(1 << 18, MOST_ELEMENTS[kind] // width))
        res = rng.choice(["", dtype, "fp32"])
        case = dict(kind=kind, rows=rows, width=width, dtype=dtype, res=res, gate=rng.random() < 0.6,
                    post=rng.random() < 0.7, scale=rng.random() < 0.5, normed=rng.random() < 0.7)
        case["normed"] = case["normed"] or not case["post"]  # a norm before, after, or both
        return case
    H, d = _log_int(rng, 1, 32), rng.choice([16, 33, 40, 64, 72, 96, 128, 128])
    case = dict(kind=kind, N=1, H=H, d=d, dtype=dtype, gate=rng.choice(["fp32", "bf16", "logit"]),
                write=rng.choice(["one", "complement"]))
    if kind == "step":
        case["N"] = _log_int(rng, 1, 256)
        return case
    most = min(1 << 18, MOST_ELEMENTS[kind] // (H * d))
    case["T"] = _log_int(rng, 1, most)
    case["N"] = _log_int(rng, 1, min(64, case["T"]))
    case["ragged"] = rng.random() < 0.6
    if not case["ragged"]:
        case["T"] -= case["T"] % case["N"]
    return case


def _lengths(case):
    """Tokens of each sequence: log-uniform shares of T (some may be 0), or T / N each."""
    N, T = case["N"], case["T"]
    if not case["ragged"]:
        return [T // N] * N
    r = random.Random(31 * T + N)
    share = [math.exp(r.uniform(0.0, math.log(64.0))) for _ in range(N)]
    lens = [int(T * s / sum(share)) for s in share]
    lens[-1] += T - sum(lens)
    return lens


# ----------------------------------------------------------------- the inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=torch.float32, mean=0.0, std=1.0):
        return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.float32).mul_(std).add_(mean).to(dtype)

    s = {"case": dict(case)}
    if case["kind"].startswith("norm"):
        rows, width = case["rows"], case["width"]
        s["y"] = normal(rows, width, dtype=dt)
        s["gate"] = normal(rows, width, dtype=dt) if case["gate"] else None
        s["post_weight"] = normal(width, mean=1.0, std=0.2) if case["post"] else None
        s["scale"] = normal(width, mean=0.5, std=0.2) if case["scale"] else None
        s["pre_weight"] = normal(width, mean=1.0, std=0.2) if case["normed"] else None
        rdt = DTYPES[case["res"]] if case["res"] else dt
        s["residual"] = normal(rows, width, dtype=rdt, std=2.0) if case["res"] else None
        if case["kind"] == "norm_train":
            s["d_out"] = normal(rows, width, dtype=rdt)
            s["d_normed"] = normal(rows, width, dtype=dt) if case["normed"] else None
        return s
    N, H, d = case["N"], case["H"], case["d"]
    tokens = N if case["kind"] == "step" else case["T"]
    s["x"] = normal(tokens, H, d, dtype=dt)
    if case["gate"] == "logit":
        # decays between a few and a few hundred tokens of memory
        s["decay"] = normal(tokens, H, d, dtype=dt, mean=-4.0, std=2.0)
        s["A_log"] = torch.empty(H, device=DEV).uniform_(-0.5, 0.5, generator=gen)
    else:
        u = torch.empty(tokens, H, d, device=DEV).uniform_(math.log(1e-3), 0.0, generator=gen)
        s["decay"] = u.exp_().neg_().to(DTYPES[case["gate"]])
        s["A_log"] = None
    s["state"] = normal(N, H, d)
    if case["kind"] == "step":
        s["state_out"] = torch.empty_like(s["state"])
        return s
    cu = [0]
    for n in _lengths(case):
        cu.append(cu[-1] + n)
    s["longest"] = max(b - a for a, b in zip(cu, cu[1:]))
    s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    if case["kind"] == "scan_train":
        s["d_out"] = normal(tokens, H, d, dtype=dt)
        s["d_final_state"] = normal(N, H, d)
    return s


# ------------------------------------------------------------- the plain forms

def _decay(s):
    """log-decay in fp32, and its derivative by the logit where there is one."""
    if s["A_log"] is None:
        return s["decay"].float(), None
    e = torch.exp(s["A_log"])[:, None]
    sig = 1.0 / (1.0 + torch.exp(-e * s["decay"].float()))
    return G_MIN * sig, G_MIN * sig * (1.0 - sig) * e


def _prefix(a, b, longest):
    """b_t + a_t b_{t-1} + a_t a_{t-1} b_{t-2} + ... along dim 0, by doubling."""
    step = 1
    while step < longest:
        b = torch.cat([b[:step], torch.addcmul(b[step:], a[step:], b[:-step])])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def _plain_scan(s, train):
    x, cu = s["x"].float(), s["cu_seqlens"].long()
    T = x.shape[0]
    g, slope = _decay(s)
    comp = s["case"]["write"] == "complement"
    a, w = torch.exp(g), (-torch.expm1(g) if comp else torch.ones((), device=x.device))
    some = (cu[1:] > cu[:-1])[:, None, None]
    first, last = cu[:-1].clamp(max=T - 1), (cu[1:] - 1).clamp(min=0)
    heads = torch.zeros_like(a[:, :1, :1]).index_add_(0, first, some.float())  # 1 at the first token of a sequence
    b = (w * x).index_add_(0, first, torch.where(some, a[first] * s["state"], 0.0))
    cut = torch.where(heads > 0, 0.0, a)
    h = _prefix(cut, b, s["longest"])
    res = {"out": h.to(s["x"].dtype), "final_state": torch.where(some, h[last], s["state"])}
    if not train:
        return res
    do = s["d_out"].float().index_add(0, last, torch.where(some, s["d_final_state"], 0.0))
    nxt = torch.cat([cut[1:], torch.zeros_like(cut[:1])])
    D = _prefix(nxt.flip(0), do.flip(0), s["longest"]).flip(0)
    h0 = torch.zeros_like(h).index_add_(0, first, torch.where(some, s["state"], 0.0))
    prev = torch.where(heads > 0, h0, torch.cat([torch.zeros_like(h[:1]), h[:-1]]))
    dg = D * a * (prev - x if comp else prev)
    res["dx"] = (D * w).to(s["x"].dtype)
    res["d_initial_state"] = torch.where(some, a[first] * D[first], s["d_final_state"])
    if slope is None:
        res["d_decay"] = dg.to(s["decay"].dtype)
    else:
        dz = dg * slope
        res["d_decay"] = dz.to(s["decay"].dtype)
        res["dA_log"] = (dz * s["decay"].float()).sum(dim=(0, 2), dtype=torch.float64).float()
    return res


def _plain_step(s):
    g, _ = _decay(s)
    x = s["x"].float()
    w = -torch.expm1(g) if s["case"]["write"] == "complement" else 1.0
    torch.add(torch.exp(g) * s["state"], w * x, out=s["state_out"])
    return {"out": s["state_out"].to(s["x"].dtype), "state": s["state_out"]}


def _plain_norm(s, train):
    y, res = s["y"].float(), s["residual"]
    odt = s["y"].dtype if res is None else res.dtype
    one = torch.ones((), device=y.device)
    w1, w2, sc = (one if s[n] is None else s[n] for n in ("post_weight", "pre_weight", "scale"))
    post, normed = s["case"]["post"], s["case"]["normed"]
    r1 = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS_POST) if post else one
    yh = y * r1
    u = yh * w1
    sig = one if s["gate"] is None else 1.0 / (1.0 + torch.exp(-s["gate"].float()))
    b = u * sig
    out = b * sc if res is None else res.float() + b * sc
    ans = {"out": out.to(odt)}
    if normed:
        r2 = torch.rsqrt((out * out).mean(-1, keepdim=True) + EPS_PRE)
        oh = out * r2
        ans["normed"] = (oh * w2).to(s["y"].dtype)
    if not train:
        return ans
    D = s["d_out"].float()
    if normed:
        dn = s["d_normed"].float()
        do = dn * w2
        D = D + r2 * (do - oh * (do * oh).mean(-1, keepdim=True))
        ans["d_pre_weight"] = (dn * oh).sum(0, dtype=torch.float64).float()
    if res is not None:
        ans["d_residual"] = D.to(odt)
    if s["scale"] is not None:
        ans["d_scale"] = (D * b).sum(0, dtype=torch.float64).float()
    db = D * sc
    du = db * sig
    if s["gate"] is not None:
        ans["d_gate"] = (db * u * sig * (1.0 - sig)).to(s["y"].dtype)
    if post:
        ans["d_post_weight"] = (du * yh).sum(0, dtype=torch.float64).float()
        dy = du * w1
        du = r1 * (dy - yh * (dy * yh).mean(-1, keepdim=True))
    ans["d_y"] = du.to(s["y"].dtype)
    return ans


# ------------------------------------------------------------ the library's way

def _own_scan(s, train):
    kda, wr = _lib(), s["case"]["write"]
    if not train:
        out, fs = kda.kda_scan_fwd(s["x"], s["decay"], s["A_log"], G_MIN, initial_state=s["state"],
                                   cu_seqlens=s["cu_seqlens"], write=wr)
        return {"out": out, "final_state": fs}
    out, fs, states = kda.kda_scan_fwd(s["x"], s["decay"], s["A_log"], G_MIN, initial_state=s["state"],
                                       cu_seqlens=s["cu_seqlens"], write=wr, want_states=True)
    gr = kda.kda_scan_bwd(s["x"], s["decay"], s["d_out"], s["A_log"], G_MIN, initial_state=s["state"],
                          d_final_state=s["d_final_state"], cu_seqlens=s["cu_seqlens"], states=states, write=wr)
    res = {"out": out, "final_state": fs, "dx": gr["dx"], "d_decay": gr["d_decay"],
           "d_initial_state": gr["d_initial_state"]}
    if s["A_log"] is not None:
        res["dA_log"] = gr["dA_log"]
    return res


def _own_step(s):
    out, state = _lib().kda_scan_step(s["x"], s["decay"], s["state"], s["A_log"], G_MIN, state_out=s["state_out"],
                                      write=s["case"]["write"])
    return {"out": out, "state": state}


def _own_norm(s, train):
    kda, c = _lib(), s["case"]
    parts = dict(residual=s["residual"], gate=s["gate"], post_norm=c["post"], post_weight=s["post_weight"],
                 scale=s["scale"], pre_weight=s["pre_weight"], post_eps=EPS_POST, pre_eps=EPS_PRE)
    out, normed = kda.kda_block_norm_fwd(s["y"], want_normed=c["normed"], **parts)
    ans = {"out": out}
    if c["normed"]:
        ans["normed"] = normed
    if train:
        gr = kda.kda_block_norm_bwd(s["y"], s["d_out"], s["d_normed"], **parts)
        ans.update({k: v for k, v in gr.items() if v is not None})
    return ans


def run(state):
    kind = state["case"]["kind"]
    if kind == "step":
        return _own_step(state) if own else _plain_step(state)
    if kind.startswith("scan"):
        return (_own_scan if own else _plain_scan)(state, kind == "scan_train")
    return (_own_norm if own else _plain_norm)(state, kind == "norm_train")


# -------------------------------------------------------------------- the work

def work(case):
    size = {"bf16": 2, "fp32": 4}
    e = size[case["dtype"]]
    if case["kind"].startswith("norm"):
        n, width = case["rows"] * case["width"], case["width"]
        r = size[case["res"]] if case["res"] else 0
        vectors = sum((case["post"], case["scale"], case["normed"]))
        total = n * (e + r + (e if case["gate"] else 0) + (r or e) + (e if case["normed"] else 0)) + 4 * width * vectors
        flops = n * 12
        if case["kind"] == "norm_train":  # and d_out, d_normed read; d_y, d_gate, d_residual, weight gradients written
            total += n * ((r or e) + (e if case["normed"] else 0) + e + (e if case["gate"] else 0) + r)
            total += 4 * width * vectors
            flops = n * 42
        return {"bytes": total, "flops": flops}
    D = case["H"] * case["d"]
    ge = e if case["gate"] == "logit" else size[case["gate"]]
    small = 8 * case["N"] * D + (4 * case["H"] if case["gate"] == "logit" else 0)
    if case["kind"] == "step":
        n = case["N"] * D
        return {"bytes": n * (2 * e + ge) + small, "flops": 8 * n}
    n = case["T"] * D
    if case["kind"] == "scan":
        return {"bytes": n * (2 * e + ge) + small + 4 * (case["N"] + 1), "flops": 8 * n}
    return {"bytes": n * (4 * e + 2 * ge) + 2 * small + 4 * (case["N"] + 1), "flops": 24 * n}


# ---------------------------------------------------------- the definition, fp64

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"].startswith("norm"):
        return _exact_norm(case, s)
    if case["kind"] != "step" and s["longest"] > 300000:
        return None
    x, z = s["x"].double(), s["decay"].double()
    scale = None
    if s["A_log"] is not None:
        scale = s["A_log"].double().exp()[None, :, None]
        sig = torch.sigmoid(scale * z)
        z = G_MIN * sig
    alpha = z.exp()
    put = 1.0 - alpha if case["write"] == "complement" else torch.ones_like(alpha)
    u = put * x
    h0 = s["state"].double()
    if case["kind"] == "step":
        h = alpha * h0 + u
        return {"out": h, "state": h}
    cu = s["cu_seqlens"].tolist()
    N, longest = case["N"], s["longest"]
    # every sequence in a column of its own, padded at its end with tokens that leave the state alone
    where = torch.full((longest, N), -1, dtype=torch.long, device=DEV)
    for n in range(N):
        where[:cu[n + 1] - cu[n], n] = torch.arange(cu[n], cu[n + 1], device=DEV)
    pad = where < 0
    at = where.clamp(min=0)
    A = torch.where(pad[..., None, None], 1.0, alpha[at])
    U = torch.where(pad[..., None, None], 0.0, u[at])
    Hs = torch.empty(longest + 1, *h0.shape, dtype=torch.float64, device=DEV)
    Hs[0] = h0
    for t in range(longest):
        torch.addcmul(U[t], A[t], Hs[t], out=Hs[t + 1])
    del U
    live = (~pad)
    out = torch.empty_like(x)
    out[where[live]] = Hs[1:][live]
    ans = {"out": out, "final_state": Hs[longest].clone()}
    if case["kind"] == "scan":
        return ans
    # adjoint of the loop: c is the gradient of the state that leaves token t
    dO = torch.where(pad[..., None, None], 0.0, s["d_out"].double()[at])
    c = s["d_final_state"].double()
    dH = torch.empty_like(A)
    for t in range(longest - 1, -1, -1):
        torch.add(dO[t], c, out=dH[t])
        c = A[t] * dH[t]
    ans["d_initial_state"] = c
    dh, prev = torch.empty_like(x), torch.empty_like(x)
    dh[where[live]], prev[where[live]] = dH[live], Hs[:-1][live]
    ans["dx"] = put * dh
    dg = dh * alpha * (prev - x) if case["write"] == "complement" else dh * alpha * prev
    if scale is None:
        ans["d_decay"] = dg
    else:
        dlogit = dg * G_MIN * sig * (1.0 - sig)  # by exp(A) z
        ans["d_decay"] = dlogit * scale
        ans["dA_log"] = (dlogit * scale * s["decay"].double()).sum(2).sum(0)
    return ans


def _exact_norm(case, s):
    with torch.enable_grad():
        leaf = {n: s[n].double().requires_grad_() for n in
                ("y", "residual", "gate", "post_weight", "scale", "pre_weight") if s[n] is not None}
        t = leaf["y"]
        if case["post"]:
            t = leaf["post_weight"] * t / torch.sqrt(t.pow(2).mean(1, keepdim=True) + EPS_POST)
        if "gate" in leaf:
            t = t * torch.sigmoid(leaf["gate"])
        if "scale" in leaf:
            t = t * leaf["scale"]
        if "residual" in leaf:
            t = t + leaf["residual"]
        ans = {"out": t}
        loss = (t * s["d_out"].double()).sum() if "d_out" in s else None
        if case["normed"]:
            n = leaf["pre_weight"] * t / torch.sqrt(t.pow(2).mean(1, keepdim=True) + EPS_PRE)
            ans["normed"] = n
            if loss is not None:
                loss = loss + (n * s["d_normed"].double()).sum()
        if loss is not None:
            for name, g in zip(leaf, torch.autograd.grad(loss, list(leaf.values()))):
                ans["d_" + name] = g
    return {k: v.detach() for k, v in ans.items()}
