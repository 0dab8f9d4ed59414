"""fp64 definitions of the gated linear recurrence and of the block norms, with
bounds on what fp32 arithmetic may be off by.

Every bound is a running one: next to a value v the reference carries E, the
most that fp32 evaluation may miss it by, built from the same recurrence with
absolute values.  U = 2^-24 is half a step of fp32 relative to the value (one
rounding).  K counts the roundings of one token's update; see scan().
"""
import numpy as np
import torch

U = 2.0 ** -24
# One token: g (a bf16/fp32 value, or 6 roundings of the gate: product, exp of 2, sum, quotient, product; each
# shifts alpha by at most |g| <= 5 times itself relative, so 30), exp or expm1 (CUDA documents 1 and 2 ulp: 4
# roundings), w, w x, fma, add: 5 more.  Kernels that join tiles add at most one exp, one sum of 16 logs and three
# operations per 16 tokens.  K = 64 covers all of it.
K = 64.0
# half a step of each output type, relative to the value
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def rounding(ref, dtype):
    return HALF[dtype] * np.abs(ref)


def assert_within(got, ref, bound, dtype, what):
    """|got - ref| <= bound + the output type's rounding of anything within bound of ref."""
    got = np64(got)
    assert got.shape == ref.shape, f"{what}: shape {got.shape} != {ref.shape}"
    ok = np.isfinite(ref)
    assert np.array_equal(np.isnan(ref), np.isnan(got)), f"{what}: NaN in other places"
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), f"{what}: infinities differ"
    err = np.abs(got - ref)[ok]
    lim = (bound + HALF[dtype] * (np.abs(ref) + bound))[ok] + 1e-37
    worst = float(np.max(err / lim)) if err.size else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3g} times its bound"


def gate(z, A_log, g_min):
    """g, dg/dz of the decay gate; z [.., H, d], A_log [H]."""
    s = np.exp(A_log)[:, None]
    with np.errstate(over="ignore", invalid="ignore"):
        p = 1.0 / (1.0 + np.exp(-s * z))
        q = 1.0 / (1.0 + np.exp(s * z))
    return g_min * p, g_min * p * q * s


def scan(x, decay, A_log=None, g_min=-5.0, s0=None, cu=None, write="one", d_out=None, dST=None):
    """The recurrence and its reverse mode in fp64, token by token.

    Arrays are fp64 numpy: x, decay, d_out [T, H, d]; s0, dST [N, H, d]; cu a
    list.  Returns {name: (value, bound)} for out, final_state and, with
    d_out, dx, d_decay, dA_log, d_initial_state.  Rows outside every sequence
    are NaN."""
    T, H, d = x.shape
    N = len(cu) - 1
    g, slope = (decay, None) if A_log is None else gate(decay, A_log, g_min)
    a = np.exp(g)
    w = -np.expm1(g) if write == "complement" else np.ones_like(g)
    comp = write == "complement"
    s0 = np.zeros((N, H, d)) if s0 is None else s0
    dST = np.zeros((N, H, d)) if dST is None else dST
    out, eo = np.full_like(x, np.nan), np.zeros_like(x)
    res = {"out": (out, eo), "final_state": (s0.copy(), np.zeros_like(s0))}
    if d_out is not None:
        for n in ("dx", "d_decay"):
            res[n] = (np.full_like(x, np.nan), np.zeros_like(x))
        res["d_initial_state"] = (dST.copy(), np.zeros_like(dST))
        if A_log is not None:
            res["dA_log"] = (np.zeros(H), np.zeros(H))
    for n in range(N):
        h, m, e = s0[n].copy(), np.abs(s0[n]), np.zeros((H, d))
        prev, eprev = [], []
        for t in range(cu[n], cu[n + 1]):
            prev.append(h)
            eprev.append(e)
            u = w[t] * x[t]
            h = a[t] * h + u
            m = a[t] * m + np.abs(u)          # the sum with absolute values
            e = a[t] * e + K * U * m
            out[t], eo[t] = h, e
        res["final_state"][0][n], res["final_state"][1][n] = h, e
        if d_out is None:
            continue
        c, mc, ec = dST[n].copy(), np.abs(dST[n]), np.zeros((H, d))
        terms = 0
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            i = t - cu[n]
            D, mD, eD = d_out[t] + c, np.abs(d_out[t]) + mc, ec + U * (np.abs(d_out[t]) + mc)
            res["dx"][0][t], res["dx"][1][t] = w[t] * D, w[t] * eD + K * U * np.abs(w[t] * D)
            p = prev[i] - x[t] if comp else prev[i]
            pm = np.abs(prev[i]) + (np.abs(x[t]) if comp else 0.0)
            dg = a[t] * D * p
            edg = a[t] * (eD * (pm + eprev[i]) + np.abs(D) * eprev[i] + K * U * mD * pm)
            if A_log is not None:
                dz = dg * slope[t]
                # the slope's factors: 12 more roundings of its value, and |s z| e^.. moves with exp's argument
                # (an infinite z has slope 0, exactly)
                fin = np.isfinite(decay[t])
                zt = np.where(fin, decay[t], 0.0)
                edz = np.abs(slope[t]) * (edg + (K + 8 * np.abs(np.exp(A_log)[:, None] * zt)) * U * np.abs(dg))
                res["dA_log"][0][:] += np.sum(np.where(fin, dz, 0.0) * zt, axis=1)
                terms += 1
                res["dA_log"][1][:] += np.sum(edz * np.abs(zt) + (T + 64) * U * np.abs(dz * zt), axis=1)
                dg, edg = dz, edz
            res["d_decay"][0][t], res["d_decay"][1][t] = dg, edg
            c = a[t] * D
            mc = a[t] * mD
            ec = a[t] * eD + K * U * mc
        res["d_initial_state"][0][n], res["d_initial_state"][1][n] = c, ec
    return res


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def block_norm(y, residual=None, gate=None, post=True, w1=None, scale=None, w2=None, e1=1e-6, e2=1e-6, normed=True,
               d_out=None, d_normed=None):
    """The block norms and their reverse mode in fp64 on rows [R, W], each with
    a bound.  n below counts the roundings of a row sum: at most W / 32 + 32
    sequential additions, 2 per product; S = 16 + n those of a scalar (rsqrt 2
    ulp) and the few factors around it; the gate's exponential moves with its
    argument."""
    R, W = y.shape
    n = W / 32.0 + 32.0
    S = (16.0 + n) * U
    one = np.ones((1, W))
    w1_, sc, w2_ = (one if v is None else v[None, :] for v in (w1, scale, w2))
    g = 0.0 * y if gate is None else gate
    sg, sq = (np.ones_like(y), np.zeros_like(y)) if gate is None else (sigmoid(gate), sigmoid(-gate))
    G = (8.0 + np.abs(g)) * U  # relative error of the sigmoid
    r1 = 1.0 / np.sqrt(np.mean(y * y, 1, keepdims=True) + e1) if post else np.ones((R, 1))
    yh = y * r1
    u = yh * w1_
    b = u * sg
    out = b * sc + (0.0 if residual is None else residual)
    mag = np.abs(b * sc) + (0.0 if residual is None else np.abs(residual))
    eb = np.abs(b) * (S + G)
    eo = eb * np.abs(sc) + 4 * U * mag
    res = {"out": (out, eo)}
    r2 = 1.0 / np.sqrt(np.mean(out * out, 1, keepdims=True) + e2)
    # relative error of r2: half of that of the mean square, from out's own errors and the sum
    er2 = S + np.mean(np.abs(out) * eo, 1, keepdims=True) * r2 * r2
    oh = out * r2
    eoh = eo * r2 + np.abs(oh) * (er2 + 4 * U)
    if normed:
        res["normed"] = (oh * w2_, np.abs(w2_) * eoh + 4 * U * np.abs(oh * w2_))
    if d_out is None and d_normed is None:
        return res
    D = np.zeros_like(y) if d_out is None else d_out.copy()
    mD, eD = np.abs(D), np.zeros_like(y)
    if d_normed is not None:
        dn = d_normed * w2_
        dot = np.mean(dn * oh, 1, keepdims=True)
        adot = np.mean(np.abs(dn * oh), 1, keepdims=True)
        edot = np.mean(np.abs(dn) * eoh, 1, keepdims=True) + S * adot
        D = D + r2 * (dn - oh * dot)
        part = r2 * (np.abs(dn) + np.abs(oh) * adot)
        mD = mD + part
        eD = part * (er2 + S) + r2 * (eoh * adot + np.abs(oh) * edot)
        rows = (R + 64.0) * U
        res["d_pre_weight"] = (np.sum(d_normed * oh, 0),
                               np.sum(np.abs(d_normed) * (eoh + rows * np.abs(oh)), 0))
    eD = eD + 4 * U * mD
    rows = (R + 64.0) * U
    if residual is not None:
        res["d_residual"] = (D, eD)
    res["d_scale"] = (np.sum(D * b, 0), np.sum(eD * (np.abs(b) + eb) + np.abs(D) * eb + rows * np.abs(D * b), 0))
    db, edb = D * sc, np.abs(sc) * eD + U * np.abs(D * sc)
    if gate is not None:
        f = u * sg * sq
        res["d_gate"] = (db * f, np.abs(f) * edb + np.abs(db * f) * (S + 2 * G))
    du, edu = db * sg, edb * sg + np.abs(db * sg) * G
    if post:
        eyh = np.abs(yh) * S
        res["d_post_weight"] = (np.sum(du * yh, 0),
                                np.sum(edu * np.abs(yh) + np.abs(du) * eyh + rows * np.abs(du * yh), 0))
        dy, edy = du * w1_, edu * np.abs(w1_) + U * np.abs(du * w1_)
        m = np.mean(dy * yh, 1, keepdims=True)
        am = np.mean(np.abs(dy * yh), 1, keepdims=True)
        em = np.mean(edy * np.abs(yh) + np.abs(dy) * eyh, 1, keepdims=True) + S * am
        du = r1 * (dy - yh * m)
        edu = r1 * (edy + eyh * am + np.abs(yh) * em + (S + 4 * U) * (np.abs(dy) + np.abs(yh) * am))
    res["d_y"] = (du, edu)
    return res
