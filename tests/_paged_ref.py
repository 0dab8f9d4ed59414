"""fp64 definitions of the norm and rotation, the append to a paged cache and the
attention over it, each with a bound on what fp32 arithmetic may be off by.

U = 2^-24 is half a step of fp32 relative to the value (one rounding).
Everything runs on the CPU, in plain loops over sequences and heads.
"""
import math

import torch

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return None if t is None else t.detach().double().cpu()


def assert_within(got, ref, bound, dtype, what):
    """|got - ref| <= bound + the output type's rounding of anything within bound of ref; NaN and
    infinities in the same places."""
    got = f64(got)
    assert got.shape == ref.shape, f"{what}: shape {tuple(got.shape)} != {tuple(ref.shape)}"
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    ok = torch.isfinite(ref)
    assert bool(torch.isfinite(got[ok]).all()), f"{what}: infinite where the definition is finite"
    err, lim = (got - ref).abs()[ok], (bound + HALF[dtype] * (ref.abs() + bound))[ok] + 1e-37
    worst = float((err / lim).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3g} times its bound"
    return worst


# ---------------------------------------------------------- norm and rotation
#
# Bounds.  The norm: a sum of d squares by 8 fused multiply-adds a lane and at most
# 4 steps over lanes, + eps: 14 U relative, half of it through the root; rsqrtf is
# documented to 2 ulp (4 U): r is off by 11 U, and u = x (r w) by 13 U.  The
# angle in half turns is an fp32 value of magnitude at most 1 (pi U) after a
# reduction that is off by 2^-30 turns (2 pi 2^-30 < U / 2); sincospif is
# documented to 1 ulp (2 U); a product with rot_scale: 7 U of |rot_scale| in all, and a
# product and a fused product with u 3 U more.  24 U of (|a| + |b|) |rot_scale| covers it.

def _pairs(rot, layout):
    i = torch.arange(rot // 2)
    return (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)


def _angles(positions, inv_freq):
    f = positions.double()[:, None] * inv_freq.double()
    return torch.cos(f)[:, None], torch.sin(f)[:, None]


def turn(x, w, positions, inv_freq, layout="half", rot_scale=1.0, norm=True, eps=1e-6, dy=None):
    """x, dy [T, H, d] fp64; returns (y, bound) and, with dy, ((dx, bound), (dw, bound))."""
    T, H, d = x.shape
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    w = torch.ones(d, dtype=torch.float64) if w is None else w
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) if norm else torch.ones(T, H, 1, dtype=torch.float64)
    u = x * r * w if norm else x
    y, e = u.clone(), (14 * U if norm else 0.0) * u.abs()
    if rot:
        a, b = _pairs(rot, layout)
        c, s = _angles(positions, inv_freq)
        y[..., a] = rot_scale * (u[..., a] * c - u[..., b] * s)
        y[..., b] = rot_scale * (u[..., b] * c + u[..., a] * s)
        e[..., a] = e[..., b] = 24 * U * abs(rot_scale) * (u[..., a].abs() + u[..., b].abs())
    if dy is None:
        return y, e
    g, eg = dy.clone(), torch.zeros_like(dy)
    if rot:
        g[..., a] = rot_scale * (dy[..., a] * c + dy[..., b] * s)
        g[..., b] = rot_scale * (dy[..., b] * c - dy[..., a] * s)
        eg[..., a] = eg[..., b] = 11 * U * abs(rot_scale) * (dy[..., a].abs() + dy[..., b].abs())
    if not norm:
        return (y, e), (g, eg), None
    gw = g * w
    m = (gw * x).sum(-1, keepdim=True) * r * r / d
    # its terms' own error, 14 roundings of their sum, 2 x 11 of r^2, 3 products
    mag = (gw * x).abs().sum(-1, keepdim=True) * r * r / d
    em = (eg * (w * x).abs()).sum(-1, keepdim=True) * r * r / d + 40 * U * mag
    dx = r * (gw - x * m)
    edx = r * (eg * w.abs() + x.abs() * em) + 16 * U * r * (gw.abs() + x.abs() * mag)
    # Terms that one lane sums: one token of each 16 or fewer (`per`), of every so-many-th such group of tokens,
    # with up to all its heads; then the block's lanes, and up to 39 blocks and 7 halves.  A tensor has at least
    # 118 of the 4864 blocks here, where no head stands against more than 40 of the other tensor.
    per = 1
    while per < 16 and T // (2 * per) >= 608:
        per *= 2
    n = -(-(-(-T // per)) // 118) * H + 256 // (d // 8) + 46
    dw = (g * x * r).sum((0, 1))
    edw = ((eg * x.abs() * r).sum((0, 1)) + (13 + n) * U * (g * x * r).abs().sum((0, 1)))
    return (y, e), (dx, edx), (dw, edw)


# ---------------------------------------------------------------- paged cache

def sequences(T, N, lens, cu):
    """(first new token, new tokens, length) of each sequence."""
    if cu is None:
        return [(n * (T // N), T // N, int(lens[n])) for n in range(N)]
    return [(int(cu[n]), int(cu[n + 1]) - int(cu[n]), int(lens[n])) for n in range(N)]


def token_positions(T, N, lens, cu):
    """Position of each token, and None for those of no sequence."""
    pos = [None] * T
    for bos, new, kv in sequences(T, N, lens, cu):
        for i in range(new):
            pos[bos + i] = kv - new + i
    return pos


def slots(table, n, page, positions):
    """(page, slot) of positions of sequence n."""
    pos = torch.as_tensor(positions, dtype=torch.long)
    return table[n].long()[pos // page], pos % page


def attention(q, kc, vc, table, lens, cu=None, causal=True, scale=None, bf16=False):
    """q [T, Hq, d], caches [pages, Hk, page, d], all fp64 on the CPU.  Returns
    (out, bound, lse, bound); rows of no sequence are NaN.

    Bounds.  A score is a sum of d products: (d + 4) U of scale sum |q k|, and as much again for
    tensor cores that keep fewer guard bits than a rounding to nearest needs.  Its
    difference to the running maximum, in powers of two, is one rounding of either term; 2^x is
    documented to 2 ulp (4 U), each rescaling takes a product and another 2^x, and a
    probability is rescaled at most once for each of its tile's successors and
    joins.  A sum of n terms adds n U.  bf16 probabilities are rounded: 2^-8."""
    T, Hq, d = q.shape
    pages, Hk, page, _ = kc.shape
    G, scale = Hq // Hk, d ** -0.5 if scale is None else scale
    nan = float("nan")
    out = torch.full_like(q, nan)
    lse = torch.full((T, Hq), nan, dtype=torch.float64)
    eo, el = torch.zeros_like(out), torch.zeros_like(lse)
    for n, (bos, new, kv) in enumerate(sequences(T, len(lens), lens, cu)):
        if new == 0:
            continue
        at = slots(table, n, page, range(kv))
        pos = torch.arange(kv - new, kv)
        see = torch.arange(kv)[None] <= pos[:, None] if causal else torch.ones(new, kv, dtype=torch.bool)
        for h in range(Hk):
            k, v = kc[at[0], h, at[1]], vc[at[0], h, at[1]]
            for g in range(h * G, (h + 1) * G):
                qh = q[bos:bos + new, g]
                s = (qh @ k.T * scale).masked_fill(~see, -math.inf)
                # products of hidden keys take no part, not even as 0 times a value that is not finite
                top = s.amax(-1, keepdim=True) if kv else torch.full((new, 1), -math.inf, dtype=torch.float64)
                none = ~see.any(-1, keepdim=True) if kv else torch.ones(new, 1, dtype=torch.bool)
                p = torch.exp(s - torch.where(none, 0.0, top))
                z = p.sum(-1, keepdim=True)
                odd = ~torch.isfinite(v)
                o = p @ v.masked_fill(odd, 0.0)
                if bool(odd.any()):  # sums of p v over the seen keys of each channel that has any
                    for j in torch.nonzero(odd.any(-1))[:, 0].tolist():
                        o = o + torch.where(see[:, j, None] & odd[j], v[j], 0.0)
                out[bos:bos + new, g] = torch.where(none, 0.0, o / z)
                lse[bos:bos + new, g] = torch.where(none, -math.inf, top + torch.log(z))[:, 0]
                es = (2 * (d + 4) * U * scale * (qh.abs() @ k.abs().T)).masked_fill(~see, 0.0)
                es = es.nan_to_num(0.0, 0.0, 0.0).amax(-1, keepdim=True) if kv else torch.zeros(new, 1, dtype=torch.float64)
                big = s.masked_fill(~see, 0.0).nan_to_num(0.0, 0.0, 0.0).abs().amax(-1, keepdim=True) if kv else 0.0
                delta = es + 4 * U * big + (8 + kv // 4 + 16) * U
                va = v.masked_fill(odd, 0.0).abs()
                mean = torch.where(none, 0.0, (p @ va) / z).nan_to_num(0.0, 0.0, 0.0)
                eo[bos:bos + new, g] = mean * (2 * delta + 2 * kv * U + (2.0 ** -8 if bf16 else 0.0))
                el[bos:bos + new, g] = (delta + kv * U + 8 * U * (1.0 + big))[:, 0] if kv else 0.0
    return out, eo, lse, el
