"""Plain 64-bit implementations of the block operators (rotary positions,
top-k router with balance loss, group norm with SiLU) for the tests, and the
bounds that their binary32 arithmetic has to keep.  Runs on any device."""
from fractions import Fraction

import torch

U = 2.0 ** -24  # half a step of binary32, relative


def half_step(v, dtype):
    """Largest rounding error of storing v (64-bit) as dtype."""
    f = torch.finfo(dtype)
    return v.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2


# --------------------------------------------------------------------------
PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


def angles(pos, freq):
    """pos·freq modulo a turn, [*pos.shape, R/2]: the exact rational product,
    reduced by 2π to 60 digits, rounded to 64 bits once.  (The 64-bit product
    alone is off by position·2^-53 radians.)"""
    turn = 2 * PI
    fs = [Fraction(f) for f in freq.double().tolist()]
    a = [[float(Fraction(p) * f % turn) for f in fs] for p in pos.reshape(-1).tolist()]
    return torch.tensor(a, dtype=torch.float64, device=pos.device).view(*pos.shape, len(fs))


def rotary(x, pos, freq, scale, inter, sign=1.0, th=None):
    """x [B, S, H, D]; th: angles [B or 1, S, 1, R/2] in place of the 64-bit
    products pos·freq; returns (y, bound) for kernel outputs of x's type.

    cos and sin: the reduced angle (|a| <= π/4) is a 30-bit integer rounded to
    binary32 and scaled, two roundings, 2·U·π/4; the series adds a few U; the
    scale another: 6·U·scale in all.  A product and a sum: 2 more roundings,
    so 8·U·scale·(|x_a| + |x_b|), then the store."""
    R = 2 * freq.numel()
    x64 = x.double()
    if th is None:
        th = pos.double().reshape(-1, x.shape[1], 1, 1) * freq.double()
    c, s = th.cos() * scale, th.sin() * scale * sign
    y, mag = x64.clone(), torch.zeros_like(x64)
    a, b = (slice(0, R, 2), slice(1, R, 2)) if inter else (slice(0, R // 2), slice(R // 2, R))
    y[..., a] = x64[..., a] * c - x64[..., b] * s
    y[..., b] = x64[..., b] * c + x64[..., a] * s
    m = (x64[..., a].abs() + x64[..., b].abs()) * abs(scale) * 8 * U
    mag[..., a] = m
    mag[..., b] = m
    return y, torch.where(mag > 0, mag + half_step(y, x.dtype), mag)


# --------------------------------------------------------------------------
def choose(logits, k):
    """The k largest of each row, largest first, equal ones in index order."""
    return torch.sort(logits.double() + 0.0, dim=1, descending=True, stable=True)[1][:, :k]


def router(logits, k, mask=None, renorm=False, dgates=None, dloss=0.0, counts=None):
    """dict of gates, ids, counts, loss, dlogits and bounds *_tol.

    A softmax term is 2^t, t = (l − m)·log2 e of magnitude |t| rounded twice
    and scaled by ln 2, and the hardware's exponential is good to 2^-22: a
    relative error of (2·|t| + 8)·U; a row's sum and its reciprocal have that
    of their largest terms and log2 E + 4 roundings (24·U).  A probability is
    thus within (2·|t| + 32)·U of itself; a normalised gate adds as much.  The
    hardware's exponential gives 0 below 2^-126 (the row's largest term is 1
    and the sum at least 1), an absolute error of at most 2^-126 a
    probability, which a gradient multiplies by the terms it stands beside."""
    T, E = logits.shape
    l = logits.double()
    valid = torch.ones(T, dtype=torch.bool, device=l.device) if mask is None else mask.bool()
    valid = valid & (l > -torch.inf).any(1)
    ids = choose(logits, k)
    safe = torch.where(valid[:, None], l, torch.zeros_like(l))
    p = torch.softmax(safe, 1) * valid[:, None]
    t = (safe - safe.amax(1, keepdim=True)) * 1.4427
    rel = (2 * t.abs().clamp(max=200) + 32) * U
    g = p.gather(1, ids)
    gr = rel.gather(1, ids)
    if renorm:
        g = torch.where(valid[:, None], g / g.sum(1, keepdim=True), torch.zeros_like(g))
        gr = 2 * gr + 8 * U
    own = torch.zeros(E + 1, dtype=torch.int64, device=l.device)
    own.index_add_(0, torch.where(valid[:, None], ids, torch.full_like(ids, E)).reshape(-1),
                   torch.ones(T * k, dtype=torch.int64, device=l.device))
    own = own[:E]
    c = own if counts is None else counts.long()
    V = max(float(c.sum()) / k, 1.0)
    loss = float(E * (own.double() * p.sum(0)).sum() / (k * max(float(own.sum()) / k, 1.0) ** 2))
    out = dict(gates=g, gates_tol=gr * g + 2.0 ** -126, counts=own, loss=loss,
               ids=torch.where(valid[:, None], ids, torch.full_like(ids, -1)),
               # p's errors, and at most 2 + log2 of the rows' additions a column
               loss_tol=loss * (64 + 2 * max(T, 1).bit_length() + T / 64) * U)
    if dgates is not None or dloss:
        a = float(dloss) * E * c.double() / (k * V * V)
        u = torch.zeros_like(p)
        dg = torch.zeros_like(g) if dgates is None else dgates.double()
        if renorm:
            dot = (dg * g).sum(1, keepdim=True)
            add = g * (dg - dot)
            u.scatter_(1, ids, add)
            dl = p * (a - (p * a).sum(1, keepdim=True)) + u
            big = p * (a.abs() + (p * a.abs()).sum(1, keepdim=True))
            mg = torch.zeros_like(p).scatter_(1, ids, g * (dg.abs() + (dg.abs() * g).sum(1, keepdim=True)))
            big = big + 2 * mg
            beside = a.abs().max() + (dg.abs() + (dg.abs() * g).sum(1, keepdim=True)).amax(1, keepdim=True)
        else:
            u.scatter_(1, ids, dg)
            w = a + u
            dl = p * (w - (p * w).sum(1, keepdim=True))
            big = p * (w.abs() + (p * w.abs()).sum(1, keepdim=True))
            beside = w.abs().amax(1, keepdim=True)
        dl = torch.where(valid[:, None], dl, torch.zeros_like(dl))
        # two probabilities' errors and a handful of roundings of each term
        tol = torch.where(valid[:, None], big * 3 * (rel + 8 * U) + 2.0 ** -126 * 2 * beside, torch.zeros_like(big))
        out.update(dlogits=dl, dlogits_tol=tol + half_step(dl, logits.dtype))
    return out


# --------------------------------------------------------------------------
def groupnorm(x, w, b, G, eps, silu, dy=None):
    """dict of y, mean, rstd, dx, grad_w, grad_b and bounds *_tol.

    K = 128·U bounds the relative error of everything that leads to a
    normalised value: at most 64 values a thread about a shift (64·U; tests of
    longer samples keep to tiles of 64 rows a thread), joined
    over threads and tiles by trees (20·U), the square root, the division and
    the products of a value (10·U), and the 16-bit path's exponential and
    reciprocal (2^-21 = 8·U, and 2·|z|·U)."""
    K = 128 * U
    N, S, C = x.shape
    xs = x.double().view(N, S, G, C // G)
    M = S * (C // G)
    mu = xs.mean((1, 3), keepdim=True)
    var = ((xs - mu) ** 2).mean((1, 3), keepdim=True)
    r = 1 / torch.sqrt(var + eps)
    spread = (var.sqrt() + (mu.abs() * 2.0 ** -6)).expand(N, S, G, C // G).reshape(N, S, C)
    xh = ((xs - mu) * r).view(N, S, C)
    rr = r.expand(N, S, G, C // G).reshape(N, S, C)
    w, b = w.double(), b.double()
    z = xh * w + b
    q = torch.sigmoid(z)
    y = z * q if silu else z
    zs = ((xs - mu).abs().view(N, S, C) + spread) * rr * w.abs() + b.abs()
    out = dict(y=y, mean=mu.view(N, G), rstd=r.view(N, G))
    out["y_tol"] = K * 1.1 * zs * (1 + (z.abs() * q if silu else 0)) + half_step(y, x.dtype)
    out["mean_tol"] = K * (spread.view(N, S, G, C // G)[:, 0, :, 0] if S else 0) + 2 * U * mu.view(N, G).abs()
    out["rstd_tol"] = K * out["rstd"]
    if dy is None:
        return out
    dy = dy.double()
    dz = dy * (q + z * q * (1 - q)) if silu else dy
    g = (dz * w).view(N, S, G, C // G)
    xg = xh.view(N, S, G, C // G)
    m1, m2 = g.mean((1, 3), keepdim=True), (g * xg).mean((1, 3), keepdim=True)
    dx = (r * (g - m1 - xg * m2)).view(N, S, C)
    # |error of dz| <= K·D, of x̂ <= K·X
    D = dy.abs() * (1 + z.abs() + zs)
    X = xh.abs() + spread * rr
    gm = (D * w.abs()).view(N, S, G, C // G)
    xm = X.view(N, S, G, C // G)
    dxs = r * (gm + gm.mean((1, 3), keepdim=True) + 2 * xm * (gm * (1 + xm)).mean((1, 3), keepdim=True))
    out.update(dx=dx, grad_w=(dz * xh).sum((0, 1)), grad_b=dz.sum((0, 1)),
               dx_tol=2 * K * dxs.view(N, S, C) + half_step(dx, x.dtype),
               grad_w_tol=2 * K * (D * X).sum((0, 1)), grad_b_tol=2 * K * D.sum((0, 1)))
    return out


def worst(got, want, tol):
    """Largest |got − want| / tol (0/0 counts as 0, a NaN on one side only as inf)."""
    got, want, tol = got.double(), torch.as_tensor(want).double().to(got.device), torch.as_tensor(tol).double().to(got.device)
    e = (got - want).abs()
    e = torch.where(torch.isnan(got) & torch.isnan(want), torch.zeros_like(e), e)
    e = torch.where(torch.isnan(e), torch.full_like(e, torch.inf), e)
    q = torch.where(e == 0, torch.zeros_like(e), e / tol)
    return float(q.max()) if q.numel() else 0.0
