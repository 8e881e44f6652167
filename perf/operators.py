"""Cases of the block operators: rotary positions, group norm with an
activation, and the top-k router with its balance loss.

Each case is one pass through one operator, forward, backward or (router)
both, on inputs made on the GPU from a seed.  ``run`` computes it in plain
torch operations, or, where ``own`` is true, through the calls a user makes.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5


def listed():
    return [
        # rotary: one decode step of 64 sequences, each at a position of its own
        dict(name="rotary decode", op="rotary", dir="fwd", dt="bf16", B=64, S=1, Hq=32, Hk=8, D=128, R=128,
             inter=False, lay="tokens", last=131072, pos64=False),
        # rotary: prompts of 4096 tokens, q and k inside one packed projection
        dict(name="rotary prompt", op="rotary", dir="fwd", dt="bf16", B=8, S=4096, Hq=32, Hk=8, D=128, R=128,
             inter=False, lay="packed", last=4096, pos64=True),
        # rotary: training backward, heads before tokens, half of each head rotated, scaled frequencies
        dict(name="rotary backward", op="rotary", dir="bwd", dt="f16", B=2, S=4096, Hq=32, Hk=32, D=128, R=64,
             inter=True, lay="heads", last=65536, pos64=False),
        # rotary: odd lengths and head sizes in binary32
        dict(name="rotary ragged", op="rotary", dir="fwd", dt="f32", B=3, S=1021, Hq=12, Hk=12, D=80, R=40,
             inter=False, lay="tokens", last=8192, pos64=True),
        # router: one decode step
        dict(name="router decode", op="router", dir="fwd", dt="f32", T=64, E=64, k=8, renorm=True, pad=0.0),
        # router: a training micro-batch, normalised gates
        dict(name="router step", op="router", dir="step", dt="bf16", T=16384, E=128, k=8, renorm=True, pad=0.0),
        # router: a large training batch over many experts
        dict(name="router large", op="router", dir="step", dt="bf16", T=262144, E=256, k=8, renorm=False, pad=0.0),
        # router: a padded batch, an odd number of tokens and experts, gates as they are
        dict(name="router ragged", op="router", dir="step", dt="f16", T=30011, E=60, k=4, renorm=False, pad=0.2),
        # group norm: per-head norm of one decode step
        dict(name="groupnorm decode", op="groupnorm", dir="fwd", dt="bf16", N=64, S=1, C=4096, G=32, act=True),
        # group norm: per-head norm of a training batch, backward
        dict(name="groupnorm heads", op="groupnorm", dir="bwd", dt="bf16", N=32768, S=1, C=4096, G=32, act=True),
        # group norm: a batch of 64 x 64 feature maps, groups of 10 channels
        dict(name="groupnorm maps", op="groupnorm", dir="fwd", dt="bf16", N=32, S=4096, C=320, G=32, act=True),
        # group norm: 512 x 512 feature maps, groups of 4 channels, backward
        dict(name="groupnorm images", op="groupnorm", dir="bwd", dt="f16", N=4, S=262144, C=128, G=32, act=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "router", "groupnorm"])
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    most = (400 << 20) // ES[dt]  # elements of the largest tensor
    if op == "rotary":
        D = rng.choice([32, 64, 64, 80, 96, 128, 128, 192, 256])
        R = rng.choice([D, D, D // 2, D // 4 // 2 * 2])
        Hq = rng.choice([1, 8, 12, 16, 32, 40, 64])
        Hk = rng.choice([h for h in (1, 4, 8, 12, 16, 32) if h <= Hq])
        B = _log(rng, 1, 64)
        S = _log(rng, 1, max(1, min(65536, most // 2 // (B * (Hq + Hk) * D))))
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), dt=dt, B=B, S=S, Hq=Hq, Hk=Hk, D=D, R=R,
                    inter=rng.random() < 0.4, lay=rng.choice(["tokens", "packed", "heads"]),
                    last=max(S, _log(rng, 1, 1 << 20)), pos64=rng.random() < 0.5)
    if op == "router":
        E = rng.choice([8, 16, 32, 60, 64, 64, 72, 128, 128, 160, 256, 384, 512])
        k = rng.choice([q for q in (1, 2, 4, 6, 8, 10) if q <= E])
        return dict(op=op, dir=rng.choice(["fwd", "step", "step"]), dt=dt, T=_log(rng, 1, 33554432 // E), E=E, k=k,
                    renorm=rng.random() < 0.5, pad=rng.choice([0.0, 0.0, 0.1, 0.3]))
    d = rng.choice(["fwd", "bwd"])
    if rng.random() < 0.4:
        G = rng.choice([8, 16, 32, 40, 64])
        C = G * rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
        S, N = 1, _log(rng, 1, min(32768, most // 4 // C))
    else:
        G = rng.choice([1, 8, 16, 32, 32, 32])
        C = G * (rng.choice([2, 4, 8, 10, 16, 20, 30, 40]) if G > 1 else rng.choice([64, 200, 384]))
        h = _log(rng, 4, 512)
        S = h * rng.choice([h, h, h + 1, max(1, h - 3)])
        N = _log(rng, 1, max(1, min(64, most // 4 // (S * C))))
    return dict(op=op, dir=d, dt=dt, N=N, S=S, C=C, G=G, act=rng.random() < 0.7)


# ---------------------------------------------------------------------------
# inputs

def _heads(case, H, randn):
    """[B, S, H, D] values in the case's memory layout."""
    B, S, D = case["B"], case["S"], case["D"]
    if case["lay"] == "heads":
        return randn(B, H, S, D).to(DT[case["dt"]]).transpose(1, 2)
    return randn(B, S, H, D).to(DT[case["dt"]])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[case["dt"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = {"case": case}
    if case["op"] == "rotary":
        B, S, Hq, Hk, D, R = (case[n] for n in ("B", "S", "Hq", "Hk", "D", "R"))
        if case["lay"] == "packed":
            packed = randn(B, S, (Hq + 2 * Hk) * D).to(dt).view(B, S, Hq + 2 * Hk, D)
            s["q"], s["k"] = packed[:, :, :Hq], packed[:, :, Hq:Hq + Hk]
        else:
            s["q"], s["k"] = _heads(case, Hq, randn), _heads(case, Hk, randn)
        start = torch.randint(0, case["last"] - S + 1, (B, 1), generator=gen, device="cuda")
        s["pos"] = (start + torch.arange(S, device="cuda")).to(torch.int64 if case["pos64"] else torch.int32)
        f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / max(R, 1))
        s["freq"] = (f / 4 if case["inter"] else f).float()  # positions four times further apart than trained
        s["scale"] = 0.1 * math.log(4.0) + 1.0 if case["inter"] else 1.0
    elif case["op"] == "router":
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = (1.5 * randn(T, E) + 0.5 * randn(E)).to(dt)  # some experts are liked more than others
        s["mask"] = None
        if case["pad"]:
            s["mask"] = torch.rand(T, generator=gen, device="cuda") >= case["pad"]
        up = 65536.0 if case["dt"] == "f16" else 1.0  # loss scaling of binary16 training
        s["dgates"] = randn(T, k) * (up / T)
        s["dloss"] = torch.full((), 0.01 * up, device="cuda")
    else:
        N, S, C, G = (case[n] for n in ("N", "S", "C", "G"))
        s["x"] = (randn(N, S, C) * (1 + 0.3 * randn(N, 1, C)) + 0.5 * randn(N, 1, C)).to(dt)
        s["w"], s["b"] = 1 + 0.1 * randn(C), 0.1 * randn(C)
        if case["dir"] == "bwd":
            s["dy"] = randn(N, S, C).to(dt)
            s["mean"] = torch.empty(N, G, device="cuda")
            s["rstd"] = torch.empty(N, G, device="cuda")
            for n in range(0, N, 1024):  # what the forward left, slice by slice
                x = s["x"][n:n + 1024].double().view(-1, S, G, C // G)
                v, m = torch.var_mean(x, dim=(1, 3), correction=0)
                s["mean"][n:n + 1024], s["rstd"][n:n + 1024] = m, (v + EPS).rsqrt()
    return s


# ---------------------------------------------------------------------------
# one pass

def run(state):
    op = state["case"]["op"]
    if op == "rotary":
        return _rotary(state)
    if op == "router":
        return _router(state)
    return _groupnorm(state)


def _turn(x, cos, sin, R, inter):
    x = x.float()
    h, rest = x[..., :R], x[..., R:]
    if inter:
        a, b = h[..., 0::2], h[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = h[..., :R // 2], h[..., R // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, rest), -1)


def _rotary(s):
    c = s["case"]
    if own:
        import backward_ws_fwd_gb300 as wsf
        call = wsf.rotary_fwd if c["dir"] == "fwd" else wsf.rotary_bwd
        return call(s["q"], s["k"], s["pos"], s["freq"], scale=s["scale"], interleaved=c["inter"])
    angle = s["pos"].double()[:, :, None, None] * s["freq"].double()
    cos, sin = (angle.cos() * s["scale"]).float(), (angle.sin() * s["scale"]).float()
    if c["dir"] == "bwd":
        sin = -sin
    return tuple(_turn(x, cos, sin, c["R"], c["inter"]).to(x.dtype) for x in (s["q"], s["k"]))


def _router(s):
    c = s["case"]
    l, k, E = s["logits"], c["k"], c["E"]
    if own:
        import backward_ws_fwd_gb300 as wsf
        gates, ids, counts, loss = wsf.router_fwd(l, k, mask=s["mask"], renormalize=c["renorm"])
        if c["dir"] == "fwd":
            return gates, ids, counts, loss
        dl = wsf.router_bwd(l, ids, counts, s["dgates"], s["dloss"], renormalize=c["renorm"])
        return gates, ids, counts, loss, dl
    x = l.float()
    e = (x - x.amax(1, keepdim=True)).exp()
    p = e / e.sum(1, keepdim=True)
    ids = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :k]
    gates = p.gather(1, ids)
    if c["renorm"]:
        gates = gates / gates.sum(1, keepdim=True)
    if s["mask"] is not None:
        keep = s["mask"][:, None]
        p, gates, ids = p * keep, gates * keep, torch.where(keep, ids, torch.full_like(ids, E))
    counts = torch.zeros(E + 1, dtype=torch.int64, device=l.device).index_add_(
        0, ids.reshape(-1), torch.ones_like(ids.reshape(-1)))[:E]
    V = counts.sum().float() / k
    share = counts.float() * E / (k * V.clamp(min=1) ** 2)
    loss = (share * p.sum(0)).sum()
    told = torch.where(ids == E, torch.full_like(ids, -1), ids).int()
    if c["dir"] == "fwd":
        return gates, told, counts.int(), loss
    dg = s["dgates"]
    up = (s["dloss"] * share).expand_as(p)
    add = torch.zeros(p.shape[0], E + 1, device=l.device)
    if c["renorm"]:
        dl = p * (up - (up * p).sum(1, keepdim=True))
        add.scatter_(1, ids, gates * (dg - (gates * dg).sum(1, keepdim=True)))
        dl = dl + add[:, :E]
    else:
        add.scatter_(1, ids, dg)
        up = up + add[:, :E]
        dl = p * (up - (up * p).sum(1, keepdim=True))
    return gates, told, counts.int(), loss, dl.to(l.dtype)


def _groupnorm(s):
    c = s["case"]
    x, w, b = s["x"], s["w"], s["b"]
    N, S, C, G = c["N"], c["S"], c["C"], c["G"]
    if own:
        import backward_ws_fwd_gb300 as wsf
        act = "silu" if c["act"] else None
        if c["dir"] == "fwd":
            return wsf.groupnorm_fwd(x, w, b, G, eps=EPS, act=act)
        return wsf.groupnorm_bwd(x, w, b, s["mean"], s["rstd"], s["dy"], G, act=act)
    f = x.float().view(N, S, G, C // G)
    if c["dir"] == "fwd":
        mean = f.mean((1, 3), keepdim=True)
        d = f - mean
        rstd = (d.square().mean((1, 3), keepdim=True) + EPS).rsqrt()
        z = (d * rstd).view(N, S, C) * w + b
        y = z / (1 + (-z).exp()) if c["act"] else z
        return y.to(x.dtype), mean.view(N, G), rstd.view(N, G)
    rstd = s["rstd"].view(N, 1, G, 1)
    xh = ((f - s["mean"].view(N, 1, G, 1)) * rstd).view(N, S, C)
    dz = s["dy"].float()
    if c["act"]:
        z = xh * w + b
        q = 1 / (1 + (-z).exp())
        dz = dz * (q + z * q * (1 - q))
    gw, gb = (dz * xh).sum((0, 1)), dz.sum((0, 1))
    g = (dz * w).view(N, S, G, C // G)
    xh = xh.view(N, S, G, C // G)
    dx = rstd * (g - g.mean((1, 3), keepdim=True) - xh * (g * xh).mean((1, 3), keepdim=True))
    return dx.view(N, S, C).to(x.dtype), gw, gb


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    es = ES[case["dt"]]
    if case["op"] == "rotary":
        n = case["B"] * case["S"] * (case["Hq"] + case["Hk"])
        return {"bytes": 2 * n * case["D"] * es + case["B"] * case["S"] * (8 if case["pos64"] else 4) + 2 * case["R"],
                "flops": 3 * n * case["R"]}
    if case["op"] == "router":
        T, E, k = case["T"], case["E"], case["k"]
        fwd = T * E * es + 8 * T * k + 4 * E + (T if case["pad"] else 0)
        bwd = 2 * T * E * es + 8 * T * k + 4 * E  # logits, ids, upstream gates; the gradient of the logits
        return {"bytes": fwd + (bwd if case["dir"] == "step" else 0),
                "flops": T * E * (5 + k) + (T * E * 8 if case["dir"] == "step" else 0)}
    n = case["N"] * case["S"] * case["C"]
    bwd = case["dir"] == "bwd"
    return {"bytes": (3 if bwd else 2) * n * es + (16 if bwd else 8) * case["C"] + 8 * case["N"] * case["G"],
            "flops": (30 if bwd else 14) * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        R, inter = case["R"], case["inter"]
        angle = s["pos"].double()[:, :, None, None] * s["freq"].double()
        unit = torch.polar(torch.full_like(angle, s["scale"]), -angle if case["dir"] == "bwd" else angle)

        def spin(x):
            x = x.double()
            pairs = x[..., :R].unflatten(-1, (R // 2, 2) if inter else (2, R // 2))
            if not inter:
                pairs = pairs.transpose(-1, -2)
            t = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit)
            if not inter:
                t = t.transpose(-1, -2)
            return torch.cat((t.flatten(-2), x[..., R:]), -1)

        return spin(s["q"]), spin(s["k"])
    if case["op"] == "router":
        E, k = case["E"], case["k"]
        l = s["logits"].double().requires_grad_()
        kth = torch.topk(l.detach(), k, dim=1).values[:, -1:]
        above, at = l.detach() > kth, l.detach() == kth
        chosen = above | (at & (at.cumsum(1) <= k - above.sum(1, keepdim=True)))
        ids = chosen.nonzero()[:, 1].view(-1, k)  # ascending; then by value, the first of equals first
        order = torch.sort(l.detach().gather(1, ids), dim=1, descending=True, stable=True)[1]
        ids = ids.gather(1, order)
        valid = (torch.ones_like(l[:, 0]) if s["mask"] is None else s["mask"].double()).detach()[:, None]
        V = max(float(valid.sum()), 1.0)
        p = torch.softmax(l, 1) * valid
        gates = p.gather(1, ids)
        if case["renorm"]:
            gates = torch.softmax(l.gather(1, ids), 1) * valid
        share = (chosen * valid).sum(0) / (k * V)
        loss = E * (share * p.sum(0) / V).sum()
        if case["dir"] == "fwd":
            return gates.detach(), None, None, loss.detach()
        (dl,) = torch.autograd.grad((gates * s["dgates"].double()).sum() + loss * s["dloss"].double(), l)
        return gates.detach(), None, None, loss.detach(), dl
    N, S, C, G = (case[n] for n in ("N", "S", "C", "G"))
    bwd = case["dir"] == "bwd"
    w, b = (s[n].double().requires_grad_(bwd) for n in ("w", "b"))
    outs, gw, gb = [], 0, 0
    step = max(1, (1 << 27) // (S * C))
    for n in range(0, N, step):  # slices of the batch, for the memory that autograd keeps
        x = s["x"][n:n + step].double().requires_grad_(bwd)
        v, m = torch.var_mean(x.view(-1, S, G, C // G), dim=(1, 3), correction=0, keepdim=True)
        z = ((x.view(-1, S, G, C // G) - m) / torch.sqrt(v + EPS)).reshape(x.shape) * w + b
        y = z * torch.sigmoid(z) if case["act"] else z
        if bwd:
            dx, dw, db = torch.autograd.grad(y, (x, w, b), s["dy"][n:n + step].double())
            outs.append(dx)
            gw, gb = gw + dw, gb + db
        else:
            outs.append((y, m.view(-1, G), (v + EPS).rsqrt().view(-1, G)))
    if bwd:
        return torch.cat(outs), gw, gb
    return tuple(torch.cat(o) for o in zip(*outs))
