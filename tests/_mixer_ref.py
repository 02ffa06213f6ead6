"""The causal convolution, the selective scan and the layer norm in 64 bits, with error bounds.

Each function evaluates an operator's formulas (forward and gradients) in float64 on the CPU and,
beside every output, a first-order bound of what an fp32 evaluation of the same formulas may be off
by, as a multiple of u = 2^-24 (half a step of fp32).  The bounds follow the data: ``E`` of a
quantity is built from the ``E`` of its inputs and the magnitudes that its sums run over (formulas
with every term's absolute value), so they hold for any input.  The local error constants:

* a sum of n products: (n + 1) u times the sum of the products' absolute values;
* softplus and the two-argument logistic: 8 u relative (expf and log1pf are within 2 steps);
* the fast sigmoid 1 / (1 + 2^(-x log2 e)): (8 + 2 |x|) u relative (rounding the product
  x log2 e moves the exponent by |x| log2 e u, the two approximate functions give 2^-22);
* a decay e = 2^(D a2), a2 = -expf(a_log) log2 e: (6 + 8 |D A|) u relative (ex2 2^-22; D, expf,
  the constant and the product each off by a few u of the exponent).

``check`` compares: |got - ref| <= 2 E + h (|ref| + 2 E), h half a step of the output's type relative to its
value (2^-8 bf16, 2^-24 fp32); the factor 2 covers the second-order terms.
"""
import torch

U = 2.0 ** -24


def d64(t):
    return None if t is None else t.detach().cpu().double()


def check(got, ref, err, what):
    g = d64(got)
    assert tuple(g.shape) == tuple(ref.shape), (what, g.shape, ref.shape)
    h = torch.finfo(got.dtype).eps / 2
    bound = 2 * err + h * (ref.abs() + 2 * err) + 1e-36  # 1e-36: results at the bottom of fp32's range
    bad = ~((g - ref).abs() <= bound)
    if bad.any():
        r = ((g - ref).abs() / bound).nan_to_num(nan=float("inf"))
        i = int(r.argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, worst {r.flatten()[i]:.3g} "
                             f"times it: got {g.flatten()[i]!r} ref {ref.flatten()[i]!r}")


def check_all(got, ref, what=""):
    """got: name -> tensor; ref: name -> (value, bound)."""
    for name, t in got.items():
        if t is not None:
            check(t, ref[name][0], ref[name][1], f"{what}{name}")


# ------------------------------------------------------------------ causal convolution
def conv(x, w, bias=None, state=None, silu=False, gy=None, gstate=None):
    x, w, bias, state, gy, gstate = map(d64, (x, w, bias, state, gy, gstate))
    B, T, C = x.shape
    W = w.shape[1]
    head = state if state is not None else x.new_zeros(B, W - 1, C)
    xp = torch.cat([head, x], dim=1)
    b0 = bias if bias is not None else x.new_zeros(C)
    pre, mag = b0.expand(B, T, C).clone(), b0.abs().expand(B, T, C).clone()
    for j in range(W):
        pre = pre + xp[:, j: j + T] * w[:, j]
        mag = mag + (xp[:, j: j + T] * w[:, j]).abs()
    epre = (W + 2) * U * mag
    out = {}
    if silu:
        s = torch.sigmoid(pre)
        y, dy = pre * s, s * (1 + pre * (1 - s))
        es = (8 + 2 * pre.abs()) * U
        out["y"] = (y, 1.1 * epre + (es + 2 * U) * y.abs())  # |silu'| <= 1.1
        # |silu''| <= 0.5; s and 1 - s carry es and 2 u / es s each, times (1 + |pre|)
        edy = 0.5 * epre + (2 * es + 4 * U) * s * (1 + pre.abs())
    else:
        y, dy, edy = pre, torch.ones_like(pre), torch.zeros_like(pre)
        out["y"] = (y, epre)
    out["state"] = (xp[:, T:], torch.zeros(B, W - 1, C, dtype=torch.float64))
    if gy is None:
        return out
    g, eg = gy * dy, gy.abs() * edy + 2 * U * (gy * dy).abs()
    gx, mx, ex = (torch.zeros(B, T + W - 1, C, dtype=torch.float64) for _ in range(3))
    gw, ew = torch.zeros(C, W, dtype=torch.float64), torch.zeros(C, W, dtype=torch.float64)
    n = B * T
    for j in range(W):
        gx[:, j: j + T] += g * w[:, j]
        mx[:, j: j + T] += (g * w[:, j]).abs()
        ex[:, j: j + T] += eg * w[:, j].abs()
        t = xp[:, j: j + T]
        gw[:, j] = (g * t).sum(dim=(0, 1))
        ew[:, j] = (eg * t.abs()).sum(dim=(0, 1)) + (n + 2) * U * (g * t).abs().sum(dim=(0, 1))
    if gstate is not None:
        gx[:, T:] += gstate
        mx[:, T:] += gstate.abs()
    ex += (W + 2) * U * mx
    out["gx"], out["gstate_in"] = (gx[:, W - 1:], ex[:, W - 1:]), (gx[:, : W - 1], ex[:, : W - 1])
    out["gw"] = (gw, ew)
    out["gbias"] = (g.sum(dim=(0, 1)), eg.sum(dim=(0, 1)) + (n + 2) * U * g.abs().sum(dim=(0, 1)))
    return out


# ------------------------------------------------------------------ selective scan
def scan(x, dt, b, c, a_log, d=None, dt_bias=None, z=None, h_in=None, gy=None, gh_out=None):
    x, dt, b, c, a_log, d, dt_bias, z, h_in, gy, gh_out = map(
        d64, (x, dt, b, c, a_log, d, dt_bias, z, h_in, gy, gh_out))
    B, T, C = x.shape
    N = a_log.shape[1]
    A = -torch.exp(a_log)
    v = dt + (dt_bias if dt_bias is not None else 0.0)
    # dt + dt_bias rounds; softplus' <= min(1, softplus(v) + small): take e^-|..| scale via softplus itself
    delta = torch.nn.functional.softplus(v, threshold=1e9)
    sig = torch.sigmoid(v)
    ev = U * v.abs()
    edelta = sig * ev + 8 * U * delta
    esig = 8 * U * sig + sig * (1 - sig) * ev
    dd = d if d is not None else x.new_zeros(C)
    dx = delta * x
    edx = edelta * x.abs() + U * dx.abs()
    h = h_in if h_in is not None else x.new_zeros(B, C, N)
    hm, eh = h.abs(), torch.zeros_like(h)
    H, HM, EH, DEC, EDEC = [h], [hm], [eh], [], []
    p, ep, pm = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    for t in range(T):
        dA = delta[:, t, :, None] * A
        e = torch.exp(dA)
        ee = e * ((6 + 8 * dA.abs()) * U + edelta[:, t, :, None] * A.abs())
        bt = b[:, t, None, :]
        eh = e * eh + ee * hm + edx[:, t, :, None] * bt.abs()
        h, hm = e * h + dx[:, t, :, None] * bt, e * hm + (dx[:, t, :, None] * bt).abs()
        eh = eh + 3 * U * hm
        ct = c[:, t, None, :]
        p[:, t] = (h * ct).sum(-1) + dd * x[:, t]
        pm[:, t] = (hm * ct.abs()).sum(-1) + (dd * x[:, t]).abs()
        ep[:, t] = (eh * ct.abs()).sum(-1) + (N + 3) * U * pm[:, t]
        H.append(h), HM.append(hm), EH.append(eh), DEC.append(e), EDEC.append(ee)
    if z is not None:
        s = torch.sigmoid(z)
        gate, egate = z * s, (z * s).abs() * (10 + 2 * z.abs()) * U
        dgate = s * (1 + z * (1 - s))
        edgate = (20 + 4 * z.abs()) * U * s * (1 + z.abs())
    else:
        gate, egate = torch.ones_like(x), torch.zeros_like(x)
    out = dict(y=(p * gate, ep * gate.abs() + egate * p.abs() + 2 * U * (p * gate).abs()), h=(h, eh))
    ck = list(range(0, T, 16))
    if ck:
        out["ckpt"] = (torch.stack([H[i] for i in ck]), torch.stack([EH[i] for i in ck]))
    if gy is None:
        return out
    g, eg = gy * gate, gy.abs() * egate + 2 * U * (gy * gate).abs()
    G = gh_out if gh_out is not None else x.new_zeros(B, C, N)
    GM, EG = G.abs(), torch.zeros_like(G)
    z_ = lambda t: torch.zeros_like(t)
    gx, ex, gdt, edt = z_(x), z_(x), z_(x), z_(x)
    gb, eb, gc, ec = z_(b), z_(b), z_(c), z_(c)
    gA, mA, eA = z_(a_log), z_(a_log), z_(a_log)
    n = B * T
    for t in reversed(range(T)):
        bt, ct, gt, egt = b[:, t, None, :], c[:, t, None, :], g[:, t, :, None], eg[:, t, :, None]
        EG = EG + egt * ct.abs()
        G, GM = G + gt * ct, GM + (gt * ct).abs()
        EG = EG + 2 * U * GM
        hc, hcm, ehc = H[t + 1], HM[t + 1], EH[t + 1]
        gc[:, t] = (gt * hc).sum(1)
        ec[:, t] = (egt * hcm + gt.abs() * ehc).sum(1) + (C + 4) * U * (gt.abs() * hcm).sum(1)
        dxt, edxt = dx[:, t, :, None], edx[:, t, :, None]
        gb[:, t] = (G * dxt).sum(1)
        eb[:, t] = (EG * dxt.abs() + GM * edxt).sum(1) + (C + 4) * U * (GM * dxt.abs()).sum(1)
        s1, s1m = (G * bt).sum(-1), (GM * bt.abs()).sum(-1)
        es1 = (EG * bt.abs()).sum(-1) + (N + 2) * U * s1m
        e, ee, hp, hpm, ehp = DEC[t], EDEC[t], H[t], HM[t], EH[t]
        q, qm = G * e * hp, GM * e * hpm
        eq = EG * e * hpm + GM * ee * hpm + GM * e * ehp + 4 * U * qm
        s2, s2m = (q * A).sum(-1), (qm * A.abs()).sum(-1)
        es2 = (eq * A.abs()).sum(-1) + (N + 8) * U * s2m
        dl, edl, xt = delta[:, t], edelta[:, t], x[:, t]
        gx[:, t] = dl * s1 + dd * g[:, t]
        ex[:, t] = edl * s1m + dl * es1 + dd.abs() * eg[:, t] + 4 * U * (dl * s1m + (dd * g[:, t]).abs())
        gd_, gdm = xt * s1 + s2, xt.abs() * s1m + s2m
        gdt[:, t] = sig[:, t] * gd_
        edt[:, t] = sig[:, t] * (xt.abs() * es1 + es2 + 4 * U * gdm) + esig[:, t] * gdm
        gA += (q * dl[..., None]).sum(0)
        mA += (qm * dl[..., None]).sum(0)
        eA += (eq * dl[..., None] + qm * edl[..., None]).sum(0)
        G, GM, EG = G * e, GM * e, EG * e + GM * ee + U * GM * e
    out["gx"], out["gdt"], out["gb"], out["gc"] = (gx, ex), (gdt, edt), (gb, eb), (gc, ec)
    out["ga_log"] = (gA * A, A.abs() * (eA + (n + 8) * U * mA))
    out["gd"] = ((g * x).sum(dim=(0, 1)),
                 (eg * x.abs()).sum(dim=(0, 1)) + (n + 2) * U * (g * x).abs().sum(dim=(0, 1)))
    out["gdt_bias"] = (gdt.sum(dim=(0, 1)), edt.sum(dim=(0, 1)) + (n + 2) * U * gdt.abs().sum(dim=(0, 1)))
    out["gh_in"] = (G, EG)
    if z is not None:
        out["gz"] = (gy * p * dgate, gy.abs() * (ep * dgate.abs() + pm * edgate) + 4 * U * (gy * pm * dgate).abs())
    return out


# ------------------------------------------------------------------ layer norm
def norm(x, w, bias=None, gate=None, groups=1, eps=1e-5, gy=None):
    shape = x.shape
    x, w, bias, gate, gy = map(d64, (x, w, bias, gate, gy))
    C = shape[-1]
    N = C // groups
    r = lambda t: None if t is None else t.reshape(-1, groups, N)
    x, gate, gy = r(x), r(gate), r(gy)
    w = w.reshape(groups, N)
    b0 = bias.reshape(groups, N) if bias is not None else torch.zeros_like(w)
    M = x.shape[0]
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    var = (xc * xc).mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    emean = (N + 2) * U * x.abs().mean(-1, keepdim=True)
    exc = emean + U * xc.abs()
    # var: each square off by 2 |xc| exc, the sum of N squares by (N + 2) u of itself
    evar = 2 * (xc.abs() * exc).mean(-1, keepdim=True) + (N + 3) * U * var + exc.pow(2).mean(-1, keepdim=True)
    erstd = rstd * (0.5 * evar / (var + eps) + 4 * U)
    xh = xc * rstd
    exh = exc * rstd + xc.abs() * erstd + U * xh.abs()
    l, lm = xh * w + b0, (xh * w).abs() + b0.abs()
    el = exh * w.abs() + 3 * U * lm
    if gate is not None:
        s = torch.sigmoid(gate)
        f, ef = gate * s, (gate * s).abs() * (10 + 2 * gate.abs()) * U
        df, edf = s * (1 + gate * (1 - s)), (20 + 4 * gate.abs()) * U * s * (1 + gate.abs())
    else:
        f, ef = torch.ones_like(x), torch.zeros_like(x)
    out = dict(y=((l * f).reshape(shape), (el * f.abs() + ef * lm + 2 * U * (l * f).abs()).reshape(shape)))
    if gy is None:
        return out
    g, eg = gy * f, gy.abs() * ef + 2 * U * (gy * f).abs()
    u, eu = g * w, eg * w.abs() + U * (g * w).abs()
    mu, mum = u.mean(-1, keepdim=True), u.abs().mean(-1, keepdim=True)
    emu = eu.mean(-1, keepdim=True) + (N + 2) * U * mum
    mx, mxm = (u * xh).mean(-1, keepdim=True), (u * xh).abs().mean(-1, keepdim=True)
    emx = (eu * xh.abs() + u.abs() * exh).mean(-1, keepdim=True) + (N + 2) * U * mxm
    inner, innerm = u - mu - xh * mx, u.abs() + mum + xh.abs() * mxm
    einner = eu + emu + exh * mxm + xh.abs() * emx + 4 * U * innerm
    out["gx"] = ((rstd * inner).reshape(shape), (rstd * einner + erstd * innerm).reshape(shape))
    out["gw"] = ((g * xh).sum(0).reshape(C),
                 ((eg * xh.abs() + g.abs() * exh).sum(0) + (M + 2) * U * (g * xh).abs().sum(0)).reshape(C))
    out["gbias"] = (g.sum(0).reshape(C), (eg.sum(0) + (M + 2) * U * g.abs().sum(0)).reshape(C))
    if gate is not None:
        out["ggate"] = ((gy * l * df).reshape(shape),
                        (gy.abs() * (el * df.abs() + lm * edf) + 4 * U * (gy * lm * df).abs()).reshape(shape))
    return out


# ------------------------------------------------------------------ inputs
def scan_inputs(B, T, C, N, seed, dtype=torch.float32, gate=True, extras=True, wide=False, grads=True, states=True):
    """Inputs of the distributions a trained layer has: steps from 1e-3 to 1e-1, rates 1 .. N."""
    import math

    g = torch.Generator().manual_seed(seed)

    def normal(*shape, scale=1.0, shift=0.0):
        return torch.randn(*shape, generator=g) * scale + shift

    def rows(*shape):
        if wide:  # a part of a wider tensor's rows
            t = normal(*shape[:-1], 2 * shape[-1] + 8).to(dtype)
            return t, (lambda q: q[..., 8: 8 + shape[-1]])
        return normal(*shape).to(dtype), (lambda q: q)

    p = {}
    views = {}
    for name, width in (("x", C), ("dt", C), ("b", N), ("c", N)) + ((("z", C),) if gate else ()):
        p[name], views[name] = rows(B, T, width)
    p["a_log"] = torch.log(torch.arange(1, N + 1).float()) + normal(C, N, scale=0.2)
    if extras:
        step = torch.exp(torch.rand(C, generator=g) * math.log(100.0) + math.log(1e-3))
        p["dt_bias"] = step + torch.log(-torch.expm1(-step))
        p["d"] = normal(C, scale=0.2, shift=1.0)
    if states:
        p["h_in"] = normal(B, C, N, scale=0.5)
    if grads:
        p["gy"] = normal(B, T, C).to(dtype)
        if states:
            p["gh_out"] = normal(B, C, N)
    return p, views
