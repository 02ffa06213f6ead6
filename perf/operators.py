"""Cases of the token-mixing block's operators: the short causal convolution, the selective
state space scan and the layer norm, each in its prompt, training and single-token form.

``run`` computes them in plain torch operations, or, with ``own`` set, through the library's
entry points; ``exact`` computes them in 64 bits from their definitions.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a short fp32 prompt of an odd length going on from a kept state: launch latency
        dict(name="conv_prompt_1x37x768_f32", kind="conv_fwd", B=1, T=37, C=768, W=4, dtype="f32", wide=False),
        # one training layer's convolution: x is one half of a projection twice as wide
        dict(name="conv_train_4x4096x2560_bf16", kind="conv_train", B=4, T=4096, C=2560, W=4, dtype="bf16",
             wide=True),
        # decode of 512 streams
        dict(name="conv_step_512x2560_bf16", kind="conv_step", B=512, T=1, C=2560, W=4, dtype="bf16", wide=False),
        # a short fp32 prompt, one row: few channels, latency
        dict(name="scan_prompt_1x129x1024_f32", kind="scan_fwd", B=1, T=129, C=1024, N=16, dtype="f32", gate=True,
             wide=False),
        # one long prompt: few rows, a long axis
        dict(name="scan_prompt_1x8192x2048_bf16", kind="scan_fwd", B=1, T=8192, C=2048, N=16, dtype="bf16", gate=True,
             wide=True),
        # one training layer: forward and backward
        dict(name="scan_train_4x4096x2560_bf16", kind="scan_train", B=4, T=4096, C=2560, N=16, dtype="bf16", gate=True,
             wide=True),
        # a small ragged training batch in fp32, half the states, no gate, odd length and channels
        dict(name="scan_train_2x333x521x8_f32", kind="scan_train", B=2, T=333, C=521, N=8, dtype="f32", gate=False,
             wide=False),
        # decode of 512 streams
        dict(name="scan_step_512x2560_bf16", kind="scan_step", B=512, T=1, C=2560, N=16, dtype="bf16", gate=True,
             wide=False),
        # the pre-norm of a four-stream decode step: latency
        dict(name="norm_4x2048_bf16", kind="norm_fwd", M=4, G=1, N=2048, dtype="bf16", gate=False),
        # the norm over each head of an Eagle or Finch layer's output, with its gate: prompts
        dict(name="norm_heads_16384x40x64_bf16", kind="norm_fwd", M=16384, G=40, N=64, dtype="bf16", gate=True),
        # a small model's pre-norm in training, fp32
        dict(name="norm_train_8192x768_f32", kind="norm_train", M=8192, G=1, N=768, dtype="f32", gate=False),
        # the norm over heads with its gate in training
        dict(name="norm_train_heads_16384x40x64_bf16", kind="norm_train", M=16384, G=40, N=64, dtype="bf16",
             gate=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["conv_fwd", "conv_train", "conv_step", "scan_fwd", "scan_fwd", "scan_train", "scan_train",
                       "scan_step", "norm_fwd", "norm_train"])
    dtype = rng.choice(["f32", "bf16"])
    wide = rng.random() < 0.5
    limit = 4 * 4096 * 2560 // (2 if dtype == "f32" else 1)  # elements of the largest listed case, by bytes
    if kind.startswith("norm"):
        gate = rng.random() < 0.5
        if rng.random() < 0.5:
            G, N = 1, _log_int(rng, 64, 8192)
        else:
            G, N = rng.randint(2, 64), rng.choice([32, 64, 80, 128])
        M = _log_int(rng, 1, max(1, min(16384, limit // (G * N))))
        return dict(kind=kind, M=M, G=G, N=N, dtype=dtype, gate=gate)
    C = _log_int(rng, 96, 5120)
    if rng.random() < 0.7:
        C = (C + 7) // 8 * 8
    if kind.endswith("step"):
        B, T = _log_int(rng, 1, 512), 1
        B = max(1, min(B, 512 * 2560 // C))
    else:
        B = rng.randint(1, 8)
        T = _log_int(rng, 1, 8192 if kind != "scan_train" else 4096)
        T = max(1, min(T, limit // (B * C)))
    case = dict(kind=kind, B=B, T=T, C=C, dtype=dtype, wide=wide)
    if kind.startswith("conv"):
        case["W"] = rng.choice([2, 3, 4])
    else:
        case["N"] = rng.choice([8, 16, 16, 16, 32])
        case["gate"] = rng.random() < 0.7
        if case["N"] == 32:
            case["T"] = max(1, case["T"] // 2)
    return case


def _seed(case, seed):
    return (seed * 1000003 + sum(ord(ch) * (i + 1) for i, ch in enumerate(case["kind"]))) & 0x7FFFFFFF


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(_seed(case, seed))
    dt = _DT[case["dtype"]]

    def normal(*shape, scale=1.0, shift=0.0):
        return torch.randn(*shape, generator=g, device=dev).mul_(scale).add_(shift)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    def rows(*shape, scale=1.0):
        # an activation; in a wide case it is the first part of rows twice as wide (a projection's output)
        if case.get("wide"):
            return normal(*shape[:-1], 2 * shape[-1], scale=scale).to(dt)[..., : shape[-1]]
        return normal(*shape, scale=scale).to(dt)

    s = dict(case=case)
    kind = case["kind"]
    if kind.startswith("norm"):
        M, G, N = case["M"], case["G"], case["N"]
        s["x"] = normal(M, G * N, scale=1.5, shift=0.2).to(dt)
        s["w"] = normal(G * N, scale=0.1, shift=1.0)
        s["b"] = normal(G * N, scale=0.1)
        s["gate"] = normal(M, G * N).to(dt) if case["gate"] else None
        s["gy"] = normal(M, G * N).to(dt) if kind == "norm_train" else None
        return s
    B, T, C = case["B"], case["T"], case["C"]
    if kind.startswith("conv"):
        W = case["W"]
        s["w"] = normal(C, W, scale=W ** -0.5)
        s["bias"] = normal(C, scale=0.1)
        if kind == "conv_step":
            s["x"] = rows(B, C)
            s["state"] = normal(B, W - 1, C).to(dt)
            s["state_out"] = torch.empty_like(s["state"])
            return s
        s["x"] = rows(B, T, C)
        s["state"] = normal(B, W - 1, C).to(dt) if kind == "conv_fwd" else None
        s["gy"] = normal(B, T, C).to(dt) if kind == "conv_train" else None
        return s
    N = case["N"]
    s["a_log"] = torch.log(torch.arange(1, N + 1, device=dev, dtype=torch.float32)) + normal(C, N, scale=0.1)
    step = torch.exp(uniform(C) * math.log(100.0) + math.log(1e-3))  # steps from 1e-3 to 1e-1 at dt = 0
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["d"] = normal(C, scale=0.1, shift=1.0)
    lead = (B, C) if kind == "scan_step" else (B, T, C)
    nlead = lead[:-1] + (N,)
    s["x"] = rows(*lead)
    s["dt"] = normal(*lead, scale=0.5).to(dt)
    s["B"] = rows(*nlead)
    s["C"] = rows(*nlead)
    s["z"] = rows(*lead) if case["gate"] else None
    if kind != "scan_train":
        s["h"] = normal(B, C, N, scale=0.3)
    if kind == "scan_step":
        s["h_out"] = torch.empty_like(s["h"])
    if kind == "scan_train":
        s["gy"] = normal(B, T, C).to(dt)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import rwkv_wkv_recurrence_b200 as rw

    case = s["case"]
    kind = case["kind"]
    if kind == "conv_fwd":
        return rw.rwkv_causal_conv_forward(s["x"], s["w"], s["bias"], s["state"], silu=True, return_state=True)
    if kind == "conv_train":
        y = rw.rwkv_causal_conv_forward(s["x"], s["w"], s["bias"], silu=True)
        return (y,) + rw.rwkv_causal_conv_backward(s["x"], s["w"], s["gy"], s["bias"], silu=True)
    if kind == "conv_step":
        y = rw.rwkv_causal_conv_step(s["x"], s["w"], s["state"], s["bias"], silu=True, state_out=s["state_out"])
        return y, s["state_out"]
    if kind == "scan_fwd":
        return rw.rwkv_selective_scan_forward(s["x"], s["dt"], s["B"], s["C"], s["a_log"], s["d"], s["dt_bias"],
                                              s["z"], s["h"], return_state=True)
    if kind == "scan_train":
        y, ckpt = rw.rwkv_selective_scan_forward(s["x"], s["dt"], s["B"], s["C"], s["a_log"], s["d"], s["dt_bias"],
                                                 s["z"], checkpoints=True)
        grads = rw.rwkv_selective_scan_backward(s["x"], s["dt"], s["B"], s["C"], s["a_log"], s["gy"], s["d"],
                                                s["dt_bias"], s["z"], ckpt)
        return (y,) + tuple(t for t in grads if t is not None)
    if kind == "scan_step":
        y = rw.rwkv_selective_scan_step(s["x"], s["dt"], s["B"], s["C"], s["a_log"], s["h"], s["d"], s["dt_bias"],
                                        s["z"], state_out=s["h_out"])
        return y, s["h_out"]
    y = rw.rwkv_layer_norm_forward(s["x"], s["w"], s["b"], s["gate"], groups=case["G"], eps=1e-5)
    if kind == "norm_fwd":
        return y
    grads = rw.rwkv_layer_norm_backward(s["x"], s["w"], s["gy"], s["b"], s["gate"], groups=case["G"], eps=1e-5)
    return (y,) + tuple(t for t in grads if t is not None)


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _run_plain(s):
    case = s["case"]
    kind = case["kind"]
    dt = _DT[case["dtype"]]
    if kind == "conv_step":
        win = torch.cat([s["state"], s["x"][:, None]], dim=1)  # [B,W,C]
        pre = (win.float() * s["w"].t()).sum(dim=1) + s["bias"]
        return (pre * _sigmoid(pre)).to(dt), win[:, 1:].contiguous()
    if kind.startswith("conv"):
        return _plain_conv(s, dt)
    if kind == "scan_step":
        x = s["x"].float()
        delta = _softplus(s["dt"].float() + s["dt_bias"])
        e = torch.exp(delta[..., None] * -torch.exp(s["a_log"]))
        h = e * s["h"] + (delta * x)[..., None] * s["B"].float()[:, None, :]
        p = (h * s["C"].float()[:, None, :]).sum(-1) + s["d"] * x
        if s["z"] is not None:
            z = s["z"].float()
            p = p * z * _sigmoid(z)
        return p.to(dt), h
    if kind.startswith("scan"):
        return _plain_scan(s, dt)
    return _plain_norm(s, dt)


def _plain_conv(s, dt):
    case = s["case"]
    B, T, C, W = case["B"], case["T"], case["C"], case["W"]
    head = s["state"] if s["state"] is not None else torch.zeros(B, W - 1, C, dtype=dt, device=s["x"].device)
    xp = torch.cat([head, s["x"]], dim=1)
    xf = xp.float()
    pre = s["bias"].expand(B, T, C)
    for j in range(W):
        pre = pre + xf[:, j: j + T] * s["w"][:, j]
    sg = _sigmoid(pre)
    y = (pre * sg).to(dt)
    if case["kind"] == "conv_fwd":
        return y, xp[:, T:].contiguous()
    g = s["gy"].float() * sg * (1.0 + pre * (1.0 - sg))
    gx = torch.zeros(B, T + W - 1, C, device=g.device)
    gw = []
    for j in range(W):
        gx[:, j: j + T] += g * s["w"][:, j]
        gw.append((g * xf[:, j: j + T]).sum(dim=(0, 1)))
    return y, gx[:, W - 1:].to(dt), torch.stack(gw, dim=1), g.sum(dim=(0, 1))


def _softplus(v):
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-torch.abs(v)))


_BLOCK = 64  # tokens whose decays and increments the plain scan forms at once


def _plain_scan(s, dt):
    case = s["case"]
    B, T, C, N = case["B"], case["T"], case["C"], case["N"]
    dev = s["x"].device
    A = -torch.exp(s["a_log"])
    train = case["kind"] == "scan_train"

    def block(t0):
        t1 = min(T, t0 + _BLOCK)
        x = s["x"][:, t0:t1].float()
        v = s["dt"][:, t0:t1].float() + s["dt_bias"]
        delta = _softplus(v)
        e = torch.exp(delta[..., None] * A)
        bt, ct = s["B"][:, t0:t1].float(), s["C"][:, t0:t1].float()
        return t1, x, v, delta, e, bt, ct

    def states(h, e, delta, x, bt):  # [B,L+1,C,N]: before the block's first token, then after each
        out = torch.empty(B, e.shape[1] + 1, C, N, device=dev)
        out[:, 0] = h
        inc = (delta * x)[..., None] * bt[:, :, None, :]
        for i in range(e.shape[1]):
            torch.addcmul(inc[:, i], e[:, i], out[:, i], out=out[:, i + 1])
        return out

    y = torch.empty(B, T, C, dtype=dt, device=dev)
    h = torch.zeros(B, C, N, device=dev) if train else s["h"]
    starts = []
    for t0 in range(0, T, _BLOCK):
        starts.append(h)
        t1, x, _, delta, e, bt, ct = block(t0)
        hs = states(h, e, delta, x, bt)
        h = hs[:, -1].clone()
        p = (hs[:, 1:] * ct[:, :, None, :]).sum(-1) + s["d"] * x
        if s["z"] is not None:
            z = s["z"][:, t0:t1].float()
            p = p * (z * _sigmoid(z))
        y[:, t0:t1] = p.to(dt)
    if not train:
        return y, h
    gx, gdt = torch.empty_like(y), torch.empty_like(y)
    gz = torch.empty_like(y) if s["z"] is not None else None
    gB = torch.empty(B, T, N, dtype=dt, device=dev)
    gC = torch.empty_like(gB)
    gA = torch.zeros(C, N, device=dev)
    gd, gbias = torch.zeros(C, device=dev), torch.zeros(C, device=dev)
    carry = torch.zeros(B, C, N, device=dev)
    for k in reversed(range(len(starts))):
        t0 = k * _BLOCK
        t1, x, v, delta, e, bt, ct = block(t0)
        hs = states(starts[k], e, delta, x, bt)
        g = s["gy"][:, t0:t1].float()
        if gz is not None:
            z = s["z"][:, t0:t1].float()
            sz = _sigmoid(z)
            p = (hs[:, 1:] * ct[:, :, None, :]).sum(-1) + s["d"] * x
            gz[:, t0:t1] = (g * p * sz * (1.0 + z * (1.0 - sz))).to(dt)
            g = g * z * sz
        gh = g[..., None] * ct[:, :, None, :]
        gC[:, t0:t1] = (g[..., None] * hs[:, 1:]).sum(2).to(dt)
        gh[:, -1] += carry
        for i in range(t1 - t0 - 1, 0, -1):
            gh[:, i - 1].addcmul_(e[:, i], gh[:, i])
        carry = e[:, 0] * gh[:, 0]
        gB[:, t0:t1] = (gh * (delta * x)[..., None]).sum(2).to(dt)
        s1 = (gh * bt[:, :, None, :]).sum(-1)
        q = gh * e * hs[:, :-1]
        gv = (x * s1 + (q * A).sum(-1)) * _sigmoid(v)
        gx[:, t0:t1] = (delta * s1 + s["d"] * g).to(dt)
        gdt[:, t0:t1] = gv.to(dt)
        gA += (q * delta[..., None]).sum(dim=(0, 1))
        gd += (g * x).sum(dim=(0, 1))
        gbias += gv.sum(dim=(0, 1))
    out = (y, gx, gdt, gB, gC, gA * A, gd, gbias)
    return out + (gz,) if gz is not None else out


def _plain_norm(s, dt):
    case = s["case"]
    M, G, N = case["M"], case["G"], case["N"]
    x = s["x"].float().view(M, G, N)
    w, b = s["w"].view(G, N), s["b"].view(G, N)
    mean = x.sum(-1, keepdim=True) / N
    xc = x - mean
    rstd = 1.0 / torch.sqrt((xc * xc).sum(-1, keepdim=True) / N + 1e-5)
    xh = xc * rstd
    ln = xh * w + b
    if s["gate"] is not None:
        gate = s["gate"].float().view(M, G, N)
        sg = _sigmoid(gate)
        y = ln * (gate * sg)
    else:
        y = ln
    y = y.view(M, G * N).to(dt)
    if case["kind"] == "norm_fwd":
        return y
    g = s["gy"].float().view(M, G, N)
    ggate = None
    if s["gate"] is not None:
        ggate = (g * ln * sg * (1.0 + gate * (1.0 - sg))).view(M, G * N).to(dt)
        g = g * gate * sg
    u = g * w
    gx = rstd * (u - u.sum(-1, keepdim=True) / N - xh * ((u * xh).sum(-1, keepdim=True) / N))
    out = (y, gx.view(M, G * N).to(dt), (g * xh).sum(0).view(-1), g.sum(0).view(-1))
    return out + (ggate,) if ggate is not None else out


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = {k: (v.double() if isinstance(v, torch.Tensor) else v) for k, v in s.items()}
    kind = case["kind"]
    if kind.startswith("norm"):
        return _exact_norm(case, d)
    if kind.startswith("conv"):
        return _exact_conv(case, d)
    return _exact_scan(case, d)


def _exact_norm(case, d):
    M, G, N = case["M"], case["G"], case["N"]
    x = d["x"].reshape(M, G, N)
    leaves = [x, d["w"].reshape(G, N), d["b"].reshape(G, N)]
    if d["gate"] is not None:
        leaves.append(d["gate"].reshape(M, G, N))
    train = case["kind"] == "norm_train"
    if train:
        leaves = [t.clone().requires_grad_() for t in leaves]
    x, w, b = leaves[:3]
    var, mean = torch.var_mean(x, dim=-1, unbiased=False, keepdim=True)
    y = (x - mean) * torch.rsqrt(var + 1e-5) * w + b
    if len(leaves) == 4:
        y = y * leaves[3] * torch.sigmoid(leaves[3])
    if not train:
        return y.reshape(M, G * N)
    grads = torch.autograd.grad(y, leaves, d["gy"].reshape(M, G, N))
    out = [y.detach().reshape(M, G * N), grads[0].reshape(M, G * N), grads[1].reshape(-1), grads[2].reshape(-1)]
    return tuple(out + [grads[3].reshape(M, G * N)] if len(leaves) == 4 else out)


def _exact_conv(case, d):
    B, T, C, W = case["B"], case["T"], case["C"], case["W"]
    x = d["x"].reshape(B, T, C)
    head = d["state"] if d.get("state") is not None else x.new_zeros(B, W - 1, C)
    train = case["kind"] == "conv_train"
    leaves = [x, d["w"], d["bias"]]
    if train:
        leaves = [t.clone().requires_grad_() for t in leaves]
    xp = torch.cat([head, leaves[0]], dim=1)
    pre = sum(xp[:, j: j + T] * leaves[1][:, j] for j in range(W)) + leaves[2]
    y = pre * torch.sigmoid(pre)
    if train:
        return (y.detach(),) + torch.autograd.grad(y, leaves, d["gy"])
    tail = xp[:, T:].contiguous()
    return (y[:, 0], tail) if case["kind"] == "conv_step" else (y, tail)


def _exact_scan(case, d):
    # the recurrence token by token, and its chain rule token by token backwards
    B, T, C, N = case["B"], case["T"], case["C"], case["N"]
    x, dt = d["x"].reshape(B, T, C), d["dt"].reshape(B, T, C)
    bt, ct = d["B"].reshape(B, T, N), d["C"].reshape(B, T, N)
    z = d["z"].reshape(B, T, C) if d["z"] is not None else None
    A = -torch.exp(d["a_log"])
    v = dt + d["dt_bias"]
    delta = torch.logaddexp(v, torch.zeros_like(v))
    train = case["kind"] == "scan_train"
    h = x.new_zeros(B, C, N) if train else d["h"]
    keep = torch.empty(T + 1 if train else 1, B, C, N, dtype=torch.float64, device=x.device)
    keep[0] = h
    p = torch.empty_like(x)
    for t in range(T):
        h = torch.exp(delta[:, t, :, None] * A) * h + (delta[:, t] * x[:, t])[..., None] * bt[:, t, None, :]
        p[:, t] = torch.einsum("bcn,bn->bc", h, ct[:, t]) + d["d"] * x[:, t]
        if train:
            keep[t + 1] = h
    gate = z * torch.sigmoid(z) if z is not None else 1.0
    y = p * gate
    if not train:
        return (y[:, 0], h) if case["kind"] == "scan_step" else (y, h)
    gy = d["gy"]
    g = gy * gate
    gx, gdelta = torch.empty_like(x), torch.empty_like(x)
    gB, gC = torch.empty_like(bt), torch.empty_like(ct)
    gA = torch.zeros_like(A)
    G = x.new_zeros(B, C, N)
    for t in reversed(range(T)):
        G = G + g[:, t, :, None] * ct[:, t, None, :]
        gC[:, t] = torch.einsum("bc,bcn->bn", g[:, t], keep[t + 1])
        gB[:, t] = torch.einsum("bcn,bc->bn", G, delta[:, t] * x[:, t])
        s1 = torch.einsum("bcn,bn->bc", G, bt[:, t])
        gx[:, t] = delta[:, t] * s1
        G = G * torch.exp(delta[:, t, :, None] * A)
        q = G * keep[t]
        gdelta[:, t] = x[:, t] * s1 + (q * A).sum(-1)
        gA += (q * delta[:, t, :, None]).sum(0)
    gx += d["d"] * g
    gv = gdelta * torch.sigmoid(v)
    out = (y, gx, gv, gB, gC, gA * A, (g * x).sum(dim=(0, 1)), gv.sum(dim=(0, 1)))
    if z is None:
        return out
    sz = torch.sigmoid(z)
    return out + (gy * p * sz * (1.0 + z * (1.0 - sz)),)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    esz = 4 if case["dtype"] == "f32" else 2
    kind = case["kind"]
    if kind.startswith("norm"):
        E, cols = case["M"] * case["G"] * case["N"], case["G"] * case["N"]
        if kind == "norm_fwd":
            return dict(bytes=E * esz * (3 if case["gate"] else 2) + 8 * cols, flops=E * (13 if case["gate"] else 8))
        # x, gy (, gate) in; y, gx (, ggate) out; gw and gb
        return dict(bytes=E * esz * (6 if case["gate"] else 4) + 16 * cols, flops=E * (38 if case["gate"] else 22))
    E, cols = case["B"] * case["T"] * case["C"], case["C"]
    if kind.startswith("conv"):
        W = case["W"]
        state = case["B"] * (W - 1) * case["C"] * esz
        par = (W + 1) * cols * 4
        if kind == "conv_train":  # x, gy in; y, gx out
            return dict(bytes=4 * E * esz + 2 * par, flops=E * (6 * W + 18))
        return dict(bytes=2 * E * esz + 2 * state + par, flops=E * (2 * W + 5))
    N = case["N"]
    bc = case["B"] * case["T"] * N * esz
    par = (N + 2) * cols * 4
    acts = 4 if case["gate"] else 3  # x, dt (, z) in and y out
    flops = E * (7 * N + 14)
    if kind == "scan_train":  # gy in, gx, gdt (, gz) and gB, gC out besides
        return dict(bytes=E * esz * (2 * acts) + 4 * bc + 2 * par, flops=flops + E * (17 * N + 24))
    state = case["B"] * case["C"] * N * 4
    return dict(bytes=E * esz * acts + 2 * bc + 2 * state + par, flops=flops)
