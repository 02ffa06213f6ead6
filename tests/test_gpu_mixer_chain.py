"""The operators around the recurrence used together: a scan block (norm, convolution, scan) as prompt, in
single tokens and in training, and the head norm with its gate behind the Eagle operator; on side streams and
in captured graphs."""
import pytest
import torch

import _mixer_ref as ref
import oracle
import rwkv_wkv_recurrence_b200 as rw
import wkv_inputs as wi

pytestmark = pytest.mark.gpu


def _block(B, T, C, N, W, seed, dev, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    p, _ = ref.scan_inputs(B, T, C, N, seed + 1, dtype=dtype, states=False)
    p = {k: v for k, v in p.items() if k != "x"}
    p.update(u=n(B, T, C).to(dtype), nw=n(C) * 0.1 + 1, nb=n(C) * 0.1, cw=n(C, W) * 0.5, cb=n(C) * 0.1)
    return {k: v.to(dev) for k, v in p.items()}


def _prompt(q, **kw):
    x = rw.rwkv_layer_norm_forward(q["u"], q["nw"], q["nb"])
    v = rw.rwkv_causal_conv_forward(x, q["cw"], q["cb"], silu=True)
    return x, v, rw.rwkv_selective_scan_forward(v, q["dt"], q["b"], q["c"], q["a_log"], q["d"], q["dt_bias"], q["z"],
                                                checkpoints=True, **kw)


def _reference(q):
    c = {k: v.detach().cpu().double() for k, v in q.items()}
    xs = c["u"]
    m = xs.mean(-1, keepdim=True)
    x = (xs - m) / torch.sqrt(xs.var(-1, unbiased=False, keepdim=True) + 1e-5) * c["nw"] + c["nb"]
    v = ref.conv(x, c["cw"], c["cb"], silu=True)["y"][0]
    y = ref.scan(v, c["dt"], c["b"], c["c"], c["a_log"], c["d"], c["dt_bias"], c["z"])["y"][0]
    return x, v, y


def test_block_prompt_and_tokens(cuda_device):
    B, T, C, N, W = 2, 40, 48, 16, 4
    q = _block(B, T, C, N, W, 51, cuda_device)
    _, _, (y, _) = _prompt(q)
    want = _reference(q)[2].to(cuda_device)
    # three fp32 operators in a row, each within a few hundred half-steps of values of order 1 .. 10
    assert torch.allclose(y.double(), want, rtol=1e-4, atol=1e-4)
    conv = torch.zeros(B, W - 1, C, device=cuda_device)
    state = torch.zeros(B, C, N, device=cuda_device)
    for t in range(T):
        x = rw.rwkv_layer_norm_forward(q["u"][:, t].contiguous(), q["nw"], q["nb"])
        v = rw.rwkv_causal_conv_step(x, q["cw"], conv, q["cb"], silu=True)
        yt = rw.rwkv_selective_scan_step(v, q["dt"][:, t], q["b"][:, t], q["c"][:, t], q["a_log"], state, q["d"],
                                         q["dt_bias"], q["z"][:, t])
        assert torch.allclose(yt.double(), want[:, t], rtol=1e-4, atol=1e-4), t


def test_block_gradients(cuda_device):
    # the chained backward against float64 autograd of the chained formulas, relative to each gradient's
    # largest entry: three fp32 backward passes, sums over at most B T = 60 tokens and 24 channels
    B, T, C, N, W = 2, 30, 24, 8, 4
    q = _block(B, T, C, N, W, 52, cuda_device)
    x, v, (y, ck) = _prompt(q)
    gv, gdt, gb, gc, ga, gd, gbias, gz = rw.rwkv_selective_scan_backward(
        v, q["dt"], q["b"], q["c"], q["a_log"], q["gy"], q["d"], q["dt_bias"], q["z"], ck)
    gx, gcw, gcb = rw.rwkv_causal_conv_backward(x, q["cw"], gv, q["cb"], silu=True)
    gu, gnw, gnb, _ = rw.rwkv_layer_norm_backward(q["u"], q["nw"], gx, q["nb"])
    got = dict(u=gu, nw=gnw, nb=gnb, cw=gcw, cb=gcb, dt=gdt, b=gb, c=gc, a_log=ga, d=gd, dt_bias=gbias, z=gz)
    leaf = {k: t.detach().cpu().double().requires_grad_() for k, t in q.items() if k in got}
    xs = leaf["u"]
    xr = (xs - xs.mean(-1, keepdim=True)) / torch.sqrt(xs.var(-1, unbiased=False, keepdim=True) + 1e-5)
    xr = xr * leaf["nw"] + leaf["nb"]
    xp = torch.cat([xr.new_zeros(B, W - 1, C), xr], 1)
    vr = torch.nn.functional.silu(sum(xp[:, j: j + T] * leaf["cw"][:, j] for j in range(W)) + leaf["cb"])
    dl = torch.nn.functional.softplus(leaf["dt"] + leaf["dt_bias"])
    h, loss = torch.zeros(B, C, N, dtype=torch.float64), 0.0
    for t in range(T):
        h = torch.exp(dl[:, t, :, None] * -torch.exp(leaf["a_log"])) * h \
            + (dl[:, t] * vr[:, t])[..., None] * leaf["b"][:, t, None]
        yt = torch.einsum("bcn,bn->bc", h, leaf["c"][:, t]) + leaf["d"] * vr[:, t]
        loss = loss + (yt * torch.nn.functional.silu(leaf["z"][:, t]) * q["gy"][:, t].cpu().double()).sum()
    want = torch.autograd.grad(loss, list(leaf.values()))
    for k, w in zip(leaf, want):
        err = (got[k].cpu().double() - w).abs().max() / w.abs().max()
        assert err <= 1e-4, (k, float(err))


def test_head_norm_behind_eagle(cuda_device):
    # y = eagle(r, k, v), o = head norm of y times silu(g), and the gradient back into r, k, v
    B, T, H, N = 1, 70, 3, 64
    p = wi.wkv5_problem(B, T, H, N, seed=53)
    c = {k: t.to(cuda_device) for k, t in p.items()}
    g = torch.Generator().manual_seed(54)
    w, b = torch.randn(H * N, generator=g) * 0.1 + 1, torch.randn(H * N, generator=g) * 0.1
    gate, go = (torch.randn(B, T, H * N, generator=g).bfloat16() for _ in range(2))
    wd, bd, gated, god = (t.to(cuda_device) for t in (w, b, gate, go))
    y = rw.rwkv_wkv5_forward(c["r"], c["k"], c["v"], c["omega"], c["u"]).view(B, T, H * N)
    o = rw.rwkv_layer_norm_forward(y, wd, bd, gated, groups=H)
    r = ref.norm(y, w, b, gate, H, 1e-5, go)  # the norm's own part, on the very y it read
    ref.check(o, *r["y"], "o")
    gy, gw, gb, gg = rw.rwkv_layer_norm_backward(y, wd, god, bd, gated, groups=H)
    ref.check_all(dict(gx=gy, gw=gw, gbias=gb, ggate=gg), r)
    gr, gk, gv, gom, gu = rw.rwkv_wkv5_backward(c["r"], c["k"], c["v"], c["omega"], c["u"], gy.view(B, T, H, N))
    rw.rwkv_check_device_error()
    rr, rk, rv, rom, ru, _ = oracle.wkv5_backward(p["r"], p["k"], p["v"], p["omega"], p["u"],
                                                  gy.view(B, T, H, N).cpu(), s_in=None, gs_out=None)
    from _parity import TOL_BF16, assert_close_rms
    for got, want, name in ((gr, rr, "gr"), (gk, rk, "gk"), (gv, rv, "gv"), (gom, rom, "gomega"), (gu, ru, "gu")):
        assert_close_rms(got.cpu(), want, TOL_BF16, name)


def _everything(q, stream=None):
    x = rw.rwkv_layer_norm_forward(q["u"], q["nw"], q["nb"], stream=stream)
    v = rw.rwkv_causal_conv_forward(x, q["cw"], q["cb"], silu=True, stream=stream)
    y, ck = rw.rwkv_selective_scan_forward(v, q["dt"], q["b"], q["c"], q["a_log"], q["d"], q["dt_bias"], q["z"],
                                           checkpoints=True, stream=stream)
    g = rw.rwkv_selective_scan_backward(v, q["dt"], q["b"], q["c"], q["a_log"], q["gy"], q["d"], q["dt_bias"], q["z"],
                                        ck, stream=stream)
    gc = rw.rwkv_causal_conv_backward(x, q["cw"], g[0], q["cb"], silu=True, stream=stream)
    gn = rw.rwkv_layer_norm_backward(q["u"], q["nw"], gc[0], q["nb"], stream=stream)
    return [t for t in (x, v, y, *g, *gc, *gn) if t is not None]


def test_two_streams_at_once(cuda_device):
    # two chains in flight on two streams, neither the current one, with their own workspaces
    qs = [_block(1, 500, 64, 16, 4, 55 + i, cuda_device, torch.bfloat16) for i in range(2)]
    want = [_everything(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [_everything(q, s) for _ in range(3) for q, s in zip(qs, streams)]
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for i, out in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(out, want[i % 2]))


def test_captured_training_step(cuda_device):
    # a captured forward and backward, replayed on new inputs, gives what eager calls give; two graphs
    # replayed together keep apart
    qs = [_block(1, 300, 40, 16, 4, 57 + i, cuda_device) for i in range(2)]
    side = torch.cuda.Stream()
    graphs, outs, ins = [], [], []
    for q in qs:
        s = {k: torch.zeros_like(v) for k, v in q.items()}
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _everything(s)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = _everything(s)
        graphs.append(g), outs.append(o), ins.append(s)
    for turn in range(2):
        for s, q in zip(ins, qs):
            for k in s:
                s[k].copy_(q[k])
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, q in zip(outs, qs):
            assert all(torch.equal(a, b) for a, b in zip(o, _everything(q)))
        qs = [{k: v.flip(0) if v.dim() == 1 else v * 0.5 for k, v in q.items()} for q in qs]


def test_captured_decode(cuda_device):
    B, C, N, W = 3, 40, 16, 4
    q = _block(B, 6, C, N, W, 59, cuda_device)
    one = [{k: (v[:, t].contiguous() if v.dim() == 3 else v) for k, v in q.items()} for t in range(6)]

    def steps(conv, state):
        ys = []
        for s in one:
            x = rw.rwkv_layer_norm_forward(s["u"], s["nw"], s["nb"])
            v = rw.rwkv_causal_conv_step(x, s["cw"], conv, s["cb"], silu=True)
            ys.append(rw.rwkv_selective_scan_step(v, s["dt"], s["b"], s["c"], s["a_log"], state, s["d"], s["dt_bias"],
                                                  s["z"]))
        return ys

    zero = lambda: (torch.zeros(B, W - 1, C, device=cuda_device), torch.zeros(B, C, N, device=cuda_device))
    c0, s0 = zero()
    want = steps(c0, s0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        steps(*zero())
    torch.cuda.current_stream().wait_stream(side)
    c1, s1 = zero()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = steps(c1, s1)
    c1.zero_(), s1.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and torch.equal(c0, c1) and torch.equal(s0, s1)
