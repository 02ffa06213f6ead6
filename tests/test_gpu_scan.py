"""The selective scan's forward, backward and step on the GPU against the 64-bit reference, within the
bounds of fp32 arithmetic that it derives (tests/_mixer_ref.py)."""
import pytest
import torch

import _mixer_ref as ref
import rwkv_wkv_recurrence_b200 as rw
from test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu
DT = pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
INPUTS = ("x", "dt", "b", "c", "a_log", "d", "dt_bias", "z", "h_in")


def _dev(p, views, dev):
    return {k: views.get(k, lambda t: t)(v.to(dev)) for k, v in p.items()}


def _cpu(p, views):
    return {k: views.get(k, lambda t: t)(v) for k, v in p.items()}


def _forward(q, **kw):
    return rw.rwkv_selective_scan_forward(*(q[k] for k in INPUTS[:5]), q.get("d"), q.get("dt_bias"), q.get("z"),
                                          q.get("h_in"), **kw)


def _backward(q, ckpt=None):
    out = rw.rwkv_selective_scan_backward(*(q[k] for k in INPUTS[:5]), q["gy"], q.get("d"), q.get("dt_bias"),
                                          q.get("z"), ckpt, q.get("h_in"), q.get("gh_out"), want_gh_in=True)
    return dict(zip(("gx", "gdt", "gb", "gc", "ga_log", "gd", "gdt_bias", "gz", "gh_in"), out))


# lengths of one token, below, at and above the 16-token checkpoints and 32-token tiles; channels that fill,
# part-fill and pass a CTA's; every state size
SHAPES = [(1, 1, 8, 16), (2, 5, 3, 16), (1, 16, 64, 16), (2, 33, 72, 16), (1, 100, 65, 16), (2, 47, 130, 8),
          (1, 31, 40, 32), (2, 64, 19, 64), (1, 17, 1, 8), (3, 2, 24, 64)]


@DT
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_backward(cuda_device, shape, dtype):
    for full in (True, False):
        p, v = ref.scan_inputs(*shape, seed=21, dtype=dtype, gate=full, extras=full, states=full)
        r = ref.scan(**_cpu(p, v))
        q = _dev(p, v, cuda_device)
        y, h, ck = _forward(q, return_state=True, checkpoints=True)
        ref.check_all(dict(y=y, h=h, ckpt=ck), r, f"full={full} ")
        with_ck, without = _backward(q, ck), _backward(q)
        ref.check_all(with_ck, r, f"full={full} ")
        assert all(a is None if b is None else torch.equal(a, b) for a, b in zip(with_ck.values(), without.values()))
        assert (with_ck["gz"] is None) == (with_ck["gd"] is None) == (not full)


@DT
def test_time_in_segments(cuda_device, dtype):
    # few channels and a long sequence: the segmented schedule, asked for and chosen, and whatever the
    # backward chooses; states in and out on both sides
    p, v = ref.scan_inputs(1, 421, 24, 16, seed=22, dtype=dtype)
    r = ref.scan(**_cpu(p, v))
    q = _dev(p, v, cuda_device)
    for algo in (rw.ALGO_SEQUENTIAL, rw.ALGO_CHUNKED, rw.ALGO_AUTO):
        y, h, ck = _forward(q, return_state=True, checkpoints=True, algo=algo)
        ref.check_all(dict(y=y, h=h, ckpt=ck), r, f"algo {algo} ")
        ref.check_all(_backward(q, ck), r, f"algo {algo} ")
    h2 = rw.lib().rwkv_selective_scan_forward_workspace_bytes(1, 421, 24, 16, rw.ALGO_AUTO)
    assert h2 > 0  # the cases above did cut time


@DT
@pytest.mark.parametrize("shape", [(2, 70, 64, 16), (1, 40, 33, 8)], ids=str)
def test_parts_of_wider_tensors(cuda_device, shape, dtype):
    p, v = ref.scan_inputs(*shape, seed=23, dtype=dtype, wide=True)
    r = ref.scan(**_cpu(p, v))
    q = _dev(p, v, cuda_device)
    assert not q["x"].is_contiguous() and not q["b"].is_contiguous()
    y, h, ck = _forward(q, return_state=True, checkpoints=True)
    ref.check_all(dict(y=y, h=h), r)
    ref.check_all(_backward(q, ck), r)


@pytest.mark.parametrize("at", [1, 3])
def test_b_and_c_off_the_16_byte_grid(cuda_device, at):
    # b and c as parts of rows at an odd place (single accesses) beside x, dt, z in wide ones
    p, v = ref.scan_inputs(2, 40, 48, 16, seed=36, dtype=torch.bfloat16)
    r = ref.scan(**p)
    q = _dev(p, v, cuda_device)
    rows = torch.zeros(2, 40, 48, dtype=torch.bfloat16, device=cuda_device)
    rows[..., at: at + 16], rows[..., 24 + at: 40 + at] = q["b"], q["c"]
    q["b"], q["c"] = rows[..., at: at + 16], rows[..., 24 + at: 40 + at]
    y, h, ck = _forward(q, return_state=True, checkpoints=True)
    ref.check_all(dict(y=y, h=h), r)
    ref.check_all(_backward(q, ck), r)


@DT
@pytest.mark.parametrize("shape", [(2, 300, 97, 16), (1, 517, 131, 8), (2, 90, 35, 32), (1, 70, 21, 64)], ids=str)
def test_rows_that_start_anywhere(cuda_device, shape, dtype):
    # every array a part of rows of an odd length at an odd place, over several tiles and segments: single
    # accesses, in bf16 as halves of 32-bit words; NaN around the parts stays there
    p, v = ref.scan_inputs(*shape, seed=38, dtype=dtype)
    r = ref.scan(**_cpu(p, v))
    q = _dev(p, v, cuda_device)
    B, T, C, _ = shape
    for n, (k, at) in enumerate((("x", 1), ("dt", 2), ("z", 3))):
        rows = torch.full((B, T, C + 4 + n % 2), float("nan"), dtype=dtype, device=cuda_device)
        rows[..., at: at + C] = q[k]
        q[k] = rows[..., at: at + C]
    y, h, ck = _forward(q, return_state=True, checkpoints=True)
    ref.check_all(dict(y=y, h=h), r)
    ref.check_all(_backward(q, ck), r)


def test_step_of_many_streams(cuda_device):
    # more streams than the grid's second dimension holds; rows of every part against single-stream calls
    B, C, N = 70001, 4, 8
    p, v = ref.scan_inputs(B, 1, C, N, seed=37, grads=False)
    q = {k: (t[:, 0] if t.dim() == 3 and k != "h_in" else t) for k, t in _dev(p, v, cuda_device).items()}
    so = torch.empty_like(q["h_in"])
    y = rw.rwkv_selective_scan_step(*(q[k] for k in INPUTS[:5]), q["h_in"], q["d"], q["dt_bias"], q["z"], state_out=so)
    for b in (0, 1, 2, 65534, 65535, 65536, 70000):
        one = {k: (t[b: b + 1].contiguous() if k in ("x", "dt", "b", "c", "z", "h_in") else t) for k, t in q.items()}
        s1 = torch.empty_like(one["h_in"])
        y1 = rw.rwkv_selective_scan_step(*(one[k] for k in INPUTS[:5]), one["h_in"], one["d"], one["dt_bias"], one["z"],
                                         state_out=s1)
        assert torch.equal(y[b], y1[0]) and torch.equal(so[b], s1[0]), b


def test_many_segments(cuda_device):
    # one channel tile over a long sequence: as many segments as there are tiles, folded in order
    p, v = ref.scan_inputs(1, 1500, 5, 8, seed=38)
    r = ref.scan(**p)
    q = _dev(p, v, cuda_device)
    y, h, ck = _forward(q, return_state=True, checkpoints=True)
    ref.check_all(dict(y=y, h=h, ckpt=ck), r)
    ref.check_all(_backward(q, ck), r)


@DT
@pytest.mark.parametrize("shape", [(1, 1, 1, 8), (3, 1, 40, 16), (5, 1, 77, 32), (130, 1, 24, 64)], ids=str)
def test_step(cuda_device, shape, dtype):
    for full in (True, False):
        p, v = ref.scan_inputs(*shape, seed=24, dtype=dtype, gate=full, extras=full, grads=False)
        r = ref.scan(**p)
        q = _dev(p, v, cuda_device)
        one = {k: (t[:, 0] if k in ("x", "dt", "b", "c", "z") else t) for k, t in q.items()}
        st = q["h_in"].clone()
        so = torch.empty_like(st)
        args = [one[k] for k in INPUTS[:5]]
        opt = [one.get("d"), one.get("dt_bias"), one.get("z")]
        y = rw.rwkv_selective_scan_step(*args, st, *opt, state_out=so)
        ref.check(y, r["y"][0][:, 0], r["y"][1][:, 0], "y")
        ref.check(so, *r["h"], "state")
        assert torch.equal(st, q["h_in"])
        y2 = rw.rwkv_selective_scan_step(*args, st, *opt)
        assert torch.equal(y, y2) and torch.equal(st, so)


def test_prompt_then_steps(cuda_device):
    # a prompt in two parts, then single tokens, equals the whole prompt
    p, v = ref.scan_inputs(2, 50, 40, 16, seed=25, grads=False)
    r = ref.scan(**p)
    q = _dev(p, v, cuda_device)
    cut = lambda a, b: {k: (t[:, a:b].contiguous() if k in ("x", "dt", "b", "c", "z") else t) for k, t in q.items()}
    y0, h = _forward(dict(cut(0, 19)), return_state=True)
    y1, h = _forward(dict(cut(19, 45), h_in=h), return_state=True)
    ys = [y0, y1]
    for t in range(45, 50):
        one = {k: (s[:, t] if k in ("x", "dt", "b", "c", "z") else s) for k, s in q.items()}
        ys.append(rw.rwkv_selective_scan_step(*(one[k] for k in INPUTS[:5]), h, one["d"], one["dt_bias"],
                                              one["z"])[:, None])
    ref.check(torch.cat(ys, 1), *r["y"], "y")
    ref.check(h, *r["h"], "h")


def test_gradients_against_differences(cuda_device):
    # directional central differences of the kernel's own fp32 forward.  With |loss| ~ a sum of n ~ 1500
    # terms of order 1 rounded at 2^-24 each, a step of 2^-6 and the 2^-12 / 6 |f'''| of the formula: 1 %
    p, v = ref.scan_inputs(1, 24, 16, 8, seed=26)
    q = _dev(p, v, cuda_device)
    g = _backward(q)
    key = dict(x="gx", dt="gdt", b="gb", c="gc", a_log="ga_log", d="gd", dt_bias="gdt_bias", z="gz", h_in="gh_in")

    def loss(s):
        y, h = _forward(s, return_state=True)
        return float((y.double() * q["gy"].double()).sum() + (h.double() * q["gh_out"].double()).sum())

    gen = torch.Generator().manual_seed(5)
    for name, gname in key.items():
        d = torch.randn(q[name].shape, generator=gen).to(cuda_device)
        want = float((g[gname].double() * d.double()).sum())
        step = 2.0 ** -6
        num = (loss(dict(q, **{name: q[name] + step * d})) - loss(dict(q, **{name: q[name] - step * d}))) / (2 * step)
        scale = float((g[gname].double() * d.double()).abs().sum())
        assert abs(num - want) <= 0.01 * scale + 1e-3, (name, num, want, scale)


def test_state_updated_in_place(cuda_device):
    # h_out may be h_in on both schedules; gh_in may be gh_out
    p, v = ref.scan_inputs(1, 300, 24, 16, seed=27)
    q = _dev(p, v, cuda_device)
    h, P, S = rw.lib(), rw._ptr, rw._stream(None)
    B, T, C, N = 1, 300, 24, 16
    for algo in (rw.ALGO_SEQUENTIAL, rw.ALGO_CHUNKED):
        y0, h0, ck = _forward(q, return_state=True, checkpoints=True, algo=algo)
        st, y = q["h_in"].clone(), torch.empty_like(y0)
        wsb = int(h.rwkv_selective_scan_forward_workspace_bytes(B, T, C, N, algo))
        ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=cuda_device)
        assert h.rwkv_selective_scan_forward(B, T, C, N, 0, P(q["a_log"]), P(q["d"]), P(q["dt_bias"]), P(q["x"]), C,
                                             P(q["dt"]), C, P(q["b"]), N, P(q["c"]), N, P(q["z"]), C, P(y), P(st),
                                             P(st), None, 16, algo, P(ws), wsb, S) == 0
        assert torch.equal(y, y0) and torch.equal(st, h0)
    want = _backward(q, ck)
    gst = q["gh_out"].clone()
    outs = {k: torch.empty_like(t) for k, t in want.items() if k != "gh_in"}
    wsb = int(h.rwkv_selective_scan_backward_workspace_bytes(B, T, C, N, 16, 1))
    ws = torch.empty(wsb, dtype=torch.uint8, device=cuda_device)
    assert h.rwkv_selective_scan_backward(B, T, C, N, 0, P(q["a_log"]), P(q["d"]), P(q["dt_bias"]), P(q["x"]), C,
                                          P(q["dt"]), C, P(q["b"]), N, P(q["c"]), N, P(q["z"]), C, P(q["gy"]), None,
                                          P(gst), P(ck), 16, P(outs["gx"]), P(outs["gdt"]), P(outs["gb"]),
                                          P(outs["gc"]), P(outs["gz"]), P(outs["ga_log"]), P(outs["gd"]),
                                          P(outs["gdt_bias"]), P(gst), P(ws), wsb, S) == 0
    assert torch.equal(gst, want["gh_in"])
    assert all(torch.equal(outs[k], want[k]) for k in outs)


@pytest.mark.parametrize("dtype,shape,off", [(torch.float32, (2, 40, 24, 16), 0), (torch.float32, (1, 35, 33, 8), 1),
                                             (torch.bfloat16, (2, 50, 40, 32), 0),
                                             (torch.bfloat16, (1, 300, 20, 16), 3)])
def test_writes_only_its_outputs(cuda_device, dtype, shape, off):
    B, T, C, N = shape
    p, v = ref.scan_inputs(*shape, seed=28, dtype=dtype)
    q = _dev(p, v, cuda_device)
    r = ref.scan(**p)
    h, P, S = rw.lib(), rw._ptr, rw._stream(None)
    code = rw.F32 if dtype == torch.float32 else rw.BF16
    f32 = torch.float32
    btc = {k: Guarded((B, T, C), dtype, cuda_device, off) for k in ("y", "gx", "gdt", "gz")}
    btn = {k: Guarded((B, T, N), dtype, cuda_device, off) for k in ("gb", "gc")}
    st = {k: Guarded((B, C, N), f32, cuda_device) for k in ("h", "gh_in")}
    par = {"ga_log": Guarded((C, N), f32, cuda_device), "gd": Guarded((C,), f32, cuda_device),
           "gdt_bias": Guarded((C,), f32, cuda_device), "ckpt": Guarded(((T + 15) // 16, B, C, N), f32, cuda_device)}
    al = {**btc, **btn, **st, **par}
    rows = (P(q["x"]), C, P(q["dt"]), C, P(q["b"]), N, P(q["c"]), N, P(q["z"]), C)
    wsb = int(h.rwkv_selective_scan_forward_workspace_bytes(B, T, C, N, rw.ALGO_CHUNKED))
    ws = Guarded((max(wsb // 4, 4),), f32, cuda_device)
    assert h.rwkv_selective_scan_forward(B, T, C, N, code, P(q["a_log"]), P(q["d"]), P(q["dt_bias"]), *rows,
                                         al["y"].ptr(), P(q["h_in"]), al["h"].ptr(), al["ckpt"].ptr(), 16,
                                         rw.ALGO_CHUNKED, ws.ptr(), wsb, S) == 0
    ws.check("forward workspace")
    wsb = int(h.rwkv_selective_scan_backward_workspace_bytes(B, T, C, N, 16, 0))
    ws = Guarded((wsb // 4,), f32, cuda_device)
    assert h.rwkv_selective_scan_backward(B, T, C, N, code, P(q["a_log"]), P(q["d"]), P(q["dt_bias"]), *rows,
                                          P(q["gy"]), P(q["h_in"]), P(q["gh_out"]), None, 16, al["gx"].ptr(),
                                          al["gdt"].ptr(), al["gb"].ptr(), al["gc"].ptr(), al["gz"].ptr(),
                                          al["ga_log"].ptr(), al["gd"].ptr(), al["gdt_bias"].ptr(),
                                          al["gh_in"].ptr(), ws.ptr(), wsb, S) == 0
    rw.rwkv_check_device_error()
    ws.check("backward workspace")
    for k, b_ in al.items():
        b_.check(k)
        ref.check(b_.t, *r[k], k)


def test_fast_and_slow_decays(cuda_device):
    # steps so large that a state forgets within a token (the decay underflows to 0), so small that it
    # never does, and dt at the ends of softplus
    p, v = ref.scan_inputs(1, 90, 32, 16, seed=29)
    p["dt"][:, ::3] += 30.0
    p["dt"][:, 1::7] -= 60.0
    p["a_log"][:8] += 6.0
    p["a_log"][8:16] -= 12.0
    r = ref.scan(**p)
    q = _dev(p, v, cuda_device)
    y, h, ck = _forward(q, return_state=True, checkpoints=True)
    ref.check_all(dict(y=y, h=h, ckpt=ck), r)
    ref.check_all(_backward(q, ck), r)


def test_nan_stays_with_its_channel(cuda_device):
    p, v = ref.scan_inputs(1, 70, 24, 16, seed=30, grads=False)
    q = _dev(p, v, cuda_device)
    clean, hc = _forward(q, return_state=True)
    q["x"][0, 20, 5] = float("nan")
    y, h = _forward(q, return_state=True)
    keep = torch.ones(24, dtype=torch.bool, device=cuda_device)
    keep[5] = False
    assert torch.equal(y[..., keep], clean[..., keep]) and torch.equal(h[:, keep], hc[:, keep])
    assert torch.equal(y[:, :20], clean[:, :20]) and torch.isnan(y[0, 20:, 5]).all() and torch.isnan(h[0, 5]).all()


def test_endless_rate(cuda_device):
    # a_log = inf: the state forgets at once, and a ragged tile's end leaves it alone
    p, v = ref.scan_inputs(1, 21, 8, 16, seed=31, grads=False)
    q = _dev(p, v, cuda_device)
    q["a_log"][3] = float("inf")
    y, h = _forward(q, return_state=True)
    dl = torch.nn.functional.softplus(q["dt"][0, -1, 3] + q["dt_bias"][3])
    assert torch.allclose(h[0, 3], dl * q["x"][0, -1, 3] * q["b"][0, -1], rtol=1e-5)
    assert torch.isfinite(y).all() and torch.isfinite(h).all()


def test_empty(cuda_device):
    p, v = ref.scan_inputs(2, 0, 8, 16, seed=32)
    q = _dev(p, v, cuda_device)
    y, h, ck = _forward(q, return_state=True, checkpoints=True)
    assert y.shape == (2, 0, 8) and ck.shape[0] == 0 and torch.equal(h, q["h_in"])
    g = _backward(q, ck)
    assert not g["ga_log"].any() and not g["gd"].any() and torch.equal(g["gh_in"], q["gh_out"])
    _, h = _forward(dict(q, h_in=None), return_state=True)
    assert torch.equal(h, torch.zeros_like(h))


def test_same_bits_twice(cuda_device):
    p, v = ref.scan_inputs(2, 300, 200, 16, seed=33, dtype=torch.bfloat16)
    q = _dev(p, v, cuda_device)
    a, b = _backward(q), _backward(q)
    assert all(torch.equal(a[k], b[k]) for k in a)
