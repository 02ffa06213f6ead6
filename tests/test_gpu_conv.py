"""The causal convolution's forward, backward and step on the GPU against the 64-bit reference, within
the bounds of fp32 arithmetic that it derives (tests/_mixer_ref.py)."""
import pytest
import torch

import _mixer_ref as ref
import rwkv_wkv_recurrence_b200 as rw
from test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu


def _inputs(B, T, C, W, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    return dict(x=n(B, T, C).to(dtype), w=n(C, W) * 0.6, bias=n(C) * 0.3, state=n(B, W - 1, C).to(dtype),
                gy=n(B, T, C).to(dtype), gstate=n(B, W - 1, C).to(dtype))


# lengths below, at and above the window, the forward's 32-token and the backward's 64-token stretches and
# its 512-token groups of them; channel counts on and off the 16-byte accesses
SHAPES = [(1, 1, 8), (2, 2, 16), (1, 3, 5), (2, 33, 24), (3, 64, 7), (1, 67, 40), (2, 130, 264), (1, 530, 33),
          (1, 1100, 8)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_backward(cuda_device, shape, W, dtype):
    B, T, C = shape
    p = _inputs(B, T, C, W, 11, dtype)
    q = {k: v.to(cuda_device) for k, v in p.items()}
    for silu, full in ((True, True), (False, True), (True, False)):
        bias, st, gs = ("bias", "state", "gstate") if full else (None, None, None)
        r = ref.conv(p["x"], p["w"], p.get(bias), p.get(st), silu, p["gy"], p.get(gs))
        y, so = rw.rwkv_causal_conv_forward(q["x"], q["w"], q.get(bias), q.get(st), silu=silu, return_state=True)
        gx, gw, gb, gsi = rw.rwkv_causal_conv_backward(q["x"], q["w"], q["gy"], q.get(bias), q.get(st), q.get(gs),
                                                       silu=silu, want_gstate_in=True)
        ref.check_all(dict(y=y, state=so, gx=gx, gw=gw, gbias=gb, gstate_in=gsi), r, f"silu={silu} full={full} ")
        assert (gb is None) == (not full)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_rows_of_a_wider_tensor(cuda_device, dtype):
    # x is the middle of rows 3 C + 8 wide (wide accesses) and of rows off the 16-byte grid
    for C, pad, at in ((64, 136, 64), (64, 75, 3), (33, 40, 5)):
        p = _inputs(2, 70, C, 4, 12, dtype)
        wide = torch.zeros(2, 70, C + pad, dtype=dtype)
        wide[..., at: at + C] = p["x"]
        xv = wide.to(cuda_device)[..., at: at + C]
        q = {k: v.to(cuda_device) for k, v in p.items()}
        r = ref.conv(p["x"], p["w"], p["bias"], None, True, p["gy"])
        y = rw.rwkv_causal_conv_forward(xv, q["w"], q["bias"], silu=True)
        gx, gw, gb = rw.rwkv_causal_conv_backward(xv, q["w"], q["gy"], q["bias"], silu=True)
        ref.check_all(dict(y=y, gx=gx, gw=gw, gbias=gb), r)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("BC", [(1, 1), (3, 40), (5, 77), (130, 264)], ids=str)
def test_step(cuda_device, BC, W, dtype):
    B, C = BC
    p = _inputs(B, 1, C, W, 13, dtype)
    q = {k: v.to(cuda_device) for k, v in p.items()}
    r = ref.conv(p["x"], p["w"], p["bias"], p["state"], True)
    st = q["state"].clone()
    so = torch.empty_like(st)
    y = rw.rwkv_causal_conv_step(q["x"][:, 0], q["w"], st, q["bias"], silu=True, state_out=so)
    ref.check(y, r["y"][0][:, 0], r["y"][1][:, 0], "y")
    ref.check(so, *r["state"], "state")
    assert torch.equal(st, q["state"])
    y2 = rw.rwkv_causal_conv_step(q["x"][:, 0], q["w"], st, q["bias"], silu=True)  # in place
    assert torch.equal(y, y2) and torch.equal(st, so)


def test_prompt_in_parts_is_the_prompt(cuda_device):
    # bit for bit: the window's sums do not depend on where the prompt was cut
    p = _inputs(2, 100, 48, 4, 14, torch.bfloat16)
    q = {k: v.to(cuda_device) for k, v in p.items()}
    y, so = rw.rwkv_causal_conv_forward(q["x"], q["w"], q["bias"], q["state"], silu=True, return_state=True)
    st, parts = q["state"], []
    for a, b in ((0, 1), (1, 3), (3, 40), (40, 98)):
        yy, st = rw.rwkv_causal_conv_forward(q["x"][:, a:b].contiguous(), q["w"], q["bias"], st, silu=True,
                                             return_state=True)
        parts.append(yy)
    for t in (98, 99):
        parts.append(rw.rwkv_causal_conv_step(q["x"][:, t], q["w"], st, q["bias"], silu=True)[:, None])
    assert torch.equal(torch.cat(parts, 1), y) and torch.equal(st, so)


def test_token_shift(cuda_device):
    # W = 2 with weight (1 - mu, mu) is the token shift
    x = torch.randn(2, 50, 32, device=cuda_device)
    mu = torch.rand(32, device=cuda_device)
    y = rw.rwkv_causal_conv_forward(x, torch.stack([1 - mu, mu], 1))
    prev = torch.cat([torch.zeros_like(x[:, :1]), x[:, :-1]], 1)
    assert torch.allclose(y, mu * x + (1 - mu) * prev, rtol=1e-6, atol=1e-6)


@pytest.mark.parametrize("dtype,C,off", [(torch.float32, 40, 0), (torch.float32, 33, 1), (torch.bfloat16, 40, 0),
                                         (torch.bfloat16, 12, 3)])
def test_writes_only_its_outputs(cuda_device, dtype, C, off):
    B, T, W = 2, 70, 4
    p = {k: v.to(cuda_device) for k, v in _inputs(B, T, C, W, 15, dtype).items()}
    h, P, S = rw.lib(), rw._ptr, rw._stream(None)
    code = rw.F32 if dtype == torch.float32 else rw.BF16
    y, gx = (Guarded((B, T, C), dtype, cuda_device, off) for _ in range(2))
    so, gs = (Guarded((B, W - 1, C), dtype, cuda_device, off) for _ in range(2))
    gw, gb = Guarded((C, W), torch.float32, cuda_device), Guarded((C,), torch.float32, cuda_device)
    wsb = int(h.rwkv_causal_conv_backward_workspace_bytes(B, T, C, W))
    ws = Guarded((wsb // 4,), torch.float32, cuda_device)
    assert h.rwkv_causal_conv_forward(B, T, C, W, code, P(p["w"]), P(p["bias"]), 1, P(p["x"]), C, y.ptr(),
                                      P(p["state"]), so.ptr(), S) == 0
    assert h.rwkv_causal_conv_backward(B, T, C, W, code, P(p["w"]), P(p["bias"]), 1, P(p["x"]), C, P(p["state"]),
                                       P(p["gy"]), P(p["gstate"]), gx.ptr(), gw.ptr(), gb.ptr(), gs.ptr(), ws.ptr(),
                                       wsb, S) == 0
    rw.rwkv_check_device_error()
    for b_, name in ((y, "y"), (so, "state"), (gx, "gx"), (gs, "gstate"), (gw, "gw"), (gb, "gb"), (ws, "workspace")):
        b_.check(name)


def test_nan_and_inf_stay_in_their_window(cuda_device):
    x = torch.randn(1, 80, 16, device=cuda_device)
    w = torch.randn(16, 4, device=cuda_device)
    clean = rw.rwkv_causal_conv_forward(x, w, silu=True)
    x[0, 30, 5], x[0, 60, 7] = float("nan"), float("inf")
    y = rw.rwkv_causal_conv_forward(x, w, silu=True)
    touched = torch.zeros_like(x, dtype=torch.bool)
    touched[0, 30:34, 5] = touched[0, 60:64, 7] = True
    assert torch.equal(y[~touched], clean[~touched])
    assert torch.isnan(y[0, 30:34, 5]).all()


def test_empty(cuda_device):
    x = torch.zeros(2, 0, 8, device=cuda_device)
    w = torch.ones(8, 4, device=cuda_device)
    st = torch.randn(2, 3, 8, device=cuda_device)
    y, so = rw.rwkv_causal_conv_forward(x, w, state_in=st, return_state=True)
    assert y.shape == x.shape and torch.equal(so, st)
    _, so = rw.rwkv_causal_conv_forward(x, w, return_state=True)
    assert torch.equal(so, torch.zeros_like(so))
    gx, gw, gb, gs = rw.rwkv_causal_conv_backward(x, w, x, torch.ones(8, device=cuda_device), None, st,
                                                  want_gstate_in=True)
    assert gx.shape == x.shape and not gw.any() and not gb.any() and torch.equal(gs, st)
    y = rw.rwkv_causal_conv_forward(torch.zeros(0, 5, 8, device=cuda_device), w)
    assert y.shape == (0, 5, 8)


def test_same_bits_twice(cuda_device):
    p = {k: v.to(cuda_device) for k, v in _inputs(2, 700, 264, 4, 16, torch.bfloat16).items()}
    a = rw.rwkv_causal_conv_backward(p["x"], p["w"], p["gy"], p["bias"], silu=True)
    b = rw.rwkv_causal_conv_backward(p["x"], p["w"], p["gy"], p["bias"], silu=True)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("C,pad,at", [(66, 0, 0), (10, 4, 2), (2, 0, 0), (66, 3, 0), (65, 0, 0), (63, 2, 1), (1, 0, 0)])
def test_two_channels_a_thread(cuda_device, C, pad, at, W, dtype):
    # even channel counts that are no multiple of 4 (neighbours in one access), odd ones and odd rows (a
    # channel of each half); forward, backward and step, states in and out, the step's in place
    p = _inputs(2, 70, C, W, 16, dtype)
    wide = torch.full((2, 70, C + pad), float("nan"), dtype=dtype)
    wide[..., at: at + C] = p["x"]
    xv = wide.to(cuda_device)[..., at: at + C]
    q = {k: v.to(cuda_device) for k, v in p.items()}
    r = ref.conv(p["x"], p["w"], p["bias"], p["state"], True, p["gy"], p["gstate"])
    y, so = rw.rwkv_causal_conv_forward(xv, q["w"], q["bias"], q["state"], silu=True, return_state=True)
    gx, gw, gb, gs = rw.rwkv_causal_conv_backward(xv, q["w"], q["gy"], q["bias"], q["state"], q["gstate"], silu=True,
                                                  want_gstate_in=True)
    ref.check_all(dict(y=y, state=so, gx=gx, gw=gw, gbias=gb, gstate_in=gs), r)
    st = q["state"].clone()
    for t in range(3):
        yt = rw.rwkv_causal_conv_step(xv[:, t].contiguous(), q["w"], st, q["bias"], silu=True)
        assert torch.equal(yt, y[:, t]), t
