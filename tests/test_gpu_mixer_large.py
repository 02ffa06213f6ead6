"""The convolution, the selective scan and the layer norm on tensors of more than 2^31 elements: the parts at the
highest offsets equal, bit for bit, what a call on those parts alone gives."""
import pytest
import torch

import rwkv_wkv_recurrence_b200 as rw

pytestmark = pytest.mark.gpu
B, T, C = 520, 2048, 2056  # 2.19e9 elements


def _act(dev, *shape, scale=1.0):
    t = torch.empty(*shape, dtype=torch.bfloat16, device=dev)
    for part in t.split(64):  # bounds the fp32 temporaries of the generator
        part.normal_().mul_(scale)
    return t


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


def test_conv(cuda_device):
    x, gy = _act(cuda_device, B, T, C), _act(cuda_device, B, T, C)
    w, bias = torch.randn(C, 4, device=cuda_device), torch.randn(C, device=cuda_device)
    y, st = rw.rwkv_causal_conv_forward(x, w, bias, silu=True, return_state=True)
    gx = rw.rwkv_causal_conv_backward(x, w, gy, bias, silu=True)[0]
    for b in (0, B - 1):
        one = x[b: b + 1]
        y1, st1 = rw.rwkv_causal_conv_forward(one, w, bias, silu=True, return_state=True)
        gx1 = rw.rwkv_causal_conv_backward(one, w, gy[b: b + 1], bias, silu=True)[0]
        assert torch.equal(y[b], y1[0]) and torch.equal(st[b], st1[0]) and torch.equal(gx[b], gx1[0])


def test_norm(cuda_device):
    x, gy = _act(cuda_device, B * T, C), _act(cuda_device, B * T, C)
    w, bias = torch.randn(C, device=cuda_device), torch.randn(C, device=cuda_device)
    y = rw.rwkv_layer_norm_forward(x, w, bias, groups=8)
    gx = rw.rwkv_layer_norm_backward(x, w, gy, bias, groups=8)[0]
    for sl in (slice(0, 100), slice(B * T - 100, B * T)):
        assert torch.equal(y[sl], rw.rwkv_layer_norm_forward(x[sl], w, bias, groups=8))
        assert torch.equal(gx[sl], rw.rwkv_layer_norm_backward(x[sl], w, gy[sl], bias, groups=8)[0])


def test_scan(cuda_device):
    N = 8
    x, dt, gy = (_act(cuda_device, B, T, C, scale=s) for s in (1.0, 0.5, 1.0))
    b, c = _act(cuda_device, B, T, N), _act(cuda_device, B, T, N)
    a_log = torch.log(torch.arange(1, N + 1, device=cuda_device).float()).expand(C, N).contiguous()
    bias = torch.full((C,), -3.0, device=cuda_device)
    y, h = rw.rwkv_selective_scan_forward(x, dt, b, c, a_log, dt_bias=bias, return_state=True)
    i = B - 1
    last = [t[i:].contiguous() for t in (x, dt, b, c)]
    y1, h1 = rw.rwkv_selective_scan_forward(*last, a_log, dt_bias=bias, return_state=True, algo=rw.ALGO_SEQUENTIAL)
    assert torch.equal(y[i], y1[0]) and torch.equal(h[i], h1[0])
    del y
    g = rw.rwkv_selective_scan_backward(x, dt, b, c, a_log, gy, dt_bias=bias)
    g1 = rw.rwkv_selective_scan_backward(*last, a_log, gy[i:].contiguous(), dt_bias=bias)
    # the two calls cut time differently: fp32 sums in another order, then one rounding to bf16 (2^-8 of the value)
    for k, name in enumerate(("gx", "gdt", "gb", "gc")):
        a, want = g[k][i].float(), g1[k][0].float()
        assert ((a - want).abs() <= 2 * 2.0 ** -8 * want.abs() + 1e-4 * want.abs().max()).all(), name
