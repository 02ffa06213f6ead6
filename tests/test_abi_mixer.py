"""Refusals of the convolution, the selective scan and the layer norm, all on the host: the C calls answer
before any CUDA work, the Python binding before it calls them."""
import ctypes

import pytest
import torch

import rwkv_wkv_recurrence_b200 as rw

P = ctypes.c_void_p
F = P(0x1000)  # never dereferenced: every call below fails validation first
BIG = 1 << 40


def _conv_fwd(B=2, T=5, C=8, W=4, dt=0, w=F, bias=F, act=1, x=F, ldx=None, y=F, si=None, so=None):
    return rw.lib().rwkv_causal_conv_forward(B, T, C, W, dt, w, bias, act, x, C if ldx is None else ldx, y, si, so,
                                             None)


def _conv_bwd(B=2, T=5, C=8, W=4, dt=0, w=F, act=1, x=F, ldx=None, gy=F, gx=F, gw=F, gb=F, gs=None, ws=F, wsb=BIG):
    return rw.lib().rwkv_causal_conv_backward(B, T, C, W, dt, w, F, act, x, C if ldx is None else ldx, None, gy, None,
                                              gx, gw, gb, gs, ws, wsb, None)


def test_conv():
    assert _conv_fwd(B=-1) == 1 and _conv_fwd(T=1 << 31) == 1 and _conv_fwd(C=-8, ldx=8) == 1
    assert _conv_fwd(dt=2) == 1 and _conv_fwd(act=2) == 1 and _conv_fwd(ldx=7) == 1
    assert _conv_fwd(W=1) == 2 and _conv_fwd(W=5) == 2 and _conv_fwd(W=-4) == 1
    assert _conv_fwd(w=None) == 1 and _conv_fwd(x=None) == 1 and _conv_fwd(y=None) == 1
    assert _conv_fwd(x=P(0x1002)) == 2 and _conv_fwd(y=P(0x1001), dt=1) == 2 and _conv_fwd(so=P(0x1001), dt=1) == 2
    assert _conv_fwd(w=P(0x1002)) == 2
    assert _conv_fwd(B=0) == 0 and _conv_fwd(C=0, ldx=0) == 0 and _conv_fwd(T=0) == 0
    assert _conv_fwd(B=1 << 20, T=1 << 20, C=1 << 12) == 2  # more blocks than a grid holds
    assert _conv_bwd(W=5) == 2 and _conv_bwd(gw=None) == 1 and _conv_bwd(gx=None) == 1 and _conv_bwd(gy=None) == 1
    assert _conv_bwd(ws=None) == 3 and _conv_bwd(wsb=4) == 3 and _conv_bwd(ws=P(0x1002)) == 2
    assert _conv_bwd(gs=P(0x1003), dt=1) == 2 and _conv_bwd(ldx=3) == 1
    h = rw.lib()
    step = lambda **k: h.rwkv_causal_conv_step(k.get("B", 2), 8, k.get("W", 4), 0, F, F, k.get("act", 1), F,
                                               k.get("ldx", 8), F, None, k.get("so", F), None)
    assert step(so=None) == 1 and step(W=6) == 2 and step(ldx=4) == 1 and step(act=-1) == 1 and step(B=0) == 0
    assert h.rwkv_causal_conv_backward_workspace_bytes(2, 513, 8, 4) == 2 * 2 * 5 * 8 * 4
    assert h.rwkv_causal_conv_backward_workspace_bytes(2, 0, 8, 4) == 0


def _scan_rows(C, N, x=F, dt=F, b=F, c=F, z=None, ldx=None, ldb=None, ldz=None):
    return (x, C if ldx is None else ldx, dt, C, b, N if ldb is None else ldb, c, N, z, C if ldz is None else ldz)


def _scan_fwd(B=2, T=5, C=8, N=16, dt=0, a=F, y=F, hi=None, ho=None, ck=None, cl=16, algo=0, ws=None, wsb=0, **rows):
    return rw.lib().rwkv_selective_scan_forward(B, T, C, N, dt, a, None, None, *_scan_rows(C, N, **rows), y, hi, ho,
                                                ck, cl, algo, ws, wsb, None)


def _scan_bwd(B=2, T=5, C=8, N=16, dt=0, a=F, gy=F, gh=None, ck=F, cl=16, gx=F, gb=F, gz=None, ga=F, ghi=None, ws=F,
              wsb=BIG, **rows):
    return rw.lib().rwkv_selective_scan_backward(B, T, C, N, dt, a, None, None, *_scan_rows(C, N, **rows), gy, None,
                                                 gh, ck, cl, gx, F, gb, F, gz, ga, None, None, ghi, ws, wsb, None)


def test_scan():
    assert _scan_fwd(B=-2) == 1 and _scan_fwd(T=1 << 31) == 1 and _scan_fwd(dt=5) == 1 and _scan_fwd(algo=3) == 1
    for n in (0, 4, 12, 17, 128):
        assert _scan_fwd(N=n) == 2
    assert _scan_fwd(ldx=7) == 1 and _scan_fwd(ldb=15) == 1 and _scan_fwd(z=F, ldz=0) == 1
    assert _scan_fwd(a=None) == 1 and _scan_fwd(x=None) == 1 and _scan_fwd(b=None) == 1
    assert _scan_fwd(y=None) == 1  # nothing asked for
    assert _scan_fwd(cl=12, ck=F) == 1 and _scan_fwd(cl=32, ck=F) == 2
    assert _scan_fwd(hi=P(0x1004)) == 2 and _scan_fwd(ho=P(0x1008)) == 2 and _scan_fwd(ck=P(0x1004)) == 2
    assert _scan_fwd(x=P(0x1002)) == 2 and _scan_fwd(dt=1, b=P(0x1001)) == 2
    assert _scan_fwd(T=600, algo=rw.ALGO_CHUNKED) == 3 and _scan_fwd(T=600, algo=rw.ALGO_CHUNKED, ws=F, wsb=8) == 3
    assert _scan_fwd(T=600, algo=rw.ALGO_CHUNKED, ws=P(0x1004), wsb=BIG) == 2
    assert _scan_fwd(B=0) == 0 and _scan_fwd(C=0) == 0 and _scan_fwd(T=0) == 0
    assert _scan_fwd(B=1 << 20, T=1 << 20, C=1 << 12) == 2
    assert _scan_bwd(N=24) == 2 and _scan_bwd(cl=8) == 1 and _scan_bwd(cl=48) == 2 and _scan_bwd(ga=None) == 1
    assert _scan_bwd(gy=None) == 1 and _scan_bwd(gx=None) == 1 and _scan_bwd(gb=None) == 1
    assert _scan_bwd(z=F) == 1  # a gate without room for its gradient
    assert _scan_bwd(ws=None) == 3 and _scan_bwd(wsb=64) == 3 and _scan_bwd(ws=P(0x1008)) == 2
    assert _scan_bwd(gh=P(0x1004)) == 2 and _scan_bwd(ck=P(0x1004)) == 2 and _scan_bwd(ghi=P(0x1008)) == 2
    h = rw.lib()
    step = lambda **k: h.rwkv_selective_scan_step(k.get("B", 2), 8, k.get("N", 16), 0, F, None, None,
                                                  *_scan_rows(8, k.get("N", 16), ldx=k.get("ldx")), F,
                                                  k.get("hi"), k.get("ho", F), None)
    assert step(N=10) == 2 and step(ho=None) == 1 and step(ldx=2) == 1 and step(hi=P(0x1004)) == 2 and step(B=0) == 0


def test_scan_workspace_queries():
    h = rw.lib()
    q = h.rwkv_selective_scan_forward_workspace_bytes
    assert q(8, 4096, 2048, 16, rw.ALGO_AUTO) == 0  # enough channels: whole sequences
    assert q(1, 8192, 768, 16, rw.ALGO_SEQUENTIAL) == 0
    assert q(1, 8192, 768, 16, rw.ALGO_AUTO) > 0  # few: segments
    assert q(1, 32, 8, 16, rw.ALGO_CHUNKED) == 0  # one tile
    assert q(1, 100, 8, 12, rw.ALGO_CHUNKED) == 0 and q(0, 100, 8, 16, 0) == 0
    b = h.rwkv_selective_scan_backward_workspace_bytes
    assert b(4, 512, 640, 16, 16, 0) >= b(4, 512, 640, 16, 16, 1) + 32 * 4 * 640 * 16 * 4
    assert b(4, 0, 640, 16, 16, 0) == 0


def test_norm():
    h = rw.lib()

    def fwd(M=3, G=2, N=8, dt=0, w=F, eps=1e-5, x=F, y=F):
        return h.rwkv_layer_norm_forward(M, G, N, dt, w, F, eps, x, None, y, None)

    def bwd(M=3, G=2, N=8, dt=0, eps=1e-5, gate=None, gy=F, gx=F, gg=None, gw=F, ws=F, wsb=BIG):
        return h.rwkv_layer_norm_backward(M, G, N, dt, F, F, eps, F, gate, gy, gx, gg, gw, F, ws, wsb, None)

    assert fwd(M=-1) == 1 and fwd(G=-1) == 1 and fwd(N=1 << 31) == 1 and fwd(dt=3) == 1
    assert fwd(eps=-1e-9) == 1 and fwd(eps=float("nan")) == 1 and fwd(eps=float("inf")) == 1
    assert fwd(w=None) == 1 and fwd(x=None) == 1 and fwd(y=None) == 1
    assert fwd(x=P(0x1002)) == 2 and fwd(dt=1, y=P(0x1001)) == 2 and fwd(G=1 << 16, N=1 << 15) == 2
    assert fwd(M=0) == 0 and fwd(G=0) == 0 and fwd(N=0) == 0
    assert bwd(gw=None) == 1 and bwd(gy=None) == 1 and bwd(gx=None) == 1 and bwd(gate=F) == 1
    assert bwd(ws=None) == 3 and bwd(wsb=16) == 3 and bwd(ws=P(0x1004)) == 2 and bwd(G=0) == 0
    assert h.rwkv_layer_norm_backward_workspace_bytes(0, 2, 8, 0) == 0
    assert h.rwkv_layer_norm_backward_workspace_bytes(64, 2, 8, 0) >= 2 * 2 * 8 * 4


def test_binding_refuses():
    x, w = torch.zeros(2, 5, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="CUDA"):
        rw.rwkv_causal_conv_forward(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        rw.rwkv_selective_scan_forward(x, x, x, x, w)
    with pytest.raises(ValueError, match="CUDA"):
        rw.rwkv_layer_norm_forward(x, w)
    rows = lambda t, shape=None: rw._rows("t", t, t.shape if shape is None else shape, torch.float32, -1)
    wide = torch.zeros(3, 4, 20)
    assert rows(wide) == 20 and rows(wide[..., 3:11]) == 20 and rows(wide[:, :1, :8]) == 80
    assert rows(wide[:1, :1, 2:4]) == 2 and rows(torch.zeros(0, 4, 6)) == 6 and rows(wide[..., :1]) == 20
    assert rows(wide[0, :, 5:9]) == 20
    with pytest.raises(ValueError, match="dense"):
        rows(wide[..., ::2])
    with pytest.raises(ValueError, match="equal distances"):
        rows(wide[:, :3])
    with pytest.raises(ValueError, match="equal distances"):
        rows(wide.transpose(0, 1))
    with pytest.raises(ValueError, match="overlap"):
        rows(torch.zeros(1, 8).expand(4, 8))
    with pytest.raises(ValueError, match="shape"):
        rows(wide, (3, 4, 21))
    with pytest.raises(ValueError, match="contiguous"):
        rw._dense("t", wide[..., :8], (3, 4, 8), torch.float32, -1)
    with pytest.raises(ValueError, match="groups"):
        rw._norm_args(x, torch.zeros(8), None, None, 3, -1)
    with pytest.raises(TypeError):
        rw._io_code("x", x.half())
