"""The layer norm's forward and backward on the GPU against the 64-bit reference, within the bounds of
fp32 arithmetic that it derives (tests/_mixer_ref.py)."""
import pytest
import torch

import _mixer_ref as ref
import rwkv_wkv_recurrence_b200 as rw
from test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu
DT = pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])


def _inputs(M, C, seed, dtype, shift=0.2):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    return dict(x=(n(M, C) * 1.5 + shift).to(dtype), w=n(C) * 0.3 + 1, bias=n(C) * 0.3, gate=(n(M, C) * 2).to(dtype),
                gy=n(M, C).to(dtype))


def _run(q, groups, gate, bias, eps=1e-5):
    z, b = q["gate"] if gate else None, q["bias"] if bias else None
    y = rw.rwkv_layer_norm_forward(q["x"], q["w"], b, z, groups=groups, eps=eps)
    gx, gw, gb, gg = rw.rwkv_layer_norm_backward(q["x"], q["w"], q["gy"], b, z, groups=groups, eps=eps)
    assert (gb is None) == (not bias) and (gg is None) == (not gate)
    return dict(y=y, gx=gx, gw=gw, gbias=gb, ggate=gg)


# (rows, groups, columns): every team shape (8 to 512 threads, one to three vectors) in wide and
# in single accesses, the wide kernel, rows that do and do not fill a launch, one column
SHAPES = [(1, 1, 1), (3, 1, 5), (5, 40, 64), (70, 3, 64), (9, 2, 77), (4, 1, 96), (33, 2, 128), (7, 1, 200),
          (5, 3, 256), (2, 1, 520), (6, 1, 768), (3, 1, 1000), (2, 2, 1001), (2, 1, 2048), (3, 1, 4096),
          (2, 1, 8192), (2, 1, 8200), (1, 1, 2500), (5, 2, 1400), (40, 1, 300)]


@DT
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_backward(cuda_device, shape, dtype):
    M, G, N = shape
    p = _inputs(M, G * N, 41, dtype)
    q = {k: v.to(cuda_device) for k, v in p.items()}
    for gate, bias in ((True, True), (False, True), (True, False), (False, False)):
        r = ref.norm(p["x"], p["w"], p["bias"] if bias else None, p["gate"] if gate else None, G, 1e-5, p["gy"])
        ref.check_all(_run(q, G, gate, bias), r, f"gate={gate} bias={bias} ")


@DT
@pytest.mark.parametrize("shape", [(20000, 1, 64), (3000, 40, 64), (5000, 1, 768), (3001, 1, 512)], ids=str)
def test_many_rows(cuda_device, shape, dtype):
    # teams take several rows each
    M, G, N = shape
    p = _inputs(M, G * N, 42, dtype)
    q = {k: v.to(cuda_device) for k, v in p.items()}
    r = ref.norm(p["x"], p["w"], p["bias"], p["gate"], G, 1e-5, p["gy"])
    ref.check_all(_run(q, G, True, True), r)


@DT
@pytest.mark.parametrize("shape", [(620, 1, 6832), (320, 1, 12296), (9, 1, 16384), (3, 2, 10000), (5, 1, 16383),
                                   (4, 1, 16400), (330, 1, 5003)], ids=str)
def test_wide_rows(cuda_device, shape, dtype):
    # the widest teams, with several rows each, and rows wider than they hold
    M, G, N = shape
    p = _inputs(M, G * N, 52, dtype)
    q = {k: v.to(cuda_device) for k, v in p.items()}
    for gate, bias in ((True, True), (False, True)):
        r = ref.norm(p["x"], p["w"], p["bias"] if bias else None, p["gate"] if gate else None, G, 1e-5, p["gy"])
        ref.check_all(_run(q, G, gate, bias), r, f"gate={gate} ")


def test_off_the_16_byte_grid(cuda_device):
    # bases one element off: single accesses, and columns so wide that they take the wide kernel then
    for M, G, N, dtype in ((5, 4, 64, torch.bfloat16), (3, 1, 768, torch.float32), (2, 1, 4096, torch.bfloat16)):
        p = _inputs(M, G * N, 43, dtype)
        q = {}
        for k, v in p.items():
            buf = torch.empty(v.numel() + 8, dtype=v.dtype, device=cuda_device)
            q[k] = buf[1: 1 + v.numel()].view(v.shape)
            q[k].copy_(v)
        r = ref.norm(p["x"], p["w"], p["bias"], p["gate"], G, 1e-5, p["gy"])
        ref.check_all(_run(q, G, True, True), r)


def test_large_mean_and_constant_rows(cuda_device):
    p = _inputs(8, 256, 44, torch.float32, shift=300.0)
    p["x"][3] = 7.0  # a row without variance: x - mean is 0 and rstd 1 / sqrt(eps)
    q = {k: v.to(cuda_device) for k, v in p.items()}
    r = ref.norm(p["x"], p["w"], p["bias"], p["gate"], 1, 1e-3, p["gy"])
    ref.check_all(_run(q, 1, True, True, eps=1e-3), r)


def test_nan_stays_in_its_group(cuda_device):
    p = {k: v.to(cuda_device) for k, v in _inputs(40, 4 * 64, 45, torch.float32).items()}
    clean = _run(p, 4, False, True)
    p["x"][11, 70] = float("nan")
    got = _run(p, 4, False, True)
    for k in ("y", "gx"):
        hit = torch.zeros(40, 256, dtype=torch.bool, device=cuda_device)
        hit[11, 64:128] = True
        assert torch.isnan(got[k][hit]).all() and torch.equal(got[k][~hit], clean[k][~hit])


def test_heads_of_a_4d_tensor(cuda_device):
    # groups over the last dimension of any leading shape
    p = _inputs(6, 3 * 64, 46, torch.bfloat16)
    q = {k: v.to(cuda_device) for k, v in p.items()}
    a = rw.rwkv_layer_norm_forward(q["x"].view(2, 3, 192), q["w"], q["bias"], q["gate"].view(2, 3, 192), groups=3)
    assert torch.equal(a.view(6, 192), _run(q, 3, True, True)["y"])


@pytest.mark.parametrize("dtype,G,N,off", [(torch.float32, 3, 64, 0), (torch.float32, 2, 33, 1),
                                           (torch.bfloat16, 1, 264, 0), (torch.bfloat16, 5, 12, 3),
                                           (torch.bfloat16, 1, 8200, 0)])
def test_writes_only_its_outputs(cuda_device, dtype, G, N, off):
    M, C = 9, G * N
    q = {k: v.to(cuda_device) for k, v in _inputs(M, C, 47, dtype).items()}
    h, P, S = rw.lib(), rw._ptr, rw._stream(None)
    code = rw.F32 if dtype == torch.float32 else rw.BF16
    y, gx, gg = (Guarded((M, C), dtype, cuda_device, off) for _ in range(3))
    gw, gb = Guarded((C,), torch.float32, cuda_device), Guarded((C,), torch.float32, cuda_device)
    wsb = int(h.rwkv_layer_norm_backward_workspace_bytes(M, G, N, code))
    ws = Guarded((wsb // 4,), torch.float32, cuda_device)
    assert h.rwkv_layer_norm_forward(M, G, N, code, P(q["w"]), P(q["bias"]), 1e-5, P(q["x"]), P(q["gate"]), y.ptr(),
                                     S) == 0
    assert h.rwkv_layer_norm_backward(M, G, N, code, P(q["w"]), P(q["bias"]), 1e-5, P(q["x"]), P(q["gate"]),
                                      P(q["gy"]), gx.ptr(), gg.ptr(), gw.ptr(), gb.ptr(), ws.ptr(), wsb, S) == 0
    rw.rwkv_check_device_error()
    for b_, name in ((y, "y"), (gx, "gx"), (gg, "ggate"), (gw, "gw"), (gb, "gbias"), (ws, "workspace")):
        b_.check(name)


def test_empty(cuda_device):
    w = torch.ones(8, device=cuda_device)
    x = torch.zeros(0, 8, device=cuda_device)
    assert rw.rwkv_layer_norm_forward(x, w).shape == (0, 8)
    gx, gw, gb, _ = rw.rwkv_layer_norm_backward(x, w, x, w)
    assert gx.shape == (0, 8) and not gw.any() and not gb.any()


def test_same_bits_twice(cuda_device):
    q = {k: v.to(cuda_device) for k, v in _inputs(3000, 320, 48, torch.bfloat16).items()}
    a, b = _run(q, 5, True, True), _run(q, 5, True, True)
    assert all(torch.equal(a[k], b[k]) for k in a)


@DT
@pytest.mark.parametrize("shape", [(20000, 1, 37), (3001, 40, 67), (1, 1, 333), (2, 3, 9), (7, 2, 4091), (1500, 1, 2050),
                                   (300, 1, 4100), (64, 5, 1023)], ids=str)
def test_rows_that_start_anywhere(cuda_device, shape, dtype):
    # rows share 16-byte vectors with their neighbours; a team's rows all lie alike
    M, G, N = shape
    p = _inputs(M, G * N, 49, dtype)
    q = {k: v.to(cuda_device) for k, v in p.items()}
    for gate, bias in ((True, True), (False, False)):
        r = ref.norm(p["x"], p["w"], p["bias"] if bias else None, p["gate"] if gate else None, G, 1e-5, p["gy"])
        ref.check_all(_run(q, G, gate, bias), r, f"gate={gate} bias={bias} ")


@DT
@pytest.mark.parametrize("N", [33, 77, 600])
def test_nan_stays_in_its_row_where_vectors_are_shared(cuda_device, N, dtype):
    p = {k: v.to(cuda_device) for k, v in _inputs(40, 4 * N, 50, dtype).items()}
    clean = _run(p, 4, True, True)
    hit = torch.zeros(40, 4 * N, dtype=torch.bool, device=cuda_device)
    for m in (0, 11, 12, 39):
        for name in ("x", "gate"):
            p[name][m, N: 2 * N] = float("nan") if m % 2 else float("inf")
        hit[m, N: 2 * N] = True
    got = _run(p, 4, True, True)
    for k in ("y", "gx", "ggate"):
        assert not torch.isfinite(got[k][hit]).any() and torch.equal(got[k][~hit], clean[k][~hit]), k


@DT
@pytest.mark.parametrize("G,N", [(3, 33), (1, 264), (2, 64), (1, 1001), (4, 12)])
@pytest.mark.parametrize("M", [1, 2, 50])
def test_all_bases_off_the_grid_alike(cuda_device, M, G, N, dtype):
    C = G * N
    p = _inputs(M, C, 51, dtype)
    code = rw.F32 if dtype == torch.float32 else rw.BF16
    for off in (1, 3):
        q = {}
        for k, v in p.items():
            buf = Guarded(tuple(v.shape), v.dtype, cuda_device, off)  # its surroundings are not the operator's
            buf.t.copy_(v)
            q[k] = buf
        h, P, S = rw.lib(), rw._ptr, rw._stream(None)
        y, gx, gg = (Guarded((M, C), dtype, cuda_device, off) for _ in range(3))
        gw, gb = Guarded((C,), torch.float32, cuda_device), Guarded((C,), torch.float32, cuda_device)
        wsb = int(h.rwkv_layer_norm_backward_workspace_bytes(M, G, N, code))
        ws = Guarded((wsb // 4,), torch.float32, cuda_device)
        ptr = lambda k: q[k].ptr()
        assert h.rwkv_layer_norm_forward(M, G, N, code, ptr("w"), ptr("bias"), 1e-5, ptr("x"), ptr("gate"), y.ptr(),
                                         S) == 0
        assert h.rwkv_layer_norm_backward(M, G, N, code, ptr("w"), ptr("bias"), 1e-5, ptr("x"), ptr("gate"), ptr("gy"),
                                          gx.ptr(), gg.ptr(), gw.ptr(), gb.ptr(), ws.ptr(), wsb, S) == 0
        rw.rwkv_check_device_error()
        for b_, name in ((y, "y"), (gx, "gx"), (gg, "ggate"), (gw, "gw"), (gb, "gbias"), (ws, "workspace")):
            b_.check(name)
        r = ref.norm(p["x"], p["w"], p["bias"], p["gate"], G, 1e-5, p["gy"])
        ref.check_all(dict(y=y.t, gx=gx.t, gw=gw.t, gbias=gb.t, ggate=gg.t), r, f"off={off} ")
