"""The selective scan over the longest sequence that a call accepts: its segments reach to within a tile of 2^31
tokens, and the tokens at each segment's ends come out as in a call on the tokens around them."""
import pytest
import torch

import rwkv_wkv_recurrence_b200 as rw

pytestmark = pytest.mark.gpu
T, C, N = 2 ** 31 - 1 - 64, 1, 8
WARM, LEN = 512, 1024  # tokens before the compared ones, tokens of a short call


def test_forward(cuda_device):
    if torch.cuda.mem_get_info()[0] < 95 << 30:
        pytest.skip("needs 82 GB for the inputs")
    bf16 = torch.bfloat16
    act = lambda w: torch.empty(1, T, w, dtype=bf16, device=cuda_device).normal_()
    x, dt, b, c = act(C), act(C).mul_(0.5), act(N), act(N)
    a_log = torch.log(torch.arange(1, N + 1, device=cuda_device).float()).expand(C, N).contiguous()
    d, bias = torch.ones(C, device=cuda_device), torch.ones(C, device=cuda_device)
    y = torch.full((1, T, C), float("nan"), dtype=bf16, device=cuda_device)
    _, h = rw.rwkv_selective_scan_forward(x, dt, b, c, a_log, d, bias, return_state=True, out=y)
    seg = (T + 1183) // 1184 // 32 * 32 + 32  # 8 CTAs on each of 148 SMs, in whole tiles
    starts = [0] + [k * seg - LEN // 2 for k in (1, 2, 600, 1183)] + [T - LEN]
    for t0 in starts:
        cut = [t[:, t0: t0 + LEN].contiguous() for t in (x, dt, b, c)]
        want, hw = rw.rwkv_selective_scan_forward(*cut, a_log, d, bias, return_state=True, algo=rw.ALGO_SEQUENTIAL)
        warm = 0 if t0 == 0 else WARM - 64
        # steps of softplus(1 + dt / 2), above 0.2 where |dt| < 5: the 448 tokens before leave less than e^-80
        # of what came earlier, so both round the same sums to bf16, at most one step (2^-7 of the value) apart
        a, w = y[:, t0 + warm: t0 + LEN].float(), want[:, warm:].float()
        assert ((a - w).abs() <= 2.0 ** -7 * w.abs() + 1e-5).all(), t0
    # the state: fp32 sums of the same terms in the same order behind the forgotten part
    assert torch.allclose(h, hw, rtol=1e-5, atol=1e-6)
    del x, dt, b, c, y
    torch.cuda.empty_cache()
