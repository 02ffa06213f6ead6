"""The largest sizes of the convolution, the selective scan and the layer norm, on the host: what a call refuses,
its workspace query answers with 0, and both do before any CUDA work."""
import ctypes

import rwkv_wkv_recurrence_b200 as rw

F = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails validation first
BIG = 1 << 62
INT_MAX = 2 ** 31 - 1


def test_conv_longest_sequence():
    h = rw.lib()
    query = h.rwkv_causal_conv_backward_workspace_bytes

    def bwd(T):
        return h.rwkv_causal_conv_backward(1, T, 8, 4, 0, F, None, 0, F, 8, None, F, None, F, F, None, None, F, BIG, None)

    for T in (INT_MAX - 63, INT_MAX - 62, INT_MAX):
        assert query(1, T, 8, 4) == 0 and bwd(T) == 2
    # parts of 512 tokens, 5 sums each for 8 channels
    assert query(1, INT_MAX - 64, 8, 4) == ((INT_MAX - 64 + 511) // 512) * 5 * 8 * 4


def test_conv_most_channels():
    h = rw.lib()
    fwd = lambda C: h.rwkv_causal_conv_forward(1, 1, C, 2, 1, F, None, 0, F, C, F, None, None, None)
    step = lambda C: h.rwkv_causal_conv_step(1, C, 2, 1, F, None, 0, F, C, F, None, F, None)
    bwd = lambda C: h.rwkv_causal_conv_backward(1, 1, C, 2, 1, F, None, 0, F, C, None, F, None, F, F, None, None, F,
                                                BIG, None)
    for C in (INT_MAX - 127, INT_MAX - 1, INT_MAX):
        assert fwd(C) == 2 and step(C) == 2 and bwd(C) == 2
        assert h.rwkv_causal_conv_backward_workspace_bytes(1, 1, C, 2) == 0


def test_scan_most_channels():
    h = rw.lib()
    for C in (INT_MAX - 127, INT_MAX - 1, INT_MAX):
        rows = (F, C, F, C, F, 8, F, 8, None, C)
        assert h.rwkv_selective_scan_forward(1, 1, C, 8, 1, F, None, None, *rows, F, None, None, None, 16, 0, None, 0,
                                             None) == 2
        assert h.rwkv_selective_scan_backward(1, 1, C, 8, 1, F, None, None, *rows, F, None, None, F, 16, F, F, F, F,
                                              None, F, None, None, None, F, BIG, None) == 2
        assert h.rwkv_selective_scan_step(1, C, 8, 1, F, None, None, *rows, F, None, F, None) == 2
        assert h.rwkv_selective_scan_forward_workspace_bytes(1, 1, C, 8, rw.ALGO_CHUNKED) == 0
        assert h.rwkv_selective_scan_backward_workspace_bytes(1, 1, C, 8, 16, 1) == 0
