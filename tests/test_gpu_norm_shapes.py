"""The layer norm's teams, one by one: for each width of a team and each way of access, the narrowest and the widest
rows that take it, in both types, gated and not, first a few rows against the 64-bit reference, then so many that every
team takes several."""
import pytest
import torch

import _mixer_ref as ref
import rwkv_wkv_recurrence_b200 as rw

pytestmark = pytest.mark.gpu

# vectors a row up to which a team of so many threads serves it (csrc/norm.cu, team_shape)
TEAMS = [(8, 8), (16, 16), (32, 32), (64, 32), (128, 64), (192, 64), (256, 128), (384, 128), (512, 256), (768, 256),
         (1024, 512), (1536, 512), (2048, 512)]
ROWS = 16  # a whole number of shift periods: copies of these rows lie on the 16-byte grid as they do


def _cases():
    for dtype, V in ((torch.float32, 4), (torch.bfloat16, 8)):
        low = 1
        for top, threads in TEAMS:
            for gate, nv in ((True, top), (False, top), (True, low), (False, low)):
                name = f"{'bf16' if V == 8 else 'f32'}-{top}x{threads}-{nv}{'-gated' if gate else ''}"
                # rows in whole vectors; rows that share vectors with their neighbours (at any shift they touch nv);
                # single elements
                yield pytest.param(dtype, "aligned", nv * V, threads, gate, id=name + "-aligned")
                if nv > 1:
                    yield pytest.param(dtype, "shifted", nv * V - V + 1, threads, gate, id=name + "-shifted")
                yield pytest.param(dtype, "single", nv, threads, gate, id=name + "-single")
            low = top + 1


def _place(t, off):
    buf = torch.empty(t.numel() + 8, dtype=t.dtype, device=t.device)
    buf[off: off + t.numel()] = t.flatten()
    return buf[off: off + t.numel()].view(t.shape)


def _run(q):
    y = rw.rwkv_layer_norm_forward(q["x"], q["w"], q["bias"], q["gate"])
    gx, gw, gb, gg = rw.rwkv_layer_norm_backward(q["x"], q["w"], q["gy"], q["bias"], q["gate"])
    return dict(y=y, gx=gx, gw=gw, gbias=gb, ggate=gg)


@pytest.mark.parametrize("dtype,access,N,threads,gate", list(_cases()))
def test_team(cuda_device, dtype, access, N, threads, gate):
    g = torch.Generator().manual_seed(61)
    n = lambda *s: torch.randn(*s, generator=g)
    p = dict(x=(n(ROWS, N) * 1.5 + 0.2).to(dtype), w=n(N) * 0.3 + 1, bias=n(N) * 0.3,
             gate=(n(ROWS, N) * 2).to(dtype) if gate else None, gy=n(ROWS, N).to(dtype))
    dev = {k: None if v is None else v.to(cuda_device) for k, v in p.items()}
    off = 1 if access == "single" else 0  # x lies elsewhere on the 16-byte grid than the rest
    q = dict(dev, x=_place(dev["x"], off))
    r = ref.norm(p["x"], p["w"], p["bias"], p["gate"], 1, 1e-5, p["gy"])
    few = _run(q)
    ref.check_all(few, r)

    # 148 SMs hold at most 2048 threads each: with more rows than that many teams each takes at least two
    k = 2 * 148 * 2048 // threads // ROWS + 1
    many = {name: t if t is None or name in ("w", "bias") else t.repeat(k, 1) for name, t in dev.items()}
    many["x"] = _place(many["x"], off)
    got = _run(many)
    for name in ("y", "gx", "ggate"):
        if few[name] is not None:
            assert torch.equal(got[name].view(k, ROWS, N), few[name].expand(k, ROWS, N)), name
    # the parameters' gradients: k times those of the few rows.  The rows' own errors are k times theirs; the sum
    # runs over k ROWS terms, which adds (k ROWS + 2) u of their absolute values, k times those of the few rows
    x = p["x"].double()
    xh = (x - x.mean(1, keepdim=True)) / (x.var(1, unbiased=False, keepdim=True) + 1e-5).sqrt()
    z = p["gate"].double() if gate else None
    gr = p["gy"].double() * (z * torch.sigmoid(z) if gate else 1.0)
    for name, mag in (("gw", (gr * xh).abs().sum(0)), ("gbias", gr.abs().sum(0))):
        ref.check(got[name], k * r[name][0], k * r[name][1] + (k * ROWS + 2) * ref.U * k * mag, f"many rows {name}")
