"""The 64-bit references of the convolution, the selective scan and the layer norm (tests/_mixer_ref.py):
their gradients against torch's autograd of the forward formula in float64 and against central
differences, and the scan's recurrence against its explicit sum over past tokens."""
import pytest
import torch

import _mixer_ref as ref


def _rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def _close(a, b, tol=1e-10):
    assert torch.allclose(a, b, rtol=tol, atol=tol), (a - b).abs().max()


def _grads_agree(forward, leaves, outs_grads, named):
    """autograd of sum(g * out), and central differences along a random direction of every leaf."""
    ls = [t.clone().requires_grad_() for t in leaves]
    loss = sum((g * o).sum() for g, o in zip(outs_grads, forward(*ls)) if g is not None)
    for (name, want), got in zip(named, torch.autograd.grad(loss, ls)):
        _close(got, want)
    for i, (name, want) in enumerate(named):
        v = _rand(77 + i, *leaves[i].shape)
        f = []
        for sgn in (1, -1):
            moved = [t if j != i else t + sgn * 1e-5 * v for j, t in enumerate(leaves)]
            f.append(sum((g * o).sum() for g, o in zip(outs_grads, forward(*moved)) if g is not None))
        num = (f[0] - f[1]) / 2e-5
        assert abs(num - (want * v).sum()) <= 1e-6 * max(1.0, abs(num)), name


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("W,T", [(2, 7), (3, 1), (4, 2), (4, 11)])
def test_conv_gradients(W, T, silu):
    B, C = 2, 3
    x, w, bias, st = _rand(1, B, T, C), _rand(2, C, W), _rand(3, C), _rand(4, B, W - 1, C)
    gy, gs = _rand(5, B, T, C), _rand(6, B, W - 1, C)
    out = ref.conv(x, w, bias, st, silu, gy, gs)

    def fwd(x, w, bias, st):
        xp = torch.cat([st, x], 1)
        pre = torch.stack([sum(w[:, j] * xp[:, t + j] for j in range(W)) + bias for t in range(T)], 1)
        return (torch.nn.functional.silu(pre) if silu else pre), xp[:, T:]

    _close(out["y"][0], fwd(x, w, bias, st)[0])
    _grads_agree(fwd, [x, w, bias, st], [gy, gs],
                 [("gx", out["gx"][0]), ("gw", out["gw"][0]), ("gbias", out["gbias"][0]),
                  ("gstate", out["gstate_in"][0])])


@pytest.mark.parametrize("gate", [False, True])
def test_scan_gradients(gate):
    B, T, C, N = 2, 9, 3, 4
    names = ["x", "dt", "b", "c", "a_log", "d", "dt_bias", "h_in"] + (["z"] if gate else [])
    shapes = dict(x=(B, T, C), dt=(B, T, C), b=(B, T, N), c=(B, T, N), a_log=(C, N), d=(C,), dt_bias=(C,),
                  h_in=(B, C, N), z=(B, T, C))
    v = {n: _rand(10 + i, *shapes[n]) for i, n in enumerate(names)}
    gy, gh = _rand(30, B, T, C), _rand(31, B, C, N)
    out = ref.scan(**v, gy=gy, gh_out=gh)

    def fwd(*a):
        q = dict(zip(names, a))
        dl = torch.nn.functional.softplus(q["dt"] + q["dt_bias"])
        h, ys = q["h_in"], []
        for t in range(T):
            h = torch.exp(dl[:, t, :, None] * -torch.exp(q["a_log"])) * h \
                + (dl[:, t] * q["x"][:, t])[..., None] * q["b"][:, t, None]
            y = torch.einsum("bcn,bn->bc", h, q["c"][:, t]) + q["d"] * q["x"][:, t]
            ys.append(y * torch.nn.functional.silu(q["z"][:, t]) if gate else y)
        return torch.stack(ys, 1), h

    y, h = fwd(*v.values())
    _close(out["y"][0], y)
    _close(out["h"][0], h)
    key = dict(x="gx", dt="gdt", b="gb", c="gc", a_log="ga_log", d="gd", dt_bias="gdt_bias", h_in="gh_in", z="gz")
    _grads_agree(fwd, list(v.values()), [gy, gh], [(n, out[key[n]][0]) for n in names])


def test_scan_is_the_explicit_sum():
    B, T, C, N = 1, 6, 2, 3
    x, dt, b, c, al = _rand(1, B, T, C), _rand(2, B, T, C), _rand(3, B, T, N), _rand(4, B, T, N), _rand(5, C, N)
    out = ref.scan(x, dt, b, c, al)
    dl, A = torch.log1p(torch.exp(dt)), -torch.exp(al)
    for t in range(T):
        want = torch.zeros(B, C, dtype=torch.float64)
        for i in range(t + 1):
            dec = torch.exp(dl[:, i + 1: t + 1].sum(1)[..., None] * A)
            want += (dec * (dl[:, i] * x[:, i])[..., None] * b[:, i, None] * c[:, t, None]).sum(-1)
        _close(out["y"][0][:, t], want)


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("G,N", [(1, 7), (3, 4), (2, 1)])
def test_norm_gradients(G, N, gate):
    M, C = 5, G * N
    x, w, b = _rand(1, M, C), _rand(2, C), _rand(3, C)
    z = [_rand(4, M, C)] if gate else []
    gy = _rand(5, M, C)
    out = ref.norm(x, w, b, z[0] if gate else None, G, 1e-3, gy)

    def fwd(x, w, b, *z):
        xs = x.reshape(M, G, N)
        y = (xs - xs.mean(-1, keepdim=True)) / torch.sqrt(xs.var(-1, unbiased=False, keepdim=True) + 1e-3)
        y = y.reshape(M, C) * w + b
        return (y * torch.nn.functional.silu(z[0]) if z else y,)

    _close(out["y"][0], fwd(x, w, b, *z)[0])
    named = [("gx", out["gx"][0]), ("gw", out["gw"][0]), ("gb", out["gbias"][0])]
    _grads_agree(fwd, [x, w, b] + z, [gy], named + ([("ggate", out["ggate"][0])] if gate else []))


def test_bounds_cover_an_fp32_evaluation():
    # the same formulas in torch's fp32 stay within the bounds (and the bounds are of fp32's size)
    p, _ = ref.scan_inputs(1, 60, 5, 8, seed=3)
    r = ref.scan(**p)
    dl = torch.nn.functional.softplus(p["dt"] + p["dt_bias"])
    h = p["h_in"]
    ys = []
    for t in range(60):
        h = torch.exp(dl[:, t, :, None] * -torch.exp(p["a_log"])) * h \
            + (dl[:, t] * p["x"][:, t])[..., None] * p["b"][:, t, None]
        ys.append((torch.einsum("bcn,bn->bc", h, p["c"][:, t]) + p["d"] * p["x"][:, t])
                  * torch.nn.functional.silu(p["z"][:, t]))
    ref.check(torch.stack(ys, 1), *r["y"], "y")
    ref.check(h, *r["h"], "h")
    assert float((r["y"][1] / (r["y"][0].abs() + 1)).max()) < 1e-3
