"""Prefill and backward with sinks on the GPU against 64 bits, the gradients against the formulas (64-bit autograd of
the plain form) and against differences.

Bounds are the framework's own for these kernels: the forward rounds P and the output to bf16 (rms 1.66e-3 each: 2.4e-3
together) and is held to rel_rms 5e-3 and 2e-2 of the largest value; each gradient carries about three bf16 roundings
(dH, P or dS, itself: 2.9e-3) and is held to the same."""
import pytest
import torch

import differential_latent_attention_b200 as gdla
import gdla_inputs as gi
from _paged import plain_prefill

pytestmark = pytest.mark.gpu

NAMES = ("q_sig", "q_noise", "k", "v", "lam", "gate")
GRADS = ("dq_sig", "dq_noise", "dk", "dv", "dlambda", "dgate")


def _fwd(t, seqlens, window, sinks, **kw):
    out = gdla.attn_fwd(*[t[x] for x in NAMES], seqlens, window, sinks=sinks, **kw)
    torch.cuda.synchronize()
    assert gdla.device_error() == 0
    return out


def _bwd(t, dout, seqlens, window, sinks, **kw):
    g = gdla.attn_bwd(*[t[x] for x in NAMES], dout, seqlens, window, sinks=sinks, **kw)
    torch.cuda.synchronize()
    assert gdla.device_error() == 0
    return g


# A row that sees one key alone has dS = P (dP - rowsum(dH H)) = 0 in exact arithmetic, and so dK and dQ of a sequence of
# one token. In fp32 the two sums of 128 products of unit normals run in different orders: partial sums of size
# sqrt(128) = 11, each addition off by 2^-24 of that, 128 of them at random: sqrt(128) * 11 * 2^-24 = 7.5e-6 a sum, 1.1e-5
# for the difference; dK adds five heads of it times q / sqrt(192): 1.1e-5 * sqrt(5) / 13.9 = 1.7e-6 rms. Six of those.
ZERO = 1e-5


def _near(got, ref, what, rel=5e-3):
    got = got.double()
    assert torch.isfinite(got).all(), what
    off, size = got - ref, ref.numel() ** 0.5
    worst, rms = float(off.abs().max()), float(off.norm()) / size
    assert rms <= rel * float(ref.norm()) / size + ZERO and worst <= 4 * rel * float(ref.abs().max()) + ZERO, (what, worst, rms)


def _same(a, b):
    v = {torch.bfloat16: torch.int16, torch.float32: torch.int32}
    return torch.equal(a.view(v[a.dtype]), b.view(v[b.dtype]))


# windows of both schedules (to 256 and over); sinks within a tile's spare columns, over them, whole tiles, the most
SHAPES = [
    ((9, 0, 23, 1, 130, 64), 2, 4, 1),
    ((700, 333), 2, 128, 4),
    ((700,), 1, 128, 16),
    ((700, 5), 1, 128, 17),
    ((513,), 2, 1, 1),
    ((450, 129), 1, 100, 64),
    ((450,), 1, 30, 65),
    ((600,), 1, 200, 128),
    ((900, 17), 2, 300, 9),
    ((1300,), 1, 257, 128),
    ((800, 200), 16, 128, 4),
]


@pytest.mark.parametrize("seqlens, heads, window, sinks", SHAPES)
def test_forward(seqlens, heads, window, sinks):
    t = gi.make_prefill_inputs(seqlens, heads, 7 + window, device="cuda")
    _near(_fwd(t, seqlens, window, sinks), plain_prefill(t, seqlens, window, sinks), (seqlens, window, sinks))


def _plain_grads(t, dout, seqlens, window, sinks):
    leaves = {x: t[x].double().requires_grad_() for x in NAMES}
    g = torch.autograd.grad(plain_prefill(leaves, seqlens, window, sinks), list(leaves.values()), dout.double())
    return dict(zip(GRADS, g))


@pytest.mark.parametrize("seqlens, heads, window, sinks", SHAPES + [
    ((2500, 100, 1400), 1, 64, 5), ((3001,), 2, 128, 100),      # key tiles in 2 parts and more, and later chunks
    ((1, 129, 257, 90, 1000), 1, 1000, 3), ((5000,), 1, 40, 128),
    ((300,) * 60, 1, 100, 4)])                                  # enough tiles: not cut
def test_backward(seqlens, heads, window, sinks):
    t = gi.make_prefill_inputs(seqlens, heads, 7 + window, device="cuda")
    dout = gi.make_prefill_grad(seqlens, heads, 7 + window, device="cuda")
    g, ref = _bwd(t, dout, seqlens, window, sinks), _plain_grads(t, dout, seqlens, window, sinks)
    for name in GRADS:
        _near(g[name], ref[name], (name, seqlens, window, sinks))
    # The sinks' own rows, which the other rows' number would hide. Short sequences cancel in them: with one visible key
    # dv = sum_i dD_i (1 - lambda_i) is made of four signal rows and the noise row -sum lambda_i dD_i, whose squares sum to
    # (4 * 0.29 + 4 * 0.29 / 3) / (4 * 0.29 / 3) = 4 times the result's (dD = dout sigmoid(g) has 0.29, lambda^2 and
    # (1 - lambda)^2 have 1/3 in the mean), so the roundings of P and dH (1.66e-3 each) show twice as large there:
    # sqrt(2 * (2 * 1.66e-3)^2 + 1.66e-3^2) = 5e-3 in the mean; twice that for so few values.
    s0 = 0
    for n in seqlens:
        r = slice(s0, s0 + min(n, sinks))
        s0 += n
        if n:
            for name in ("dk", "dv"):
                _near(g[name][r], ref[name][r], (name, "sinks", seqlens, window, sinks), 1e-2)


def test_gradients_against_differences():
    """Along random directions, (f(x + h) - f(x - h)) / 2 of the 64-bit form. h = 1e-4 leaves the difference 1e-8 off;
    the kernel's gradient has rms 5e-3, so along a random direction it is off by at most 5e-3 |g| |d| / sqrt(n) times a
    normal variable: six of those."""
    seqlens, heads, window, sinks = (300, 77), 1, 40, 6
    t = gi.make_prefill_inputs(seqlens, heads, 3, device="cuda")
    dout = gi.make_prefill_grad(seqlens, heads, 3, device="cuda")
    g = _bwd(t, dout, seqlens, window, sinks)
    for i, (x, name) in enumerate(zip(NAMES, GRADS)):
        gen = torch.Generator(device="cuda").manual_seed(50 + i)
        d = torch.randn(t[x].shape, generator=gen, device="cuda", dtype=torch.float64)
        f = []
        for sign in (1, -1):
            moved = {k: v.double() for k, v in t.items()}
            moved[x] = moved[x] + sign * 1e-4 * d
            f.append(float((plain_prefill(moved, seqlens, window, sinks) * dout.double()).sum()))
        want = (f[0] - f[1]) / 2e-4
        got = float((g[name].double() * d).sum())
        assert abs(got - want) <= 6 * 5e-3 * float(g[name].double().norm()), (name, got, want)


@pytest.mark.parametrize("window", [0, 128, 300])
def test_no_sinks_is_the_plain_call(window):
    seqlens = (700, 33)
    t = gi.make_prefill_inputs(seqlens, 2, 11, device="cuda")
    dout = gi.make_prefill_grad(seqlens, 2, 11, device="cuda")
    lib, arr = gdla.library(), torch.tensor(seqlens, dtype=torch.int32)
    ref = _fwd(t, seqlens, window, 0)
    out = torch.empty_like(ref)
    assert lib.gdla_attn_fwd_sinks(*[t[x].data_ptr() for x in NAMES], out.data_ptr(), 2, arr.data_ptr(), 2, window, 0,
                                   torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert _same(out, ref)
    a = _bwd(t, dout, seqlens, window, 0)
    assert all(_same(a[n], x) for n, x in _bwd(t, dout, seqlens, window, 0).items())


def test_windows_that_cover_everything_are_full_attention():
    """window >= the longest sequence, up to the largest int: the causal result, bit for bit."""
    seqlens = (400, 33)
    t = gi.make_prefill_inputs(seqlens, 2, 12, device="cuda")
    dout = gi.make_prefill_grad(seqlens, 2, 12, device="cuda")
    ref, g = _fwd(t, seqlens, 0, 0), _bwd(t, dout, seqlens, 0, 0)
    for window in (400, 100_000, 2 ** 31 - 1):
        assert _same(_fwd(t, seqlens, window, 5), ref)
        h = _bwd(t, dout, seqlens, window, 5)
        assert all(_same(h[n], g[n]) for n in GRADS)
    # and a shorter window with sinks on every key before it sees everything too
    _near(_fwd(t, seqlens, 300, 128), plain_prefill(t, seqlens, 0, 0), "sinks reach the window")


def test_a_sink_that_takes_all():
    """One sink with by far the largest score: every row past it is the sink's value."""
    n, heads = 600, 1
    t = gi.make_prefill_inputs((n,), heads, 13, device="cuda")
    t["q_sig"][:], t["q_noise"][:] = 1.0, -1.0
    t["k"][:] = 0.0
    t["k"][2] = 8.0
    out = _fwd(t, (n,), 64, 3).double()
    v = t["v"].double()
    rows = torch.arange(100, n, device="cuda")
    # signal heads: all weight on key 2; the noise head: none on it, so the mean of the rest it sees
    u = torch.arange(n, device="cuda")
    see = ((rows[:, None] - u[None] < 64) & (u[None] <= rows[:, None])) | (u[None] < 2)
    see[:, 2] = False
    noise = see.double() @ v[:, 0] / see.sum(1, keepdim=True)
    want = torch.sigmoid(t["gate"].double()[rows]) * (v[2, 0] - t["lam"].double()[rows, :, None] * noise[:, None])
    assert float((out[rows] - want).abs().max()) <= 2e-2 * float(want.abs().max())


def test_many_sequences():
    """More sequences than one launch's plan holds, most with chunks of later rows."""
    seqlens = tuple(100 + 7 * (i % 40) for i in range(270))
    t = gi.make_prefill_inputs(seqlens, 1, 14, device="cuda")
    dout = gi.make_prefill_grad(seqlens, 1, 14, device="cuda")
    _near(_fwd(t, seqlens, 16, 3), plain_prefill(t, seqlens, 16, 3), "fwd")
    g, ref = _bwd(t, dout, seqlens, 16, 3), _plain_grads(t, dout, seqlens, 16, 3)
    for name in GRADS:
        _near(g[name], ref[name], name)


def test_deterministic_own_buffers_and_streams():
    seqlens, window, sinks = (1500, 40), 64, 7
    t = gi.make_prefill_inputs(seqlens, 2, 15, device="cuda")
    dout = gi.make_prefill_grad(seqlens, 2, 15, device="cuda")
    a = _bwd(t, dout, seqlens, window, sinks)
    need = gdla.attn_bwd_sinks_workspace_bytes(seqlens, 2, window, sinks)
    ws = torch.full((need // 4 + 64,), float("nan"), device="cuda").view(torch.uint8)[:need]
    grads = {n: torch.full_like(x, float("nan")) for n, x in a.items()}
    b = _bwd(t, dout, seqlens, window, sinks, workspace=ws, grads=grads)
    assert all(_same(a[n], b[n]) for n in GRADS)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = _bwd(t, dout, seqlens, window, sinks, stream=side)
    assert all(_same(a[n], c[n]) for n in GRADS)
    assert _same(_fwd(t, seqlens, window, sinks, stream=side), _fwd(t, seqlens, window, sinks))
    with pytest.raises(gdla.GDLAError):
        _bwd(t, dout, seqlens, window, sinks, workspace=ws[:need - 256])


@pytest.mark.parametrize("window, sinks", [(64, 7), (300, 4), (64, 0)])
def test_buffers_on_16_byte_boundaries(window, sinks):
    """Every buffer 16 bytes past a 32-byte boundary: the same bits."""
    seqlens = (500, 33)
    t = gi.make_prefill_inputs(seqlens, 2, 18, device="cuda")
    dout = gi.make_prefill_grad(seqlens, 2, 18, device="cuda")

    def shift(x):
        step = 16 // x.element_size()
        y = torch.empty(x.numel() + 2 * step, dtype=x.dtype, device="cuda")
        off = step if y.data_ptr() % 32 == 0 else 0
        y = y[off:off + x.numel()].view(x.shape)
        assert y.data_ptr() % 32 == 16
        return y.copy_(x)

    moved = {n: shift(x) for n, x in t.items()}
    a = _bwd(t, dout, seqlens, window, sinks)
    grads = {n: shift(x) for n, x in a.items()}
    b = _bwd(moved, shift(dout), seqlens, window, sinks, grads=grads)
    assert all(_same(a[n], b[n]) for n in GRADS)
    out = shift(t["gate"])
    assert _same(_fwd(moved, seqlens, window, sinks, out=out), _fwd(t, seqlens, window, sinks))


def test_captured_forward_and_backward():
    seqlens, window, sinks = (700, 100), 128, 4
    t = gi.make_prefill_inputs(seqlens, 2, 16, device="cuda")
    dout = gi.make_prefill_grad(seqlens, 2, 16, device="cuda")
    out = torch.empty_like(t["gate"])
    ws = torch.empty(gdla.attn_bwd_sinks_workspace_bytes(seqlens, 2, window, sinks), dtype=torch.uint8, device="cuda")
    grads = {n: torch.zeros_like(x) for n, x in _bwd(t, dout, seqlens, window, sinks).items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdla.attn_fwd(*[t[x] for x in NAMES], seqlens, window, out=out, sinks=sinks)
        gdla.attn_bwd(*[t[x] for x in NAMES], dout, seqlens, window, grads=grads, workspace=ws, sinks=sinks)
    other = gi.make_prefill_inputs(seqlens, 2, 17, device="cuda")
    for x in NAMES:
        t[x].copy_(other[x])
    g.replay()
    torch.cuda.synchronize()
    assert _same(out, _fwd(other, seqlens, window, sinks))
    want = _bwd(other, dout, seqlens, window, sinks)
    assert all(_same(grads[n], want[n]) for n in GRADS)
