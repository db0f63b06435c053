"""Plain 64-bit forms of the paged-cache operators and of attention with sinks, and the
inputs of their tests (torch, on whatever device the tensors are on)."""
import math

import torch

GROUP, NOPE, ROPE, DQK, DV = 4, 128, 64, 192, 128
MIN_EXP = -110
BF16_HALF = 2.0 ** -8   # largest relative error of one rounding to bf16
E4M3_HALF = 2.0 ** -4   # .. to a normal e4m3 number; below 2^-6 the step is 2^-9 (half: 2^-10)


def rand(shape, seed, scale=1.0, dtype=torch.bfloat16, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=device) * scale).to(dtype)


def turn(x, pos):
    """Rotary embedding of x [n, ..., 64] (pairs i, i + 32, base 10000) at positions pos, in 64 bits."""
    freq = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device=x.device) / 32)
    a = pos.double()[:, None] * freq
    shape = (x.shape[0],) + (1,) * (x.dim() - 2) + (32,)
    c, s = a.cos().view(shape), a.sin().view(shape)
    lo, hi = x.double()[..., :32], x.double()[..., 32:]
    return torch.cat([lo * c - hi * s, lo * s + hi * c], -1)


def exponent(amax):
    """The smallest e >= MIN_EXP with amax <= 448 * 2^e, by comparisons."""
    e = MIN_EXP
    if amax > 0:
        e = max(MIN_EXP, math.frexp(amax)[1] - 9)
        while amax > 448.0 * 2.0 ** e:
            e += 1
        while e > MIN_EXP and amax <= 448.0 * 2.0 ** (e - 1):
            e -= 1
    return e


def e4m3(x):
    """float64 -> e4m3 codes (uint8), nearest even, what is not finite -> NaN. |x| <= 448."""
    y = torch.where(torch.isfinite(x), x, torch.full_like(x, float("nan")))
    return y.to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)


def new_pool(pages, heads, page, kind, seed, device="cuda"):
    """A pool full of somebody's old values (e4m3: arbitrary finite codes, scales around one)."""
    g = torch.Generator(device=device).manual_seed(seed)
    out = {}
    for name, dim in (("k", DQK), ("v", DV)):
        x = torch.randn((pages, heads, page, dim), generator=g, device=device)
        if kind == "bf16":
            out[name + "_pages"], out[name + "_scale"] = x.to(torch.bfloat16), None
        else:
            s = torch.exp2(torch.randint(-9, -5, (pages, heads), generator=g, device=device).float())
            out[name + "_pages"] = (x / s[..., None, None] * 0.9).clamp(-448, 448).to(torch.float8_e4m3fn)
            out[name + "_scale"] = s
    return out


def table_of(lengths, page, pages, width=None, seed=0, device="cuda"):
    """A block table [B, width] of distinct shuffled pages; entries past a sequence's pages are -1."""
    each = [(n + page - 1) // page for n in lengths]
    width = width or max(1, max(each))
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    assert sum(each) <= pages
    t = torch.full((len(lengths), width), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(each):
        t[b, :m] = order[at:at + m].to(torch.int32)
        at += m
    return t.to(device)


def plain_append(pool, table, page, k_nope, k_rope, v, new, total, rotate):
    """The pool after the append: pages as values (bf16 case: float64 before rounding, NaN where nothing was written)
    or, for e4m3, codes and scales. new / total: tokens appended per sequence and their lengths afterwards."""
    h = k_nope.shape[1]
    eight = pool["k_scale"] is not None
    out = {}
    for name in ("k", "v"):
        pages = pool[name + "_pages"]
        out[name] = pages.clone().view(torch.uint8) if eight else torch.full_like(pages, float("nan"), dtype=torch.float64)
        out[name + "_scale"] = pool[name + "_scale"].clone() if eight else None
    at = 0
    for b, (n, length) in enumerate(zip(new, total)):
        if n == 0:
            continue
        before = length - n
        rows = slice(at, at + n)
        at += n
        pos = torch.arange(before, length, device=v.device)
        rope = k_rope[rows].double()
        if rotate:
            rope = turn(rope, pos)
        k = torch.cat([k_nope[rows].double(), rope[:, None].expand(n, h, ROPE)], -1)
        for j in range(before // page, (length - 1) // page + 1):
            p = int(table[b, j])
            lo, hi = max(before, j * page), min(length, (j + 1) * page)
            a, c = lo - j * page, hi - j * page
            for name, x in (("k", k), ("v", v[rows].double())):
                y = x[lo - before:hi - before].transpose(0, 1)      # [H, rows, dim]
                if not eight:
                    out[name][p, :, a:c] = y
                    continue
                for head in range(h):
                    fin = y[head][torch.isfinite(y[head])]
                    e = exponent(float(fin.abs().max()) if fin.numel() else 0.0)
                    if a > 0:
                        was = int(math.frexp(float(pool[name + "_scale"][p, head]))[1]) - 1
                        e = max(e, was)
                        old = out[name][p, head, :a].view(torch.float8_e4m3fn).double() * 2.0 ** (was - e)
                        out[name][p, head, :a] = e4m3(old)
                    out[name][p, head, a:c] = e4m3(y[head] * 2.0 ** -e)
                    out[name + "_scale"][p, head] = 2.0 ** e
    return out


def plain_decode(q_sig, q_noise, pool, table, page, lens, lam, gate, window=0, sinks=0, rotate=False):
    """Decode over the pages, sequence by sequence in 64 bits."""
    h = q_noise.shape[1]
    num = pool["k_pages"].shape[0]
    out = torch.zeros((len(lens), GROUP * h, DV), dtype=torch.float64, device=q_sig.device)
    for b, n in enumerate(lens):
        if n <= 0:
            continue
        pos = torch.arange(n, device=q_sig.device)
        if window > 0:
            pos = pos[(pos >= n - window) | (pos < sinks)]
        at = table[b].long()[pos // page]
        pos, at = pos[(at >= 0) & (at < num)], at[(at >= 0) & (at < num)]
        if pos.numel() == 0:
            continue
        q = torch.cat([q_sig[b].double().view(h, GROUP, DQK), q_noise[b].double().view(h, 1, DQK)], 1)
        if rotate:
            r = turn(q[..., NOPE:].reshape(1, 5 * h, ROPE), torch.tensor([n - 1], device=q.device)).view(h, 5, ROPE)
            q = torch.cat([q[..., :NOPE], r], -1)
        kv = []
        for name in ("k", "v"):
            pages, scale = pool[name + "_pages"], pool[name + "_scale"]
            raw = pages.view(torch.uint8) if scale is not None else pages
            x = raw[at, :, pos % page]
            x = x.view(torch.float8_e4m3fn).double() * scale.double()[at][..., None] if scale is not None else x.double()
            kv.append(x)
        a = torch.softmax(torch.einsum("hid,nhd->hin", q, kv[0]) / math.sqrt(DQK), -1)
        hd = torch.einsum("hin,nhd->hid", a, kv[1])
        d = hd[:, :GROUP] - lam[b].double().view(h, GROUP, 1) * hd[:, GROUP:]
        out[b] = torch.sigmoid(gate[b].double()) * d.reshape(GROUP * h, DV)
    return out


def decode_inputs(batch, heads, seed, device="cuda"):
    hs = GROUP * heads
    g = torch.Generator(device=device).manual_seed(seed + 1)
    return {"q_sig": rand((batch, hs, DQK), seed + 2, device=device), "q_noise": rand((batch, heads, DQK), seed + 3, device=device),
            "lam": torch.rand((batch, hs), generator=g, device=device) * 0.98 + 0.01,
            "gate": rand((batch, hs, DV), seed + 4, device=device)}


def check_decode(got, ref, what=""):
    """One decode output against 64 bits.

    The kernels hold scores, statistics and O in fp32; what they round are the probabilities (bf16 with its remainder:
    2^-16; f16: 2^-12), turned queries (2^-16 with the remainder, f16: 2^-12) and the output (2^-8 at most, rms
    2^-8 / sqrt(12) * 1.44 = 1.63e-3 over evenly spread significands). A score is off by at most
    |q| |k| (192 * 2^-24 + 2^-12) / sqrt(192) <= 20 * 20 * 2.6e-4 / 13.9 = 7.5e-3 in the worst case and by some 1e-4
    in the mean, so: each value within 2^-8 of itself and 2e-2 of the largest, and the rms within
    sqrt(1.66e-3^2 + (2^-12 * 4)^2) = 1.93e-3 < 2.2e-3."""
    got = got.double()
    assert torch.isfinite(got).all(), what
    diff = (got - ref).abs()
    top = float(ref.abs().max())
    assert bool((diff <= BF16_HALF * ref.abs() + 2e-2 * top).all()), (what, float(diff.max()), top)
    if top > 0:
        rms = float(diff.norm() / ref.norm())
        assert rms <= 2.2e-3, (what, rms)


def visible(n, window, sinks, device):
    t = torch.arange(n, device=device)
    near = (t[:, None] - t[None]) < window if window > 0 else torch.ones((n, n), dtype=torch.bool, device=device)
    return (t[None] <= t[:, None]) & (near | (t[None] < (sinks if window > 0 else 0)))


def plain_prefill(t, seqlens, window, sinks):
    """Output of the packed prefill in 64 bits (differentiable)."""
    h = t["k"].shape[1]
    outs, s0 = [], 0
    for n in seqlens:
        r = slice(s0, s0 + n)
        s0 += n
        if n == 0:
            continue
        q = torch.cat([t["q_sig"][r].double().view(n, h, GROUP, DQK), t["q_noise"][r].double()[:, :, None]], 2)
        s = torch.einsum("thid,uhd->hitu", q, t["k"][r].double()) / math.sqrt(DQK)
        s = s.masked_fill(~visible(n, window, sinks, s.device), -math.inf)
        hd = torch.einsum("hitu,uhd->thid", torch.softmax(s, -1), t["v"][r].double())
        d = hd[:, :, :GROUP] - t["lam"][r].double().view(n, h, GROUP, 1) * hd[:, :, GROUP:]
        outs.append(torch.sigmoid(t["gate"][r].double()) * d.reshape(n, GROUP * h, DV))
    return torch.cat(outs)
