"""The serving and training operators around a paged KV cache, as measured cases.

Four operators of grouped differential attention (per KV head 4 signal query heads and
1 noise head over one K of 192 dims, 128 content and 64 rotary, and one V of 128):

  append    new keys and values into a paged cache, the shared rotary key turned to its
            position on the way; pages in bf16, or in e4m3 with one power-of-two scale per
            page and KV head (a page that grows its scale has its older tokens re-encoded)
  decode    one query per sequence over that cache, full context or a sliding window with
            the first `sinks` tokens still visible
  prefill   packed sequences, sliding window and sinks
  backward  the gradients of that prefill

Every case is plain numbers; lengths come from the case alone (`lens`), values from the
seed. `own` selects the framework's kernels instead of the plain forms below.
"""
import math
import random

import numpy as np
import torch

own = False

GROUP, NOPE, ROPE, DV = 4, 128, 64, 128
DQK = NOPE + ROPE
SCALE = 1.0 / math.sqrt(DQK)
BASE = 10000.0
E4M3_MAX = 448.0
MIN_EXP = -110          # exponent of an all-zero page's scale


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def listed():
    append = dict(op="append", rotate=True)
    decode = dict(op="decode", rotate=True)
    return [
        # one request's next token, bf16 pages: the smallest call there is
        dict(append, name="append_b1_step", batch=1, new_lo=1, new_hi=1, old_lo=1000, old_hi=1000, heads=16,
             page=64, cache="bf16", lens=1),
        # a decode step of a full batch into 8-bit pages that are partly filled
        dict(append, name="append_b64_step_e4m3", batch=64, new_lo=1, new_hi=1, old_lo=1, old_hi=4000, heads=16,
             page=64, cache="e4m3", lens=2),
        # eight ragged prompts of some thousand tokens after their prefill, 8-bit pages
        dict(append, name="append_prompts_e4m3", batch=8, new_lo=3800, new_hi=4400, old_lo=0, old_hi=50, heads=16,
             page=64, cache="e4m3", lens=3),
        # ragged chunks of prompts into small bf16 pages, keys already turned by the prologue
        dict(append, name="append_chunks_bf16", batch=13, new_lo=0, new_hi=777, old_lo=0, old_hi=999, heads=5,
             page=16, cache="bf16", rotate=False, lens=4),
        # one request over a few thousand tokens: latency, split over the whole card
        dict(decode, name="decode_b1_L4096", batch=1, len_lo=4096, len_hi=4096, heads=16, page=64, cache="bf16",
             window=0, sinks=0, lens=5),
        # the decode batch of the repository's benchmark (64 requests of 1,024 to 32,768 tokens), 8-bit pages
        dict(decode, name="decode_b64_e4m3", batch=64, len_lo=1024, len_hi=32768, heads=16, page=64, cache="e4m3",
             window=0, sinks=0, lens=6),
        # its sliding-window layers (window 128) with four sinks, bf16 pages
        dict(decode, name="decode_b64_w128_s4", batch=64, len_lo=1024, len_hi=8192, heads=16, page=64, cache="bf16",
             window=128, sinks=4, lens=7),
        # a ragged batch, odd head count, small 8-bit pages, a wide window with odd sinks
        dict(decode, name="decode_b9_w1000_s5_e4m3", batch=9, len_lo=0, len_hi=5001, heads=3, page=16, cache="e4m3",
             window=1000, sinks=5, lens=8),
        # sliding-window layer of a training or prefill batch: two packed sequences of 8,192
        dict(op="prefill", name="prefill_B2_T8192_w128_s4", batch=2, len_lo=8192, len_hi=8192, heads=16, window=128,
             sinks=4, lens=9),
        # ragged short prompts, odd sizes, a window that is no multiple of a tile
        dict(op="prefill", name="prefill_ragged_w200_s17", batch=7, len_lo=1, len_hi=700, heads=3, window=200,
             sinks=17, lens=10),
        # the same layer's backward, one sequence of 4,096
        dict(op="backward", name="backward_T4096_w128_s4", batch=1, len_lo=4096, len_hi=4096, heads=16, window=128,
             sinks=4, lens=11),
        # ragged, a long window and odd sinks
        dict(op="backward", name="backward_ragged_w333_s9", batch=5, len_lo=1, len_hi=900, heads=2, window=333,
             sinks=9, lens=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "decode", "prefill", "backward"))
    lens = rng.randrange(1 << 30)
    heads = rng.choice((1, 2, 3, 4, 5, 8, 16))
    if op == "append":
        batch = _log_int(rng, 1, 64)
        step = rng.random() < 0.4
        hi = 1 if step else min(4400, max(2, _log_int(rng, 2, 35000) // batch))
        return dict(op=op, batch=batch, new_lo=1 if step else rng.randrange(0, hi), new_hi=hi, old_lo=0,
                    old_hi=_log_int(rng, 1, 4000), heads=heads, page=rng.choice((16, 32, 64, 128)),
                    cache=rng.choice(("bf16", "e4m3")), rotate=rng.random() < 0.7, lens=lens)
    if op == "decode":
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, min(32768, 1000000 // batch))
        sliding = rng.random() < 0.5
        return dict(op=op, batch=batch, len_lo=rng.randrange(0, hi + 1), len_hi=hi, heads=heads,
                    page=rng.choice((16, 32, 64, 128)), cache=rng.choice(("bf16", "e4m3")),
                    window=_log_int(rng, 16, 2000) if sliding else 0, sinks=rng.randrange(0, 65) if sliding else 0,
                    rotate=rng.random() < 0.7, lens=lens)
    tokens = _log_int(rng, 40, 16384 if op == "prefill" else 4096)
    batch = min(tokens, _log_int(rng, 1, 12))
    hi = tokens // batch
    return dict(op=op, batch=batch, len_lo=rng.randrange(0, hi + 1), len_hi=hi, heads=heads,
                window=_log_int(rng, 16, 1000), sinks=_log_int(rng, 1, 64), lens=lens)


def _lengths(case):
    """(lengths before or 0, new tokens or sequence lengths) of the case, from the case alone."""
    r = random.Random(case["lens"])
    if case["op"] == "append":
        old = [r.randint(case["old_lo"], case["old_hi"]) for _ in range(case["batch"])]
        return old, [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    got = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["batch"])]
    if sum(got) == 0:
        got[-1] = max(1, case["len_hi"])
    return [0] * case["batch"], got


def _pairs(lengths, window, sinks):
    """Visible (query, key) pairs of one query head."""
    total = 0
    for n in lengths:
        t = np.arange(n, dtype=np.int64)
        near = np.minimum(t + 1, window) if window > 0 else t + 1
        far = np.minimum(sinks, t + 1 - near) if window > 0 else 0
        total += int(np.sum(near + far))
    return total


def work(case):
    old, new = _lengths(case)
    h, hs = case["heads"], GROUP * case["heads"]
    n = sum(new)
    if case["op"] == "append":
        size = 2 if case["cache"] == "bf16" else 1
        pages = sum((o + k - 1) // case["page"] - o // case["page"] + 1 for o, k in zip(old, new) if k)
        moved = n * (h * (NOPE + DV) * 2 + ROPE * 2) + n * h * (DQK + DV) * size
        return {"bytes": moved + pages * (4 + (0 if size == 2 else 16 * h)), "flops": n * ROPE * 3}
    if case["op"] == "decode":
        size = 2 if case["cache"] == "bf16" else 1
        keys = sum(min(x, case["window"]) + min(case["sinks"], max(0, x - case["window"])) if case["window"] > 0 else x
                   for x in new)
        small = len(new) * (5 * h * DQK * 2 + hs * (4 + DV * 2 * 2))
        return {"bytes": keys * h * (DQK + DV) * size + small, "flops": 2 * keys * 5 * h * (DQK + DV)}
    pairs = _pairs(new, case["window"], case["sinks"])
    tensors = n * ((5 * h + h) * DQK * 2 + h * DV * 2 + hs * (4 + DV * 2))
    if case["op"] == "prefill":
        return {"bytes": tensors + n * hs * DV * 2, "flops": 2 * pairs * 5 * h * (DQK + DV)}
    # read q, k, v, lambda, gate and dout; write a gradient for each but dout; S and dP, then dQ, dK, dV
    return {"bytes": 2 * tensors + n * hs * DV * 2, "flops": 2 * pairs * 5 * h * (3 * DQK + 3 * DV)}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _normal(shape, gen, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _lam(shape, gen):
    return torch.rand(shape, generator=gen, device="cuda", dtype=torch.float32) * 0.998 + 0.001


def _cu(lengths):
    return torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32, device="cuda")


def _scale_exponent(amax):
    """Smallest e with amax <= 448 * 2^e (448 = 0.875 * 2^9), not under MIN_EXP."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp_min(MIN_EXP)


def _power(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def _pages(count, heads, page, dim, cache, gen):
    """Pages of keys or values with a spread of their own per page and head, and their scales."""
    if cache == "bf16":
        out = torch.empty((count, heads, page, dim), dtype=torch.bfloat16, device="cuda")
        scale = None
    else:
        out = torch.empty((count, heads, page, dim), dtype=torch.float8_e4m3fn, device="cuda")
        scale = torch.empty((count, heads), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (heads * page * dim))
    for a in range(0, count, step):
        b = min(count, a + step)
        x = torch.randn((b - a, heads, page, dim), generator=gen, device="cuda")
        x *= torch.exp2(torch.randn((b - a, heads, 1, 1), generator=gen, device="cuda") * 0.5)
        if cache == "bf16":
            out[a:b] = x.to(torch.bfloat16)
        else:
            s = _power(_scale_exponent(x.abs().amax((-1, -2))))
            scale[a:b] = s
            out[a:b] = (x / s[..., None, None]).to(torch.float8_e4m3fn)
    return out, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    old, new = _lengths(case)
    h, hs, batch = case["heads"], GROUP * case["heads"], case["batch"]
    st = {"case": case, "op": case["op"]}
    if case["op"] in ("append", "decode"):
        page = case["page"]
        total = [a + b for a, b in zip(old, new)]
        each = [(x + page - 1) // page for x in total]
        width, used = max(1, max(each)), sum(each)
        count = used + 3                      # a pool with pages that belong to nobody
        order = torch.randperm(count, generator=gen, device="cuda").to(torch.int32)
        table = torch.zeros((batch, width), dtype=torch.int32, device="cuda")
        at = 0
        for b, m in enumerate(each):
            table[b, :m] = order[at:at + m]
            at += m
        st["block_table"] = table
        st["seqlens_k"] = torch.tensor(total, dtype=torch.int32, device="cuda")
        st["max_seqlen_k"] = max(1, max(total))
        st["k_pages"], st["k_scale"] = _pages(count, h, page, DQK, case["cache"], gen)
        st["v_pages"], st["v_scale"] = _pages(count, h, page, DV, case["cache"], gen)
    if case["op"] == "append":
        n = sum(new)
        spread = torch.exp2(torch.randn((n, 1, 1), generator=gen, device="cuda") * 0.5)
        k = torch.randn((n, h, DQK), generator=gen, device="cuda") * spread
        if case["rotate"]:                    # a decode step's own projections
            st["k_nope"] = k[..., :NOPE].to(torch.bfloat16).contiguous()
            st["k_rope"] = k[:, 0, NOPE:].to(torch.bfloat16).contiguous()
        else:                                 # views into the prologue's keys, one turned rotary part for all heads
            k[..., NOPE:] = k[:, :1, NOPE:]
            k = k.to(torch.bfloat16)
            st["k_nope"], st["k_rope"] = k[..., :NOPE], k[:, 0, NOPE:]
        st["v"] = (torch.randn((n, h, DV), generator=gen, device="cuda") * spread).to(torch.bfloat16)
        st["cu_seqlens_new"] = _cu(new)
    elif case["op"] == "decode":
        st["q_sig"] = _normal((batch, hs, DQK), gen)
        st["q_noise"] = _normal((batch, h, DQK), gen)
        st["lam"] = _lam((batch, hs), gen)
        st["gate"] = _normal((batch, hs, DV), gen)
    else:
        n = sum(new)
        st["seqlens"] = tuple(new)
        st["q_sig"] = _normal((n, hs, DQK), gen)
        st["q_noise"] = _normal((n, h, DQK), gen)
        st["k"] = _normal((n, h, DQK), gen)
        st["v"] = _normal((n, h, DV), gen)
        st["lam"] = _lam((n, hs), gen)
        st["gate"] = _normal((n, hs, DV), gen)
        if case["op"] == "backward":
            st["dout"] = _normal((n, hs, DV), gen)
    return st


# ---------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------
def _turn(x, pos):
    """Rotary embedding of the last 64 dims (pairs i, i + 32) of x at positions pos (x: [n, ..., 64])."""
    freq = BASE ** (-torch.arange(ROPE // 2, dtype=torch.float64, device=x.device) / (ROPE // 2))
    angle = pos.double()[:, None] * freq
    c, s = angle.cos().float(), angle.sin().float()
    while c.dim() < x.dim():
        c, s = c.unsqueeze(1), s.unsqueeze(1)
    a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat([a * c - b * s, a * s + b * c], -1)


def _plain_append(st):
    case = st["case"]
    page, h = case["page"], case["heads"]
    cu, lens, table = st["cu_seqlens_new"].long(), st["seqlens_k"].long(), st["block_table"].long()
    n = st["v"].shape[0]
    tok = torch.arange(n, device="cuda")
    b = torch.searchsorted(cu[1:], tok, right=True)
    count = cu[1:] - cu[:-1]
    before = lens - count
    pos = before[b] + tok - cu[b]
    at, slot = table[b, pos // page], pos % page
    rope = st["k_rope"].float()
    if case["rotate"]:
        rope = _turn(rope, pos)
    k = torch.cat([st["k_nope"].float(), rope[:, None, :].expand(n, h, ROPE)], -1)
    v = st["v"].float()
    head = torch.arange(h, device="cuda")[None]
    if case["cache"] == "bf16":
        st["k_pages"][at[:, None], head, slot[:, None]] = k.to(torch.bfloat16)
        st["v_pages"][at[:, None], head, slot[:, None]] = v.to(torch.bfloat16)
        return {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    # the page in which each sequence goes on, with the slots that it holds already
    goes_on = (count > 0) & (before % page > 0)
    cont = table[torch.arange(len(lens), device="cuda"), (before // page).clamp_max(table.shape[1] - 1)][goes_on]
    held = (before % page)[goes_on]
    for name, x in (("k", k), ("v", v)):
        pages, scale = st[name + "_pages"], st[name + "_scale"]
        codes = pages.view(torch.uint8)
        amax = torch.zeros_like(scale).scatter_reduce_(0, at[:, None].expand(n, h), x.abs().amax(-1), "amax")
        touched = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda")
        touched[at] = True
        carry = torch.zeros_like(touched)
        carry[cont] = True
        was = torch.frexp(scale)[1] - 1
        need = _scale_exponent(amax)
        now = torch.where(carry[:, None], torch.maximum(was, need), need)
        now = torch.where(touched[:, None], now, was)
        old = pages[cont].float() * _power(was[cont] - now[cont])[..., None, None]
        keep = torch.arange(page, device="cuda")[None, None, :, None] < held[:, None, None, None]
        codes[cont] = torch.where(keep, old.to(torch.float8_e4m3fn).view(torch.uint8), codes[cont])
        new_scale = torch.where(touched[:, None], _power(now), scale)
        q = x / new_scale[at][..., None]
        codes[at[:, None], head, slot[:, None]] = q.to(torch.float8_e4m3fn).view(torch.uint8)
        scale.copy_(new_scale)
    return {"k_pages": st["k_pages"], "v_pages": st["v_pages"], "k_scale": st["k_scale"], "v_scale": st["v_scale"]}


def _visible(case, lens, width):
    """(positions, which of them are there): [B, M] of the keys that each sequence's query sees; full context takes
    every place of its pages."""
    window, longest = case["window"], max(_lengths(case)[1])
    if window <= 0:
        pos = torch.arange(width, device=lens.device)[None].expand(lens.shape[0], -1)
        return pos, pos < lens[:, None]
    lo = (lens - window).clamp_min(0)[:, None]
    near = lo + torch.arange(max(1, min(window, longest)), device=lens.device)
    far = torch.arange(case["sinks"], device=lens.device)[None].expand(lens.shape[0], -1)
    return torch.cat([far, near], 1), torch.cat([far < lo, near < lens[:, None]], 1)


def _gathered(pages, scale, table, pos, whole):
    """[B, H, M, D] in fp32: the rows of the pages at each sequence's positions (`whole`: all of them, in order)."""
    h, page, dim = pages.shape[1:]
    raw = pages.view(torch.uint8 if scale is not None else torch.bfloat16)
    if whole:
        x = raw[table].permute(0, 2, 1, 3, 4).contiguous()                                    # [B, H, W, P, D]
        x = x.float() if scale is None else x.view(torch.float8_e4m3fn).float()
        if scale is not None:
            x *= scale[table].permute(0, 2, 1)[..., None, None]
        return x.view(table.shape[0], h, -1, dim)
    at = table.gather(1, (pos // page).clamp_max(table.shape[1] - 1))
    x = raw[at, :, pos % page].transpose(1, 2)                                                # [B, H, M, D]
    if scale is None:
        return x.float()
    x = x.contiguous().view(torch.float8_e4m3fn).float()
    x *= scale[at].transpose(1, 2)[..., None]
    return x


def _plain_decode(st):
    case = st["case"]
    bsz, h = case["batch"], case["heads"]
    table, lens = st["block_table"].long(), st["seqlens_k"].long()
    q = torch.cat([st["q_sig"].float().view(bsz, h, GROUP, DQK), st["q_noise"].float()[:, :, None]], 2)
    if case["rotate"]:
        q = torch.cat([q[..., :NOPE], _turn(q[..., NOPE:], (lens - 1).clamp_min(0))], -1)
    whole = case["window"] <= 0
    pos, seen = _visible(case, lens, table.shape[1] * case["page"])
    k = _gathered(st["k_pages"], st["k_scale"], table, pos, whole)
    s = torch.matmul(q, k.transpose(-1, -2)) * SCALE
    del k
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    v = _gathered(st["v_pages"], st["v_scale"], table, pos, whole).masked_fill(~seen[:, None, :, None], 0.0)
    hd = torch.matmul(p, v)
    d = hd[:, :, :GROUP] - st["lam"].view(bsz, h, GROUP, 1) * hd[:, :, GROUP:]
    out = torch.sigmoid(st["gate"].float().view(bsz, h, GROUP, DV)) * d
    return out.view(bsz, GROUP * h, DV).to(torch.bfloat16)


def _banded(q_sig, q_noise, k, v, lam, gate, lengths, window, sinks):
    """Sliding window with sinks over packed sequences, in blocks of `window` queries against two blocks of keys
    and the first tokens of every sequence (fp32 in, fp32 out)."""
    n, h = k.shape[0], k.shape[1]
    dev = k.device
    blocks = (n + window - 1) // window
    pad = blocks * window - n
    lens = torch.tensor(lengths, device=dev)
    start = torch.cumsum(lens, 0) - lens
    seq = torch.repeat_interleave(torch.arange(len(lengths), device=dev), lens)
    at = torch.arange(blocks * window, device=dev)
    seq = torch.nn.functional.pad(seq, (0, pad), value=-1)
    q = torch.cat([q_sig.view(n, h, GROUP, DQK), q_noise[:, :, None]], 2)
    grow = lambda x: torch.nn.functional.pad(x, (0, 0) * (x.dim() - 1) + (0, pad))  # noqa: E731
    q = grow(q).view(blocks, window, h, 5, DQK).permute(0, 2, 3, 1, 4)
    two = lambda x: torch.cat([torch.cat([torch.zeros_like(x[:1]), x[:-1]]), x], 1)  # noqa: E731
    kb = two(grow(k).view(blocks, window, h, DQK)).permute(0, 2, 3, 1)
    vb = two(grow(v).view(blocks, window, h, DV)).permute(0, 2, 1, 3)
    near = torch.matmul(q.reshape(blocks, h, 5 * window, DQK), kb).view(blocks, h, 5, window, 2 * window)
    t, u = at.view(blocks, window), at.view(blocks, window)
    u = torch.cat([u - window, u], 1)
    useq = torch.cat([torch.cat([torch.full_like(seq[:window], -2), seq[:-window]]).view(blocks, window),
                      seq.view(blocks, window)], 1)
    gap = t[:, :, None] - u[:, None, :]
    seen = (gap >= 0) & (gap < window) & (useq[:, None, :] == seq.view(blocks, window)[:, :, None])
    near = near.masked_fill(~seen[:, None, None], -math.inf)
    # the first tokens of every sequence, for the queries of their own that see them no more through the window
    first = (start[:, None] + torch.arange(sinks, device=dev)[None]).reshape(-1)
    there = (torch.arange(sinks, device=dev)[None] < lens[:, None]).reshape(-1)
    fseq = torch.arange(len(lengths), device=dev)[:, None].expand(-1, sinks).reshape(-1)
    first = first.clamp_max(n - 1)
    ks, vs = k[first].permute(1, 2, 0), v[first].permute(1, 0, 2)
    far = torch.matmul(q.permute(1, 0, 2, 3, 4).reshape(h, -1, DQK), ks).view(h, blocks, 5, window, -1).transpose(0, 1)
    fsee = there & (fseq == seq[:, None]) & (at[:, None] - first >= window)
    far = far.masked_fill(~fsee.view(blocks, 1, 1, window, -1), -math.inf)
    s = torch.cat([near, far], -1) * SCALE
    top = s.amax(-1, keepdim=True).detach()
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    pn, pf = p[..., :2 * window], p[..., 2 * window:]
    hd = torch.matmul(pn.reshape(blocks, h, 5 * window, 2 * window), vb).view(blocks, h, 5, window, DV)
    hf = torch.matmul(pf.transpose(0, 1).reshape(h, -1, pf.shape[-1]), vs)
    hd = hd + hf.view(h, blocks, 5, window, DV).transpose(0, 1)
    hd = hd.permute(0, 3, 1, 2, 4).reshape(blocks * window, h, 5, DV)[:n]
    d = hd[:, :, :GROUP] - lam.view(n, h, GROUP, 1) * hd[:, :, GROUP:]
    return torch.sigmoid(gate) * d.reshape(n, GROUP * h, DV)


def _plain_prefill(st):
    case = st["case"]
    f = [st[x].float() for x in ("q_sig", "q_noise", "k", "v", "lam", "gate")]
    return _banded(*f, st["seqlens"], case["window"], case["sinks"]).to(torch.bfloat16)


NAMES = ("dq_sig", "dq_noise", "dk", "dv", "dlambda", "dgate")


def _plain_backward(st):
    case = st["case"]
    f = [st[x].float().detach().requires_grad_() for x in ("q_sig", "q_noise", "k", "v", "lam", "gate")]
    out = _banded(*f, st["seqlens"], case["window"], case["sinks"])
    g = torch.autograd.grad(out, f, st["dout"].float())
    return {name: x.to(torch.bfloat16) for name, x in zip(NAMES, g)}


def run(st):
    case, op = st["case"], st["op"]
    if not own:
        return {"append": _plain_append, "decode": _plain_decode, "prefill": _plain_prefill,
                "backward": _plain_backward}[op](st)
    import differential_latent_attention_b200 as gdla
    if op == "append":
        gdla.cache_append(st["k_nope"], st["k_rope"], st["v"], st["k_pages"], st["v_pages"], st["block_table"],
                          st["cu_seqlens_new"], st["seqlens_k"], k_scale=st["k_scale"], v_scale=st["v_scale"],
                          rotate=case["rotate"])
        names = ("k_pages", "v_pages") + (("k_scale", "v_scale") if case["cache"] == "e4m3" else ())
        return {name: st[name] for name in names}
    if op == "decode":
        return gdla.attn_decode_paged(st["q_sig"], st["q_noise"], st["k_pages"], st["v_pages"], st["block_table"],
                                      st["seqlens_k"], st["max_seqlen_k"], st["lam"], st["gate"],
                                      window=case["window"], sinks=case["sinks"], k_scale=st["k_scale"],
                                      v_scale=st["v_scale"], rotate=case["rotate"])
    args = [st[x] for x in ("q_sig", "q_noise", "k", "v", "lam", "gate")]
    if op == "prefill":
        return gdla.attn_fwd(*args, st["seqlens"], window=case["window"], sinks=case["sinks"])
    g = gdla.attn_bwd(*args, st["dout"], st["seqlens"], window=case["window"], sinks=case["sinks"])
    # lambda's projection takes its gradient in bf16, as every other projection does
    return {name: g[name].to(torch.bfloat16) for name in NAMES}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------------------
def _turn64(x, pos):
    out = x.clone()
    for i in range(ROPE // 2):
        a = pos.double() * BASE ** (-i / (ROPE // 2))
        shape = [-1] + [1] * (x.dim() - 2)
        c, s = torch.cos(a).view(shape), torch.sin(a).view(shape)
        out[..., i] = x[..., i] * c - x[..., i + ROPE // 2] * s
        out[..., i + ROPE // 2] = x[..., i] * s + x[..., i + ROPE // 2] * c
    return out


def _exact_append(case, st):
    page, h = case["page"], case["heads"]
    old, new = _lengths(case)
    eight = case["cache"] == "e4m3"
    kp, vp = st["k_pages"].double(), st["v_pages"].double()
    ks, vs = (st["k_scale"].double(), st["v_scale"].double()) if eight else (None, None)
    at = 0
    for b, (before, n) in enumerate(zip(old, new)):
        if n == 0:
            continue
        sl = slice(at, at + n)
        at += n
        pos = torch.arange(before, before + n, device="cuda")
        rope = st["k_rope"][sl].double()
        if case["rotate"]:
            rope = _turn64(rope, pos)
        k = torch.cat([st["k_nope"][sl].double(), rope[:, None].expand(n, h, ROPE)], -1).transpose(0, 1)
        v = st["v"][sl].double().transpose(0, 1)
        for j in range(before // page, (before + n - 1) // page + 1):
            lo, hi = max(before, j * page), min(before + n, (j + 1) * page)
            p, a, c = int(st["block_table"][b, j]), lo - j * page, hi - j * page
            for pool, scale, x in ((kp, ks, k), (vp, vs, v)):
                y = x[:, lo - before:hi - before]
                if eight:
                    top = y.abs().amax((1, 2))
                    want = torch.full_like(top, 2.0 ** MIN_EXP)
                    guess = torch.round(torch.log2((top / E4M3_MAX).clamp_min(1e-300)))
                    for step in (1.0, 0.0, -1.0):      # the smallest power of two that reaches the largest value
                        two = torch.ldexp(torch.ones_like(top), (guess + step).clamp_min(float(MIN_EXP)).int())
                        want = torch.where(top <= E4M3_MAX * two, two, want)
                    if a > 0:
                        want = torch.maximum(want, scale[p])
                        back = pool[p, :, :a] * (scale[p] / want)[:, None, None]
                        pool[p, :, :a] = back.to(torch.float32).to(torch.float8_e4m3fn).double()
                    scale[p] = want
                    y = (y / want[:, None, None]).to(torch.float32).to(torch.float8_e4m3fn).double()
                pool[p, :, a:c] = y
    return {"k_pages": kp, "v_pages": vp, "k_scale": ks, "v_scale": vs} if eight else {"k_pages": kp, "v_pages": vp}


def _exact_decode(case, st):
    page, h, bsz = case["page"], case["heads"], case["batch"]
    _, lens = _lengths(case)
    out = torch.zeros((bsz, h * GROUP, DV), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if n == 0:
            continue
        pos = torch.arange(n, device="cuda")
        if case["window"] > 0:
            pos = pos[(pos >= n - case["window"]) | (pos < case["sinks"])]
        at, slot = st["block_table"][b].long()[pos // page], pos % page
        qs, qn = st["q_sig"][b].double().view(h, GROUP, DQK), st["q_noise"][b].double().view(h, 1, DQK)
        q = torch.cat([qs, qn], 1)
        if case["rotate"]:
            turned = _turn64(q[..., NOPE:].reshape(-1, ROPE), torch.full((5 * h,), n - 1, device="cuda"))
            q = torch.cat([q[..., :NOPE], turned.view(h, 5, ROPE)], -1)
        kv = []
        for name in ("k", "v"):
            pages = st[name + "_pages"]
            x = pages.view(torch.uint8 if case["cache"] == "e4m3" else torch.bfloat16)[at, :, slot]
            x = x.view(pages.dtype).double()
            kv.append(x * st[name + "_scale"].double()[at][..., None] if case["cache"] == "e4m3" else x)
        a = torch.softmax(torch.einsum("hid,nhd->hin", q, kv[0]) * SCALE, -1)
        hd = torch.einsum("hin,nhd->hid", a, kv[1])
        d = hd[:, :GROUP] - st["lam"][b].double().view(h, GROUP, 1) * hd[:, GROUP:]
        out[b] = (torch.sigmoid(st["gate"][b].double()) * d.reshape(h * GROUP, DV))
    return out


def _exact_attention(case, st, backward):
    """Row blocks of each sequence against the keys that they can see, forward or with every gradient's formula."""
    h, window, sinks = case["heads"], case["window"], case["sinks"]
    n = st["k"].shape[0]
    z = lambda *s: torch.zeros(s, dtype=torch.float64, device="cuda")  # noqa: E731
    out = z(n, GROUP * h, DV)
    g = {"dq_sig": z(n, GROUP * h, DQK), "dq_noise": z(n, h, DQK), "dk": z(n, h, DQK), "dv": z(n, h, DV),
         "dlambda": z(n, GROUP * h), "dgate": z(n, GROUP * h, DV)}
    s0 = 0
    for length in st["seqlens"]:
        for r0 in range(0, length, 512):
            r1 = min(length, r0 + 512)
            lo = max(0, r0 - window + 1)
            u = torch.cat([torch.arange(min(sinks, lo), device="cuda"), torch.arange(lo, r1, device="cuda")])
            t = torch.arange(r0, r1, device="cuda")
            ok = (u[None] <= t[:, None]) & ((t[:, None] - u[None] < window) | (u[None] < sinks))
            r = t.shape[0]
            rows, keys = s0 + t, s0 + u
            q = torch.cat([st["q_sig"][rows].double().view(r, h, GROUP, DQK), st["q_noise"][rows].double()[:, :, None]], 2)
            k, v = st["k"][keys].double(), st["v"][keys].double()
            a = torch.einsum("rhid,nhd->hirn", q, k) * SCALE
            a = torch.softmax(a.masked_fill(~ok, -math.inf), -1)
            hd = torch.einsum("hirn,nhd->rhid", a, v)
            lam = st["lam"][rows].double().view(r, h, GROUP, 1)
            sg = torch.sigmoid(st["gate"][rows].double()).view(r, h, GROUP, DV)
            d = hd[:, :, :GROUP] - lam * hd[:, :, GROUP:]
            out[rows] = (sg * d).view(r, -1, DV)
            if not backward:
                continue
            go = st["dout"][rows].double().view(r, h, GROUP, DV)
            dd = go * sg
            g["dgate"][rows] = (go * d * sg * (1 - sg)).view(r, -1, DV)
            g["dlambda"][rows] = -(dd * hd[:, :, GROUP:]).sum(-1).view(r, -1)
            dh = torch.cat([dd, -(lam * dd).sum(2, keepdim=True)], 2)
            g["dv"].index_add_(0, keys, torch.einsum("hirn,rhid->nhd", a, dh))
            dp = torch.einsum("rhid,nhd->hirn", dh, v)
            ds = a * (dp - (dh * hd).sum(-1).permute(1, 2, 0)[..., None]) * SCALE
            dq = torch.einsum("hirn,nhd->rhid", ds, k)
            g["dq_sig"][rows] = dq[:, :, :GROUP].reshape(r, -1, DQK)
            g["dq_noise"][rows] = dq[:, :, GROUP]
            g["dk"].index_add_(0, keys, torch.einsum("hirn,rhid->nhd", ds, q))
        s0 += length
    return {name: g[name] for name in NAMES} if backward else out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, st)
    if case["op"] == "decode":
        return _exact_decode(case, st)
    return _exact_attention(case, st, case["op"] == "backward")
