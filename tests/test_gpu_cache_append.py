"""gdla_cache_append on the GPU against its definition in 64 bits (tests/_paged.py), bit for bit where nothing is
computed (K's content, V, scales, codes rescaled by a power of two) and within one rounding where the rotation is."""
import pytest
import torch

import differential_latent_attention_b200 as gdla
from _paged import BF16_HALF, NOPE, new_pool, plain_append, rand, table_of, turn

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _case(new, total, heads, page, kind, seed, spare=3):
    """Inputs of one append: a pool with a page table, and packed new rows whose size varies from token to token."""
    n = sum(new)
    pages = sum((t + page - 1) // page for t in total) + spare
    spread = torch.exp2(torch.randint(-4, 5, (n, 1, 1), generator=torch.Generator().manual_seed(seed)).float()).cuda()
    return {"pool": new_pool(pages, heads, page, kind, seed), "table": table_of(total, page, pages, seed=seed),
            "k_nope": (rand((n, heads, 128), seed + 1, dtype=torch.float32) * spread).to(torch.bfloat16),
            "k_rope": (rand((n, 64), seed + 2, dtype=torch.float32) * spread[:, 0]).to(torch.bfloat16),
            "v": (rand((n, heads, 128), seed + 3, dtype=torch.float32) * spread).to(torch.bfloat16),
            "cu": _i32([0] + list(torch.tensor(new).cumsum(0))), "lens": _i32(total)}


def _clone(pool):
    return {k: None if v is None else v.clone() for k, v in pool.items()}


def _run(c, pool, rotate=True, **kw):
    gdla.cache_append(kw.get("k_nope", c["k_nope"]), kw.get("k_rope", c["k_rope"]), kw.get("v", c["v"]), pool["k_pages"],
                      pool["v_pages"], kw.get("table", c["table"]), kw.get("cu", c["cu"]), kw.get("lens", c["lens"]),
                      k_scale=pool["k_scale"], v_scale=pool["v_scale"], rotate=rotate, stream=kw.get("stream"))
    torch.cuda.synchronize()
    assert gdla.device_error() == 0


def _raw(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t.view(torch.int16)


def _compare(pool, before, want, rotate):
    """The pool after the call against the plain append's."""
    eight = pool["k_scale"] is not None
    for name in ("k", "v"):
        got, ref = pool[name + "_pages"], want[name]
        if not eight:
            written = ~torch.isnan(ref)
            assert torch.equal(_raw(got)[~written], _raw(before[name + "_pages"])[~written]), name   # nothing else is touched
            exact = torch.where(written, ref, torch.zeros_like(ref))
            if name == "v" or not rotate:
                assert torch.equal(got.double()[written], exact[written])
                continue
            assert torch.equal(got.double()[..., :NOPE][written[..., :NOPE]], exact[..., :NOPE][written[..., :NOPE]])
            # one bf16 rounding of x cos - y sin, which fp32 gets to 4 * 2^-24 of |x| + |y|
            g, e, w = got.double()[..., NOPE:], exact[..., NOPE:], written[..., NOPE:]
            size = (e[..., :32].square() + e[..., 32:].square()).sqrt() * 2
            tol = BF16_HALF * e.abs() + 2.0 ** -22 * torch.cat([size, size], -1)
            assert bool(((g - e).abs() <= tol)[w].all())
            continue
        assert torch.equal(pool[name + "_scale"], want[name + "_scale"]), name
        codes = _raw(got)
        if name == "v" or not rotate:
            assert torch.equal(codes, ref)
            continue
        assert torch.equal(codes[..., :NOPE], ref[..., :NOPE])
        # a turned value next to a border between two codes may go to either: at most one code apart, and rarely
        g, e = codes[..., NOPE:], ref[..., NOPE:]
        apart = (g.view(torch.float8_e4m3fn).float() - e.view(torch.float8_e4m3fn).float()).abs()
        step = (e.view(torch.float8_e4m3fn).float().abs() * 2.0 ** -3).clamp_min(2.0 ** -9) * 1.01
        assert bool(((g == e) | (apart <= step)).all())
        assert float((g != e).float().mean()) <= 1e-4


def _check(new, total, heads, page, kind, seed, rotate=True):
    c = _case(new, total, heads, page, kind, seed)
    pool = _clone(c["pool"])
    _run(c, pool, rotate)
    want = plain_append(c["pool"], c["table"], page, c["k_nope"], c["k_rope"], c["v"], new, total, rotate)
    _compare(pool, c["pool"], want, rotate)
    return c, pool


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_steps(kind, page):
    """One token each: an empty cache, the first and last slot of a page, a sequence without a new token."""
    total = [1, page, page + 1, 2 * page - 1, 5, 3 * page, 1]
    _check([1, 1, 1, 1, 0, 1, 1], total, 3, page, kind, 10 + page)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("rotate", [True, False])
def test_ragged_prompts(kind, page, rotate):
    """Whole pages, pages that are gone on with, that end inside, and sequences with nothing."""
    new = [0, 3 * page + 5, 1, 2 * page, page - 1, 0, 7]
    old = [4, 0, page - 1, page, 1, 0, 2 * page - 3]
    _check(new, [a + b for a, b in zip(new, old)], 5, page, kind, 50 + page, rotate)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_many_sequences(kind):
    """More sequences than one round of the search tries at a time, several rounds' worth, some empty; single tokens and
    a few each (both kernels)."""
    g = torch.Generator().manual_seed(3)
    for most, batch in ((1, 1100), (2, 77), (40, 77)):
        new = torch.randint(0, most + 1, (batch,), generator=g).tolist()
        old = torch.randint(0, 50, (batch,), generator=g).tolist()
        _check(new, [a + b for a, b in zip(new, old)], 1 if batch > 1000 else 2, 16, kind, 80 + most)


@pytest.mark.parametrize("heads", [1, 4, 7, 64])
def test_head_counts(heads):
    _check([70, 1], [75, 33], heads, 64, "e4m3", 90 + heads)
    _check([1, 1], [75, 33], heads, 64, "e4m3", 91 + heads)


def test_far_positions():
    """Angles at a million tokens and more: fp32 angles would be off by 2^-4 of a turn there."""
    lens = [1 << 20, (1 << 24) + 5, (1 << 27) + 77]
    n, h, page = len(lens), 2, 128
    k_rope = rand((n, 64), 5)
    zero = torch.zeros((n, h, 128), dtype=torch.bfloat16, device="cuda")
    for i, length in enumerate(lens):      # one table row as wide as the longest would be large: one sequence at a time
        pool = new_pool(2, h, page, "bf16", 6)
        width = length // page + 1
        table = torch.full((1, width), 1, dtype=torch.int32, device="cuda")
        gdla.cache_append(zero[:1], k_rope[i:i + 1], zero[:1], pool["k_pages"], pool["v_pages"], table, _i32([0, 1]), _i32([length]))
        got = pool["k_pages"][1, 0, (length - 1) % page, NOPE:].double()
        want = turn(k_rope[i:i + 1], torch.tensor([length - 1], device="cuda"))[0]
        size = (want[:32].square() + want[32:].square()).sqrt()
        # the angle is good to 2^-24 of a turn: 2 pi 2^-24 of the pair's size, beside the rounding
        tol = BF16_HALF * want.abs() + (2 * 3.1416 * 2.0 ** -24 + 2.0 ** -22) * torch.cat([size, size])
        assert bool(((got - want).abs() <= tol).all())


def test_step_by_step_is_one_append_in_bf16():
    """Tokens one after another leave bf16 pages as all at once does, bit for bit."""
    new, page, heads = [37, 5], 16, 3
    c = _case(new, new, heads, page, "bf16", 21)
    once, steps = _clone(c["pool"]), _clone(c["pool"])
    _run(c, once)
    starts = [0, new[0]]
    for i in range(max(new)):
        rows = [starts[b] + i for b in range(2) if i < new[b]]
        cu = _i32([0, 1 if i < new[0] else 0, len(rows)])
        _run(c, steps, k_nope=c["k_nope"][rows], k_rope=c["k_rope"][rows], v=c["v"][rows], cu=cu,
             lens=_i32([min(i + 1, new[0]), min(i + 1, new[1])]))
    for name in ("k_pages", "v_pages"):
        assert torch.equal(_raw(once[name]), _raw(steps[name]))


def test_growing_scale_keeps_older_codes():
    """A page whose later tokens are larger and larger: each growth divides the older codes by a power of two, rounding
    only what falls under e4m3's smallest normal; a smaller token leaves the scale alone; a fresh page forgets."""
    page, heads = 16, 1
    pool = new_pool(2, heads, page, "e4m3", 1)
    table = _i32([[0]])
    sizes = [1e-3, 1.0, 0.01, 4000.0, 1.0, 3e38, 1e-30]
    want = None
    for i, size in enumerate(sizes):
        c = {"k_nope": rand((1, 1, 128), 100 + i, size), "k_rope": rand((1, 64), 200 + i, size), "v": rand((1, 1, 128), 300 + i, size)}
        before = _clone(pool)
        gdla.cache_append(c["k_nope"], c["k_rope"], c["v"], pool["k_pages"], pool["v_pages"], table, _i32([0, 1]), _i32([i + 1]),
                          k_scale=pool["k_scale"], v_scale=pool["v_scale"], rotate=False)
        want = plain_append(before, table, page, c["k_nope"], c["k_rope"], c["v"], [1], [i + 1], False)
        for name in ("k", "v"):
            assert torch.equal(pool[name + "_pages"].view(torch.uint8), want[name]), (i, name)
            assert torch.equal(pool[name + "_scale"], want[name + "_scale"]), (i, name)
    small = {"k_nope": rand((1, 1, 128), 7), "k_rope": rand((1, 64), 8), "v": rand((1, 1, 128), 9)}
    gdla.cache_append(small["k_nope"], small["k_rope"], small["v"], pool["k_pages"], pool["v_pages"], table, _i32([0, 1]),
                      _i32([1]), k_scale=pool["k_scale"], v_scale=pool["v_scale"], rotate=False)
    top = float(small["v"].abs().max())
    scale = float(pool["v_scale"][0, 0])
    assert scale / 2 * 448 < top <= scale * 448


@pytest.mark.parametrize("n", [1, 40])
def test_zeros_and_non_finite_values(n):
    """All-zero rows take the least scale; infinities and NaN become e4m3's NaN and leave the scale to the others; bf16
    pages hold them as they are."""
    page, heads = 64, 2
    c = _case([n], [n], heads, page, "e4m3", 31)
    for x in ("k_nope", "v"):
        c[x][:, 1] = 0
    c["k_rope"][:] = 0
    c["v"][0, 0, 3], c["v"][0, 0, 4], c["k_nope"][n - 1, 0, 7] = float("inf"), float("nan"), float("-inf")
    pool = _clone(c["pool"])
    _run(c, pool)
    want = plain_append(c["pool"], c["table"], page, c["k_nope"], c["k_rope"], c["v"], [n], [n], True)
    for name in ("k", "v"):
        assert torch.equal(pool[name + "_scale"], want[name + "_scale"])
        got, ref = pool[name + "_pages"].float(), want[name].view(torch.float8_e4m3fn).float()
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(got[~torch.isnan(got)], ref[~torch.isnan(ref)])
    p = int(c["table"][0, 0])
    assert float(pool["v_scale"][p, 1]) == 2.0 ** -110
    assert torch.isnan(pool["v_pages"].float()[p, 0, 0, 3:5]).all()
    b = _case([n], [n], heads, page, "bf16", 31)
    b["v"][0, 0, 3] = float("inf")
    pool = _clone(b["pool"])
    _run(b, pool)
    assert float(pool["v_pages"][int(b["table"][0, 0]), 0, 0, 3]) == float("inf")


def test_views_of_the_prologue_layout():
    """k as two views of [N, H, 192], V with a head stride of zero (one row for every head)."""
    n, heads, page = 50, 4, 32
    k = rand((n, heads, 192), 41)
    k[..., 128:] = k[:, :1, 128:]
    v = rand((n, 1, 128), 42).expand(n, heads, 128)
    for kind in ("bf16", "e4m3"):
        c = _case([n], [n + 9], heads, page, kind, 43)
        a, b = _clone(c["pool"]), _clone(c["pool"])
        _run(c, a, False, k_nope=k[..., :128], k_rope=k[:, 0, 128:], v=v)
        _run(c, b, False, k_nope=k[..., :128].contiguous(), k_rope=k[:, 0, 128:].contiguous(), v=v.contiguous())
        for name in ("k_pages", "v_pages"):
            assert torch.equal(_raw(a[name]), _raw(b[name]))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 50])
def test_what_does_not_fit_is_skipped(kind, n):
    """Sequences whose numbers do not fit, table entries outside the pool and rows behind the last sequence leave the
    pool as it was; the others are appended."""
    page, heads = 16, 2
    new, total = [n, n, n, n], [n, n + 5, n, n + 3]
    c = _case(new, total, heads, page, kind, 61)
    table = c["table"].clone()
    table[0, :] = c["pool"]["k_pages"].shape[0]      # past the pool
    table[1, 0] = -1                                # one page of the second
    lens = _i32([n, n + 5, n - 1, n + 3])           # the third says it holds fewer than it brings
    more = torch.cat([c["v"], c["v"]])              # rows behind the last sequence
    rows = {"k_nope": torch.cat([c["k_nope"], c["k_nope"]]), "k_rope": torch.cat([c["k_rope"], c["k_rope"]]), "v": more}
    pool = _clone(c["pool"])
    _run(c, pool, table=table, lens=lens, **rows)
    want = _clone(c["pool"])
    ok = _clone(c["pool"])
    _run(c, ok)
    pages = {int(p) for p in c["table"][3] if p >= 0} | {int(p) for p in c["table"][1, 1:] if p >= 0}
    for name in ("k_pages", "v_pages"):
        for p in range(pool[name].shape[0]):
            src = ok if p in pages else want
            assert torch.equal(_raw(pool[name])[p], _raw(src[name])[p]), (name, p)
    # a table narrower than a sequence's length, and counts that run past the rows
    pool = _clone(c["pool"])
    _run(c, pool, lens=_i32([10 ** 6] * 4))
    _run(c, pool, cu=_i32([0, 10 ** 6, 10 ** 6 + 1, 10 ** 6 + 2, 10 ** 6 + 3]))
    _run(c, pool, cu=_i32([-5, -4, -3, -2, -1]))
    least, most = -2 ** 31, 2 ** 31 - 1             # differences of these leave 32 bits
    _run(c, pool, lens=_i32([least, least + n - 1, least + n, -1]))
    _run(c, pool, lens=_i32([most, most - 1, most - n, most]))
    _run(c, pool, cu=_i32([most, least, most, least, most]))
    _run(c, pool, cu=_i32([least, most, least, most, least]))
    _run(c, pool, cu=_i32([least] * 5))
    for name in ("k_pages", "v_pages"):
        assert torch.equal(_raw(pool[name]), _raw(c["pool"][name]))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 64, 128])
def test_steps_beside_chunks(kind, page):
    """Units of one to five rows (also a chunk's last page) beside whole pages, and sequences that bring nothing for long
    stretches, so that the search for a unit's sequence starts far from it."""
    new = [1] * 20 + [page + 3, 3, 4, 5, 6, 2 * page + 4, 2 * page + 5, 1]
    old = [(7 * i) % (2 * page) for i in range(20)] + [0, page - 2, page - 4, 11, page - 1, 0, page - 3, 0]
    _check(new, [n + o for n, o in zip(new, old)], 3, page, kind, 1101)
    new = [0] * 90 + [3 * page + 1] + [0] * 60 + [1, 2, 0, page] + [0] * 50 + [1]
    _check(new, [n + (5 * i) % page for i, n in enumerate(new)], 9, page, kind, 1102)


def test_no_tokens():
    c = _case([0], [5], 2, 16, "bf16", 71)
    pool = _clone(c["pool"])
    _run(c, pool)
    assert torch.equal(_raw(pool["k_pages"]), _raw(c["pool"]["k_pages"]))


def test_pool_past_32_bit_offsets():
    """The pages in use lie behind 2^31 elements (and bytes) of the pool."""
    heads, page = 64, 128
    pages = (1 << 31) // (heads * page * 128) + 4
    c = _case([130, 1], [200, 20], heads, page, "e4m3", 81)
    pool = {"k_pages": torch.zeros((pages, heads, page, 192), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
            "v_pages": torch.zeros((pages, heads, page, 128), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
            "k_scale": torch.ones((pages, heads), device="cuda"), "v_scale": torch.ones((pages, heads), device="cuda")}
    shift = pages - c["pool"]["k_pages"].shape[0]
    for name, x in c["pool"].items():
        pool[name].view(torch.uint8 if "pages" in name else torch.float32)[shift:] = x.view(torch.uint8) if "pages" in name else x
    small = _clone(c["pool"])
    _run(c, small)
    _run(c, pool, table=torch.where(c["table"] >= 0, c["table"] + shift, c["table"]))
    for name in small:
        assert torch.equal(_raw(pool[name][shift:]) if "pages" in name else pool[name][shift:],
                           _raw(small[name]) if "pages" in name else small[name]), name
    assert int(pool["k_pages"].view(torch.uint8)[:shift].max()) == 0


def test_side_stream_and_replayed_graph():
    """On another stream, and captured once: the replays follow lengths, table and rows as they change in place."""
    new, page, heads = [1, 1, 1], 16, 2
    c = _case(new, [4, 40, 17], heads, page, "e4m3", 91)
    ref = _clone(c["pool"])
    _run(c, ref)
    pool = _clone(c["pool"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _run(c, pool, stream=side)
    for name in ("k_pages", "v_pages"):
        assert torch.equal(_raw(pool[name]), _raw(ref[name]))
    pool, eager = _clone(c["pool"]), _clone(c["pool"])
    live = {k: c[k].clone() for k in ("k_nope", "k_rope", "v", "lens", "table")}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdla.cache_append(live["k_nope"], live["k_rope"], live["v"], pool["k_pages"], pool["v_pages"], live["table"], c["cu"],
                          live["lens"], k_scale=pool["k_scale"], v_scale=pool["v_scale"])
    for name in pool:
        pool[name].view(torch.uint8 if "pages" in name else torch.float32).copy_(
            c["pool"][name].view(torch.uint8 if "pages" in name else torch.float32))
    for step in range(5):
        rows = {"k_nope": rand((3, heads, 128), 500 + step, 2.0 ** step), "k_rope": rand((3, 64), 600 + step),
                "v": rand((3, heads, 128), 700 + step)}
        lens = c["lens"] + step
        if step == 3:
            live["table"].fill_(2)           # somewhere else from now on: each sequence writes a page of its own
            live["table"][1], live["table"][2] = 3, 4
            live["table"][0] = 5
        for k, x in rows.items():
            live[k].copy_(x)
        live["lens"].copy_(lens)
        g.replay()
        torch.cuda.synchronize()
        _run(c, eager, table=live["table"].clone(), lens=lens, **rows)
        for name in ("k_pages", "v_pages"):
            assert torch.equal(_raw(pool[name]), _raw(eager[name])), step
        for name in ("k_scale", "v_scale"):
            assert torch.equal(pool[name], eager[name]), step
