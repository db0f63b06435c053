"""gdla_attn_decode_paged on the GPU against 64 bits (tests/_paged.py holds the plain form and derives the bounds)."""
import pytest
import torch

import differential_latent_attention_b200 as gdla
from _paged import check_decode, decode_inputs, new_pool, plain_decode, rand, table_of

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _run(d, pool, table, lens, most=None, **kw):
    out = gdla.attn_decode_paged(d["q_sig"], d["q_noise"], pool["k_pages"], pool["v_pages"], table,
                                 lens if torch.is_tensor(lens) else _i32(lens), most or max(1, max(lens)), d["lam"], d["gate"],
                                 k_scale=pool["k_scale"], v_scale=pool["v_scale"], **kw)
    torch.cuda.synchronize()
    assert gdla.device_error() == 0
    return out


def _case(lens, heads, page, kind, seed, spare=2):
    pages = sum((n + page - 1) // page for n in lens) + spare
    return decode_inputs(len(lens), heads, seed), new_pool(pages, heads, page, kind, seed), table_of(lens, page, pages, seed=seed)


def _check(lens, heads, page, kind, seed, most=None, **kw):
    d, pool, table = _case(lens, heads, page, kind, seed)
    if most:
        table = torch.nn.functional.pad(table, (0, max(0, (most + page - 1) // page - table.shape[1])), value=-1)
    got = _run(d, pool, table, lens, most, **kw)
    ref = plain_decode(**d, pool=pool, table=table, page=page, lens=lens, **kw)
    check_decode(got, ref, (lens, heads, page, kind, kw))
    return got


EDGES = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1000, 1023, 1025, 2049]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_edge_lengths(kind, page):
    _check(EDGES, 2, page, kind, 100 + page)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 1), (16, 4), (100, 17), (128, 4), (129, 128), (1000, 5), (5000, 64)])
def test_windows_and_sinks(kind, window, sinks):
    _check(EDGES, 3, 16, kind, 200 + window, window=window, sinks=sinks)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("window, sinks", [(0, 0), (130, 9)])
def test_turned_queries(kind, window, sinks):
    _check([1, 70, 513, 4001], 2, 64, kind, 300, window=window, sinks=sinks, rotate=True)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_every_way_to_cut_an_item(kind):
    """One CTA per item, clusters of 2, 4 and 8, and several clusters joined over the workspace."""
    _check([300] * 160, 2, 16, kind, 401)                                     # 320 items
    _check([700, 650, 900, 513] * 12, 2, 64, kind, 402)                       # 96 items: clusters
    _check([2000, 1500, 1111], 5, 64, kind, 403)
    _check([4096], 16, 64, kind, 404)
    need = gdla.decode_paged_workspace_bytes(2, 1, 20011, 0)
    assert need > 0
    _check([20011, 77], 1, 64, kind, 405)
    _check([9000], 1, 128, kind, 406, most=70000)                             # planned for more than is there


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_many_items_of_few_keys(kind):
    """More than 592 items of at most 512 keys: CTAs of two warps."""
    lens = [(37 * i) % 401 for i in range(200)]
    _check(lens, 3, 16, kind, 441)
    _check([n + 500 for n in lens], 4, 32, kind, 442, window=100, sinks=17, rotate=True)


def test_sixty_four_heads():
    _check([500, 33], 64, 32, "e4m3", 450)
    _check([500, 33], 64, 32, "bf16", 451)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_no_keys_give_zero(kind):
    """Length 0, negative or over the bound, a table without one valid page."""
    page, heads = 16, 2
    lens = [20, 30, 40, 20]
    d, pool, table = _case(lens, heads, page, kind, 501)
    table[3] = -1
    got = _run(d, pool, table, _i32([0, -3, 49, 20]), 48)
    assert torch.count_nonzero(got.float()) == 0
    got = _run(d, pool, table, _i32([20, -3, 49, 20]), 48, window=7, sinks=3)
    assert torch.count_nonzero(got[1:].float()) == 0 and torch.count_nonzero(got[0].float()) > 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("window, sinks", [(0, 0), (40, 3), (16, 0)])
def test_slots_that_are_not_seen_never_matter(kind, window, sinks):
    """NaN and infinities in every slot that the query does not see, in the same pages and blocks: not a bit changes."""
    page, heads = 32, 2
    lens = [1, 5, 17, 47, 64, 100, 333]
    d, pool, table = _case(lens, heads, page, kind, 521)
    clean = _run(d, pool, table, lens, window=window, sinks=sinks)
    dirty = {k: None if v is None else v.clone() for k, v in pool.items()}
    seen = torch.zeros((pool["k_pages"].shape[0], page), dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for u in range(n):
            if window <= 0 or u >= n - window or u < sinks:
                seen[int(table[b, u // page]), u % page] = True
    for name in ("k_pages", "v_pages"):
        x = dirty[name]
        bad = x.view(torch.uint8) if kind == "e4m3" else x
        bad.masked_fill_(~seen[:, None, :, None], 0x7F if kind == "e4m3" else float("nan"))
    assert torch.equal(_run(d, dirty, table, lens, window=window, sinks=sinks).view(torch.int16), clean.view(torch.int16))


def test_nan_in_a_seen_key_shows():
    d, pool, table = _case([40, 40], 2, 16, "bf16", 531)
    pool["v_pages"][int(table[0, 1]), 1, 3, 5] = float("nan")
    got = _run(d, pool, table, [40, 40])
    assert torch.isnan(got[0, 4:, 5].float()).all()              # head 1's signal heads, that dim
    got[0, 4:, 5] = 0
    assert torch.isfinite(got.float()).all()


def test_pages_outside_the_pool_hold_no_keys():
    page = 16
    lens = [100, 100]
    for kind in ("bf16", "e4m3"):
        d, pool, table = _case(lens, 2, page, kind, 541)
        table[0, 2], table[0, 6], table[1, 0] = pool["k_pages"].shape[0], -7, 2 ** 31 - 1
        got = _run(d, pool, table, lens)
        check_decode(got, plain_decode(**d, pool=pool, table=table, page=page, lens=lens), kind)


def test_shared_pages():
    """Two sequences over the same first pages."""
    page = 16
    d, pool, table = _case([64, 80], 2, page, "e4m3", 551)
    table[1, :4] = table[0, :4]
    got = _run(d, pool, table, [64, 80])
    check_decode(got, plain_decode(**d, pool=pool, table=table, page=page, lens=[64, 80]))


def test_scales_of_every_size():
    """Pages whose scales are up to 2^60 apart, in an order that goes up and down, and scales that are no powers of two:
    O's unit follows. The heavy pages decide the result; a second query sees the light ones alone."""
    page, heads = 16, 2
    for exps in ([0, 30, -30, 5, 5, -60, 20], [-40] * 7, [30, 30, 30, 30, 30, 30, -30], [0, 9, -9, 8, -8, 7, 0]):
        lens = [7 * page, 5 * page + 3]
        d, pool, table = _case(lens, heads, page, "e4m3", 561)
        for b in range(2):
            for j, e in enumerate(exps):
                if j < table.shape[1] and int(table[b, j]) >= 0:
                    pool["v_scale"][int(table[b, j])] = 1.37 * 2.0 ** e
        got = _run(d, pool, table, lens)
        ref = plain_decode(**d, pool=pool, table=table, page=page, lens=lens)
        check_decode(got, ref, exps)
        got = _run(d, pool, table, lens, window=page, sinks=0)
        check_decode(got, plain_decode(**d, pool=pool, table=table, page=page, lens=lens, window=page), exps)


def test_pages_of_zeros_between_large_ones():
    """A page of zeros has the least scale, 2^-110; what the pages around it gave stays finite and as it was."""
    page, heads = 16, 2
    for exps in ([32, None, 32, 30, None, None, 31], [None, -7, None, -7, -6, None, -7], [None] * 7, [-110] * 7):
        lens = [7 * page, 2 * page]
        d, pool, table = _case(lens, heads, page, "e4m3", 565)
        for b in range(2):
            for j, e in enumerate(exps):
                if j < table.shape[1] and int(table[b, j]) >= 0:
                    pool["v_scale"][int(table[b, j])] = 2.0 ** (-110 if e is None else e)
                    if e is None:
                        pool["v_pages"][int(table[b, j])] = 0
        for window in (0, page):
            got = _run(d, pool, table, lens, window=window)
            check_decode(got, plain_decode(**d, pool=pool, table=table, page=page, lens=lens, window=window), (exps, window))
    # one warp takes many blocks on both sides of the zeros: sums of 2^16 units and more
    for exp in (0, 40):
        lens = [4096] * 640
        d, pool, table = decode_inputs(640, 1, 566), new_pool(6, 1, 128, "e4m3", 566), torch.zeros((640, 32), dtype=torch.int32, device="cuda")
        table[:] = torch.arange(32, device="cuda") % 5
        table[:, 20] = 5
        pool["v_pages"].fill_(448.0)
        pool["v_scale"][:] = 2.0 ** exp
        pool["v_pages"][5], pool["v_scale"][5] = 0, 2.0 ** -110
        got = _run(d, pool, table, lens)
        some = {k: x[:4] for k, x in d.items()}
        check_decode(got[:4], plain_decode(**some, pool=pool, table=table, page=128, lens=lens[:4]), exp)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_sharp_and_growing_scores(kind):
    """Scores that grow along the sequence (the running maximum moves all the time) and one key that takes all."""
    page, n = 16, 400
    d, pool, table = _case([n], 1, page, kind, 571)
    q = d["q_noise"][0, 0].float()
    d["q_sig"][:] = d["q_noise"][:, :1]
    direction = q / q.norm()
    for u in range(n):
        p, s = int(table[0, u // page]), u % page
        row = (direction * (u / 40.0)).to(torch.bfloat16)
        if kind == "bf16":
            pool["k_pages"][p, 0, s] = row
        else:
            pool["k_scale"][p, 0] = 2.0 ** -5
            pool["k_pages"][p, 0, s] = (row.float() * 32).to(torch.float8_e4m3fn)
    got = _run(d, pool, table, [n])
    ref = plain_decode(**d, pool=pool, table=table, page=page, lens=[n])
    # four signal heads equal to the noise head: D = (1 - lambda) H
    check_decode(got, ref, kind)


def test_small_and_large_queries():
    """f16 queries are divided by a power of two per head: sizes far from one, in e4m3 caches too."""
    page, lens = 16, [90, 33]
    for kind in ("bf16", "e4m3"):
        for size in (2.0 ** -40, 2.0 ** -10, 8.0):
            d, pool, table = _case(lens, 2, page, kind, 581)
            d["q_sig"], d["q_noise"] = (d["q_sig"].float() * size).to(torch.bfloat16), (d["q_noise"].float() * size).to(torch.bfloat16)
            got = _run(d, pool, table, lens, rotate=True)
            check_decode(got, plain_decode(**d, pool=pool, table=table, page=page, lens=lens, rotate=True), (kind, size))


def test_deterministic_and_own_buffers():
    d, pool, table = _case([20000, 300], 1, 64, "e4m3", 591)
    need = gdla.decode_paged_workspace_bytes(2, 1, 20000)
    ws = torch.full((need // 4,), float("nan"), device="cuda").view(torch.uint8)      # contents do not matter
    out = torch.full((2, 4, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    a = _run(d, pool, table, [20000, 300], out=out, workspace=ws)
    assert a.data_ptr() == out.data_ptr()
    b = _run(d, pool, table, [20000, 300])
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    with pytest.raises(gdla.GDLAError):
        _run(d, pool, table, [20000, 300], workspace=ws[:256])


def test_pool_past_32_bit_offsets():
    heads, page, lens = 64, 128, [300, 129]
    pages = (1 << 31) // (heads * page * 128) + 6
    d, pool, table = _case(lens, heads, page, "e4m3", 601, spare=1)
    big = {"k_pages": torch.full((pages, heads, page, 192), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
           "v_pages": torch.full((pages, heads, page, 128), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
           "k_scale": torch.ones((pages, heads), device="cuda"), "v_scale": torch.ones((pages, heads), device="cuda")}
    shift = pages - pool["k_pages"].shape[0]
    for name, x in pool.items():
        big[name].view(torch.uint8 if "pages" in name else torch.float32)[shift:] = x.view(torch.uint8) if "pages" in name else x
    a = _run(d, pool, table, lens)
    b = _run(d, big, torch.where(table >= 0, table + shift, table), lens)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_long_context():
    """One sequence of 200,000 tokens under one KV head: many clusters, chunks of the table, far positions."""
    n, page = 200_003, 128
    d, pool, table = _case([n], 1, page, "e4m3", 611)
    got = _run(d, pool, table, [n], rotate=True)
    check_decode(got, plain_decode(**d, pool=pool, table=table, page=page, lens=[n], rotate=True))
    got = _run(d, pool, table, [n], window=4096, sinks=100)
    check_decode(got, plain_decode(**d, pool=pool, table=table, page=page, lens=[n], window=4096, sinks=100))


def test_side_stream_and_replayed_graph():
    """On another stream, and captured with room to grow: replays follow lengths and table; two graphs that share a
    workspace run one after the other."""
    page, heads = 64, 1
    lens = [9000, 40]
    d, pool, table = _case([12000, 600], heads, page, "e4m3", 621)
    most = 12000
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ref = _run(d, pool, table, lens, most)
    assert torch.equal(_run(d, pool, table, lens, most, stream=side).view(torch.int16), ref.view(torch.int16))
    ws = torch.empty(gdla.decode_paged_workspace_bytes(2, heads, most), dtype=torch.uint8, device="cuda")
    live = _i32(lens)
    outs, graphs = [torch.empty_like(d["gate"]) for _ in range(2)], []
    for out in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gdla.attn_decode_paged(d["q_sig"], d["q_noise"], pool["k_pages"], pool["v_pages"], table, live, most, d["lam"], d["gate"],
                                   k_scale=pool["k_scale"], v_scale=pool["v_scale"], out=out, workspace=ws)
        graphs.append(g)
    for step, now in enumerate(([9000, 40], [12000, 0], [1, 600], [4097, 513])):
        live.copy_(_i32(now))
        graphs[0].replay()
        if step % 2:
            table[1, :3] = table[0, 5:8]
        graphs[1].replay()
        torch.cuda.synchronize()
        check_decode(outs[1], plain_decode(**d, pool=pool, table=table, page=page, lens=now), now)
        if not step % 2:
            assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))


def test_whole_pages_equal_the_packed_decode():
    """The same keys packed and paged: both decodes against each other."""
    page, heads, lens = 64, 2, [500, 64, 1300]
    d, pool, table = _case(lens, heads, page, "bf16", 631)
    rows = [(int(table[b, u // page]), u % page) for b, n in enumerate(lens) for u in range(n)]
    at, slot = torch.tensor([r[0] for r in rows], device="cuda"), torch.tensor([r[1] for r in rows], device="cuda")
    cu = _i32([0, 500, 564, 1864])
    for window in (0, 128):
        packed = gdla.attn_decode(d["q_sig"], d["q_noise"], pool["k_pages"][at, :, slot].contiguous(),
                                  pool["v_pages"][at, :, slot].contiguous(), cu, 1300, d["lam"], d["gate"], window)
        paged = _run(d, pool, table, lens, window=window)
        # the packed decode rounds probabilities to bf16 (rms 2^-8 / sqrt(12) * 1.44 more)
        assert float((packed.double() - paged.double()).norm() / paged.double().norm()) <= 4e-3
