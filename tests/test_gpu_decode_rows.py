"""gdla_attn_decode_paged held to 64 bits sequence by sequence, and its e4m3 values over every size of V.

A batch's longest sequences have the smallest outputs (about 1 / sqrt(keys)), so one norm over the batch hardly sees
them. Here each sequence and KV head, 512 outputs, is held to its own size. The output's rounding has rms 1.63e-3 over
evenly spread significands (2^-8 / sqrt(12) * 1.44); the rms over 512 values varies by some 5 % of that, six of which make
2.1e-3; with 4 * 2^-12 for what else is rounded (f16 probabilities and turned queries, 2^-12 each, where H_S and
lambda H_N cancel by half), sqrt(2.1e-3^2 + 9.8e-4^2) = 2.33e-3."""
import pytest
import torch

from _paged import BF16_HALF, GROUP, decode_inputs, new_pool, plain_decode
from test_gpu_decode_paged import EDGES, _case, _run

pytestmark = pytest.mark.gpu

ROWS_RMS = 2.4e-3


def check_rows(got, ref, what):
    """Every (sequence, KV head) by itself; a sequence without keys is zero."""
    got = got.double()
    assert torch.isfinite(got).all(), what
    a, b = [x.view(x.shape[0], -1, GROUP * 128) for x in (got, ref)]
    norm = b.norm(dim=-1)
    assert bool((a[norm == 0] == 0).all()), what
    some = norm > 0
    rms = ((a - b).norm(dim=-1)[some] / norm[some])
    assert float(rms.max()) <= ROWS_RMS, (what, float(rms.max()))
    top = b.abs().amax(-1, keepdim=True)
    assert bool(((a - b).abs() <= BF16_HALF * b.abs() + 1e-2 * top).all()), what


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_edge_lengths(kind, page):
    d, pool, table = _case(EDGES, 2, page, kind, 700 + page)
    check_rows(_run(d, pool, table, EDGES), plain_decode(**d, pool=pool, table=table, page=page, lens=EDGES), (kind, page))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 1), (16, 4), (100, 17), (128, 4), (129, 128), (1000, 5), (5000, 64)])
def test_windows_and_sinks(kind, window, sinks):
    d, pool, table = _case(EDGES, 3, 16, kind, 800 + window)
    kw = dict(window=window, sinks=sinks)
    check_rows(_run(d, pool, table, EDGES, **kw), plain_decode(**d, pool=pool, table=table, page=16, lens=EDGES, **kw), (kind, kw))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("window, sinks", [(0, 0), (130, 9)])
def test_turned_queries(kind, window, sinks):
    lens = [1, 70, 513, 4001]
    d, pool, table = _case(lens, 2, 64, kind, 900)
    kw = dict(window=window, sinks=sinks, rotate=True)
    check_rows(_run(d, pool, table, lens, **kw), plain_decode(**d, pool=pool, table=table, page=64, lens=lens, **kw), (kind, kw))


@pytest.mark.parametrize("lens, heads", [([1, 17, 300, 2049], 2), ([4096], 16), ([20011, 77], 1), ([300] * 320, 2)])
def test_values_times_a_power_of_two(lens, heads):
    """Every V scale times 2^e: every output times 2^e, bit for bit. One CTA, clusters, several clusters, small CTAs."""
    d, pool, table = _case(lens, heads, 32, "e4m3", 921)
    ref = _run(d, pool, table, lens)
    for e in (-60, -33, -12, -9, -4, 3, 8, 40):
        moved = {**pool, "v_scale": pool["v_scale"] * 2.0 ** e}
        got = _run(d, moved, table, lens)
        assert torch.equal(got.float(), ref.float() * 2.0 ** e), e


@pytest.mark.parametrize("e", [-118, -100, 110])
def test_values_near_the_ends_of_fp32(e):
    """V scales down to 2^-127 (an fp32 subnormal, smaller than any that the append writes) and up to 2^104."""
    lens = [1, 17, 300, 2049]
    d, pool, table = _case(lens, 2, 32, "e4m3", 931)
    pool["v_scale"] *= 2.0 ** e
    check_rows(_run(d, pool, table, lens), plain_decode(**d, pool=pool, table=table, page=32, lens=lens), e)


def _dominated(above, apart, size, neighbours):
    """160 sequences of 2,000 keys (one CTA an item: every warp's sums matter) whose first key scores `above` log2 units
    over the others by dim 0 alone, and whose first page has no values and a V scale 2^apart times the other pages'."""
    page, n, batch, heads = 16, 2000, 160, 2
    d = decode_inputs(batch, heads, 941)
    pool = new_pool(n // page + 1, heads, page, "e4m3", 942)
    table = torch.randperm(n // page, device="cuda", generator=torch.Generator(device="cuda").manual_seed(943))
    table = table.to(torch.int32).expand(batch, -1).contiguous()
    first = int(table[0, 0])
    d["q_sig"][..., 0] = d["q_noise"][..., 0] = 16.0
    pool["k_pages"].view(torch.uint8)[..., 0] = 0
    pool["v_scale"][:] = 2.0 ** (size - 8)
    pool["v_scale"][first] *= 2.0 ** apart
    pool["v_pages"][first] = 0
    pool["k_scale"][first] = 2.0 ** -4
    if not neighbours:
        pool["k_pages"][first] = 0
    row = torch.zeros(192, device="cuda")
    row[0] = above * 0.6931 * 192 ** 0.5 / 16 * 16       # dim 0 of the key, in codes of the page's scale
    pool["k_pages"][first, :, 0] = row.to(torch.float8_e4m3fn)
    got = _run(d, pool, table, [n] * batch)[:3]
    some = {k: x[:3] for k, x in d.items()}
    ref = plain_decode(**some, pool=pool, table=table[:3], page=page, lens=[n] * 3)
    other = torch.arange(pool["v_pages"].shape[0], device="cuda") != first
    v = pool["v_pages"].double()[other] * pool["v_scale"].double()[other][..., None, None]
    return got, ref, n, float(v.square().mean().sqrt())


ABOVE = pytest.mark.parametrize("above", [10, 14, 18])          # of the dominating key over the others, in log2
APART = pytest.mark.parametrize("apart", [-7, -2, 0, 3, 7, 12])  # of its page's V scale over the other pages', in log2
SIZE = pytest.mark.parametrize("size", [-20, 0])               # of all V scales


@ABOVE
@APART
@SIZE
def test_a_dominating_key_without_a_value(above, apart, size):
    """One key takes nearly all of the weight and has no value, as an attention sink: the output is what the thousands of
    others, a 2^-10 to 2^-18 of the weight each, add up to."""
    got, ref, _, _ = _dominated(above, apart, size, False)
    check_rows(got, ref, (above, apart, size))


@ABOVE
@APART
@SIZE
def test_dominating_neighbours_without_a_value(above, apart, size):
    """The same with 15 neighbours in the key's page whose own scores reach a hundred log2 units in one direction or the
    other: they leave the others as little as 2^-70 of the weight, under what an f16 probability holds.

    A probability of the kernel, relative to the running maximum, is off by 2^-12 of itself or, under f16's normal
    numbers, by at most 2^-25 in f16; with the bias of 2^9 and a V scale's ratio of 2^-4 that is 2^-30 of the maximum. Over n
    keys whose values have independent signs H is off by sqrt(n) 2^-30 rms(V) (its sum of weights is at least one), D
    by sqrt(2) times that, the 512 outputs of a sequence and KV head by sqrt(512) times that in norm; twice that, as the
    four heads share 128 values. Beside ROWS_RMS of the output."""
    got, ref, n, v = _dominated(above, apart, size, True)
    got = got.double()
    assert torch.isfinite(got).all()
    a, b = [x.view(3, -1, GROUP * 128) for x in (got, ref)]
    step = 2 * (2 * n * 512) ** 0.5 * 2.0 ** -30 * v
    assert bool(((a - b).norm(dim=-1) <= ROWS_RMS * b.norm(dim=-1) + step).all()), (above, apart, size)
