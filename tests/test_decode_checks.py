"""The bounds that the paged decode is held to see a slip in the longest sequence of a batch (on the CPU: the slip is in
the oracle, the output is the right one rounded as the kernels do)."""
import pytest
import torch

from _paged import decode_inputs, new_pool, plain_decode, table_of
from test_gpu_decode_paged import EDGES
from test_gpu_decode_rows import check_rows


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 128])
def test_a_dropped_key_shows(kind, page):
    heads = 2
    pages = sum((n + page - 1) // page for n in EDGES) + 2
    d = decode_inputs(len(EDGES), heads, 700 + page, device="cpu")
    pool = new_pool(pages, heads, page, kind, 700 + page, device="cpu")
    table = table_of(EDGES, page, pages, seed=700 + page, device="cpu")
    ref = plain_decode(**d, pool=pool, table=table, page=page, lens=EDGES)
    got = ref.to(torch.bfloat16)
    check_rows(got, ref, "the right output")
    for b, n in enumerate(EDGES):
        if n < 100:
            continue
        short = list(EDGES)
        short[b] = n - 1
        with pytest.raises(AssertionError):
            check_rows(got, plain_decode(**d, pool=pool, table=table, page=page, lens=short), n)
