"""gdla_cache_append with a cu_seqlens_new that descends, which it does not take: each page of the call is appended to as
by its own sequence or left as it was, and nothing else changes."""
import pytest
import torch

import differential_latent_attention_b200 as gdla
from _paged import new_pool, rand, table_of

pytestmark = pytest.mark.gpu

N, HEADS, PAGE = 200, 2, 16


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _append(pool, table, cu, lens, rows):
    gdla.cache_append(rows["k_nope"], rows["k_rope"], rows["v"], pool["k_pages"], pool["v_pages"], table, cu, lens,
                      k_scale=pool["k_scale"], v_scale=pool["v_scale"])
    torch.cuda.synchronize()
    assert gdla.device_error() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("cu", [[0, 200, 0, 200], [0, 100, 50, 60, 200], [200, 0, 200], [0, 3, 2, 1, 0], [150, 200, 0, 150, 3, 4]])
def test_descending(kind, cu):
    batch = len(cu) - 1
    new = [b - a for a, b in zip(cu, cu[1:])]
    old = [5 * b % 23 for b in range(batch)]
    lens = [max(0, n) + o for n, o in zip(new, old)]
    pool = new_pool(sum((n + PAGE - 1) // PAGE for n in lens) + 2, HEADS, PAGE, kind, 51)
    table = table_of(lens, PAGE, pool["k_pages"].shape[0], seed=52)
    rows = {"k_nope": rand((N, HEADS, 128), 53), "k_rope": rand((N, 64), 54), "v": rand((N, HEADS, 128), 55)}
    alone = []                                   # the pool after each sequence's append alone
    for b in range(batch):
        one = {k: None if v is None else v.clone() for k, v in pool.items()}
        if new[b] > 0:
            own = {k: x[cu[b]:cu[b + 1]] for k, x in rows.items()}
            _append(one, table[b:b + 1].contiguous(), _i32([0, new[b]]), _i32([lens[b]]), own)
        alone.append(one)
    got = {k: None if v is None else v.clone() for k, v in pool.items()}
    _append(got, table, _i32(cu), _i32(lens), rows)
    owner = {int(p): b for b in range(batch) for p in table[b] if p >= 0}
    for name in ("k_pages", "v_pages", "k_scale", "v_scale"):
        if got[name] is None:
            continue
        for p in range(pool["k_pages"].shape[0]):
            x = got[name][p].contiguous().view(torch.uint8)
            same = torch.equal(x, pool[name][p].contiguous().view(torch.uint8))
            assert same or torch.equal(x, alone[owner[p]][name][p].contiguous().view(torch.uint8)), (name, p)
