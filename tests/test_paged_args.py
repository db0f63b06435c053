"""The paged-cache and sinks entry points on the CPU: argument checks of the C ABI (fake, aligned addresses that
these paths never dereference), workspace sizes, and what the binding refuses."""
import ctypes

import numpy as np
import pytest
import torch

import differential_latent_attention_b200 as gdla
from differential_latent_attention_b200 import _build

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gdla.library()


def _append(lib, **kw):
    a = dict(kn=FAKE, kn_t=128, kn_h=128, kr=FAKE, kr_t=64, v=FAKE, v_t=128, v_h=128, kp=FAKE, vp=FAKE, ks=FAKE,
             vs=FAKE, kind=1, pages=4, page=64, table=FAKE, width=2, cu=FAKE, n=1, lens=FAKE, batch=1, heads=1, rot=1)
    a.update(kw)
    return lib.gdla_cache_append(*a.values(), None)


def test_append_argument_checks(lib):
    assert _append(lib, n=0) == 0                                     # nothing to do
    for name in ("kn", "kr", "v", "kp", "vp"):
        assert _append(lib, **{name: 0}) == 1
        assert _append(lib, **{name: FAKE + 8}) == 1
    for name in ("ks", "vs", "table", "cu", "lens"):
        assert _append(lib, **{name: 0}) == 1
        assert _append(lib, **{name: FAKE + 2}) == 1
    assert _append(lib, kind=0, ks=0, vs=0, n=0) == 0                 # bf16 pages have no scales
    assert _append(lib, kind=2) == 1
    for name in ("kn_t", "kn_h", "kr_t", "v_t", "v_h"):
        assert _append(lib, **{name: -8}) == 1
        assert _append(lib, **{name: 12}) == 1
    for page in (0, 8, 48, 256):
        assert _append(lib, page=page) == 2
    assert _append(lib, heads=0) == 2
    assert _append(lib, heads=65) == 2
    for name in ("pages", "width", "batch"):
        assert _append(lib, **{name: 0}) == 1
    assert _append(lib, n=-1) == 1
    assert _append(lib, pages=2 ** 30, heads=2) == 1                  # num_pages * num_kv_heads >= 2^31
    assert _append(lib, width=2 ** 25) == 1                           # positions past 2^31
    assert _append(lib, batch=2 ** 24) == 1


def _decode(lib, **kw):
    a = dict(qs=FAKE, qn=FAKE, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, kind=1, pages=4, page=64, table=FAKE, width=2,
             lens=FAKE, most=128, lam=FAKE, gate=FAKE, out=FAKE, batch=1, heads=1, window=0, sinks=0, rot=0, ws=0, wsb=0)
    a.update(kw)
    return lib.gdla_attn_decode_paged(*a.values(), None)


def test_decode_argument_checks(lib):
    for name in ("qs", "qn", "kp", "vp", "lam", "gate", "out"):
        assert _decode(lib, **{name: 0}) == 1
        assert _decode(lib, **{name: FAKE + 8}) == 1
    for name in ("ks", "vs", "table", "lens"):
        assert _decode(lib, **{name: 0}) == 1
        assert _decode(lib, **{name: FAKE + 2}) == 1
    assert _decode(lib, page=24) == 2
    assert _decode(lib, heads=65) == 2
    assert _decode(lib, kind=-1) == 1
    assert _decode(lib, most=0) == 1
    assert _decode(lib, most=129) == 1                                # more than the table holds
    assert _decode(lib, sinks=-1) == 1
    assert _decode(lib, sinks=129) == 2
    need = lib.gdla_decode_paged_workspace_bytes(1, 1, 1 << 20, 0, 0)
    assert need > 0
    big = dict(most=1 << 20, width=1 << 14)
    assert _decode(lib, **big) == 3
    assert _decode(lib, ws=FAKE, wsb=need - 1, **big) == 3
    assert _decode(lib, ws=FAKE + 16, wsb=need, **big) == 3


def test_decode_workspace_sizes(lib):
    size = lib.gdla_decode_paged_workspace_bytes
    assert size(64, 16, 32768, 0, 0) == 0       # many items: one cluster each
    assert size(1, 16, 4096, 0, 0) == 0
    assert size(1, 1, 1 << 20, 128, 4) == 0     # a window: few keys
    per = 5 * (128 + 2) * 4                     # five heads' O, maximum and sum in fp32, per cluster
    assert size(1, 1, 1 << 20, 0, 0) % per == 0
    assert 2 * per <= size(1, 1, 1 << 20, 0, 0) <= 64 * per
    for bad in ((0, 1, 64, 0, 0), (1, 0, 64, 0, 0), (1, 65, 64, 0, 0), (1, 1, 0, 0, 0), (1, 1, 64, 0, -1), (1, 1, 64, 0, 129)):
        assert size(*bad) == 0


def _sinks(lib, lens, bwd, heads=1, window=128, sinks=4, ptrs=None, ws=FAKE, wsb=1 << 40):
    arr = np.asarray(lens, dtype=np.int32)
    p = ptrs or [FAKE] * (13 if bwd else 7)
    if bwd:
        return lib.gdla_attn_bwd_sinks(*p, len(arr), arr.ctypes.data_as(ctypes.c_void_p), heads, window, sinks, ws, wsb, None)
    return lib.gdla_attn_fwd_sinks(*p, len(arr), arr.ctypes.data_as(ctypes.c_void_p), heads, window, sinks, None)


@pytest.mark.parametrize("bwd", [False, True])
def test_sinks_argument_checks(lib, bwd):
    assert _sinks(lib, [4], bwd, heads=0) == 2
    assert _sinks(lib, [4, -1], bwd) == 1
    assert _sinks(lib, [0, 0], bwd) == 0
    assert _sinks(lib, [4], bwd, sinks=-1) == 1
    assert _sinks(lib, [4], bwd, sinks=129) == 2
    assert _sinks(lib, [24 * 2 ** 20 + 1], bwd) == 2
    for i in range(13 if bwd else 7):
        p = [FAKE] * (13 if bwd else 7)
        p[i] = 0
        assert _sinks(lib, [4], bwd, ptrs=p) == 1
        p[i] = FAKE + 8
        assert _sinks(lib, [4], bwd, ptrs=p) == 1


def test_sinks_workspace(lib):
    size = gdla.attn_bwd_sinks_workspace_bytes
    base = gdla.attn_bwd_workspace_bytes
    assert size((4096,), 16, 0, 4) == base(4096, 16)          # no window: no sinks
    assert size((4096,), 16, 5000, 4) == base(4096, 16)       # a window over everything
    assert size((200, 100) * 40, 2, 128, 4) == base(12000, 2)  # every row within the first key tile's reach
    assert size((200, 100), 2, 128, 4) > base(300, 2)          # few key tiles: cut, so with partials
    assert size((4096,), 16, 128, 4) > base(4096, 16)
    assert size((4096,), 16, 128, 8) > size((4096,), 16, 128, 4)
    assert size((4096,), 65, 128, 4) == 0
    assert size((4096,), 16, 128, 129) == 0
    assert size((-1,), 16, 128, 4) == 0
    need = size((4096,), 2, 128, 4)
    assert _sinks(lib, [4096], True, heads=2, ws=0) == 3
    assert _sinks(lib, [4096], True, heads=2, wsb=need - 1) == 3
    assert _sinks(lib, [4096], True, heads=2, ws=FAKE + 16) == 3


# The binding looks at the device last, so on host tensors every other check can be seen; a call that passes them all
# ends with the refusal of host tensors.
def _cache(dtype=torch.bfloat16, pages=2, heads=3, page=16, batch=2, width=2):
    c = dict(k_pages=torch.zeros((pages, heads, page, 192), dtype=dtype), v_pages=torch.zeros((pages, heads, page, 128), dtype=dtype),
             block_table=torch.zeros((batch, width), dtype=torch.int32), seqlens_k=torch.ones(batch, dtype=torch.int32))
    if dtype == torch.float8_e4m3fn:
        c.update(k_scale=torch.ones((pages, heads)), v_scale=torch.ones((pages, heads)))
    return c


def _new(n=5, heads=3, batch=2):
    bf = torch.bfloat16
    return dict(k_nope=torch.zeros((n, heads, 128), dtype=bf), k_rope=torch.zeros((n, 64), dtype=bf),
                v=torch.zeros((n, heads, 128), dtype=bf), cu_seqlens_new=torch.zeros(batch + 1, dtype=torch.int32))


def _query(batch=2, heads=3):
    bf = torch.bfloat16
    return dict(q_sig=torch.zeros((batch, 4 * heads, 192), dtype=bf), q_noise=torch.zeros((batch, heads, 192), dtype=bf),
                lam=torch.zeros(batch, 4 * heads), gate=torch.zeros((batch, 4 * heads, 128), dtype=bf), max_seqlen_k=16)


KINDS = [torch.bfloat16, torch.float8_e4m3fn]


@pytest.mark.parametrize("dtype", KINDS)
def test_binding_refuses_host_tensors_last(dtype):
    with pytest.raises(ValueError, match="CUDA device"):
        gdla.cache_append(**_new(), **_cache(dtype))
    with pytest.raises(ValueError, match="CUDA device"):
        gdla.attn_decode_paged(**_query(), **_cache(dtype), window=128, sinks=4, rotate=True)


@pytest.mark.parametrize("call, base", [(gdla.cache_append, _new), (gdla.attn_decode_paged, _query)])
def test_binding_checks_the_cache(call, base):
    good = {**base(), **_cache(torch.float8_e4m3fn)}
    for name, value, error in (
            ("k_pages", None, TypeError), ("block_table", 3, TypeError),
            ("k_pages", good["k_pages"][0], ValueError), ("block_table", good["block_table"][0], ValueError),
            ("k_pages", good["k_pages"].float(), TypeError),                     # neither cache type
            ("k_pages", good["k_pages"][..., :128].contiguous(), ValueError),
            ("v_pages", torch.zeros((2, 3, 16, 128), dtype=torch.bfloat16), TypeError),
            ("v_pages", good["v_pages"][:1], ValueError),
            ("v_pages", torch.zeros((2, 3, 128, 16), dtype=torch.float8_e4m3fn).transpose(2, 3), ValueError),
            ("k_scale", None, TypeError), ("v_scale", None, TypeError), ("k_scale", torch.ones(2, 4), ValueError),
            ("k_scale", torch.ones((2, 3), dtype=torch.float64), TypeError),
            ("block_table", good["block_table"].long(), TypeError),
            ("seqlens_k", good["seqlens_k"].long(), TypeError), ("seqlens_k", torch.ones(3, dtype=torch.int32), ValueError)):
        with pytest.raises(error) as e:
            call(**{**good, name: value})
        assert "CUDA device" not in str(e.value), name
    with pytest.raises(ValueError, match="e4m3"):
        call(**{**base(), **_cache(), "k_scale": torch.ones((2, 3)), "v_scale": torch.ones((2, 3))})


def test_append_checks_its_rows():
    """Dense last dimension, strides of whole 16-byte units, one row's stride says nothing."""
    wide = torch.zeros((5, 3, 192), dtype=torch.bfloat16)
    shared = torch.zeros((5, 1, 128), dtype=torch.bfloat16).expand(5, 3, 128)
    c = _cache()
    for rows in (dict(k_nope=wide[..., :128], k_rope=wide[:, 0, 128:]), dict(v=shared)):
        with pytest.raises(ValueError, match="CUDA device"):
            gdla.cache_append(**{**_new(), **rows}, **c)
    one = torch.zeros((1, 1, 131), dtype=torch.bfloat16)[..., :128]
    with pytest.raises(ValueError, match="CUDA device"):
        gdla.cache_append(**{**_new(1, 1), "k_nope": one, "v": one}, **_cache(heads=1))
    odd = torch.zeros((5, 3, 132), dtype=torch.bfloat16)[..., :128]
    for rows, error, match in (
            (dict(k_nope=odd), ValueError, "multiples of 8"), (dict(v=odd), ValueError, "multiples of 8"),
            (dict(k_rope=torch.zeros((5, 68), dtype=torch.bfloat16)[:, :64]), ValueError, "multiples of 8"),
            (dict(v=torch.zeros((5, 128, 3), dtype=torch.bfloat16).transpose(1, 2)), ValueError, "contiguous"),
            (dict(k_nope=wide[:, :2, :128]), ValueError, "k_nope: expected shape"),
            (dict(k_rope=torch.zeros((4, 64), dtype=torch.bfloat16)), ValueError, "k_rope: expected shape"),
            (dict(v=torch.zeros((5, 3, 128))), TypeError, "v: expected BFloat16"),
            (dict(v=None), TypeError, "v must be"),
            (dict(cu_seqlens_new=torch.zeros(2, dtype=torch.int32)), ValueError, "cu_seqlens_new")):
        with pytest.raises(error, match=match):
            gdla.cache_append(**{**_new(), **rows}, **c)


def test_decode_checks_its_queries():
    c, q = _cache(), _query()
    for name, value, error in (
            ("q_sig", q["q_sig"][:, :11], ValueError), ("q_noise", q["q_noise"].float(), TypeError),
            ("q_sig", torch.zeros((2, 192, 12), dtype=torch.bfloat16).transpose(1, 2), ValueError),
            ("lam", q["lam"].double(), TypeError), ("gate", q["gate"][..., :64], ValueError),
            ("max_seqlen_k", "long", TypeError), ("max_seqlen_k", 2 ** 40, ValueError), ("window", 1.5, TypeError)):
        with pytest.raises(error) as e:
            gdla.attn_decode_paged(**{**q, name: value}, **c)
        assert "CUDA device" not in str(e.value), name
