"""The paged-cache and sinks entry points on the CPU: argument checks of the C ABI (fake, aligned addresses that
these paths never dereference), workspace sizes, and what the binding refuses."""
import ctypes

import numpy as np
import pytest
import torch

import differential_latent_attention_b200 as gdla
from differential_latent_attention_b200 import _build, ops

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


def _cpu_cache(dtype=torch.bfloat16):
    return dict(k_pages=torch.zeros((2, 1, 16, 192), dtype=dtype), v_pages=torch.zeros((2, 1, 16, 128), dtype=dtype),
                block_table=torch.zeros((1, 2), dtype=torch.int32), seqlens_k=torch.ones(1, dtype=torch.int32))


def test_binding_refuses_host_tensors_and_wrong_caches():
    c = _cpu_cache()
    new = dict(k_nope=torch.zeros((1, 1, 128), dtype=torch.bfloat16), k_rope=torch.zeros((1, 64), dtype=torch.bfloat16),
               v=torch.zeros((1, 1, 128), dtype=torch.bfloat16), cu_seqlens_new=torch.tensor([0, 1], dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        gdla.cache_append(**new, **c)
    q = dict(q_sig=torch.zeros((1, 4, 192), dtype=torch.bfloat16), q_noise=torch.zeros((1, 1, 192), dtype=torch.bfloat16),
             lam=torch.zeros(1, 4), gate=torch.zeros((1, 4, 128), dtype=torch.bfloat16), max_seqlen_k=16)
    with pytest.raises(ValueError, match="CUDA"):
        gdla.attn_decode_paged(**q, **c)
    with pytest.raises(ValueError, match="expected k_pages"):
        gdla.attn_decode_paged(**q, **{**c, "k_pages": c["k_pages"][0]})
    with pytest.raises(TypeError):
        gdla.attn_decode_paged(**q, **{**c, "k_pages": None})


class _Fake(torch.Tensor):
    """A tensor that says it is on cuda:0 (no launch is reached with it)."""

    def get_device(self):
        return 0

    @property
    def is_cuda(self):
        return True


def _fake(t):
    return t.as_subclass(_Fake)


def test_row_views():
    """What the appended rows may look like: dense last dimension, strides of whole 16-byte units."""
    k = _fake(torch.zeros((5, 3, 192), dtype=torch.bfloat16))
    nope, rope = k[..., :128], k[:, 0, 128:]
    assert ops._rows(nope, "k_nope", (5, 3, 128), 0)[1:] == (576, 192)
    assert ops._rows(rope, "k_rope", (5, 64), 0)[1:] == (576, 576)
    shared = _fake(torch.zeros((5, 1, 128), dtype=torch.bfloat16)).expand(5, 3, 128)
    assert ops._rows(shared, "v", (5, 3, 128), 0)[1:] == (128, 0)
    one = _fake(torch.zeros((1, 1, 131), dtype=torch.bfloat16))[..., :128]   # a stride that is never used
    assert ops._rows(one, "v", (1, 1, 128), 0)[1:] == (0, 0)
    odd = _fake(torch.zeros((5, 3, 132), dtype=torch.bfloat16))[..., :128]
    with pytest.raises(ValueError, match="multiples of 8"):
        ops._rows(odd, "k_nope", (5, 3, 128), 0)
    with pytest.raises(ValueError, match="contiguous"):
        ops._rows(_fake(torch.zeros((5, 128, 3), dtype=torch.bfloat16)).transpose(1, 2), "v", (5, 3, 128), 0)
    with pytest.raises(ValueError, match="shape"):
        ops._rows(nope, "k_nope", (5, 2, 128), 0)
    with pytest.raises(TypeError):
        ops._rows(_fake(torch.zeros((5, 3, 128))), "v", (5, 3, 128), 0)
    with pytest.raises(ValueError, match="cuda:0"):
        ops._rows(nope, "k_nope", (5, 3, 128), 1)


def test_e4m3_cache_wants_scales_and_bf16_none():
    c = {k: _fake(v) for k, v in _cpu_cache(torch.float8_e4m3fn).items()}
    with pytest.raises(TypeError, match="k_scale"):
        ops._cache(c["k_pages"], c["v_pages"], None, None, c["block_table"], c["seqlens_k"], None)
    b = {k: _fake(v) for k, v in _cpu_cache().items()}
    s = _fake(torch.ones((2, 1)))
    with pytest.raises(ValueError, match="e4m3"):
        ops._cache(b["k_pages"], b["v_pages"], s, s, b["block_table"], b["seqlens_k"], None)
    with pytest.raises(TypeError, match="float8"):
        ops._cache(_fake(torch.zeros((2, 1, 16, 192))), b["v_pages"], None, None, b["block_table"], b["seqlens_k"], None)
