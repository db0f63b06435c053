"""Calls on a stream other than the current one: memory that a call makes itself is ordered with the launch stream before
the call, and with the current stream, where the caller has it, after."""
import pytest
import torch

import differential_latent_attention_b200 as gdla
import gdla_inputs as gi
from _paged import decode_inputs, new_pool, table_of

pytestmark = pytest.mark.gpu

NAMES = ("q_sig", "q_noise", "k", "v", "lam", "gate")
WEIGHTS = ("w_qa", "w_kva", "gamma_q", "gamma_kv", "w_qb", "w_uk", "w_uv", "w_lambda", "w_gate")
SEQLENS = (700, 333)


def _fwd(sinks):
    t = gi.make_prefill_inputs(SEQLENS, 2, 5, device="cuda")
    return lambda stream: {"out": gdla.attn_fwd(*[t[x] for x in NAMES], SEQLENS, 128, sinks=sinks, stream=stream)}


def _bwd(sinks):
    t, dout = gi.make_prefill_inputs(SEQLENS, 2, 6, device="cuda"), gi.make_prefill_grad(SEQLENS, 2, 6, device="cuda")
    return lambda stream: gdla.attn_bwd(*[t[x] for x in NAMES], dout, SEQLENS, 128, sinks=sinks, stream=stream)


def _prologue():
    t = gi.make_prologue_inputs((130,), 1, 7, device="cuda")
    return lambda stream: gdla.prologue(t["x"], *[t[w] for w in WEIGHTS], (130,), stream=stream)


def _decode():
    d = gi.make_decode_inputs((9000, 70), 1, 8, device="cuda")
    return lambda stream: {"out": gdla.attn_decode(d["q_sig"], d["q_noise"], d["k_cache"], d["v_cache"], d["cu_seqlens_k"], 9000,
                                                   d["lam"], d["gate"], stream=stream)}


def _latent():
    d = gi.make_latent_decode_inputs((9000, 70), 1, 9, device="cuda")
    return lambda stream: {"out": gdla.attn_decode_latent(d["q_abs_sig"], d["q_abs_noise"], d["ckv"], d["cu_seqlens_k"], 9000,
                                                          d["w_uv"], d["lam"], d["gate"], stream=stream)}


def _paged(kind):
    lens = [20000, 70]
    d, pool, table = decode_inputs(2, 1, 10), new_pool(320, 1, 64, kind, 10), table_of(lens, 64, 320)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    assert gdla.decode_paged_workspace_bytes(2, 1, 20000) > 0
    return lambda stream: {"out": gdla.attn_decode_paged(d["q_sig"], d["q_noise"], pool["k_pages"], pool["v_pages"], table, n, 20000,
                                                         d["lam"], d["gate"], k_scale=pool["k_scale"], v_scale=pool["v_scale"],
                                                         stream=stream)}


CALLS = {"fwd": lambda: _fwd(0), "fwd sinks": lambda: _fwd(4), "bwd": lambda: _bwd(0), "bwd sinks": lambda: _bwd(4),
         "prologue": _prologue, "decode": _decode, "latent": _latent, "paged bf16": lambda: _paged("bf16"),
         "paged e4m3": lambda: _paged("e4m3")}
BUSY = 800_000_000    # cycles, some 0.4 s


def _copies(got):
    return {n: x.clone() for n, x in got.items()}


def _same(a, b):
    return all(torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)) for n in a)


def _segment_stream(t):
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]


@pytest.mark.parametrize("name", CALLS)
def test_blocks_with_work_pending_are_left_alone(name):
    """Blocks of the sizes that the call needs were freed on the current stream while it still has to write them."""
    call, side = CALLS[name](), torch.cuda.Stream()
    ref = _copies(call(None))
    for x in call(side).values():    # the side stream's own blocks are there, and the kernels that the test runs itself
        x.view(torch.uint8).fill_(0xFF)
    torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    for attempt in range(3):
        got = call(None)
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY << attempt)
        for x in got.values():
            x.view(torch.uint8).fill_(0xFF)
        del got, x
        busy = torch.cuda.Event()
        busy.record()
        got = call(side)
        side.synchronize()
        before = not busy.query()    # the current stream had not come to its writes yet
        torch.cuda.synchronize()
        assert all(_segment_stream(x) == side.cuda_stream for x in got.values())
        assert gdla.device_error() == 0
        assert _same(got, ref)
        if before:
            return
    pytest.skip("the host was too slow for the order of writes that this test wants")


@pytest.mark.parametrize("name", CALLS)
def test_results_freed_before_they_are_read(name):
    """A result of the side stream, read late on the current one and freed at once: the next call does not write over it."""
    call, side = CALLS[name](), torch.cuda.Stream()
    ref = _copies(call(None))
    torch.cuda.synchronize()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    late = _copies(got)
    del got
    with torch.cuda.stream(side):
        for x in call(side).values():
            x.view(torch.uint8).fill_(0xFF)
    torch.cuda.synchronize()
    assert _same(late, ref)


@pytest.mark.parametrize("name", CALLS)
def test_the_current_stream_given(name):
    call = CALLS[name]()
    ref = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    assert _same(call(torch.cuda.current_stream()), ref)
    with torch.cuda.stream(side):
        got = call(None)
        again = call(side)
    side.synchronize()
    assert all(_segment_stream(x) == side.cuda_stream for x in [*got.values(), *again.values()])
    assert _same(got, ref) and _same(again, ref)
    assert gdla.device_error() == 0


@pytest.mark.parametrize("name", CALLS)
def test_captured_on_a_forked_stream(name):
    call = CALLS[name]()
    ref = _copies(call(None))
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        call(side)                    # its result and workspace are freed inside the capture
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
        late = _copies(got)
    for _ in range(2):
        for x in [*got.values(), *late.values()]:
            x.view(torch.uint8).fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert _same(got, ref) and _same(late, ref)
    assert gdla.device_error() == 0
