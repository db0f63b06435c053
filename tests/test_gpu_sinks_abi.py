"""gdla_attn_fwd_sinks and gdla_attn_bwd_sinks with nothing to add, through the C ABI (the Python calls send sinks == 0 to
the plain entry points): sinks == 0, or no window, is the plain call, workspace and all."""
import numpy as np
import pytest
import torch

import differential_latent_attention_b200 as gdla
import gdla_inputs as gi

pytestmark = pytest.mark.gpu

NAMES = ("q_sig", "q_noise", "k", "v", "lam", "gate")
GRADS = ("dq_sig", "dq_noise", "dk", "dv", "dlambda", "dgate")


@pytest.mark.parametrize("window, sinks", [(0, 0), (128, 0), (300, 0), (0, 5), (-3, 128), (700, 5)])
def test_is_the_plain_call(window, sinks):
    seqlens, heads = (700, 33), 2
    t, dout = gi.make_prefill_inputs(seqlens, heads, 31, device="cuda"), gi.make_prefill_grad(seqlens, heads, 31, device="cuda")
    lib, lens = gdla.library(), np.asarray(seqlens, dtype=np.int32)
    stream = torch.cuda.current_stream().cuda_stream
    inputs = [t[x].data_ptr() for x in NAMES]
    plain = window if sinks == 0 else 0                  # a window of 700 reaches over everything
    ref = gdla.attn_fwd(*[t[x] for x in NAMES], seqlens, plain)
    out = torch.full_like(ref, float("nan"))
    assert lib.gdla_attn_fwd_sinks(*inputs, out.data_ptr(), 2, lens.ctypes.data, heads, window, sinks, stream) == 0
    size = lib.gdla_attn_bwd_sinks_workspace_bytes(2, lens.ctypes.data, heads, window, sinks)
    assert size == lib.gdla_attn_bwd_workspace_bytes(sum(seqlens), heads)
    want = gdla.attn_bwd(*[t[x] for x in NAMES], dout, seqlens, plain)
    got = {n: torch.full_like(want[n], float("nan")) for n in GRADS}
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert lib.gdla_attn_bwd_sinks(*inputs, dout.data_ptr(), *[got[n].data_ptr() for n in GRADS], 2, lens.ctypes.data, heads,
                                   window, sinks, ws.data_ptr(), size, stream) == 0
    torch.cuda.synchronize()
    assert gdla.device_error() == 0
    for a, b in [(out, ref)] + [(got[n], want[n]) for n in GRADS]:
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
