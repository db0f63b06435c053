"""Windows far longer than every sequence, up to the largest int: the full causal result and gradients, bit for bit."""
import pytest
import torch

import differential_latent_attention_b200 as gdla
import gdla_inputs as gi
from _paged import decode_inputs, new_pool, table_of

pytestmark = pytest.mark.gpu

NAMES = ("q_sig", "q_noise", "k", "v", "lam", "gate")
WINDOWS = (1000, 2 ** 30, 2 ** 31 - 128, 2 ** 31 - 1)


def _same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("window", WINDOWS)
def test_prefill_and_backward(window):
    seqlens = (400, 33, 900)
    t, dout = gi.make_prefill_inputs(seqlens, 2, 21, device="cuda"), gi.make_prefill_grad(seqlens, 2, 21, device="cuda")
    args = [t[x] for x in NAMES]
    for sinks in (0, 7):
        out = torch.full_like(t["gate"], float("nan"))
        gdla.attn_fwd(*args, seqlens, window, out=out, sinks=sinks)
        assert _same(out, gdla.attn_fwd(*args, seqlens))
        ref = gdla.attn_bwd(*args, dout, seqlens)
        grads = {n: torch.full_like(x, float("nan")) for n, x in ref.items()}
        gdla.attn_bwd(*args, dout, seqlens, window, grads=grads, sinks=sinks)
        torch.cuda.synchronize()
        assert gdla.device_error() == 0
        for n in ref:
            assert _same(grads[n], ref[n]), (n, sinks)


@pytest.mark.parametrize("window", WINDOWS)
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_paged_decode(window, kind):
    lens = [900, 1, 333]
    d, pool, table = decode_inputs(3, 2, 22), new_pool(30, 2, 64, kind, 22), table_of(lens, 64, 30)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def run(window, sinks):
        return gdla.attn_decode_paged(d["q_sig"], d["q_noise"], pool["k_pages"], pool["v_pages"], table, n, 900, d["lam"],
                                      d["gate"], window=window, sinks=sinks, k_scale=pool["k_scale"], v_scale=pool["v_scale"])
    for sinks in (0, 7):
        assert _same(run(window, sinks), run(0, 0))
