"""Packed sequences side by side: what one holds, infinities and NaN included, never shows in another's results or
gradients, not in one bit, whatever tiles they share."""
import pytest
import torch

import differential_latent_attention_b200 as gdla
import gdla_inputs as gi

pytestmark = pytest.mark.gpu

NAMES = ("q_sig", "q_noise", "k", "v", "lam", "gate")
MASKS = [(0, 0), (40, 0), (128, 4), (128, 17), (300, 0), (300, 9)]


def _same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("window, sinks", MASKS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("seqlens", [(100, 57, 30), (1, 1, 1), (127, 129, 128), (700, 5, 390), (47, 33, 11, 64, 13, 2)])
def test_prefill_and_backward(seqlens, bad, window, sinks):
    t, dout = gi.make_prefill_inputs(seqlens, 2, 41, device="cuda"), gi.make_prefill_grad(seqlens, 2, 41, device="cuda")
    out = gdla.attn_fwd(*[t[x] for x in NAMES], seqlens, window, sinks=sinks)
    g = gdla.attn_bwd(*[t[x] for x in NAMES], dout, seqlens, window, sinks=sinks)
    start = 0
    for n in seqlens[:4]:
        own = torch.zeros(sum(seqlens), dtype=torch.bool, device="cuda")
        own[start:start + n] = True
        start += n
        dirty = {x: torch.where(own.view(-1, *[1] * (y.dim() - 1)), torch.full_like(y, bad), y) for x, y in t.items()}
        bad_dout = torch.where(own[:, None, None], torch.full_like(dout, bad), dout)
        got = gdla.attn_fwd(*[dirty[x] for x in NAMES], seqlens, window, sinks=sinks)
        grads = gdla.attn_bwd(*[dirty[x] for x in NAMES], bad_dout, seqlens, window, sinks=sinks)
        torch.cuda.synchronize()
        assert gdla.device_error() == 0
        assert _same(got[~own], out[~own]), n
        for name in g:
            assert _same(grads[name][~own], g[name][~own]), (n, name)
