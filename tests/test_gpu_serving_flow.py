"""The operators as a server uses them together: prefill of the prompts with sinks, their keys into the paged cache,
then decode steps (append one token, attend over the cache) under the same mask, eagerly and as one captured graph."""
import pytest
import torch

import differential_latent_attention_b200 as gdla
import gdla_inputs as gi
from _paged import check_decode, plain_decode, plain_prefill, rand, table_of, turn

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _layer(total, heads, seed):
    """A layer's projections for whole sequences, keys and queries before the rotation."""
    n = sum(total)
    t = gi.make_prefill_inputs(total, heads, seed, device="cuda")
    t["k_rope"] = rand((n, 64), seed + 1)
    pos = torch.cat([torch.arange(x, device="cuda") for x in total])
    raw = {"q_sig": t["q_sig"].clone(), "q_noise": t["q_noise"].clone()}
    for x in ("q_sig", "q_noise"):
        t[x][..., 128:] = turn(t[x][..., 128:], pos).to(torch.bfloat16)
    t["k"][..., 128:] = turn(t["k_rope"], pos).to(torch.bfloat16)[:, None]
    return t, raw


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("window, sinks", [(128, 4), (0, 0)])
def test_prompts_then_steps(kind, window, sinks):
    heads, page, prompt, steps = 2, 16, [200, 3, 77], 20
    total = [p + steps for p in prompt]
    t, raw = _layer(total, heads, 900)
    start = [0, total[0], total[0] + total[1]]
    whole = plain_prefill(t, total, window, sinks)
    pages = sum((x + page - 1) // page for x in total) + 2
    table = table_of(total, page, pages)
    if kind == "bf16":
        k_pages = torch.full((pages, heads, page, 192), float("nan"), dtype=torch.bfloat16, device="cuda")
        v_pages = torch.full((pages, heads, page, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        ks = vs = None
    else:
        k_pages = torch.full((pages, heads, page, 192), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        v_pages = torch.full((pages, heads, page, 128), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        ks, vs = torch.full((pages, heads), 3e30, device="cuda"), torch.full((pages, heads), 3e30, device="cuda")
    # prompts: prefill, and their keys (turned already) into the cache as views of k
    rows = torch.cat([torch.arange(s, s + p) for s, p in zip(start, prompt)]).cuda()
    part = {x: t[x][rows].contiguous() for x in ("q_sig", "q_noise", "k", "v", "lam", "gate")}
    out = gdla.attn_fwd(*part.values(), prompt, window, sinks=sinks)
    diff = (out.double() - whole[rows]).norm() / whole[rows].norm()
    assert float(diff) <= 5e-3
    gdla.cache_append(part["k"][..., :128], part["k"][:, 0, 128:], part["v"], k_pages, v_pages, table,
                      _i32([0] + list(torch.tensor(prompt).cumsum(0))), _i32(prompt), k_scale=ks, v_scale=vs, rotate=False)
    # steps: one graph, captured on the first, replayed for the others
    lens, cu = _i32(prompt), _i32([0, 1, 2, 3])
    live = {"k_nope": torch.empty((3, heads, 128), dtype=torch.bfloat16, device="cuda"),
            "k_rope": torch.empty((3, 64), dtype=torch.bfloat16, device="cuda"),
            "v": torch.empty((3, heads, 128), dtype=torch.bfloat16, device="cuda"),
            "q_sig": torch.empty((3, 4 * heads, 192), dtype=torch.bfloat16, device="cuda"),
            "q_noise": torch.empty((3, heads, 192), dtype=torch.bfloat16, device="cuda"),
            "lam": torch.empty((3, 4 * heads), device="cuda"),
            "gate": torch.empty((3, 4 * heads, 128), dtype=torch.bfloat16, device="cuda")}
    result = torch.empty_like(live["gate"])

    def step():
        lens.add_(1)
        gdla.cache_append(live["k_nope"], live["k_rope"], live["v"], k_pages, v_pages, table, cu, lens, k_scale=ks, v_scale=vs)
        gdla.attn_decode_paged(live["q_sig"], live["q_noise"], k_pages, v_pages, table, lens, max(total), live["lam"],
                               live["gate"], window=window, sinks=sinks, k_scale=ks, v_scale=vs, rotate=True, out=result)

    def load(i):
        at = torch.tensor([s + p + i for s, p in zip(start, prompt)], device="cuda")
        live["k_nope"].copy_(t["k"][at, :, :128])
        live["k_rope"].copy_(t["k_rope"][at])
        for x in ("v", "lam", "gate"):
            live[x].copy_(t[x][at])
        for x in ("q_sig", "q_noise"):
            live[x].copy_(raw[x][at])
        return at

    graph = None
    for i in range(steps):
        at = load(i)
        if graph is None:
            step()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        now = [p + i + 1 for p in prompt]
        assert lens.tolist() == now
        pool = {"k_pages": k_pages, "v_pages": v_pages, "k_scale": ks, "v_scale": vs}
        ref = plain_decode(live["q_sig"], live["q_noise"], pool, table, page, now, live["lam"], live["gate"], window, sinks, True)
        check_decode(result, ref, (kind, i))
        if kind == "bf16":
            # and the rows of the whole prefill: queries there were rounded to bf16 after the turn, here not
            rel = float((result.double() - whole[at]).norm() / whole[at].norm())
            assert rel <= 5e-3, (i, rel)
    if kind == "e4m3":
        # e4m3's own rounding (2^-4 at most, rms 2^-4 / sqrt(12) * 1.44 = 2.6e-2) of keys and values, seen through a
        # softmax over one key and more: within a tenth of the whole
        rel = float((result.double() - whole[at]).norm() / whole[at].norm())
        assert rel <= 0.1, rel
    assert gdla.device_error() == 0


def test_prologue_into_the_cache():
    """The prologue's outputs as they come: k goes in as two views, the last token decodes to the prefill's last row."""
    seqlens, heads, page = (100, 37), 2, 32
    p = gi.make_prologue_inputs(seqlens, heads, 5, device="cuda")
    o = gdla.prologue(p["x"], *[p[w] for w in ("w_qa", "w_kva", "gamma_q", "gamma_kv", "w_qb", "w_uk", "w_uv", "w_lambda", "w_gate")],
                      seqlens)
    pages = 8
    k_pages = torch.zeros((pages, heads, page, 192), dtype=torch.bfloat16, device="cuda")
    v_pages = torch.zeros((pages, heads, page, 128), dtype=torch.bfloat16, device="cuda")
    table = table_of(seqlens, page, pages)
    gdla.cache_append(o["k"][..., :128], o["k"][:, 0, 128:], o["v"], k_pages, v_pages, table, _i32([0, 100, 137]), _i32(seqlens),
                      rotate=False)
    last = torch.tensor([99, 136], device="cuda")
    for window, sinks in ((0, 0), (16, 4)):
        pre = gdla.attn_fwd(o["q_sig"], o["q_noise"], o["k"], o["v"], o["lam"], o["gate"], seqlens, window, sinks=sinks)
        dec = gdla.attn_decode_paged(o["q_sig"][last], o["q_noise"][last], k_pages, v_pages, table, _i32(seqlens), 100,
                                     o["lam"][last], o["gate"][last], window=window, sinks=sinks)
        rel = float((dec.double() - pre[last].double()).norm() / pre[last].double().norm())
        assert rel <= 4e-3, (window, rel)
