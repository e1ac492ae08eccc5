"""A batch in pieces: rows of the router's logits, indices and weights that do
not start on 16 bytes (6 slots of 4 bytes a token), through routing and both
routed blocks, give what the whole batch gives."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("start,end", [(1, 40), (3, 4), (37, 333), (1, 2)])
@pytest.mark.parametrize("dtype,experts", [("float32", 61), ("bfloat16", 33), ("float16", 40)])
def test_rows_in_pieces(start, end, dtype, experts):
    import torch
    import test_gpu_moe as m
    import test_gpu_moe_q4 as m4
    from transformer_ffn_rmsnorm_gb300 import ffn
    rows, d, f, k = 333, 128, 192, 6
    gen = torch.Generator(device="cuda").manual_seed(experts)
    logits = torch.randn(rows, experts, generator=gen, device="cuda").to(getattr(torch, dtype))
    bias = 0.1 * torch.randn(experts, generator=gen, device="cuda")
    s = slice(start, end)
    idx, w = ffn.ffn_moe_route(logits, k, bias=bias, flags=ffn.FFN_ROUTE_RENORM)
    oi, ow = torch.full_like(idx, -5), torch.full_like(w, -5.0)
    ffn.ffn_moe_route(logits[s], k, bias=bias, flags=ffn.FFN_ROUTE_RENORM, idx=oi[s], weights=ow[s])
    assert torch.equal(oi[s], idx[s]) and torch.equal(ow[s], w[s])
    oi[s], ow[s] = -5, -5.0
    assert bool((oi == -5).all()) and bool((ow == -5).all())
    x, _, _, wg, wu, wd, res = m.make(torch, rows, d, f, experts, k, torch.bfloat16)
    y = ffn.ffn_moe_forward(x[s], idx[s], w[s], wg, wu, wd, res=res[s])
    m.check(torch, y, *m.reference(torch, x[s], idx[s], w[s], wg, wu, wd, res[s], False))
    x, _, _, packed, values, res = m4.make(torch, rows, d, f, experts, k)
    y = ffn.ffn_moe_forward_q4(x[s], idx[s], w[s], *packed, ffn=f, res=res[s])
    m4.check(torch, y, *m4.reference(torch, x[s], idx[s], w[s], values, res[s]))
    ffn.ffn_device_status()
