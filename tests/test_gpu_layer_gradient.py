"""The documented gradient of the routed 8-bit layer, run as it stands: each step against its formula in 64 bits on
what the step before wrote (tolerances: e4m3_util; the chain itself: test_layer_gradient_host)."""

import pytest

import e4m3_util as u
from readme_blocks import block

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    from transformer_ffn_rmsnorm_gb300 import ffn
    return torch, ffn


@pytest.mark.parametrize("rows", [1, 37, 700])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_example(env, rows, dtype):
    """The last rows are padding: no expert, and no gradient."""
    torch, ffn = env
    d, f, experts, k, dt = 272, 400, 12, 8, getattr(torch, dtype)
    gen = torch.Generator(device="cuda").manual_seed(rows)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")
    v = {"torch": torch, "ffn": ffn, "experts": experts, "x": rnd(rows, d).to(dt), "stream": rnd(rows, d).to(dt),
         "g": (1 + 0.1 * rnd(d)).to(dt), "logits": rnd(rows, experts), "dstream": rnd(rows, d).to(dt),
         "w_gate": rnd(experts, f, d) / d ** 0.5, "w_up": rnd(experts, f, d) / d ** 0.5,
         "w_down": rnd(experts, d, f) / f ** 0.5}
    pad = 3 if rows > 3 else 0
    if pad:
        v["logits"][-pad:] = float("-inf")
    exec(block("ffn.ffn_gateup_e4m3(xs"), v)
    exec(block("ffn.ffn_moe_unsort_backward("), v)
    used, off, pos = int(v["offsets"][-1]), v["offsets"], v["pos"]
    assert used == (rows - pad) * k
    s, at = slice(0, used), pos[:rows - pad].flatten().long()

    # w_tj dstream_t to the pairs' rows, <ys, dstream> to the weights
    g = v["dstream"][:rows - pad].double().repeat_interleave(k, dim=0)
    want = v["w"][:rows - pad].double().flatten()[:, None] * g
    half = torch.finfo(dt).eps / 2
    assert bool(((v["dys"].double()[at] - want).abs() <= want.abs() * (half + 2.0 ** -23)).all())
    t = v["ys"].double()[at] * g
    assert bool(((v["dw"][:rows - pad].double().flatten() - t.sum(1)).abs() <=
                 t.abs().sum(1) * (d / 128 + 12) * 2.0 ** -24).all())
    assert bool((v["dw"][rows - pad:] == 0).all())

    # the products, by the weights' transposes
    for name in ("gate", "up", "down"):
        q, sc = ffn.ffn_quantize_e4m3(v["w_" + name], block_rows=128)
        qt, st = v[{"gate": "wgt", "up": "wut", "down": "wdt"}[name]]
        assert torch.equal(qt.view(torch.uint8), q.view(torch.uint8).transpose(1, 2))
        assert torch.equal(st, sc.transpose(1, 2))

    def check(y, x, w, inn, res=None):
        ref, mag = u.product(torch, (x[0][s], x[1][s]), w, off)
        u.check_linear(torch, y[s], ref, mag, inn, None if res is None else res[s])
    check(v["dh"], ffn.ffn_quantize_e4m3(v["dys"]), v["wdt"], d)
    check(v["gate"], (v["xs"], v["xss"]), v["wg"], d)
    check(v["up"], (v["xs"], v["xss"]), v["wu"], d)
    dgate, dup = ffn.ffn_quantize_e4m3(v["dgate"]), ffn.ffn_quantize_e4m3(v["dup"])
    first = ffn.ffn_linear_e4m3(*dgate, v["wgt"], offsets=off, dtype=torch.float32)
    check(first, dgate, v["wgt"], f)
    check(v["dxs"], dup, v["wut"], f, first)

    # SwiGLU's derivative in 32 bits: a sigmoid and its complement within 2^-21 (4 ulp of 1), six more roundings
    gate, up, dh = (v[n][s].double() for n in ("gate", "up", "dh"))
    sig = torch.sigmoid(gate)
    scale = (dh * up).abs() * (1 + gate.abs()) * 2
    assert bool(((v["dgate"][s].double() - dh * up * sig * (1 + gate * (1 - sig))).abs() <= scale * 2.0 ** -20).all())
    assert bool(((v["dup"][s].double() - dh * gate * sig).abs() <= (dh * gate).abs() * 2.0 ** -20).all())

    # back to the tokens
    t = v["dxs"].double()[at].view(rows - pad, k, d)
    assert bool(((v["dn"][:rows - pad].double() - t.sum(1)).abs() <= t.abs().sum(1) * (k + 2) * 2.0 ** -24).all())
    assert bool((v["dn"][rows - pad:] == 0).all())
    ffn.ffn_device_status()
