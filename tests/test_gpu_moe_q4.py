"""ffn_moe_forward_q4 against the formula in 64 bits on the dequantised weights.

The bound of every element as in test_gpu_moe (products' fp32 sums, h, y),
with three more roundings to fp16, each at most half a step, 2^-11 of the
value: a weight (u - 8) s (at most 14 significant bits; below fp16's normal
range it is a multiple of 2^-24 and exact), an activation of x (a bf16 value:
exact in fp16's normal range, below it half of 2^-24), and h, stored 2^-8
(half of 2^-24 x 2^8 below the normal range).  So each product's terms carry
2^-11 for the weight beside K 2^-23 for the sum."""

import pytest

from gpu_util import BF16_MAX, BF16_MEAN

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    from transformer_ffn_rmsnorm_gb300 import ffn
    return torch, ffn


def pack(torch, q, s):
    """[..., in] codes -8..7 and [..., in/32] scales in the device layout."""
    lead, inn = q.shape[:-1], q.shape[-1]
    blocks, ngrp = inn // 32, -(-inn // 128)
    u = (q + 8).to(torch.uint8).reshape(*lead, blocks, 32)
    full = torch.zeros(*lead, 4 * ngrp, 16, dtype=torch.uint8, device=q.device)
    full[..., :blocks, :] = u[..., :16] | (u[..., 16:] << 4)
    qs = full.reshape(*lead, ngrp, 4, 4, 4).transpose(-3, -2).reshape(*lead, 64 * ngrp)
    sc = torch.zeros(*lead, 4 * ngrp, dtype=torch.float16, device=q.device)
    sc[..., :blocks] = s
    return qs.contiguous(), sc.contiguous()


def weight(torch, gen, experts, out, inn, scale=1.0):
    q = torch.randint(-8, 8, (experts, out, inn), generator=gen, device="cuda", dtype=torch.int8)
    s = ((0.5 + torch.rand(experts, out, inn // 32, generator=gen, device="cuda")) * (scale * 0.2 / inn ** 0.5)).half()
    return pack(torch, q, s), q.double() * s.double().repeat_interleave(32, dim=-1)


def make(torch, rows, d, f, experts, k, seed=0, idx=None):
    gen = torch.Generator(device="cuda").manual_seed(seed + rows)
    x = torch.randn(rows, d, generator=gen, device="cuda").bfloat16()
    res = torch.randn(rows, d, generator=gen, device="cuda").bfloat16()
    if idx is None:
        idx = torch.rand(rows, experts, generator=gen, device="cuda").topk(k, dim=1).indices
    w = torch.softmax(torch.randn(rows, k, generator=gen, device="cuda"), dim=1)
    packed, values = zip(*(weight(torch, gen, experts, o, i) for o, i in ((f, d), (f, d), (d, f))))
    return x, idx.to(torch.int32).contiguous(), w, packed, values, res


def reference(torch, x, idx, w, values, res):
    d, f = x.shape[1], values[0].shape[1]
    y = res.double().clone() if res is not None else torch.zeros_like(x, dtype=torch.float64)
    sum_abs, bound = y.abs(), torch.zeros_like(y)
    half, tiny = 2.0 ** -11, 2.0 ** -25
    x64 = x.double()
    for e in range(values[0].shape[0]):
        at, slot = torch.nonzero(idx == e, as_tuple=True)
        if not len(at):
            continue
        xs, a, b, c = x64[at], *(v[e] for v in values)
        g, u = xs @ a.T, xs @ b.T
        dg, du = (xs.abs() @ m.abs().T * (d * 2.0 ** -23 + half * 1.01) + tiny * m.abs().sum(dim=1) for m in (a, b))
        silu = g * torch.sigmoid(g)
        h = silu * u
        dh = 1.1 * dg * (u.abs() + du) + silu.abs() * du + h.abs() * 16 * 2.0 ** -24
        dh = dh + (h.abs() + dh) * half + tiny * 256
        o = h @ c.T
        do = dh @ c.abs().T * (1 + half) + (h.abs() + dh) @ c.abs().T * (f * 2.0 ** -23 + half)
        share = w[at, slot].double()[:, None]
        y.index_add_(0, at, o * share)
        bound.index_add_(0, at, do * share.abs())
        sum_abs.index_add_(0, at, (o * share).abs() + do * share.abs())
    fi = torch.finfo(x.dtype)
    bound = bound + sum_abs * (idx.shape[1] + 2) * 2.0 ** -24
    return y, bound + (y.abs() + bound) * (fi.eps / 2) + fi.tiny * fi.eps / 2


def check(torch, y, ref, bound):
    d = (y.double() - ref).abs()
    assert bool(torch.isfinite(y).all())
    assert bool((d <= bound).all()), float((d / bound).max())
    rms = float(ref.square().mean().sqrt())
    rest = float((d - ref.abs() * (torch.finfo(y.dtype).eps / 2)).max())   # y's own rounding aside (test_gpu_moe)
    assert rest <= BF16_MAX * rms and float(d.mean()) <= BF16_MEAN * rms, (rest / rms, float(d.mean()) / rms)


def run(env, args, residual=True, **kw):
    torch, ffn = env
    x, idx, w, packed, values, res = args
    res = res if residual else None
    y = ffn.ffn_moe_forward_q4(x, idx, w, *packed, ffn=values[0].shape[1], res=res, **kw)
    ffn.ffn_device_status()
    check(torch, y, *reference(torch, x, idx, w, values, res))
    return y


@pytest.mark.parametrize("rows,d,f,experts,k", [(1, 32, 32, 1, 1), (1, 128, 128, 2, 1), (1, 256, 512, 4, 2),
                                                (3, 96, 160, 3, 2), (16, 512, 320, 8, 2), (300, 256, 544, 4, 2),
                                                (1000, 288, 96, 5, 3), (700, 512, 1408, 16, 6), (64, 1024, 1024, 64, 8),
                                                (2, 2048, 2176, 4, 4)])
def test_shapes(env, rows, d, f, experts, k):
    torch, _ = env
    run(env, make(torch, rows, d, f, experts, k), residual=rows % 2 == 1)


@pytest.mark.parametrize("rows", [31, 32, 33, 64, 65, 127, 128, 129, 255, 257, 513])
def test_tile_edges(env, rows):
    torch, _ = env
    idx = torch.full((rows, 2), -1, dtype=torch.int32, device="cuda")
    idx[:, 0] = 1
    idx[::3, 1] = 3
    run(env, make(torch, rows, 192, 352, 5, 2, idx=idx))


def test_single_weights_keep_their_places(env):
    """One non-zero code in W_down per output and an h that tells the inner
    index apart: every nibble of the layout reaches its own k, and every code
    its value (the products are exact here: y = h[place] * code)."""
    torch, ffn = env
    d, f = 160, 224
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.zeros(1, d, dtype=torch.bfloat16, device="cuda")
    x[0, 0] = 1.0
    # gate: G = 32 for every feature (silu(32) = 32 to 1e-13), up: U = a small integer of the feature
    qg = torch.zeros(1, f, d, dtype=torch.int8, device="cuda")
    qg[0, :, 0] = 4
    sg = torch.full((1, f, d // 32), 8.0, device="cuda").half()
    qu = torch.zeros(1, f, d, dtype=torch.int8, device="cuda")
    qu[0, :, 0] = (torch.arange(f, device="cuda") % 15 - 7).to(torch.int8)
    su = torch.ones(1, f, d // 32, device="cuda").half()
    qd = torch.zeros(1, d, f, dtype=torch.int8, device="cuda")
    place = torch.randperm(f, generator=gen, device="cuda")[:d]
    code = torch.randint(-8, 8, (d,), generator=gen, device="cuda", dtype=torch.int8)
    qd[0, torch.arange(d, device="cuda"), place] = code
    sd = torch.ones(1, d, f // 32, device="cuda").half()
    idx = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    y = ffn.ffn_moe_forward_q4(x, idx, torch.ones(1, 1, device="cuda"), pack(torch, qg, sg), pack(torch, qu, su),
                               pack(torch, qd, sd), ffn=f)
    want = 32.0 * qu[0, place, 0].double() * code.double()
    assert torch.equal(y[0].double(), want)


def test_large_and_small_scales(env):
    """Scales from 2^-20 (codes times them are subnormal in fp16) to 16."""
    torch, ffn = env
    rows, d, f, experts = 9, 128, 192, 2
    gen = torch.Generator(device="cuda").manual_seed(21)
    x, idx, w, _, _, res = make(torch, rows, d, f, experts, 1)
    mats = []
    for (o, i), top in (((f, d), 1.0), ((f, d), 2.0 ** -14), ((d, f), 16.0)):
        q = torch.randint(-8, 8, (experts, o, i), generator=gen, device="cuda", dtype=torch.int8)
        s = (top * torch.rand(experts, o, i // 32, generator=gen, device="cuda")).half()
        mats.append((pack(torch, q, s), q.double() * s.double().repeat_interleave(32, dim=-1)))
    packed, values = zip(*mats)
    y = ffn.ffn_moe_forward_q4(x, idx, w, *packed, ffn=f)
    ref, bound = reference(torch, x, idx, w, values, None)
    assert bool(((y.double() - ref).abs() <= bound).all())


def test_skipped_experts_and_nothing_leaks(env):
    torch, ffn = env
    rows, d, f, experts = 50, 96, 160, 6
    gen = torch.Generator(device="cuda").manual_seed(1)
    idx = torch.randint(0, 3, (rows, 3), generator=gen, device="cuda", dtype=torch.int32) * 2   # 0, 2, 4; repeats
    idx[0] = -1
    idx[1] = torch.tensor([-7, 2 ** 31 - 1, experts], dtype=torch.int32)
    idx[2, 1:] = -1
    x, idx, w, packed, values, res = make(torch, rows, d, f, experts, 3, idx=idx)
    clean = torch.where((idx >= 0) & (idx < experts), w, torch.zeros_like(w))
    w[0] = float("nan")
    ref, bound = reference(torch, x, idx, clean, values, res)
    for qs, sc in packed:
        sc[1::2] = float("nan")              # unused experts
    x[17] = float("nan")
    ws = ffn.workspace(ffn.ffn_moe_q4_workspace_bytes(rows, d, f, experts, 3), "cuda").fill_(255)
    buf = torch.cat([res, res])
    y = ffn.ffn_moe_forward_q4(x, idx, w, *packed, ffn=f, res=buf[:rows], out=buf[:rows], ws=ws)
    keep = torch.arange(rows, device="cuda") != 17
    assert bool(torch.isnan(y[17].float()).all()) and torch.equal(buf[rows:], res)
    check(torch, y[keep], ref[keep], bound[keep])
    assert torch.equal(y[:2], res[:2])


def test_repeatable_streams_and_graph(env):
    torch, ffn = env
    rows, d, f, experts, k = 140, 256, 512, 8, 2
    x, idx, w, packed, values, res = make(torch, rows, d, f, experts, k)
    want = ffn.ffn_moe_forward_q4(x, idx, w, *packed, ffn=f, res=res)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [ffn.ffn_moe_forward_q4(x, idx, w, *packed, ffn=f, res=res, stream=s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    ws = ffn.workspace(ffn.ffn_moe_q4_workspace_bytes(rows, d, f, experts, k), "cuda")
    y = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ffn.ffn_moe_forward_q4(x, idx, w, *packed, ffn=f, res=res, out=y, ws=ws)
    idx.copy_((idx + 3) % experts)
    idx[5:40, 0] = 6
    graph.replay()
    check(torch, y, *reference(torch, x, idx, w, values, res))


@pytest.mark.parametrize("rows,d,f,experts,k", [(9000, 32, 64, 40, 4), (30, 32, 32, 500, 8), (400, 96, 32, 3, 1),
                                                (1, 4096, 96, 2, 2)])
def test_many_calls_in_a_row(env, rows, d, f, experts, k):
    """Rows of one to a few 128-value groups, so that every unit is one stage or
    two and the rings turn fast; queued back to back."""
    torch, ffn = env
    x, idx, w, packed, values, res = make(torch, rows, d, f, experts, k)
    want = run(env, (x, idx, w, packed, values, res))
    ws = ffn.workspace(ffn.ffn_moe_q4_workspace_bytes(rows, d, f, experts, k), "cuda")
    y = torch.empty_like(x)
    for _ in range(300):
        ffn.ffn_moe_forward_q4(x, idx, w, *packed, ffn=f, res=res, out=y, ws=ws)
    torch.cuda.synchronize()
    ffn.ffn_device_status()
    assert torch.equal(y, want)


@pytest.mark.parametrize("rows,d,f,experts,k", [(40, 640, 1408, 16, 1), (64, 2048, 4768, 24, 2), (700, 640, 4768, 12, 1),
                                                (900, 1664, 672, 24, 2), (5, 1024, 8192, 4, 2), (66, 1056, 4064, 40, 3)])
def test_long_rows_and_unequal_loads(env, rows, d, f, experts, k):
    """A call's widest tile decides how many stages are in flight: even and odd
    numbers of 128-value groups in a row, one expert with most of the tokens
    beside many with one, a split reduction, several units one after another;
    the same bits in every call, whether the weights come from memory or from
    cache."""
    torch, ffn = env
    idx = torch.rand(rows, experts, generator=torch.Generator().manual_seed(rows)).topk(k, dim=1).indices
    idx[experts:, 0] = experts // 2   # (a second slot may name it too)
    x, idx, w, packed, values, res = make(torch, rows, d, f, experts, k, idx=idx.cuda())
    want = run(env, (x, idx, w, packed, values, res))
    flush = torch.empty(200 << 20, dtype=torch.uint8, device="cuda")
    got = torch.empty(300, *x.shape, dtype=x.dtype, device="cuda")
    for i in range(300):
        if i % 2:
            flush.fill_(i % 5)
        ffn.ffn_moe_forward_q4(x, idx, w, *packed, ffn=f, res=res, out=got[i])
    assert bool((got == want).all()), int((got != want).flatten(1).any(dim=1).sum())
    ffn.ffn_device_status()


def test_range_is_reported(env):
    torch, ffn = env
    from transformer_ffn_rmsnorm_gb300 import _lib
    x, idx, w, packed, values, res = make(torch, 4, 64, 64, 4, 2)
    ffn.ffn_device_status()
    x[2, 3] = -1e6
    ffn.ffn_moe_forward_q4(x, idx, w, *packed, ffn=64)
    with pytest.raises(ffn.FFNError) as err:
        ffn.ffn_device_status()
    assert err.value.status == _lib.FFN_ERR_RANGE


def test_refused(env):
    torch, ffn = env
    x, idx, w, packed, values, res = make(torch, 4, 64, 64, 4, 2)
    need = ffn.ffn_moe_q4_workspace_bytes(4, 64, 64, 4, 2)
    with pytest.raises(ffn.FFNError):
        ffn.ffn_moe_forward_q4(x, idx, w, *packed, ffn=64, ws=ffn.workspace(need - 256, "cuda"))
    with pytest.raises(TypeError):
        ffn.ffn_moe_forward_q4(x.half(), idx, w, *packed, ffn=64)
    with pytest.raises(ValueError):
        ffn.ffn_moe_forward_q4(x, idx, w, *packed, ffn=96)


def test_agrees_with_prepared_weights(env):
    """The same weights through ffn_prepare_weights_q4 and ffn_moe_forward."""
    torch, ffn = env
    x, idx, w, packed, values, res = make(torch, 260, 256, 384, 4, 2)
    prep = [ffn.ffn_prepare_weights_q4((qs.flatten(0, 1), sc.flatten(0, 1)), v.shape[2]).view(v.shape)
            for (qs, sc), v in zip(packed, values)]
    y = ffn.ffn_moe_forward(x, idx, w, *prep, res=res, flags=ffn.FFN_PREPARED_WEIGHTS)
    check(torch, y, *reference(torch, x, idx, w, values, res))
