"""ffn_moe_forward against the formula in 64 bits.

Two bounds on every element.  (1) Worst case, from the roundings: a product of
length K in fp32 is off by at most K 2^-23 of the sum of its terms'
magnitudes; h carries the errors of G and U through silu(G) U (|silu'| <=
1.1), 16 x 2^-24 for the exponential and products, and half a step of its
16-bit type (below the normal range of fp16, where prepared weights store h
2^-8, half the smallest step); the results add k weighted terms and round
once.  (2) The tolerance of every 16-bit block here (gpu_util.assert_lowp),
max |diff| <= 2e-2 rms and mean |diff| <= 4e-3 rms, for what the rounding of
y does not explain: that alone is up to half a step, eps / 2 |y| = 2^-8 |y| in
bf16, and |y| reaches 6 rms among 10^5 elements (more where a token's weights
are unequal), 6 x 2^-8 = 2.3e-2 rms.  The roundings of h, the rest, are
independent, about 2^-8 / sqrt 3 = 2.3e-3 rms together: 2e-2 is eight of them."""

import pytest

from gpu_util import BF16_MAX, BF16_MEAN

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    from transformer_ffn_rmsnorm_gb300 import ffn
    return torch, ffn


def make(torch, rows, d, f, experts, k, dt, seed=0, idx=None):
    gen = torch.Generator(device="cuda").manual_seed(seed + rows)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")
    x = rnd(rows, d).to(dt)
    res = rnd(rows, d).to(dt)
    wg, wu = ((rnd(experts, f, d) / d ** 0.5).to(dt) for _ in range(2))
    wd = (rnd(experts, d, f) / f ** 0.5).to(dt)
    if idx is None:
        idx = torch.rand(rows, experts, generator=gen, device="cuda").topk(k, dim=1).indices
    w = torch.softmax(rnd(rows, k), dim=1)
    return x, idx.to(torch.int32).contiguous(), w, wg, wu, wd, res


def reference(torch, x, idx, w, wg, wu, wd, res, prepared):
    """(y, bound) in float64; weights [experts, ...] are widened one expert at a time."""
    d, f = x.shape[1], wg.shape[1]
    y = res.double().clone() if res is not None else torch.zeros_like(x, dtype=torch.float64)
    sum_abs, bound = y.abs(), torch.zeros_like(y)
    hi = torch.finfo(torch.float16 if prepared else x.dtype)
    step = hi.eps / 2
    least = hi.tiny * hi.eps / 2 * (256 if prepared else 1)
    x64 = x.double()
    for e in range(wg.shape[0]):
        at, slot = torch.nonzero(idx == e, as_tuple=True)
        if not len(at):
            continue
        xs, a, b, c = x64[at], wg[e].double(), wu[e].double(), wd[e].double()
        g, u = xs @ a.T, xs @ b.T
        dg, du = (xs.abs() @ m.abs().T * (d * 2.0 ** -23) for m in (a, b))
        silu = g * torch.sigmoid(g)
        h = silu * u
        dh = 1.1 * dg * (u.abs() + du) + silu.abs() * du + h.abs() * 16 * 2.0 ** -24
        dh = dh + (h.abs() + dh) * step + least
        o = h @ c.T
        do = dh @ c.abs().T + (h.abs() + dh) @ c.abs().T * (f * 2.0 ** -23)
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
    rest = float((d - ref.abs() * (torch.finfo(y.dtype).eps / 2)).max())
    assert rest <= BF16_MAX * rms and float(d.mean()) <= BF16_MEAN * rms, (rest / rms, float(d.mean()) / rms)


def run(env, args, residual=True, prepared=False, **kw):
    torch, ffn = env
    x, idx, w, wg, wu, wd, res = args
    res = res if residual else None
    ws = [wg, wu, wd]
    if prepared:
        ws = [ffn.ffn_prepare_weights(t) for t in ws]
    y = ffn.ffn_moe_forward(x, idx, w, *ws, res=res, flags=ffn.FFN_PREPARED_WEIGHTS if prepared else 0, **kw)
    ffn.ffn_device_status()
    check(torch, y, *reference(torch, x, idx, w, wg, wu, wd, res, prepared))
    return y


@pytest.mark.parametrize("dtype,prepared", [("bfloat16", False), ("float16", False), ("bfloat16", True),
                                            ("float16", True)])
@pytest.mark.parametrize("rows,d,f,experts,k", [(1, 64, 64, 1, 1), (1, 128, 72, 4, 2), (2, 8, 8, 2, 1),
                                                (5, 136, 264, 3, 2), (33, 512, 320, 8, 2), (300, 256, 520, 4, 2),
                                                (1000, 264, 136, 5, 3), (700, 512, 1408, 16, 6), (64, 1024, 1024, 64, 8)])
def test_shapes(env, rows, d, f, experts, k, dtype, prepared):
    torch, _ = env
    args = make(torch, rows, d, f, experts, k, getattr(torch, dtype))
    run(env, args, residual=rows % 2 == 1, prepared=prepared)


@pytest.mark.parametrize("rows", [15, 16, 17, 31, 32, 33, 64, 65, 80, 127, 128, 129, 255, 256, 257, 300, 513, 1025])
def test_tile_edges(env, rows):
    """Every token to expert 1 and every third one to expert 3 as well: token
    tiles that end at, before and after their limits; two experts unused."""
    torch, _ = env
    idx = torch.full((rows, 2), -1, dtype=torch.int32, device="cuda")
    idx[:, 0] = 1
    idx[::3, 1] = 3
    args = make(torch, rows, 192, 320, 5, 2, torch.bfloat16, idx=idx)
    run(env, args)


def test_skipped_out_of_range_and_repeated_experts(env):
    torch, ffn = env
    rows, experts = 50, 6
    gen = torch.Generator(device="cuda").manual_seed(1)
    idx = torch.randint(0, experts, (rows, 3), generator=gen, device="cuda", dtype=torch.int32)   # repeats in a row
    idx[0] = -1
    idx[1] = torch.tensor([-7, 2 ** 31 - 1, experts], dtype=torch.int32)
    idx[2, 1:] = -1
    args = list(make(torch, rows, 128, 256, experts, 3, torch.float16, idx=idx))
    args[2][0] = float("nan")                # weights of skipped slots are not used
    args[2][2, 1:] = float("inf")
    x, idx, w, wg, wu, wd, res = args
    clean = torch.where((idx >= 0) & (idx < experts), w, torch.zeros_like(w))
    y = ffn.ffn_moe_forward(x, idx, w, wg, wu, wd, res=res)
    check(torch, y, *reference(torch, x, idx, clean, wg, wu, wd, res, False))
    assert torch.equal(y[:2], res[:2])
    y = ffn.ffn_moe_forward(x, idx, w, wg, wu, wd)
    assert bool((y[:2] == 0).all())
    none = torch.full_like(idx, -1)
    assert torch.equal(ffn.ffn_moe_forward(x, none, w, wg, wu, wd, res=res), res)


def test_nothing_leaks_between_tokens_and_experts(env):
    """NaN in one token's x, in an unused expert's weights (the rows next to
    the last ones of a ragged tile) and in the workspace stay where they are."""
    torch, ffn = env
    rows, d, f, experts = 70, 136, 200, 4
    idx = torch.randint(0, 2, (rows, 1), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)) * 2
    x, idx, w, wg, wu, wd, res = make(torch, rows, d, f, experts, 1, torch.bfloat16, idx=idx)
    ref, bound = reference(torch, x, idx, w, wg, wu, wd, res, False)
    x[17] = float("nan")
    for t in (wg, wu, wd):
        t[1] = float("nan")
        t[3] = float("nan")
    ws = ffn.workspace(ffn.ffn_moe_workspace_bytes(rows, d, f, experts, 1, x.dtype), "cuda").fill_(255)
    y = ffn.ffn_moe_forward(x, idx, w, wg, wu, wd, res=res, ws=ws)
    keep = torch.arange(rows, device="cuda") != 17
    assert bool(torch.isnan(y[17].float()).all())
    check(torch, y[keep], ref[keep], bound[keep])


def test_in_place_rows_behind_and_repeatable(env):
    torch, ffn = env
    x, idx, w, wg, wu, wd, res = make(torch, 90, 256, 384, 8, 4, torch.bfloat16)
    want = ffn.ffn_moe_forward(x, idx, w, wg, wu, wd, res=res)
    for _ in range(3):
        assert torch.equal(ffn.ffn_moe_forward(x, idx, w, wg, wu, wd, res=res), want)
    buf = torch.cat([res, res])
    y = ffn.ffn_moe_forward(x, idx, w, wg, wu, wd, res=buf[:90], out=buf[:90])
    assert torch.equal(y, want) and torch.equal(buf[90:], res)


def test_small_workspace_is_refused(env):
    torch, ffn = env
    x, idx, w, wg, wu, wd, res = make(torch, 4, 64, 64, 4, 2, torch.bfloat16)
    need = ffn.ffn_moe_workspace_bytes(4, 64, 64, 4, 2, x.dtype)
    with pytest.raises(ffn.FFNError):
        ffn.ffn_moe_forward(x, idx, w, wg, wu, wd, ws=ffn.workspace(need - 256, "cuda"))
    with pytest.raises(ValueError):
        ffn.ffn_moe_forward(x, idx, w, wg, wu[:3], wd)
    with pytest.raises(TypeError):
        ffn.ffn_moe_forward(x, idx.long(), w, wg, wu, wd)
    with pytest.raises(TypeError):
        ffn.ffn_moe_forward(x.float(), idx, w, wg, wu, wd)


def test_range_is_reported(env):
    """A bf16 x beyond fp16's range on prepared weights records FFN_ERR_RANGE."""
    torch, ffn = env
    from transformer_ffn_rmsnorm_gb300 import _lib
    x, idx, w, wg, wu, wd, res = make(torch, 4, 64, 64, 4, 2, torch.bfloat16)
    prep = [ffn.ffn_prepare_weights(t) for t in (wg, wu, wd)]
    ffn.ffn_device_status()
    x[2, 3] = 1e6
    ffn.ffn_moe_forward(x, idx, w, *prep, flags=ffn.FFN_PREPARED_WEIGHTS)
    with pytest.raises(ffn.FFNError) as err:
        ffn.ffn_device_status()
    assert err.value.status == _lib.FFN_ERR_RANGE


def test_captured_with_other_experts_at_replay(env):
    """The graph holds no choice of experts: replayed with other indices (and
    other loads of the experts) it computes the new ones; two graphs in turn
    share one workspace."""
    torch, ffn = env
    rows, d, f, experts, k = 200, 256, 320, 8, 2
    x, idx, w, wg, wu, wd, res = make(torch, rows, d, f, experts, k, torch.bfloat16)
    ws = ffn.workspace(ffn.ffn_moe_workspace_bytes(rows, d, f, experts, k, x.dtype), "cuda")
    y, y1 = torch.empty_like(x), torch.empty_like(x[:1])
    ffn.ffn_moe_forward(x, idx, w, wg, wu, wd, res=res, out=y, ws=ws)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        ffn.ffn_moe_forward(x, idx, w, wg, wu, wd, res=res, out=y, ws=ws)
    with torch.cuda.graph(graphs[1]):
        ffn.ffn_moe_forward(x[:1], idx[:1], w[:1], wg, wu, wd, out=y1, ws=ws)
    for seed in (5, 6):
        x2, idx2, w2, *_ = make(torch, rows, d, f, experts, k, torch.bfloat16, seed=seed)
        if seed == 6:
            idx2 = torch.zeros_like(idx2)
            idx2[:, 1] = 7
        x.copy_(x2)
        idx.copy_(idx2)
        w.copy_(w2)
        y.zero_()
        graphs[0].replay()
        graphs[1].replay()
        check(torch, y, *reference(torch, x2, idx2, w2, wg, wu, wd, res, False))
        assert torch.equal(y1, ffn.ffn_moe_forward(x2[:1], idx2[:1], w2[:1], wg, wu, wd))


@pytest.mark.parametrize("rows,d,f,experts,k", [(40000, 64, 72, 100, 8), (5000, 64, 64, 1000, 4), (64, 64, 64, 1024, 32),
                                                (300, 64, 64, 7, 1), (70000, 8, 8, 3, 2), (2, 4096, 8, 3, 3)])
def test_many_pairs_and_many_experts(env, rows, d, f, experts, k):
    """Chunks of more than 256 pairs, a thread an expert in the scan, fewer
    pairs than experts, tiny and lopsided sizes; skipped slots among them."""
    torch, _ = env
    args = list(make(torch, rows, d, f, experts, k, torch.float16))
    args[1][::7, 0] = -1
    run(env, args)


def test_host_threads(env):
    """Calls from several host threads, each on its own stream and workspace."""
    import threading
    torch, ffn = env
    sets = [make(torch, 40 * (i + 1), 256, 512, 4, 2, torch.bfloat16, seed=i) for i in range(4)]
    want = [ffn.ffn_moe_forward(*a[:6], res=a[6]) for a in sets]
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(20):
            got[i] = ffn.ffn_moe_forward(*sets[i][:6], res=sets[i][6], stream=s)
        s.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("rows,experts", [(96, 2), (128, 3), (40, 1), (20, 8), (300, 4)])
def test_many_calls_in_a_row(env, rows, experts):
    """Calls queued back to back: each one's kernels start while the ones
    before still hold some multiprocessors (small plans, CTA pairs and single
    CTAs), where a pair's allocation of tensor memory has to wait for both."""
    torch, ffn = env
    x, idx, w, wg, wu, wd, res = make(torch, rows, 512, 1024, experts, min(2, experts), torch.bfloat16)
    want = ffn.ffn_moe_forward(x, idx, w, wg, wu, wd, res=res)
    ws = ffn.workspace(ffn.ffn_moe_workspace_bytes(rows, 512, 1024, experts, min(2, experts), x.dtype), "cuda")
    y = torch.empty_like(x)
    for _ in range(600):
        ffn.ffn_moe_forward(x, idx, w, wg, wu, wd, res=res, out=y, ws=ws)
    torch.cuda.synchronize()
    ffn.ffn_device_status()
    assert torch.equal(y, want)


def test_streams_with_their_own_workspaces(env):
    torch, ffn = env
    sets = [make(torch, 150 + 30 * i, 256, 512, 8, 2, torch.bfloat16, seed=i) for i in range(3)]
    want = [ffn.ffn_moe_forward(*a[:6], res=a[6]) for a in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[ffn.ffn_moe_forward(*a[:6], res=a[6], stream=s) for a, s in zip(sets, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(p, q) for p, q in zip(g, want))


@pytest.mark.slow
def test_weights_beyond_32_bit_offsets(env):
    """160 experts of 4096 x 4096: element offsets pass 2^31 in every weight."""
    torch, ffn = env
    experts, d, f = 160, 4096, 4096
    idx = torch.tensor([[159, 0], [158, 129], [159, 128]], dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(8)
    ws = []
    for _ in range(3):
        w = torch.zeros(experts, f, d, dtype=torch.bfloat16, device="cuda")
        for e in torch.unique(idx).tolist():
            w[e] = torch.randn(f, d, generator=gen, device="cuda") / 64
        ws.append(w)
    x = torch.randn(3, d, generator=gen, device="cuda").bfloat16()
    share = torch.rand(3, 2, generator=gen, device="cuda")
    y = ffn.ffn_moe_forward(x, idx, share, *ws)
    check(torch, y, *reference(torch, x, idx, share, *ws, None, False))
    del ws


def test_layer_norm_route_experts(env):
    """The operators together, as a layer runs them, captured in a graph:
    r = x + res and its norm, router logits, routing, the experts on the norm,
    added to r."""
    torch, ffn = env
    rows, d, f, experts, k = 130, 512, 384, 16, 4
    x, _, _, wg, wu, wd, res = make(torch, rows, d, f, experts, k, torch.bfloat16)
    gen = torch.Generator(device="cuda").manual_seed(12)
    g = (1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).bfloat16()
    router = torch.randn(experts, d, generator=gen, device="cuda").bfloat16() / d ** 0.5
    bias = 0.05 * torch.randn(experts, generator=gen, device="cuda")

    def layer(x, res):
        r, n = ffn.ffn_add_rmsnorm(x, g, 1e-6, res=res)
        logits = (n @ router.T).float()
        idx, w = ffn.ffn_moe_route(logits, k, bias=bias, groups=4, topk_groups=2,
                                   flags=ffn.FFN_ROUTE_SIGMOID | ffn.FFN_ROUTE_RENORM)
        return r, n, logits, idx, w, ffn.ffn_moe_forward(n, idx, w, wg, wu, wd, res=r, out=r)

    layer(x, res)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, n, logits, idx, w, y = layer(x, res)
    graph.replay()
    torch.cuda.synchronize()
    r_ref = (x.float() + res.float()).bfloat16()
    ri, rw = ffn.ffn_moe_route(logits, k, bias=bias, groups=4, topk_groups=2,
                               flags=ffn.FFN_ROUTE_SIGMOID | ffn.FFN_ROUTE_RENORM)
    assert torch.equal(ri, idx) and torch.equal(rw, w)
    assert torch.equal(n, ffn.ffn_add_rmsnorm(r_ref, g, 1e-6)[1])
    check(torch, y, *reference(torch, n, idx, w, wg, wu, wd, r_ref, False))
    ffn.ffn_device_status()
