"""The operators of the 8-bit layer one after the other, as they are used: dense, routed,
a routed layer's gradients, captured in graphs, on other streams and host threads, and beyond
2^31 elements.  Each step is compared with its formula in 64 bits on what the step before
wrote (tolerances: e4m3_util), so that no step's error is another's tolerance."""

import threading

import pytest

import e4m3_util as u

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def env():
    import torch
    from transformer_ffn_rmsnorm_gb300 import ffn
    return torch, ffn


def weights(torch, ffn, experts, out, inn, seed, transpose=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lead = (experts,) if experts else ()
    w = torch.randn(*lead, out, inn, generator=gen, device="cuda") / inn ** 0.5
    q = ffn.ffn_quantize_e4m3(w, block_rows=128)
    return (q, ffn.ffn_quantize_e4m3(w, block_rows=128, transpose=True)) if transpose else q


def check_norm(torch, n, scales, r, g):
    r64 = r.double()
    v = r64 / torch.sqrt((r64 * r64).mean(dim=1, keepdim=True) + EPS) * g.double()
    u.check_quantized(torch, n, scales, v, v.abs() * 60 * 2.0 ** -24)


@pytest.mark.parametrize("rows", [1, 5, 40, 300])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
def test_dense_layer(env, rows, dtype):
    torch, ffn = env
    d, f, dt = 400, 1008, getattr(torch, dtype)
    x, stream, g = torch.randn(rows, d, device="cuda").to(dt), torch.randn(rows, d, device="cuda").to(dt), \
        (1 + 0.1 * torch.randn(d, device="cuda")).to(dt)
    wg, wu = weights(torch, ffn, 0, f, d, 1), weights(torch, ffn, 0, f, d, 2)
    wd = weights(torch, ffn, 0, d, f, 3)
    r, n, ns = ffn.ffn_add_rmsnorm_e4m3(x, g, EPS, res=stream, group=128)
    check_norm(torch, n, ns, r, g)
    h, hs = ffn.ffn_gateup_e4m3(n, ns, wg, wu)
    u.check_gateup(torch, h, hs, (n, ns), wg, wu, d)
    y = ffn.ffn_linear_e4m3(h, hs, wd, res=r)
    ref, mag = u.product(torch, (h, hs), wd)
    u.check_linear(torch, y, ref, mag, f, r)
    ffn.ffn_device_status()


class Routed:
    """A routed layer's weights and buffers; forward() as a program calls it."""

    def __init__(self, torch, ffn, rows, d, f, experts, k, dt=None, seed=0):
        self.torch, self.ffn, self.k, self.experts, self.d, self.f = torch, ffn, k, experts, d, f
        dt = dt or torch.bfloat16
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.x, self.res = (torch.randn(rows, d, generator=gen, device="cuda").to(dt) for _ in range(2))
        self.logits = torch.randn(rows, experts, generator=gen, device="cuda")
        self.g = torch.ones(d, device="cuda", dtype=dt)
        self.wg, self.wu = (weights(torch, ffn, experts, f, d, seed + i) for i in (1, 2))
        self.wd = weights(torch, ffn, experts, d, f, seed + 3)
        self.xs = torch.zeros(rows * k, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        self.xss = torch.zeros(rows * k, -(-d // 128), device="cuda")
        self.h = torch.zeros(rows * k, f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        self.hs = torch.zeros(rows * k, -(-f // 128), device="cuda")
        self.ys = torch.zeros(rows * k, d, dtype=dt, device="cuda")
        self.ws = ffn.workspace(ffn.ffn_moe_sort_workspace_bytes(rows, experts, k), "cuda")

    def forward(self):
        ffn = self.ffn
        self.r, self.n, self.ns = ffn.ffn_add_rmsnorm_e4m3(self.x, self.g, EPS, res=self.res, group=128)
        self.idx, self.w = ffn.ffn_moe_route(self.logits, self.k, flags=ffn.FFN_ROUTE_RENORM)
        _, _, self.pos, self.off = ffn.ffn_moe_sort(self.n, self.idx, self.experts, x_scales=self.ns, out=self.xs,
                                                    scales=self.xss, ws=self.ws)
        ffn.ffn_gateup_e4m3(self.xs, self.xss, self.wg, self.wu, offsets=self.off, out=self.h, scales=self.hs)
        ffn.ffn_linear_e4m3(self.h, self.hs, self.wd, offsets=self.off, out=self.ys)
        self.y = ffn.ffn_moe_unsort(self.ys, self.pos, self.w, res=self.r)
        return self.y

    def check(self):
        torch = self.torch
        check_norm(torch, self.n, self.ns, self.r, self.g)
        rows, k = self.idx.shape
        used = int(self.off[-1])
        assert used == int((self.idx >= 0).sum())
        at = self.pos.flatten().long()
        live = at >= 0
        e = torch.repeat_interleave(torch.arange(self.experts, device="cuda"),
                                    (self.off[1:] - self.off[:-1]).long())
        assert torch.equal(e[at[live]], self.idx.flatten()[live].long())
        token = torch.arange(rows * k, device="cuda")[live] // k
        assert torch.equal(self.xs.view(torch.uint8)[at[live]], self.n.view(torch.uint8)[token])
        assert torch.equal(self.xss[at[live]], self.ns[token])
        s = slice(0, used)
        u.check_gateup(torch, self.h, self.hs, (self.xs, self.xss), self.wg, self.wu, self.d, self.off, s)
        ref, mag = u.product(torch, (self.h, self.hs), self.wd, self.off)
        u.check_linear(torch, self.ys[s], ref[s], mag[s], self.f)
        t = torch.where(live[:, None], self.ys.double()[at.clamp(min=0)], 0.0).view(rows, k, -1)
        t = t * self.w.double()[:, :, None]
        y, m = t.sum(1) + self.r.double(), t.abs().sum(1) + self.r.double().abs()
        fi = torch.finfo(self.y.dtype)
        tol = m * (2 * k + 4) * 2.0 ** -24 + y.abs() * fi.eps / 2 + fi.tiny
        assert bool(((self.y.double() - y).abs() <= tol).all())


@pytest.mark.parametrize("rows,experts,k", [(1, 8, 2), (16, 8, 2), (37, 64, 6), (600, 5, 2), (300, 3, 3)])
def test_routed_layer(env, rows, experts, k):
    """The last rows are padding: no expert, y is r."""
    torch, ffn = env
    m = Routed(torch, ffn, rows, 272, 400, experts, k, seed=rows)
    if rows > 3:
        m.logits[-3:] = float("-inf")
    m.forward()
    m.check()
    if rows > 3:
        assert torch.equal(m.y[-3:], m.r[-3:])
    ffn.ffn_device_status()


def test_routed_layer_captured(env):
    """Two captured layers of shared weights, replayed with other inputs and routes, one after the other and
    at the same time: the bits of eager calls."""
    torch, ffn = env
    shapes = [(24, 64, 6), (700, 64, 6)]
    layers = [Routed(torch, ffn, r, 256, 384, e, k, seed=7) for r, e, k in shapes]
    graphs, streams = [], []
    for m in layers:
        m.forward()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.forward()
        graphs.append(g)
        streams.append(torch.cuda.Stream())
    for turn in range(4):
        want = []
        for m in layers:
            m.x.copy_(torch.randn_like(m.x))
            m.logits.copy_(torch.randn_like(m.logits))
            if turn == 2:
                m.logits[1:] = float("-inf")       # one token alone has experts
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            if turn % 2:
                with torch.cuda.stream(s):
                    g.replay()
            else:
                g.replay()
        torch.cuda.synchronize()
        for m in layers:
            got = m.y.clone()
            m.check()
            y_graph, m_y = got, m.y
            fresh = Routed.__new__(Routed)
            fresh.__dict__.update(m.__dict__)
            fresh.ys = torch.zeros_like(m.ys)
            assert torch.equal(fresh.forward(), y_graph)
            m.y = m_y
    ffn.ffn_device_status()


def test_streams_and_host_threads(env):
    """Calls from four host threads on streams of their own, and the stream argument."""
    torch, ffn = env
    layers = [Routed(torch, ffn, r, 256, 384, 16, 4, seed=20 + r) for r in (3, 50, 260, 900)]
    want = [m.forward().clone() for m in layers]
    torch.cuda.synchronize()
    bad = []

    def work(m, ref):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                if not torch.equal(m.forward(), ref):
                    bad.append(m)
        s.synchronize()
    threads = [threading.Thread(target=work, args=a) for a in zip(layers, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    s = torch.cuda.Stream()
    m = layers[1]
    s.wait_stream(torch.cuda.current_stream())
    n, ns = ffn.ffn_quantize_e4m3(m.x, stream=s)
    xs, xss, pos, off = ffn.ffn_moe_sort(n, m.idx, 16, x_scales=ns, stream=s)
    h, hs = ffn.ffn_gateup_e4m3(xs, xss, m.wg, m.wu, offsets=off, stream=s)
    y = ffn.ffn_moe_unsort(ffn.ffn_linear_e4m3(h, hs, m.wd, offsets=off, stream=s), pos, m.w, stream=s)
    dys, dw = ffn.ffn_moe_unsort_backward(y, torch.zeros_like(m.ys), pos, m.w, stream=s)
    s.synchronize()
    n2, ns2 = ffn.ffn_quantize_e4m3(m.x)
    xs, xss, pos, off = ffn.ffn_moe_sort(n2, m.idx, 16, x_scales=ns2)
    h, hs = ffn.ffn_gateup_e4m3(xs, xss, m.wg, m.wu, offsets=off)
    y2 = ffn.ffn_moe_unsort(ffn.ffn_linear_e4m3(h, hs, m.wd, offsets=off), pos, m.w)
    assert torch.equal(y, y2) and bool((dw == 0).all())
    ffn.ffn_device_status()


@pytest.mark.parametrize("rows,experts,k", [(5, 4, 2), (333, 6, 3)])
def test_routed_linear_training_step(env, rows, experts, k):
    """y = res + sum_j w_j W[e_j] x: the gradients of x, of the router's weights and of res through the
    operators' own backward calls and the transposed weights."""
    torch, ffn = env
    d, f = 272, 400
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, d, generator=gen, device="cuda").bfloat16()
    dy = torch.randn(rows, f, generator=gen, device="cuda").bfloat16()
    idx, w = ffn.ffn_moe_route(torch.randn(rows, experts, generator=gen, device="cuda"), k)
    wq, wt = weights(torch, ffn, experts, f, d, 5, transpose=True)
    xs, _, pos, off = ffn.ffn_moe_sort(x, idx, experts)
    q, s = ffn.ffn_quantize_e4m3(xs)
    ys = ffn.ffn_linear_e4m3(q, s, wq, offsets=off)
    dys, dw = ffn.ffn_moe_unsort_backward(dy, ys, pos, w)
    at = pos.flatten().long()
    token = torch.arange(rows * k, device="cuda") // k
    g = dy.double()[token]
    v = ys.double()[at] * g
    assert bool(((dw.double().flatten() - v.sum(1)).abs() <= v.abs().sum(1) * (f / 128 + 12) * 2.0 ** -24).all())
    want = w.double().flatten()[:, None] * g
    assert bool(((dys.double()[at] - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -23)).all())
    dq, ds = ffn.ffn_quantize_e4m3(dys)
    dxs = ffn.ffn_linear_e4m3(dq, ds, wt, offsets=off, dtype=torch.float32)
    vq = u.values(dq, ds, 1)
    ref, mag = torch.zeros(rows * k, d, device="cuda", dtype=torch.float64), torch.zeros(rows * k, d, device="cuda",
                                                                                         dtype=torch.float64)
    o = off.tolist()
    for e in range(experts):
        m = u.values(wq[0][e], wq[1][e], 128)
        r = slice(o[e], o[e + 1])
        ref[r], mag[r] = vq[r] @ m, vq[r].abs() @ m.abs()
    u.check_linear(torch, dxs, ref, mag, f)
    dx = ffn.ffn_moe_unsort(dxs, pos)
    t = dxs.double()[at].view(rows, k, d)
    assert bool(((dx.double() - t.sum(1)).abs() <= t.abs().sum(1) * (k + 2) * 2.0 ** -24).all())
    ffn.ffn_device_status()


def test_rows_times_features_beyond_32_bits(env):
    """More than 2^31 outputs and inputs: the last rows."""
    torch, ffn = env
    rows, out = 70000, 32768
    x = torch.zeros(rows, 16, device="cuda")
    x[-300:] = torch.randn(300, 16, device="cuda")
    xq = ffn.ffn_quantize_e4m3(x)
    w = weights(torch, ffn, 0, out, 16, 9)
    y = ffn.ffn_linear_e4m3(*xq, w)
    tail = (xq[0][-300:], xq[1][-300:])
    ref, mag = u.product(torch, tail, w)
    u.check_linear(torch, y[-300:], ref, mag, 16)
    assert bool((y[:rows - 300:997] == 0).all())
    q, s = ffn.ffn_quantize_e4m3(y)
    u.check_quantized(torch, q[-300:], s[-300:], y[-300:].double(), torch.zeros(300, out, device="cuda"))
    del q, s
    qt, st = ffn.ffn_quantize_e4m3(y.view(2, 35000, out)[:, :34992].contiguous(), block_rows=128, transpose=True)
    part = y[35000 + 34992 - 48:35000 + 34992].double().abs()     # a last block of 48 rows
    a = part.view(48, out // 128, 128).amax(dim=(0, 2)).clamp(min=2.0 ** -100) / 448
    assert bool(((st[1, :, -1].double() - a).abs() <= a * 3 * 2.0 ** -24).all())
    got = qt[1, :, -48:].double() * st[1, :, -1].double().repeat_interleave(128)[:, None]
    assert bool(((got.T.abs() - part).abs() <= part * 2.0 ** -4 * 1.001 + a.repeat_interleave(128) * 2.0 ** -9).all())
    del qt, st
    wg = weights(torch, ffn, 0, out, 16, 10)
    h, hs = ffn.ffn_gateup_e4m3(*xq, w, wg)
    u.check_gateup(torch, h[-300:], hs[-300:], tail, w, wg, 16)
    assert bool((h[:rows - 300:997].float() == 0).all())
    ffn.ffn_device_status()


def test_sorted_rows_beyond_32_bits(env):
    torch, ffn = env
    rows, d, k, experts = 36000, 8192, 8, 16
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randint(0, 255, (rows, d), generator=gen, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
    idx = torch.randint(0, experts, (rows, k), generator=gen, device="cuda", dtype=torch.int32)
    xs, _, pos, off = ffn.ffn_moe_sort(x, idx, experts)
    for j in range(k):
        for t in range(j, rows, 6007):
            assert torch.equal(xs.view(torch.uint8)[pos[t, j].long()], x.view(torch.uint8)[t])
    ys = torch.zeros(rows * k, d, dtype=torch.float16, device="cuda")
    at = pos[-5:].flatten().long()
    ys[at] = torch.randn(len(at), d, device="cuda").half()
    w = torch.rand(rows, k, device="cuda")
    y = ffn.ffn_moe_unsort(ys, pos, w)
    t = ys[at].double().view(5, k, d) * w[-5:].double()[:, :, None]
    assert bool(((y[-5:].double() - t.sum(1)).abs() <= t.abs().sum(1) * 12 * 2.0 ** -24 + t.sum(1).abs() * 2.0 ** -11 +
                 2.0 ** -25).all())
    assert bool((y[:-5:501] == 0).all())
    dys, dw = ffn.ffn_moe_unsort_backward(y, ys, pos, w, dys=ys)
    g = w[-5:].double()[:, :, None] * y[-5:].double()[:, None, :]
    assert bool(((dys[at].double().view(5, k, d) - g).abs() <= g.abs() * (2.0 ** -11 + 2.0 ** -23) + 2.0 ** -25).all())
    ffn.ffn_device_status()
