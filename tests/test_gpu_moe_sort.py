"""ffn_moe_sort, ffn_moe_unsort and their gradients against plain loops.

Tolerances: positions, offsets and sorted rows are compared bit for bit.  A sum of k
products in fp32 is off by at most (k + 2) * 2^-24 of its terms' magnitudes, a dot
product over d by d / 128 + 12 such steps (a thread's share of a row, then the
CTA's); outputs of fewer bits add half a step."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    from transformer_ffn_rmsnorm_gb300 import ffn
    return torch, ffn


def order(torch, idx, experts):
    """Positions and offsets, pair by pair."""
    flat = idx.cpu().flatten().tolist()
    lists = [[] for _ in range(experts)]
    for i, e in enumerate(flat):
        if 0 <= e < experts:
            lists[e].append(i)
    pos, off = [-1] * len(flat), [0]
    for pairs in lists:
        for i, p in enumerate(pairs):
            pos[p] = off[-1] + i
        off.append(off[-1] + len(pairs))
    return (torch.tensor(pos, dtype=torch.int32).view(idx.shape), torch.tensor(off, dtype=torch.int32))


def choose(torch, rows, experts, k, seed, kind):
    gen = torch.Generator().manual_seed(seed)
    idx = torch.randint(0, experts, (rows, k), generator=gen)
    if kind == "holes":
        idx[torch.rand(rows, k, generator=gen) < 0.3] = -1
        idx[torch.rand(rows, k, generator=gen) < 0.05] = experts + 3
    elif kind == "none":
        idx[:] = -1
    elif kind == "one":
        idx[:] = experts - 1
    return idx.to(torch.int32).cuda()


CASES = [(1, 1, 1), (1, 8, 2), (16, 8, 2), (5, 1024, 32), (32, 64, 8), (256, 3, 1), (257, 3, 1), (100, 64, 6),
         (700, 1024, 8), (4099, 61, 6), (9000, 16, 1)]


@pytest.mark.parametrize("rows,experts,k", CASES)
@pytest.mark.parametrize("kind", ["all", "holes", "none", "one"])
def test_sort(env, rows, experts, k, kind):
    torch, ffn = env
    d = 144
    idx = choose(torch, rows, experts, k, rows + k, kind)
    ref_pos, ref_off = order(torch, idx, experts)
    x = torch.randn(rows, d, device="cuda")
    live = ref_pos.flatten() >= 0
    token = torch.arange(rows * k)[live] // k
    at = ref_pos.flatten()[live].long()
    for dt in (torch.float32, torch.float16, torch.bfloat16, torch.float8_e4m3fn):
        v = x.to(dt)
        raw = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[v.element_size()]
        out = torch.full((rows * k, d), 9.0, device="cuda").to(dt)
        want = out.view(raw).cpu().clone()
        want[at] = v.view(raw).cpu()[token]
        sc = out_sc = None
        if dt is torch.float8_e4m3fn:
            sc = torch.rand(rows, 3, device="cuda")
            out_sc = torch.full((rows * k, 3), 4.0, device="cuda")
            want_sc = out_sc.cpu().clone()
            want_sc[at] = sc.cpu()[token]
        xs, scales, pos, off = ffn.ffn_moe_sort(v, idx, experts, x_scales=sc, out=out, scales=out_sc)
        assert torch.equal(pos.cpu(), ref_pos) and torch.equal(off.cpu(), ref_off)
        assert torch.equal(xs.view(raw).cpu(), want)
        if sc is not None:
            assert torch.equal(scales.cpu(), want_sc)


@pytest.mark.parametrize("pieces", [1, 2, 5])
def test_sort_many_chunks(env, pieces):
    """More than 512 chunks of 1024 pairs: chunks grow."""
    torch, ffn = env
    rows, k, experts = 120000 * pieces // 5 + 1, 6, 37
    idx = choose(torch, rows, experts, k, pieces, "holes")
    x = torch.randn(rows, 16, device="cuda").to(torch.float8_e4m3fn)
    _, _, pos, off = ffn.ffn_moe_sort(x, idx, experts)
    flat = idx.flatten().long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    o = key.sort(stable=True).indices
    want = torch.empty_like(flat)
    want[o] = torch.arange(len(flat), device="cuda")
    want[key == experts] = -1
    assert torch.equal(pos.flatten().long(), want)
    assert torch.equal(off[1:].long(), torch.bincount(key, minlength=experts + 1)[:experts].cumsum(0))


def refs(torch, pos, ys, w, res):
    rows, k = pos.shape
    f = pos.flatten().long()
    live = (f >= 0)[:, None]
    v = torch.where(live, ys.double()[f.clamp(min=0)], 0.0).view(rows, k, -1)
    t = v if w is None else torch.where(live.view(rows, k, 1), v * w.double()[:, :, None], 0.0)
    y, mag = t.sum(dim=1), t.abs().sum(dim=1)
    return (y, mag, v) if res is None else (y + res.double(), mag + res.double().abs(), v)


@pytest.mark.parametrize("rows,experts,k", [(1, 1, 1), (1, 8, 2), (16, 8, 2), (5, 64, 32), (300, 64, 6), (1025, 9, 9)])
@pytest.mark.parametrize("d", [8, 128, 1032, 5120])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
def test_unsort_and_gradient(env, rows, experts, k, d, dtype):
    torch, ffn = env
    dt = getattr(torch, dtype)
    idx = choose(torch, rows, experts, k, rows + k + d, "holes")
    pos = order(torch, idx, experts)[0].cuda()
    ys, res, dy = (torch.randn(n, d, device="cuda").to(dt) for n in (rows * k, rows, rows))
    w = torch.rand(rows, k, device="cuda")
    w[pos < 0] = float("nan")                       # not read
    ys[int((pos >= 0).sum()):] = float("nan")       # nor these
    half, tiny = torch.finfo(dt).eps / 2, torch.finfo(dt).tiny * torch.finfo(dt).eps / 2
    e = (k + 2) * 2.0 ** -24
    for wt, r in ((w, res), (w, None), (None, None), (None, res)):
        y = ffn.ffn_moe_unsort(ys, pos, wt, res=r)
        ref, mag, _ = refs(torch, pos, ys, wt, r)
        assert bool(((y.double() - ref).abs() <= mag * e * 2 + ref.abs() * half + tiny).all())
    z = res.clone()
    assert ffn.ffn_moe_unsort(ys, pos, w, res=z, out=z) is z
    assert torch.equal(z, ffn.ffn_moe_unsort(ys, pos, w, res=res))
    # gradients
    dys = torch.full_like(ys, 3.0)
    dys, dw = ffn.ffn_moe_unsort_backward(dy, ys, pos, w, dys=dys)
    _, _, v = refs(torch, pos, ys, None, None)
    g = dy.double()
    want = (v * g[:, None, :]).sum(dim=2)
    mags = (v.abs() * g.abs()[:, None, :]).sum(dim=2)
    assert bool(((dw.double() - want).abs() <= mags * (d / 128 + 12) * 2.0 ** -24).all())
    assert bool((dw[pos < 0] == 0).all())
    want = torch.full(ys.shape, 3.0, dtype=torch.float64, device="cuda")
    live = pos >= 0
    want[pos[live].long()] = (w.double()[:, :, None] * g[:, None, :])[live]
    assert bool(((dys.double() - want).abs() <= want.abs() * (half + 2.0 ** -24) + tiny).all())
    # in ys' place
    both, dw2 = ffn.ffn_moe_unsort_backward(dy, ys, pos, w, dys=ys)
    assert both is ys and torch.equal(dw2, dw) and torch.equal(ys[pos[live].long()], dys[pos[live].long()])


def test_positions_out_of_range_count_nothing(env):
    torch, ffn = env
    pos = torch.tensor([[0, 6], [-7, 2], [5, 1 << 30]], dtype=torch.int32, device="cuda")
    ys = torch.randn(6, 8, device="cuda")
    y = ffn.ffn_moe_unsort(ys, pos)
    assert torch.equal(y, ys[[0, 2, 5]])
    w = torch.ones(3, 2, device="cuda")
    dys, dw = ffn.ffn_moe_unsort_backward(y, ys, pos, w)
    assert torch.equal(dys[[0, 2, 5]], y) and bool((dys[[1, 3, 4]] == 0).all())
    assert bool((dw.flatten()[[1, 2, 5]] == 0).all())


def test_gradients_against_differences(env):
    """sort, a weighted unsort: L = <c, y>; its differences in x, the rows and the weights."""
    torch, ffn = env
    rows, experts, k, d = 40, 7, 3, 64
    idx = choose(torch, rows, experts, k, 1, "holes")
    gen = torch.Generator(device="cuda").manual_seed(2)

    def rnd(*s):
        return torch.randn(*s, generator=gen, device="cuda")
    x, w, c = rnd(rows, d), torch.rand(rows, k, generator=gen, device="cuda"), rnd(rows, d)

    def loss(x, w):
        xs, _, pos, off = ffn.ffn_moe_sort(x, idx, experts)
        return (c.double() * ffn.ffn_moe_unsort(2 * xs, pos, w).double()).sum(), xs, pos

    base, xs, pos = loss(x, w)
    dys, dw = ffn.ffn_moe_unsort_backward(c, 2 * xs, pos, w)
    dx = ffn.ffn_moe_unsort(2 * dys, pos)
    ex, ew = rnd(rows, d), rnd(rows, k)
    # L is linear in x and in w: the difference of whole steps is the gradient's product
    for got, want in ((loss(x + ex, w)[0] - base, (dx.double() * ex.double()).sum()),
                      (loss(x, w + ew)[0] - base, (dw.double() * ew.double()).sum())):
        assert abs(float(got - want)) <= 1e-5 * float((c.abs() * 2 * k * 16).sum())
