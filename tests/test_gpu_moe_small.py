"""The routed blocks whose h is fp16 (Q4 and prepared weights, fp16 storage) on
small and large hidden values: h = silu(G) U goes with the square of x, out of
fp16's normal range (2^-14 to 2^16) at an x of rms 0.01 or weights of as small a
gain, and beyond it at one of 300.

Every row of y is held to the tolerances of the other 16-bit blocks relative to
its own rms, and every element to the bound of test_gpu_moe and test_gpu_moe_q4
with another last term for h.  A row is stored times a power of two, 2^(16 l),
with l = 0 if its largest value m is in [2^-12, 2^15) and the one that brings it
to [2^-12, 2^4) if below and to [2^-1, 2^15) if above; so the steps below fp16's
normal range, 2^-24, are of h 2^-24 min(1, 2^12 m), or 2^-24 x 2 m above, and h
is rounded at most twice."""

import pytest

from gpu_util import BF16_MAX, BF16_MEAN
from test_gpu_moe_q4 import pack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    from transformer_ffn_rmsnorm_gb300 import ffn
    return torch, ffn


KINDS = ["q4", "prepared", "float16"]


def make(torch, kind, rows, d, f, experts, k, gain=1.0, feature_gain=None, seed=0):
    """(x of unit rms, idx, w, the call's weights, their values); weights of unit
    gain times `gain` in gate and up, `feature_gain` [f] more in up.  fp16
    storage: w_down of gain 2^10, which keeps small outputs in fp16's range."""
    gen = torch.Generator(device="cuda").manual_seed(seed + rows)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")
    x = rnd(rows, d)
    idx = torch.rand(rows, experts, generator=gen, device="cuda").topk(k, dim=1).indices.to(torch.int32).contiguous()
    w = torch.softmax(rnd(rows, k), dim=1)
    fg = torch.ones(f, device="cuda") if feature_gain is None else feature_gain
    mats = []
    for i, (o, n) in enumerate(((f, d), (f, d), (d, f))):
        scale = (gain if i < 2 else 1024.0 if kind == "float16" else 1.0) / n ** 0.5
        row = (fg if i == 1 else torch.ones(o, device="cuda"))[None, :, None]
        if kind == "q4":
            q = torch.randint(-8, 8, (experts, o, n), generator=gen, device="cuda", dtype=torch.int8)
            s = ((0.5 + torch.rand(experts, o, n // 32, generator=gen, device="cuda")) * (0.2 * scale) * row).half()
            mats.append((pack(torch, q, s), q.double() * s.double().repeat_interleave(32, dim=-1)))
        else:
            m = (rnd(experts, o, n) * scale * row).to(torch.float16 if kind == "float16" else torch.bfloat16)
            mats.append((m, m.double()))
    weights, values = zip(*mats)
    return x, idx, w, weights, values


def call(env, kind, x, idx, w, weights, f, **kw):
    torch, ffn = env
    if kind == "q4":
        return ffn.ffn_moe_forward_q4(x, idx, w, *weights, ffn=f, **kw)
    if kind == "prepared":
        prep = [ffn.ffn_prepare_weights(m) for m in weights]
        return ffn.ffn_moe_forward(x, idx, w, *prep, flags=ffn.FFN_PREPARED_WEIGHTS, **kw)
    return ffn.ffn_moe_forward(x, idx, w, *weights, **kw)


def reference(torch, kind, x, idx, w, values):
    d, f = x.shape[1], values[0].shape[1]
    y = torch.zeros_like(x, dtype=torch.float64)
    sum_abs, bound = torch.zeros_like(y), torch.zeros_like(y)
    half = 2.0 ** -11
    wh = half * 1.01 if kind == "q4" else 0.0                     # a dequantised weight in fp16
    xt = 0.0 if kind == "float16" else 2.0 ** -25                 # x in fp16, below its normal range
    x64 = x.double()
    for e in range(values[0].shape[0]):
        at, slot = torch.nonzero(idx == e, as_tuple=True)
        if not len(at):
            continue
        xs, a, b, c = x64[at], *(v[e] for v in values)
        g, u = xs @ a.T, xs @ b.T
        dg, du = (xs.abs() @ m.abs().T * (d * 2.0 ** -23 + wh) + xt * m.abs().sum(dim=1) for m in (a, b))
        silu = g * torch.sigmoid(g)
        h = silu * u
        dh = 1.1 * dg * (u.abs() + du) + silu.abs() * du + h.abs() * 16 * 2.0 ** -24
        m = 1.1 * h.abs().amax(dim=1, keepdim=True)
        dh = dh + (h.abs() + dh) * 2 * half + 2.0 ** -24 * (torch.clamp(m * 2.0 ** 12, max=1.0) + 2 * m)
        o = h @ c.T
        do = dh @ c.abs().T * (1 + half) + (h.abs() + dh) @ c.abs().T * (f * 2.0 ** -23 + (half if wh else 0.0))
        share = w[at, slot].double()[:, None]
        y.index_add_(0, at, o * share)
        bound.index_add_(0, at, do * share.abs())
        sum_abs.index_add_(0, at, (o * share).abs() + do * share.abs())
    fi = torch.finfo(x.dtype)
    bound = bound + sum_abs * (idx.shape[1] + 2) * 2.0 ** -24
    return y, bound + (y.abs() + bound) * (fi.eps / 2) + fi.tiny * fi.eps / 2


def check_rows(torch, y, ref, bound):
    d = (y.double() - ref).abs()
    assert bool(torch.isfinite(y).all())
    assert bool((d <= bound).all()), float((d / bound).max())
    fi = torch.finfo(y.dtype)
    rms = ref.square().mean(dim=1).sqrt()
    rest = (d - ref.abs() * (fi.eps / 2) - fi.tiny * fi.eps / 2).clamp(min=0)   # y's own rounding aside (test_gpu_moe)
    assert bool((rest.amax(dim=1) <= BF16_MAX * rms).all()), float((rest.amax(dim=1) / rms).max())
    lost = d.mean(dim=1) - fi.tiny * fi.eps / 2
    assert bool((lost <= BF16_MEAN * rms).all()), float((lost / rms).max())


def storage(torch, kind):
    return torch.float16 if kind == "float16" else torch.bfloat16


@pytest.mark.parametrize("rms", [1.0, 0.1, 0.01, 1e-3, 1e-4])
@pytest.mark.parametrize("rows,d,f,experts,k", [(1, 512, 320, 4, 2), (20, 512, 1408, 8, 2), (300, 256, 544, 3, 2)])
@pytest.mark.parametrize("kind", KINDS)
def test_small_x(env, kind, rows, d, f, experts, k, rms):
    """(300 rows of 3 experts: CTA pairs, several tiles an expert)"""
    torch, ffn = env
    x, idx, w, weights, values = make(torch, kind, rows, d, f, experts, k)
    x = (x * rms).to(storage(torch, kind))
    y = call(env, kind, x, idx, w, weights, f)
    ffn.ffn_device_status()
    check_rows(torch, y, *reference(torch, kind, x, idx, w, values))


@pytest.mark.parametrize("gain", [0.1, 0.02, 2e-3])
@pytest.mark.parametrize("rows", [2, 260])
@pytest.mark.parametrize("kind", KINDS)
def test_small_weights(env, kind, rows, gain):
    torch, ffn = env
    x, idx, w, weights, values = make(torch, kind, rows, 384, 416, 3, 2, gain=gain)
    x = x.to(storage(torch, kind))
    y = call(env, kind, x, idx, w, weights, 416)
    check_rows(torch, y, *reference(torch, kind, x, idx, w, values))


@pytest.mark.parametrize("rows", [9, 70, 400])
@pytest.mark.parametrize("kind", KINDS)
def test_rows_of_all_sizes_in_one_tile(env, kind, rows):
    """Each row keeps its own scale; rows of zeros, and what is captured once
    serves other sizes at replay."""
    torch, ffn = env
    d, f, experts, k = 256, 608, 2, 2
    x, idx, w, weights, values = make(torch, kind, rows, d, f, experts, k)
    sizes = torch.tensor([1.0, 0.05, 1e-3, 0.0, 4.0, 1e-4, 0.2], device="cuda")
    size = sizes[torch.arange(rows, device="cuda") % len(sizes)]
    xs = (x * size[:, None]).to(storage(torch, kind))
    y = call(env, kind, xs, idx, w, weights, f)
    ref, bound = reference(torch, kind, xs, idx, w, values)
    some = size > 0
    check_rows(torch, y[some], ref[some], bound[some])
    assert bool((y[~some] == 0).all())
    for _ in range(20):
        assert torch.equal(call(env, kind, xs, idx, w, weights, f), y)
    # a row's result does not depend on the rows beside it
    alone = call(env, kind, xs[2:3].contiguous(), idx[2:3].contiguous(), w[2:3].contiguous(), weights, f)
    check_rows(torch, alone, ref[2:3], bound[2:3])
    buf, out = xs.clone(), torch.empty_like(xs)
    if kind == "prepared":
        weights = [ffn.ffn_prepare_weights(m) for m in weights]
        need = ffn.ffn_moe_workspace_bytes(rows, d, f, experts, k, xs.dtype, ffn.FFN_PREPARED_WEIGHTS)
        ws = ffn.workspace(need, "cuda")
        def go(): ffn.ffn_moe_forward(buf, idx, w, *weights, flags=ffn.FFN_PREPARED_WEIGHTS, out=out, ws=ws)
    elif kind == "q4":
        ws = ffn.workspace(ffn.ffn_moe_q4_workspace_bytes(rows, d, f, experts, k), "cuda")
        def go(): ffn.ffn_moe_forward_q4(buf, idx, w, *weights, ffn=f, out=out, ws=ws)
    else:
        ws = ffn.workspace(ffn.ffn_moe_workspace_bytes(rows, d, f, experts, k, xs.dtype), "cuda")
        def go(): ffn.ffn_moe_forward(buf, idx, w, *weights, out=out, ws=ws)
    ws.fill_(255)
    go()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for shift in (0, 1, 2, 0):
        buf.copy_((x * size.roll(shift)[:, None]).to(xs.dtype))
        graph.replay()
        want = call(env, kind, buf, idx, w, weights, f) if kind != "prepared" else ffn.ffn_moe_forward(
            buf, idx, w, *weights, flags=ffn.FFN_PREPARED_WEIGHTS)
        assert torch.equal(out, want)
        if shift == 0:
            assert torch.equal(out, y)


@pytest.mark.parametrize("rms", [1.0, 0.02, 1e-3])
@pytest.mark.parametrize("rows", [3, 40, 330])
@pytest.mark.parametrize("kind", KINDS)
def test_features_of_all_sizes(env, kind, rows, rms):
    """Runs of features far below the others, of zeros, and at the end of a row
    that is not a whole number of 32: one scale still holds for the row."""
    torch, ffn = env
    d, f = 256, 32 * 17 + (0 if kind == "q4" else 8)
    fg = torch.ones(f, device="cuda")
    fg[:32] = 2.0 ** -6
    fg[64:128] = 0.0
    fg[128:130] = 2.0 ** -9
    fg[192:256] = 2.0 ** -9
    fg[-24:] = 2.0 ** -5
    for gain in (fg, fg * (torch.arange(f, device="cuda") < 150)):
        x, idx, w, weights, values = make(torch, kind, rows, d, f, 3, 2, feature_gain=gain)
        x = (x * rms).to(storage(torch, kind))
        y = call(env, kind, x, idx, w, weights, f)
        check_rows(torch, y, *reference(torch, kind, x, idx, w, values))


@pytest.mark.parametrize("top", [40.0, 400.0, 8000.0])
@pytest.mark.parametrize("rows", [4, 35, 300])
@pytest.mark.parametrize("kind", KINDS)
def test_large_values_beside_small_ones(env, kind, rows, top):
    """|h| to 10^5 and 10^9 (fp16 ends at 65504) beside rows of 1e-7."""
    torch, ffn = env
    d, f = 256, 320
    x, idx, w, weights, values = make(torch, kind, rows, d, f, 2, 1)
    if kind == "float16":
        top = min(top, 400.0)
        w = w * (20.0 / top) ** 2 / 1024     # keeps y in fp16's range beside w_down's gain of 2^10
    size = torch.tensor([top, 1e-3], device="cuda")[torch.arange(rows, device="cuda") % 2]
    x = (x * size[:, None]).to(storage(torch, kind))
    y = call(env, kind, x, idx, w, weights, f)
    ref, bound = reference(torch, kind, x, idx, w, values)
    if kind == "float16":      # (the small rows' y is below fp16's range there)
        check_rows(torch, y[::2], ref[::2], bound[::2])
        assert bool(((y.double() - ref).abs() <= bound).all())
    else:
        check_rows(torch, y, ref, bound)
    ffn.ffn_device_status()


@pytest.mark.parametrize("kind", KINDS)
def test_infinities_and_nan_stay_in_their_rows(env, kind):
    torch, ffn = env
    rows, d, f = 40, 256, 320
    x, idx, w, weights, values = make(torch, kind, rows, d, f, 2, 1)
    x = (x * torch.tensor([1.0, 1e-3], device="cuda")[torch.arange(rows, device="cuda") % 2][:, None])
    x = x.to(storage(torch, kind))
    ref, bound = reference(torch, kind, x, idx, w, values)
    x[3, 5], x[8, 7] = float("inf"), float("nan")
    y = call(env, kind, x, idx, w, weights, f)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[3] = keep[8] = False
    check_rows(torch, y[keep], ref[keep], bound[keep])
    assert not bool(torch.isfinite(y[~keep]).any())


@pytest.mark.parametrize("kind", KINDS)
def test_many_calls_with_rows_of_all_sizes(env, kind):
    """Rows whose blocks have to be brought to one scale before the down product
    reads them, by whichever warp comes first: the same bits in every call, calls
    queued back to back on two streams, in turn with calls of ordinary values."""
    torch, ffn = env
    rows, d, f, experts, k = 600, 256, 1376, 6, 2
    x, idx, w, weights, values = make(torch, kind, rows, d, f, experts, k)
    size = torch.tensor([1.0, 0.02, 0.012, 0.008, 0.0, 1e-3], device="cuda")[torch.arange(rows, device="cuda") % 6]
    xs = [(x * s).to(storage(torch, kind)) for s in (size[:, None], 0.012, 1.0)]
    flags = {"flags": ffn.FFN_PREPARED_WEIGHTS} if kind == "prepared" else {}
    if kind == "prepared":
        weights = [ffn.ffn_prepare_weights(m) for m in weights]

    def go(i, **kw):
        if kind == "q4":
            return ffn.ffn_moe_forward_q4(xs[i], idx, w, *weights, ffn=f, **kw)
        return ffn.ffn_moe_forward(xs[i], idx, w, *weights, **flags, **kw)
    want = [go(i) for i in range(3)]
    for i in range(2):
        ref, bound = reference(torch, kind, xs[i], idx, w, values)
        some = xs[i].abs().amax(dim=1) > 0
        check_rows(torch, want[i][some], ref[some], bound[some])
    bytes_ = (ffn.ffn_moe_q4_workspace_bytes(rows, d, f, experts, k) if kind == "q4" else
              ffn.ffn_moe_workspace_bytes(rows, d, f, experts, k, xs[0].dtype, flags.get("flags", 0)))
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [ffn.workspace(bytes_, "cuda") for _ in streams]
    got = torch.empty(200, *xs[0].shape, dtype=xs[0].dtype, device="cuda")
    torch.cuda.synchronize()
    for i in range(200):
        go(i // 2 % 3, out=got[i], ws=ws[i % 2], stream=streams[i % 2])
    torch.cuda.synchronize()
    ffn.ffn_device_status()
    for j in range(3):
        part = torch.stack([got[i] for i in range(200) if i // 2 % 3 == j])
        assert bool((part == want[j]).all()), int((part != want[j]).flatten(1).any(dim=1).sum())


@pytest.mark.parametrize("rows,d,f,experts", [(5, 128, 4768, 2), (40, 256, 14336, 2), (300, 128, 4768, 3),
                                              (700, 64, 8224, 2), (33, 1056, 2080, 1)])
@pytest.mark.parametrize("kind", KINDS)
def test_long_rows_of_all_sizes(env, kind, rows, d, f, experts):
    """More levels a row than a warp reads at once, and down products that are
    split, so that several blocks need the same rows."""
    torch, ffn = env
    fg = torch.ones(f, device="cuda")
    fg[f // 3:f // 2] = 2.0 ** -8
    fg[f // 2:f // 2 + 640] = 0.0
    x, idx, w, weights, values = make(torch, kind, rows, d, f, experts, 1, feature_gain=fg)
    sizes = torch.tensor([0.02, 1.0, 0.0, 3.0, 0.004], device="cuda")
    size = sizes[torch.arange(rows, device="cuda") % len(sizes)]
    x = (x * size[:, None]).to(storage(torch, kind))
    y = call(env, kind, x, idx, w, weights, f)
    ref, bound = reference(torch, kind, x, idx, w, values)
    some = size > 0
    check_rows(torch, y[some], ref[some], bound[some])
    assert bool((y[~some] == 0).all())
    for _ in range(10):
        assert torch.equal(call(env, kind, x, idx, w, weights, f), y)
    ffn.ffn_device_status()


@pytest.mark.parametrize("kind", ["prepared", "float16"])
def test_a_rows_scale_does_not_depend_on_its_neighbours(env, kind):
    """The largest h of a row just below 2^-12, where rounding to fp16 reaches it
    (h = 32 U, U = 2^-17 (1 - 2^-13)), beside one of 2^-26, which is 0 at the
    scale of 2^-12 and not at the next: the same bits alone, beside smaller rows
    and beside larger ones."""
    torch, ffn = env
    d, f = 64, 64
    dt = storage(torch, kind)
    gate, up, down = (torch.zeros(1, o, i, device="cuda") for o, i in ((f, d), (f, d), (d, f)))
    gate[0, :, 0] = 32.0
    up[0, 0, 0], up[0, 0, 1], up[0, 1, 2] = 2.0 ** -17, -2.0 ** -20, 2.0 ** -20
    down[0, :, 0], down[0, ::2, 1] = 1.0, 128.0   # (prepared weights are below 256)
    x = torch.zeros(9, d, device="cuda")
    x[:, 0], x[:, 1], x[:, 2] = 1.0, 2.0 ** -10, 2.0 ** -11
    x[1:] *= 2.0 ** -4
    weights = [m.to(dt) for m in (gate, up, down)]
    idx = torch.zeros(9, 1, dtype=torch.int32, device="cuda")
    w = torch.full((9, 1), 2.0 ** 10, device="cuda")

    def first(rows):
        return call(env, kind, rows.to(dt), idx[:len(rows)], w[:len(rows)], weights, f)[0]
    alone = first(x[:1])
    assert torch.equal(first(x), alone)
    large = x.clone()
    large[1:] *= 256
    assert torch.equal(first(large), alone)
    assert bool((alone.double() - 2.0 ** -2).abs().max() <= 2.0 ** -9)
