"""ffn_add_rmsnorm and ffn_add_rmsnorm_e4m3 against the formula in 64 bits.

Tolerances, derived: r is one fp32 addition and one rounding, so it is compared
bit for bit.  v = r * rsqrt(mean r^2 + eps) * g in fp32: the sum of squares of
non-negative terms is off by at most its depth in additions (a thread's share
of the row, at most d / 256 where the row is read element by element, 32
elements where it is held in registers; then 10 levels) times 2^-24, halved by
the root; the division, eps, rsqrtf (2 ulp) and two products add at most 8 x
2^-24.  n adds the storage type's half step, a scale two more roundings, and a
code half a step of e4m3 (2^-4 of its value, 2^-10 below 2^-6) of v / scale,
which carries twice v's error."""

import pytest

pytestmark = pytest.mark.gpu

EPS = 1e-6
FLOOR = 2.0 ** -100


@pytest.fixture(scope="module")
def env():
    import torch
    from transformer_ffn_rmsnorm_gb300 import ffn
    return torch, ffn


def make(torch, rows, d, dt, seed, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(rows, d, generator=gen, device="cuda") * scale).to(dt)
    res = (torch.randn(rows, d, generator=gen, device="cuda") * 3 * scale).to(dt)
    g = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dt)
    return x, res, g


def reference(torch, x, res, g):
    r = x if res is None else (x.float() + res.float()).to(x.dtype)
    r64 = r.double()
    v = r64 / torch.sqrt((r64 * r64).mean(dim=-1, keepdim=True) + EPS) * g.double()
    return r, v


def v_err(d):
    return (max(32, -(-d // 256)) + 10) * 2.0 ** -25 + 8 * 2.0 ** -24


def check_n(torch, n, v, d):
    fi = torch.finfo(n.dtype)
    tol = v.abs() * (fi.eps / 2 + 2 * v_err(d)) + fi.tiny * fi.eps / 2
    assert bool(((n.double() - v).abs() <= tol).all())


def check_q(torch, q, scales, v, group):
    rows, d = v.shape
    group = group or d
    e = 2 * v_err(d) + 4 * 2.0 ** -24
    for j, c in enumerate(range(0, d, group)):
        part = v[:, c:c + group]
        s = part.abs().amax(dim=1).clamp(min=FLOOR) / 448.0
        assert bool(((scales[:, j].double() - s).abs() <= s * e).all()), j
        t = part / s[:, None]
        got = q[:, c:c + group].double()
        assert bool(((got - t).abs() <= torch.maximum(t.abs() * 2.0 ** -4, t.new_tensor(2.0 ** -10)) + t.abs() * 2 * e).all())
        assert bool((got.abs() <= 448).all())


SHAPES = [(1, 1), (5, 7), (3, 8), (2, 100), (9, 264), (1, 4096), (33, 5120), (700, 1024), (3, 20000), (2, 40000),
          (2, 33001)]


@pytest.mark.parametrize("rows,d", SHAPES)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("with_res", [True, False])
def test_norm(env, rows, d, dtype, with_res):
    torch, ffn = env
    x, res, g = make(torch, rows, d, getattr(torch, dtype), rows + d)
    res = res if with_res else None
    r_ref, v = reference(torch, x, res, g)
    r, n = ffn.ffn_add_rmsnorm(x, g, EPS, res=res)
    assert torch.equal(r, r_ref)
    check_n(torch, n, v, d)


@pytest.mark.parametrize("rows,d", SHAPES)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
def test_e4m3(env, rows, d, dtype, group):
    torch, ffn = env
    x, res, g = make(torch, rows, d, getattr(torch, dtype), rows + d + group)
    r_ref, v = reference(torch, x, res, g)
    r, q, scales = ffn.ffn_add_rmsnorm_e4m3(x, g, EPS, res=res, group=group)
    assert torch.equal(r, r_ref)
    assert scales.shape == (rows, -(-d // group) if group else 1)
    check_q(torch, q, scales, v, group)


@pytest.mark.parametrize("d", [4096, 4095, 40000])
@pytest.mark.parametrize("quant", [False, True])
def test_in_place(env, d, quant):
    """r in x's or res's place, n in x's: the results of separate outputs, and
    rows behind the last one untouched."""
    torch, ffn = env
    x, res, g = make(torch, 6, d, torch.bfloat16, 5)
    call = ((lambda x, res, **k: ffn.ffn_add_rmsnorm_e4m3(x, g, EPS, res=res, group=128, **k)) if quant
            else (lambda x, res, **k: ffn.ffn_add_rmsnorm(x, g, EPS, res=res, **k)))
    want = [t.clone() for t in call(x, res)]
    for place in ("x", "res"):
        full_x, full_res = torch.cat([x, x]), torch.cat([res, res])
        a, b = full_x[:6], full_res[:6]
        got = call(a, b, r_out=a if place == "x" else b)
        assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(got, want))
        assert torch.equal(full_x[6:], x) and torch.equal(full_res[6:], res)
    if not quant:
        a = x.clone()
        r, n = ffn.ffn_add_rmsnorm(a, g, EPS, res=res, out=a, r_out=torch.empty_like(x))
        assert torch.equal(r, want[0]) and torch.equal(n, want[1])


def test_same_bits_as_rmsnorm(env):
    """n is ffn_rmsnorm of r, up to the order of the row's sum: never more
    than one step of the storage type apart."""
    torch, ffn = env
    x, res, g = make(torch, 64, 4096, torch.bfloat16, 11)
    r, n = ffn.ffn_add_rmsnorm(x, g, EPS, res=res)
    other = ffn.ffn_rmsnorm(r, g, EPS)
    assert bool(((n.double() - other.double()).abs() <= other.double().abs() * torch.finfo(torch.bfloat16).eps).all())
    assert float((n == other).double().mean()) > 0.99


@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("d", [512, 509])
def test_zero_tiny_huge_and_not_finite(env, d, group):
    torch, ffn = env
    x, _, g = make(torch, 6, d, torch.float32, 3)
    x[0] = 0
    x[1] *= 1e-25                       # squares vanish: v = x / sqrt(eps)
    x[2] *= 1e18
    x[3, 5] = float("nan")
    x[4, 40] = float("inf")
    _, q, scales = ffn.ffn_add_rmsnorm_e4m3(x, g, EPS, group=group)
    _, v = reference(torch, x[:3], None, g)
    check_q(torch, q[:3], scales[:3], v, group)
    assert bool((q[0].float() == 0).all()) and bool((scales[0] > 0).all())
    assert bool(torch.isnan(scales[3]).all()) and bool(torch.isnan(q[3].float()).all())
    at = 40 // group if group else 0    # infinity: v is NaN there and 0 elsewhere
    assert bool(torch.isnan(scales[4, at]))
    if group:
        rest = [j for j in range(scales.shape[1]) if j != at]
        assert bool((scales[4, rest] > 0).all()) and bool((q[4, (at + 1) * group:].float() == 0).all())


def test_streams_graph_and_empty(env):
    torch, ffn = env
    x, res, g = make(torch, 40, 1024, torch.bfloat16, 9)
    want = ffn.ffn_add_rmsnorm(x, g, EPS, res=res)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ffn.ffn_add_rmsnorm(x, g, EPS, res=res, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    r, n = torch.empty_like(x), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ffn.ffn_add_rmsnorm(x, g, EPS, res=res, r_out=r, out=n)
    x2, res2, _ = make(torch, 40, 1024, torch.bfloat16, 10)
    x.copy_(x2)
    res.copy_(res2)
    graph.replay()
    want = ffn.ffn_add_rmsnorm(x2, g, EPS, res=res2)
    assert torch.equal(r, want[0]) and torch.equal(n, want[1])
    before = ffn.ffn_launch_count()
    r, q, sc = ffn.ffn_add_rmsnorm_e4m3(x[:0], g, EPS, res=res[:0], group=64)
    assert q.shape == (0, 1024) and sc.shape == (0, 16) and ffn.ffn_launch_count() == before
    ffn.ffn_device_status()
