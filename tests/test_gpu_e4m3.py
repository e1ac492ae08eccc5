"""ffn_quantize_e4m3, ffn_linear_e4m3 and ffn_gateup_e4m3 against their formulas in
64 bits (tolerances: e4m3_util)."""

import pytest

import e4m3_util as u

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    from transformer_ffn_rmsnorm_gb300 import ffn
    return torch, ffn


# ------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("rows,d", [(1, 1), (3, 7), (1, 128), (5, 130), (9, 264), (33, 96), (2, 4096), (300, 1000),
                                    (4099, 136)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize_rows(env, rows, d, dtype, group):
    torch, ffn = env
    gen = torch.Generator(device="cuda").manual_seed(rows + d)
    x = (torch.randn(rows, d, generator=gen, device="cuda") * 3).to(getattr(torch, dtype))
    q, s = ffn.ffn_quantize_e4m3(x, group=group)
    assert s.shape == (rows, -(-d // group))
    u.check_quantized(torch, q, s, x.double(), torch.zeros_like(x, dtype=torch.float64), group)


def blocks_of(torch, x, q, s):
    rows, d = x.shape
    for i in range(-(-rows // 128)):
        for j in range(-(-d // 128)):
            b = x[128 * i:128 * i + 128, 128 * j:128 * j + 128].double()
            c = q[128 * i:128 * i + 128, 128 * j:128 * j + 128]
            flat, z = b.reshape(1, -1), torch.zeros(1, b.numel(), device="cuda", dtype=torch.float64)
            u.check_quantized(torch, c.reshape(1, -1).float(), s[i:i + 1, j:j + 1], flat, z, flat.shape[1])


@pytest.mark.parametrize("rows,d", [(1, 16), (128, 128), (130, 144), (16, 400), (384, 272)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
def test_quantize_blocks(env, rows, d, dtype):
    torch, ffn = env
    gen = torch.Generator(device="cuda").manual_seed(rows + d)
    x = torch.randn(2, rows, d, generator=gen, device="cuda").to(getattr(torch, dtype))
    x[0, 0, 0] = 100.0
    q, s = ffn.ffn_quantize_e4m3(x, block_rows=128)
    assert s.shape == (2, -(-rows // 128), -(-d // 128))
    for e in range(2):
        blocks_of(torch, x[e], q[e], s[e])
    if rows % 16 == 0:
        qt, st = ffn.ffn_quantize_e4m3(x, block_rows=128, transpose=True)
        assert torch.equal(qt.view(torch.uint8), q.view(torch.uint8).transpose(1, 2))
        assert torch.equal(st, s.transpose(1, 2))


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("block_rows,d", [(1, 384), (128, 384), (1, 333)])
def test_quantize_special_values(env, dtype, block_rows, d):
    """Zeros, a NaN, an infinity: their blocks alone."""
    torch, ffn = env
    x = torch.ones(128, d, device="cuda").to(getattr(torch, dtype))
    x[:, 0:128] = 0
    x[5, 130] = float("nan")
    x[7, 260] = float("-inf")
    q, s = ffn.ffn_quantize_e4m3(x, block_rows=block_rows)
    v = q.float()
    assert bool((v[:, :128] == 0).all())
    assert torch.equal(s[:, 0], torch.full_like(s[:, 0], 2.0 ** -100 / 448))
    r = 5 if block_rows == 1 else 0
    assert bool(s[r, 1].isnan()) and bool(v[5, 130].isnan())
    r = 7 if block_rows == 1 else 0
    assert bool(s[r, 2].isinf()) and bool(v[7, 260].isnan()) and bool((v[7, 256:260] == 0).all())
    if block_rows == 1:
        assert bool((v[8, 128:] == 448).all())


# ------------------------------------------------------------------ products
SHAPES = [(1, 16, 8), (1, 128, 128), (1, 4096, 1000), (2, 144, 136), (15, 1040, 72), (16, 256, 384), (17, 48, 200),
          (32, 2048, 128), (33, 512, 264), (64, 1024, 640), (100, 384, 1000), (128, 4096, 256), (129, 272, 136),
          (255, 1536, 392), (300, 640, 128), (777, 1024, 520), (1030, 512, 2056)]


@pytest.mark.parametrize("rows,inn,out", SHAPES)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
def test_linear(env, rows, inn, out, dtype):
    torch, ffn = env
    dt = getattr(torch, dtype)
    x, (w,) = u.make(torch, rows, inn, [out], 0, rows + inn)
    y = ffn.ffn_linear_e4m3(*x, w, dtype=dt)
    ref, mag = u.product(torch, x, w)
    u.check_linear(torch, y, ref, mag, inn)
    res = torch.randn(rows, out, device="cuda").to(dt)
    z = res.clone()
    ffn.ffn_linear_e4m3(*x, w, res=z, out=z)      # in the residual's place
    u.check_linear(torch, z, ref, mag, inn, res)
    assert torch.equal(y, ffn.ffn_linear_e4m3(*x, w, dtype=dt))
    ffn.ffn_device_status()


@pytest.mark.parametrize("rows,inn,out", SHAPES)
def test_gateup(env, rows, inn, out):
    torch, ffn = env
    x, (wg, wu) = u.make(torch, rows, inn, [out, out], 0, rows + inn + 1)
    q, s = ffn.ffn_gateup_e4m3(*x, wg, wu)
    u.check_gateup(torch, q, s, x, wg, wu, inn)
    ffn.ffn_device_status()


def offsets_of(torch, counts, first=0):
    at = [first]
    for c in counts:
        at.append(at[-1] + c)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


COUNTS = [[1], [0, 0, 1], [3, 0, 5, 1], [16, 17, 0, 33], [1, 40, 0, 129, 2], [300, 0, 1, 257, 128], [0, 0, 0],
          [2] * 70, [7, 260, 31, 600]]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}e{sum(c)}")
@pytest.mark.parametrize("inn,out,more", [(272, 200, 0), (640, 384, 5)])
def test_by_expert(env, counts, inn, out, more):
    """Experts without rows; rows of no expert at the end are left as they were."""
    torch, ffn = env
    rows = sum(counts) + more
    if rows == 0:
        rows = more = 3
    x, (wg, wu) = u.make(torch, rows, inn, [out, out], len(counts), rows)
    off = offsets_of(torch, counts)
    y = torch.full((rows, out), 7.0, device="cuda", dtype=torch.bfloat16)
    ffn.ffn_linear_e4m3(*x, wg, offsets=off, out=y)
    ref, mag = u.product(torch, x, wg, off)
    n = rows - more
    u.check_linear(torch, y[:n], ref[:n], mag[:n], inn)
    assert bool((y[n:] == 7).all())
    q = torch.full((rows, out), 3.0, device="cuda").to(torch.float8_e4m3fn)
    s = torch.full((rows, -(-out // 128)), 5.0, device="cuda")
    ffn.ffn_gateup_e4m3(*x, wg, wu, offsets=off, out=q, scales=s)
    u.check_gateup(torch, q, s, x, wg, wu, inn, off, slice(0, n))
    assert bool((q[n:].float() == 3).all()) and bool((s[n:] == 5).all())
    ffn.ffn_device_status()


@pytest.mark.parametrize("rows", [40, 700])
def test_offsets_out_of_range(env, rows):
    """A first row behind 0, ends beyond the rows or before their starts: no row outside is written."""
    torch, ffn = env
    x, (w,) = u.make(torch, rows, 256, [136], 5, 3)
    off = torch.tensor([-5, 9, 4, 20, rows + 1000, 30], dtype=torch.int32, device="cuda")
    eff = [(0, 9), (9, 9), (4, 20), (20, rows), (rows, rows)]
    room = torch.full((rows + 64, 136), 7.0, device="cuda", dtype=torch.float32)
    ffn.ffn_linear_e4m3(*x, w, offsets=off, out=room[:rows])
    assert bool((room[rows:] == 7).all())
    for e, (a, b) in enumerate(eff):
        if e in (0, 2):      # (rows of two experts, 4 to 8, are either's)
            a, b = (0, 4) if e == 0 else (9, 20)
        if b > a:
            ref, mag = u.product(torch, (x[0][a:b], x[1][a:b]), (w[0][e], w[1][e]))
            u.check_linear(torch, room[a:b], ref, mag, 256)
    ffn.ffn_device_status()


@pytest.mark.parametrize("rows", [3, 50, 600])
def test_special_rows(env, rows):
    """A row with a NaN scale or codes stays alone; a row of zeros gives zeros."""
    torch, ffn = env
    x, (wg, wu) = u.make(torch, rows, 384, [264, 264], 0, 9)
    x[1][0, 1] = float("nan")
    x[0].view(torch.uint8)[1, 5] = 0x7F
    x[0].view(torch.uint8)[2] = 0
    y = ffn.ffn_linear_e4m3(*x, wg, dtype=torch.float32)
    assert bool(y[:2].isnan().all()) and bool((y[2] == 0).all()) and bool(y[3:].isfinite().all())
    q, s = ffn.ffn_gateup_e4m3(*x, wg, wu)
    assert bool(s[:2].isnan().all()) and bool((q[2].float() == 0).all()) and bool(s[2:].isfinite().all())
    assert torch.equal(s[2], torch.full_like(s[2], 2.0 ** -100 / 448))
    ffn.ffn_device_status()


@pytest.mark.parametrize("rows", [1, 20, 200])
def test_exact_values(env, rows):
    """Whole numbers and scales of powers of two: the sums are exact."""
    torch, ffn = env
    gen = torch.Generator(device="cuda").manual_seed(rows)
    xq = torch.randint(-8, 9, (rows, 640), generator=gen, device="cuda").float().to(torch.float8_e4m3fn)
    wq = torch.randint(-8, 9, (264, 640), generator=gen, device="cuda").float().to(torch.float8_e4m3fn)
    xs = torch.ldexp(torch.ones(rows, 5, device="cuda"), torch.randint(-2, 3, (rows, 5), generator=gen, device="cuda"))
    ws = torch.ldexp(torch.ones(3, 5, device="cuda"), torch.randint(-2, 3, (3, 5), generator=gen, device="cuda"))
    y = ffn.ffn_linear_e4m3(xq, xs, (wq, ws), dtype=torch.float32)
    assert torch.equal(y.double(), u.product(torch, (xq, xs), (wq, ws))[0])


@pytest.mark.parametrize("rows", [1, 24, 200, 600])
def test_scale_range(env, rows):
    """Tiny and huge scales beside each other."""
    torch, ffn = env
    x, (w,) = u.make(torch, rows, 512, [136], 0, 11)
    x[1][:, 0] *= 2.0 ** 60
    w[1][:, 0] *= 2.0 ** -60
    x[1][:, 2] *= 2.0 ** -100
    y = ffn.ffn_linear_e4m3(*x, w, dtype=torch.float32)
    ref, mag = u.product(torch, x, w)
    u.check_linear(torch, y, ref, mag, 512)


def test_gradient_of_x(env):
    """dX = dY W through the transposed weight, against the formula and differences of the product."""
    torch, ffn = env
    gen = torch.Generator(device="cuda").manual_seed(5)
    w = torch.randn(400, 272, generator=gen, device="cuda") / 16
    q, s = ffn.ffn_quantize_e4m3(w, block_rows=128)
    qt, st = ffn.ffn_quantize_e4m3(w, block_rows=128, transpose=True)
    dy = ffn.ffn_quantize_e4m3(torch.randn(37, 400, generator=gen, device="cuda"))
    dx = ffn.ffn_linear_e4m3(*dy, (qt, st), dtype=torch.float32)
    m, v = u.values(q, s, 128), u.values(*dy, 1)
    u.check_linear(torch, dx, v @ m, v.abs() @ m.abs(), 400)
    # the product is linear: <dy, P(x + e) - P(x)> = <dx, e>
    x = ffn.ffn_quantize_e4m3(torch.randn(2, 37, 272, generator=gen, device="cuda"))
    a, b = (ffn.ffn_linear_e4m3(x[0][i], x[1][i], (q, s), dtype=torch.float32).double() for i in range(2))
    step = u.values(x[0][0], x[1][0], 1) - u.values(x[0][1], x[1][1], 1)
    left, right = (v * (a - b)).sum(), (dx.double() * step).sum()
    mags = (v.abs() * (a.abs() + b.abs())).sum()
    assert abs(float(left - right)) <= float(mags) * 2 * u.product_err(400) * 16


@pytest.mark.parametrize("start,end", [(1, 40), (3, 4), (37, 333)])
def test_rows_in_pieces(env, start, end):
    """Rows of a batch whose scales (7 a row) do not start on 16 bytes."""
    torch, ffn = env
    x, (wg, wu) = u.make(torch, 333, 880, [264, 264], 0, 4)
    p = (x[0][start:end], x[1][start:end])
    ref, mag = u.product(torch, p, wg)
    u.check_linear(torch, ffn.ffn_linear_e4m3(*p, wg), ref, mag, 880)
    s = torch.zeros(333, 3, device="cuda")
    q, _ = ffn.ffn_gateup_e4m3(*p, wg, wu, scales=s[start:end])      # (its rows of 264 codes start on 8 bytes)
    u.check_gateup(torch, q, s[start:end], p, wg, wu, 880)
    assert bool((s[:start] == 0).all()) and bool((s[end:] == 0).all())
    h = torch.randn(333, 880, device="cuda")
    s = torch.zeros(333, 7, device="cuda")
    q, _ = ffn.ffn_quantize_e4m3(h[start:end], scales=s[start:end])
    u.check_quantized(torch, q, s[start:end], h[start:end].double(), torch.zeros(end - start, 880, device="cuda"))


SKEWED = [[0] * 20 + [500, 3] + [0] * 10, [1] * 40 + [333], [0, 0, 700, 0], [90] + [0] * 63]


@pytest.mark.parametrize("counts", SKEWED, ids=lambda c: f"{len(c)}e{max(c)}")
def test_one_expert_has_most_rows(env, counts):
    """The mean alone chooses the kernel: few rows an expert, but many of one."""
    torch, ffn = env
    rows = sum(counts)
    x, (wg, wu) = u.make(torch, rows, 400, [264, 264], len(counts), rows)
    off = offsets_of(torch, counts)
    ref, mag = u.product(torch, x, wg, off)
    u.check_linear(torch, ffn.ffn_linear_e4m3(*x, wg, offsets=off), ref, mag, 400)
    q, s = ffn.ffn_gateup_e4m3(*x, wg, wu, offsets=off)
    u.check_gateup(torch, q, s, x, wg, wu, 400, off)
    ffn.ffn_device_status()


@pytest.mark.parametrize("counts", [[3, 0, 5, 1], [40, 0, 61], [300, 0, 1, 257], [0, 90] + [0] * 62],
                         ids=lambda c: f"{len(c)}e{sum(c)}")
@pytest.mark.parametrize("out", [136, 384])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
def test_residual_by_expert(env, counts, out, dtype):
    """Elsewhere and in place; rows of no expert keep what they hold, the residual or not."""
    torch, ffn = env
    dt, n, more = getattr(torch, dtype), sum(counts), 6
    x, (w,) = u.make(torch, n + more, 272, [out], len(counts), n)
    off = offsets_of(torch, counts)
    ref, mag = u.product(torch, x, w, off)
    res = torch.randn(n + more, out, device="cuda").to(dt)
    y = torch.full_like(res, 7.0)
    ffn.ffn_linear_e4m3(*x, w, offsets=off, res=res, out=y)
    u.check_linear(torch, y[:n], ref[:n], mag[:n], 272, res[:n])
    assert bool((y[n:] == 7).all())
    z = res.clone()
    ffn.ffn_linear_e4m3(*x, w, offsets=off, res=z, out=z)
    assert torch.equal(z[:n], y[:n]) and torch.equal(z[n:], res[n:])
    ffn.ffn_device_status()


@pytest.mark.parametrize("rows,inn,out", [(257, 2048, 264), (300, 1296, 392), (512, 4096, 1024), (511, 144, 72),
                                          (640, 4096, 4096), (1500, 1024, 4104)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
def test_linear_of_few_and_many_units(env, rows, inn, out, dtype):
    """Units of 128 and of 256 features, whole and cut at the edges, with and without a residual."""
    torch, ffn = env
    dt = getattr(torch, dtype)
    x, (w,) = u.make(torch, rows, inn, [out], 0, rows + out)
    ref, mag = u.product(torch, x, w)
    room = torch.full((rows + 8, out), 7.0, device="cuda", dtype=dt)
    ffn.ffn_linear_e4m3(*x, w, out=room[:rows])
    u.check_linear(torch, room[:rows], ref, mag, inn)
    assert bool((room[rows:] == 7).all())
    res = torch.randn(rows, out, device="cuda").to(dt)
    u.check_linear(torch, ffn.ffn_linear_e4m3(*x, w, res=res), ref, mag, inn, res)
    ffn.ffn_device_status()
