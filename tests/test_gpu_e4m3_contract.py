"""What include/ffn.h says of the e4m3 operators beyond their formulas' tolerances: the codes' bits,
falling offsets, where scales and pointers may lie."""

import pytest

import e4m3_util as u

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    from transformer_ffn_rmsnorm_gb300 import ffn
    return torch, ffn


# ------------------------------------------------------------------ bits
def quantized(torch, x, block_rows, group):
    """(codes, scales) of x [rows, d] by the formula in 32 bits on the host, each step rounded to nearest even."""
    v = x.float().cpu().numpy()
    rows, d = v.shape
    q, s = v.copy(), []
    for r in range(0, rows, block_rows):
        line = []
        for c in range(0, d, group):
            b = v[r:r + block_rows, c:c + group]
            one = b.dtype.type
            a = max(abs(b).max(), one(2.0 ** -100))
            line.append(a / one(448))
            q[r:r + block_rows, c:c + group] = b * (one(448) / a)
        s.append(line)
    q = torch.from_numpy(q).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).cuda(), torch.tensor(s, dtype=torch.float32, device="cuda")


@pytest.mark.parametrize("rows,d,block_rows,group", [(300, 1000, 1, 128), (77, 130, 1, 128), (129, 264, 1, 64),
                                                     (65, 96, 1, 32), (400, 656, 128, 128)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
def test_quantize_bit_for_bit(env, rows, d, block_rows, group, dtype):
    """Values of 16 bits lie on ties between codes, where the last bit of 448 / a decides: the quotient is the
    nearest one, not 448 times a rounded reciprocal."""
    torch, ffn = env
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = (torch.randn(rows, d, generator=gen, device="cuda") * 3).to(getattr(torch, dtype))
    q, s = ffn.ffn_quantize_e4m3(x, block_rows=block_rows, group=group)
    want, scales = quantized(torch, x, block_rows, group)
    assert torch.equal(s, scales)
    assert torch.equal(q.view(torch.uint8), want)


# ------------------------------------------------------------------ rows of a batch
@pytest.mark.parametrize("d", [1, 7, 130, 132, 136, 264, 1001])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
def test_quantize_any_rows_of_a_batch(env, d, dtype):
    """x and q begin where a row does, or where an element does if rows are read one by one; what is around stays."""
    torch, ffn = env
    dt = getattr(torch, dtype)
    x = torch.randn(10, d, device="cuda").to(dt)
    for first, rows in ((1, 4), (3, 7), (9, 1)):
        part = x[first:first + rows]
        room = torch.full((10, d), 3.0, device="cuda").to(torch.float8_e4m3fn)
        q = room[first:first + rows]
        _, s = ffn.ffn_quantize_e4m3(part, out=q)
        u.check_quantized(torch, q, s, part.double(), torch.zeros(rows, d, device="cuda", dtype=torch.float64))
        assert bool((room[:first].float() == 3).all()) and bool((room[first + rows:].float() == 3).all())
    if d * x.element_size() % 16:
        flat = torch.randn(4 * d + 1, device="cuda").to(dt)[1:].view(4, d)
        q = torch.zeros(4 * d + 3, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[3:].view(4, d)
        _, s = ffn.ffn_quantize_e4m3(flat, out=q)
        u.check_quantized(torch, q, s, flat.double(), torch.zeros(4, d, device="cuda", dtype=torch.float64))


@pytest.mark.parametrize("start,end", [(1, 30), (3, 4), (37, 333)])
@pytest.mark.parametrize("out", [264, 136])
def test_gateup_into_any_rows_of_a_batch(env, start, end, out):
    """Codes whose rows begin on 8 bytes; what is around stays."""
    torch, ffn = env
    x, (wg, wu) = u.make(torch, 333, 400, [out, out], 0, 4)
    p = (x[0][start:end], x[1][start:end])
    room = torch.full((333, out), 3.0, device="cuda").to(torch.float8_e4m3fn)
    q, s = ffn.ffn_gateup_e4m3(*p, wg, wu, out=room[start:end])
    u.check_gateup(torch, q, s, p, wg, wu, 400)
    assert bool((room[:start].float() == 3).all()) and bool((room[end:].float() == 3).all())
    whole, scales = ffn.ffn_gateup_e4m3(*p, wg, wu)
    assert torch.equal(whole.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s, scales)
    ffn.ffn_device_status()


# ------------------------------------------------------------------ offsets that fall
def falling(rows):
    """Offsets and where each expert's rows begin and end: an offset below one before it counts as that one, and what
    is beyond 0 .. rows as the nearest of the two."""
    few = [-5, 9, 4, 20, rows + 1000, 30]
    many = [min(e * 2, rows - 8) for e in range(71)]
    many[31], many[32], many[33] = rows - 20, 3, rows - 18        # falls from the 32nd expert on, and rises
    many[63], many[64], many[65] = rows - 6, -100, rows - 7        # the same at the 64th
    for e in range(34, 63):
        many[e] = rows - 30 + e // 3                               # (below what came before, then beyond it)
    for off in (few, many):
        top, at = 0, []
        for v in off:
            top = max(top, min(max(v, 0), rows))
            at.append(top)
        yield off, at


@pytest.mark.parametrize("rows", [40, 240, 900, 5000])
@pytest.mark.parametrize("experts", [5, 70])
@pytest.mark.parametrize("out", [136, 384])
def test_offsets_that_fall(env, rows, experts, out):
    """Every row is its one expert's, also across the groups of 32 experts that are looked at together; rows of no
    expert stay."""
    torch, ffn = env
    (off, at), = [c for c in falling(rows) if len(c[0]) == experts + 1]
    x, (wg, wu) = u.make(torch, rows, 256, [out, out], experts, rows)
    given = torch.tensor(off, dtype=torch.int32, device="cuda")
    counts = torch.tensor(at, dtype=torch.int32, device="cuda")
    first, end = at[0], at[-1]
    room = torch.full((rows + 64, out), 7.0, device="cuda")
    ffn.ffn_linear_e4m3(*x, wg, offsets=given, out=room[:rows])
    ref, mag = u.product(torch, x, wg, counts)
    s = slice(first, end)
    u.check_linear(torch, room[s], ref[s], mag[s], 256)
    assert bool((room[:first] == 7).all()) and bool((room[end:] == 7).all())
    codes = torch.full((rows + 64, out), 3.0, device="cuda").to(torch.float8_e4m3fn)
    sc = torch.full((rows + 64, -(-out // 128)), 5.0, device="cuda")
    ffn.ffn_gateup_e4m3(*x, wg, wu, offsets=given, out=codes[:rows], scales=sc[:rows])
    u.check_gateup(torch, codes[:rows], sc[:rows], x, wg, wu, 256, counts, s)
    assert bool((codes[end:].float() == 3).all()) and bool((sc[end:] == 5).all())
    ffn.ffn_device_status()


# ------------------------------------------------------------------ range of scales
@pytest.mark.parametrize("rows", [1, 24, 48, 200, 700])
@pytest.mark.parametrize("ex,ew", [(-63, -63), (-126, 0), (0, -126), (-90, -36), (60, 60), (110, 10)])
def test_scales_whose_product_is_at_the_end_of_its_range(env, rows, ex, ew):
    """Powers of two whose product is a normal fp32 number, the smallest among them, times whole numbers: exact."""
    torch, ffn = env
    gen = torch.Generator(device="cuda").manual_seed(rows)

    def whole(*shape):
        return torch.randint(-1, 2, shape, generator=gen, device="cuda").float().to(torch.float8_e4m3fn)
    xq, wq = whole(rows, 400), whole(264, 400)
    xs = torch.full((rows, 4), 2.0, device="cuda", dtype=torch.float64).pow(ex).float()
    ws = torch.full((3, 4), 2.0, device="cuda", dtype=torch.float64).pow(ew).float()
    xq.view(torch.uint8)[:, 60:] = 0      # |sums| <= 60 in the first block, 0 in the others
    y = ffn.ffn_linear_e4m3(xq, xs, (wq, ws), dtype=torch.float32)
    want = (xq.double() @ wq.double().T) * 2.0 ** (ex + ew)
    assert torch.equal(y.double(), want)
    ffn.ffn_device_status()


@pytest.mark.parametrize("rows", [1, 200])
def test_silu_that_vanishes(env, rows):
    """Gates of -80, -88 and -96 beside an up of 2^100: the last two count 0, the first does not."""
    torch, ffn = env
    codes = torch.zeros(24, 16, device="cuda")
    codes[:, 0] = torch.tensor([-320.0, -352.0, -384.0], device="cuda").repeat_interleave(8)
    x = torch.zeros(rows, 16, device="cuda")
    x[:, 0] = 1
    one = torch.ones(1, 1, device="cuda")
    up = torch.zeros(24, 16, device="cuda")
    up[:, 0] = 1

    def e4m3(v):
        return v.to(torch.float8_e4m3fn)
    q, s = ffn.ffn_gateup_e4m3(e4m3(x), torch.ones(rows, 1, device="cuda"), (e4m3(codes), one * 0.25),
                               (e4m3(up), one * 2.0 ** 100))
    g = torch.tensor(-80.0, dtype=torch.float64)
    h = (g * torch.sigmoid(g) * 2.0 ** 100).abs()
    assert bool(((s.double().cpu() - h / 448).abs() <= h / 448 * (6 + 1.17 * 80) * 2.0 ** -23).all())
    assert bool((q[:, :8].float() == -448).all()) and bool((q[:, 8:].float() == 0).all())
    ffn.ffn_device_status()
