"""Inputs, references in 64 bits and derived tolerances of the e4m3 products.

Tolerance of a product, relative to A = the sum of the magnitudes of its terms: a
tensor-core step adds 32 exact products and the sum so far, each cut to 2^-23 of
the largest at the least: 33 * 2^-23 a step, four steps a block, under 2^-15.9 of
the block's magnitudes in all.  Blocks are added in fp32, nkb of them in up to 8
parts: (nkb + 8) * 2^-24; the scales' product, its product with the sum and res
add 4 * 2^-24.  The output's rounding is half a step of its type."""

import math

BLOCK = 128


def make(torch, rows, inn, outs, experts, seed, scale=1.0):
    """x codes and scales, and a (codes, scales) weight for each of `outs`."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kb = -(-inn // BLOCK)

    def codes(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(60).clamp_(-448, 448).to(torch.float8_e4m3fn)

    def scales(*shape):
        return (0.25 + torch.rand(*shape, generator=gen, device="cuda")) / 60
    x = codes(rows, inn), scales(rows, kb) * scale
    lead = (experts,) if experts else ()
    ws = [(codes(*lead, o, inn), scales(*lead, -(-o // BLOCK), kb) / math.sqrt(inn)) for o in outs]
    return x, ws


def values(q, s, block_rows):
    """64-bit values of codes with scales for each block_rows x 128."""
    v = q.double()
    wide = s.double().repeat_interleave(block_rows, dim=-2)[..., :q.shape[-2], :]
    return v * wide.repeat_interleave(BLOCK, dim=-1)[..., :q.shape[-1]]


def product(torch, x, w, offsets=None):
    """(y, sum of magnitudes) in 64 bits; rows of no expert are 0."""
    v = values(*x, 1)
    if offsets is None:
        m = values(*w, BLOCK)
        return v @ m.T, v.abs() @ m.abs().T
    y = v.new_zeros(len(v), w[0].shape[1])
    a = torch.zeros_like(y)
    at = offsets.tolist()
    for e in range(len(w[0])):
        r = slice(at[e], at[e + 1])
        m = values(w[0][e], w[1][e], BLOCK)
        y[r], a[r] = v[r] @ m.T, v[r].abs() @ m.abs().T
    return y, a


def product_err(inn):
    return 132 * 2.0 ** -23 + (-(-inn // BLOCK) + 8 + 4) * 2.0 ** -24


def check_linear(torch, y, ref, mag, inn, res=None):
    fi = torch.finfo(y.dtype)
    if res is not None:
        ref, mag = ref + res.double(), mag + res.double().abs()
    tol = mag * product_err(inn) * (1 + fi.eps) + ref.abs() * (fi.eps / 2) + fi.tiny * fi.eps / 2
    d = (y.double() - ref).abs()
    assert bool((d <= tol).all()), float((d / tol).max())


def check_quantized(torch, q, s, h, dh, group=BLOCK):
    """Codes and scales of h, known within dh; see ffn_quantize_e4m3."""
    for j, c in enumerate(range(0, h.shape[1], group)):
        part, err = h[:, c:c + group], dh[:, c:c + group]
        sr = part.abs().amax(dim=1).clamp(min=2.0 ** -100) / 448.0
        ds = err.amax(dim=1) / 448.0 + sr * 3 * 2.0 ** -24
        assert bool(((s[:, j].double() - sr).abs() <= ds).all()), j
        t = part / sr[:, None]
        got = q[:, c:c + group].double()
        move = err / sr[:, None] + t.abs() * (ds / sr + 3 * 2.0 ** -24)[:, None]   # of what is rounded
        half = torch.maximum((t.abs() + move) * 2.0 ** -4, t.new_tensor(2.0 ** -10))
        assert bool(((got - t).abs() <= half + move).all()), j
        assert bool((got.abs() <= 448).all())


def check_gateup(torch, q, s, x, wg, wu, inn, offsets=None, rows=None):
    g, ag = product(torch, x, wg, offsets)
    u, au = product(torch, x, wu, offsets)
    if rows is not None:
        g, ag, u, au, q, s = (v[rows] for v in (g, ag, u, au, q, s))
    e = product_err(inn)
    silu = g * torch.sigmoid(g)
    h = silu * u
    # |silu'| <= 1.1; the exponential and division: (4 + 1.17 |g|) ulp of the sigmoid
    dh = 1.1 * ag * e * (u.abs() + au * e) + silu.abs() * au * e + h.abs() * (6 + 1.17 * g.abs()) * 2.0 ** -23
    check_quantized(torch, q, s, h, dh)
