"""Refusals of the routed layer's entry points and of their Python wrappers
(CPU only: every one is found before anything is launched)."""

import ctypes

import pytest

from transformer_ffn_rmsnorm_gb300 import _lib


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def ptrs(n):
    return [ctypes.c_void_p((i + 1) << 28) for i in range(n)]   # never dereferenced


def test_add_rmsnorm_refusals(lib):
    x, res, g, r, n = ptrs(5)
    B = _lib.FFN_BF16
    f = lib.ffn_add_rmsnorm
    assert f(None, res, g, r, n, 2, 64, 1e-6, B, None) == _lib.FFN_ERR_NULL
    assert f(x, res, None, r, n, 2, 64, 1e-6, B, None) == _lib.FFN_ERR_NULL
    assert f(x, res, g, r, None, 2, 64, 1e-6, B, None) == _lib.FFN_ERR_NULL
    assert f(x, res, g, r, n, 2, 64, 1e-6, 9, None) == _lib.FFN_ERR_DTYPE
    assert f(x, res, g, r, n, -1, 64, 1e-6, B, None) == _lib.FFN_ERR_SHAPE
    assert f(x, res, g, r, n, 2, 0, 1e-6, B, None) == _lib.FFN_ERR_SHAPE
    assert f(x, res, g, r, n, 2, 1 << 30, 1e-6, B, None) == _lib.FFN_ERR_SHAPE
    odd = ctypes.c_void_p(res.value + 2)
    assert f(x, odd, g, r, n, 2, 64, 1e-6, B, None) == _lib.FFN_ERR_ALIGN
    near = ctypes.c_void_p(x.value + 16)
    assert f(x, res, g, near, n, 2, 64, 1e-6, B, None) == _lib.FFN_ERR_ALIAS
    assert f(x, res, g, r, near, 2, 64, 1e-6, B, None) == _lib.FFN_ERR_ALIAS
    assert f(x, res, g, x, x, 2, 64, 1e-6, B, None) == _lib.FFN_ERR_ALIAS
    assert f(x, res, g, g, n, 2, 64, 1e-6, B, None) == _lib.FFN_ERR_ALIAS
    assert f(x, res, g, r, n, 0, 64, 1e-6, B, None) == _lib.FFN_OK
    q, s = ptrs(7)[5:]
    f = lib.ffn_add_rmsnorm_e4m3
    assert f(x, res, g, r, q, None, 2, 64, 0, 1e-6, B, None) == _lib.FFN_ERR_NULL
    for group in (-32, 16, 48, 256):
        assert f(x, res, g, r, q, s, 2, 64, group, 1e-6, B, None) == _lib.FFN_ERR_SHAPE
    assert f(x, res, g, r, x, s, 2, 64, 0, 1e-6, B, None) == _lib.FFN_ERR_ALIAS     # codes never in place
    assert f(x, res, g, r, q, ctypes.c_void_p(q.value + 64), 2, 64, 0, 1e-6, B, None) == _lib.FFN_ERR_ALIAS
    assert f(x, res, g, r, q, s, 0, 64, 0, 1e-6, B, None) == _lib.FFN_OK


def test_route_refusals(lib):
    l, b, i, w = ptrs(4)
    f = lib.ffn_moe_route
    F = _lib.FFN_F32

    def call(logits=l, bias=b, idx=i, wt=w, rows=4, experts=64, k=6, groups=1, topk_groups=1, dtype=F, flags=0):
        return f(logits, bias, idx, wt, rows, experts, k, groups, topk_groups, 1.0, dtype, flags, None)

    assert call(logits=None) == _lib.FFN_ERR_NULL
    assert call(idx=None) == _lib.FFN_ERR_NULL
    assert call(wt=None) == _lib.FFN_ERR_NULL
    assert call(dtype=3) == _lib.FFN_ERR_DTYPE
    assert call(flags=4) == _lib.FFN_ERR_FLAGS
    for bad in ({"rows": -1}, {"experts": 0}, {"experts": 1025}, {"k": 0}, {"k": 33}, {"experts": 4, "k": 5},
                {"groups": 0}, {"groups": 3}, {"experts": 66, "groups": 33}, {"groups": 4, "topk_groups": 5},
                {"groups": 4, "topk_groups": 0}, {"groups": 16, "topk_groups": 1}):
        assert call(**bad) == _lib.FFN_ERR_SHAPE, bad
    assert call(bias=ctypes.c_void_p(b.value + 4)) == _lib.FFN_ERR_ALIGN
    assert call(wt=i) == _lib.FFN_ERR_ALIAS
    assert call(idx=ctypes.c_void_p(l.value + 64)) == _lib.FFN_ERR_ALIAS
    assert call(rows=0) == _lib.FFN_OK


def test_wrappers_refuse_what_the_library_cannot_see():
    """Host tensors never reach the library."""
    import torch
    from transformer_ffn_rmsnorm_gb300 import ffn
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ffn.ffn_add_rmsnorm(x, x[0], 1e-6)
    with pytest.raises(ValueError):
        ffn.ffn_add_rmsnorm_e4m3(x, x[0], 1e-6)
    with pytest.raises(ValueError):
        ffn.ffn_moe_route(x, 2)


def test_moe_forward_refusals(lib):
    x, idx, w, wg, wu, wd, res, y, ws = ptrs(9)
    B = _lib.FFN_BF16

    def need(rows=4, d=64, ffn=128, experts=8, k=2, dtype=B, flags=0):
        out = ctypes.c_size_t(0)
        return lib.ffn_moe_workspace_bytes(rows, d, ffn, experts, k, dtype, flags, ctypes.byref(out)), out.value

    def call(x=x, idx=idx, w=w, wg=wg, wu=wu, wd=wd, res=res, y=y, rows=4, d=64, ffn=128, experts=8, k=2, dtype=B,
             flags=0, ws=ws, bytes_=1 << 27):
        return lib.ffn_moe_forward(x, idx, w, wg, wu, wd, res, y, rows, d, ffn, experts, k, dtype, flags, ws, bytes_,
                                   None)

    assert need()[0] == _lib.FFN_OK and need()[1] >= 8 * (128 * 2 + 64 * 4)
    assert need(flags=_lib.FFN_PREPARED_WEIGHTS)[1] >= need()[1]
    assert need(rows=0) == (_lib.FFN_OK, 0)
    for name in ("x", "idx", "w", "wg", "wu", "wd", "y"):
        assert call(**{name: None}) == _lib.FFN_ERR_NULL, name
    for bad in ({"dtype": _lib.FFN_F32}, {"dtype": 5}):
        assert call(**bad) == _lib.FFN_ERR_DTYPE and need(**bad)[0] == _lib.FFN_ERR_DTYPE
    for flags in (_lib.FFN_RESIDUAL, _lib.FFN_PATH_GEMV, 1 << 20):
        assert call(flags=flags) == _lib.FFN_ERR_FLAGS
    for bad in ({"rows": -1}, {"d": 0}, {"d": 68}, {"ffn": 100}, {"experts": 0}, {"experts": 1025}, {"k": 0},
                {"k": 33}, {"rows": 1 << 30}, {"experts": 1024, "ffn": 1 << 21}, {"experts": 1024, "d": 1 << 21}):
        assert call(**bad) == _lib.FFN_ERR_SHAPE and need(**bad)[0] == _lib.FFN_ERR_SHAPE, bad
    n = need()[1]
    assert call(bytes_=n - 1) == _lib.FFN_ERR_WORKSPACE
    assert call(ws=None) == _lib.FFN_ERR_WORKSPACE
    for name, p in (("x", x), ("wg", wg), ("res", res), ("ws", ws)):
        assert call(**{name: ctypes.c_void_p(p.value + 8)}) == _lib.FFN_ERR_ALIGN, name
    for bad in (x, wd, w, ctypes.c_void_p(res.value + 16), ctypes.c_void_p(ws.value + 256)):
        assert call(y=bad) == _lib.FFN_ERR_ALIAS
    assert call(ws=wu) == _lib.FFN_ERR_ALIAS
    assert call(rows=0) == _lib.FFN_OK


def test_moe_forward_q4_refusals(lib):
    x, idx, w, a, b, c, res, y, ws = ptrs(9)
    sa, sb, sc = (ctypes.c_void_p((i + 20) << 28) for i in range(3))

    def q4(q, s):
        return _lib.Q4Weight(q.value if q else None, s.value if s else None)

    def need(rows=4, d=64, ffn=128, experts=8, k=2):
        out = ctypes.c_size_t(0)
        return lib.ffn_moe_q4_workspace_bytes(rows, d, ffn, experts, k, ctypes.byref(out)), out.value

    def call(x=x, idx=idx, w=w, a=a, b=b, c=c, sa=sa, sb=sb, sc=sc, res=res, y=y, rows=4, d=64, ffn=128, experts=8,
             k=2, ws=ws, bytes_=1 << 27):
        return lib.ffn_moe_forward_q4(x, idx, w, q4(a, sa), q4(b, sb), q4(c, sc), res, y, rows, d, ffn, experts, k, ws,
                                      bytes_, None)

    assert need()[0] == _lib.FFN_OK and need()[1] >= 8 * (128 * 2 + 64 * 4) + 4 * 64 * 2
    for name in ("x", "idx", "w", "a", "b", "c", "sa", "sb", "sc", "y"):
        assert call(**{name: None}) == _lib.FFN_ERR_NULL, name
    for bad in ({"d": 48}, {"ffn": 72}, {"rows": -1}, {"experts": 0}, {"experts": 2000}, {"k": 0}, {"k": 40},
                {"rows": 1 << 30}):
        assert call(**bad) == _lib.FFN_ERR_SHAPE and need(**bad)[0] == _lib.FFN_ERR_SHAPE, bad
    assert call(bytes_=need()[1] - 1) == _lib.FFN_ERR_WORKSPACE
    assert call(sb=ctypes.c_void_p(sb.value + 2)) == _lib.FFN_ERR_ALIGN
    for bad in (x, c, sc, ctypes.c_void_p(res.value + 16)):
        assert call(y=bad) == _lib.FFN_ERR_ALIAS
    assert call(rows=0) == _lib.FFN_OK and need(rows=0) == (_lib.FFN_OK, 0)


def workspace_query(lib, q4, flags=0):
    def need(rows, d, ffn, experts, k):
        out = ctypes.c_size_t(0)
        if q4:
            st = lib.ffn_moe_q4_workspace_bytes(rows, d, ffn, experts, k, ctypes.byref(out))
        else:
            st = lib.ffn_moe_workspace_bytes(rows, d, ffn, experts, k, _lib.FFN_BF16, flags, ctypes.byref(out))
        assert st == _lib.FFN_OK
        return out.value
    return need


@pytest.mark.parametrize("form", ["bf16", "prepared", "q4"])
@pytest.mark.parametrize("d,ffn,experts,k", [(4096, 14336, 8, 2), (5120, 2176, 32, 4), (2048, 1408, 64, 6),
                                             (64, 512, 1024, 1), (32, 32, 1, 1), (256, 4096, 3, 32)])
def test_workspace_serves_every_smaller_batch(lib, form, d, ffn, experts, k):
    """The query never falls as the rows grow, across the changes of the split
    count, of single CTAs to pairs and of the plan's chunks; and a call of fewer
    rows takes what the query gives for more (it gets as far as the alignment
    of its input, which is checked after the workspace)."""
    need = workspace_query(lib, form == "q4", _lib.FFN_PREPARED_WEIGHTS if form == "prepared" else 0)
    marks = [1024 // k, 24 * experts // k, 131072 // k, 262144 // k, 393216 // k, 131072 * 5 // k]
    near = {max(1, m + i) for m in marks for i in range(-3, 4)}
    rows = sorted(set(range(1, 700)) | near | set(range(700, 4000, 97)))
    sizes = [need(r, d, ffn, experts, k) for r in rows]
    assert all(a <= b for a, b in zip(sizes, sizes[1:])), [r for r, a, b in zip(rows, sizes, sizes[1:]) if a > b]

    x, idx, w, a, b, c, res, y, ws = ptrs(9)
    ws = ctypes.c_void_p(1 << 50)
    far = [ctypes.c_void_p((i + 1) << 44) for i in range(16)]
    odd = ctypes.c_void_p((1 << 43) + 2)

    def status(r, bytes_):
        if form == "q4":
            m = [_lib.Q4Weight(far[i].value, far[i + 3].value) for i in range(3)]
            return lib.ffn_moe_forward_q4(odd, far[6], far[7], *m, None, far[8], r, d, ffn, experts, k, ws, bytes_, None)
        return lib.ffn_moe_forward(odd, far[6], far[7], far[0], far[1], far[2], None, far[8], r, d, ffn, experts, k,
                                   _lib.FFN_BF16, _lib.FFN_PREPARED_WEIGHTS if form == "prepared" else 0, ws, bytes_, None)
    for top in (rows[-1], 456, 97, 512, 1024 // k + 1, 24 * experts // k + 1, 131072 // k + 1):
        for r in [r for r in rows if r <= top][::7] + [top]:
            assert status(r, need(top, d, ffn, experts, k)) == _lib.FFN_ERR_ALIGN, (r, top)
        assert status(top, 0) == _lib.FFN_ERR_WORKSPACE


def test_rows_of_a_batch_need_no_16_bytes(lib):
    """Logits, indices and weights are read one by one: slices of their rows are
    taken (a call of too small a workspace gets as far as that, and a call of
    logits that overlap the outputs as far as the overlap)."""
    x, idx, w, wg, wu, wd, res, y, ws = ptrs(9)

    def at(p, n):
        return ctypes.c_void_p(p.value + n)

    def route(logits=x, bias=res, i=idx, wt=w, dtype=_lib.FFN_F32):
        return lib.ffn_moe_route(logits, bias, i, wt, 4, 63, 6, 1, 1, 1.0, dtype, 0, None)
    for dtype, size in ((_lib.FFN_F32, 4), (_lib.FFN_F16, 2), (_lib.FFN_BF16, 2)):
        assert route(logits=at(x, 63 * size), i=at(x, 64 * size), dtype=dtype) == _lib.FFN_ERR_ALIAS
        assert route(logits=at(x, size // 2), dtype=dtype) == _lib.FFN_ERR_ALIGN
    assert route(i=at(idx, 24), wt=at(idx, 28)) == _lib.FFN_ERR_ALIAS
    for name in ("i", "wt"):
        assert route(**{name: at(idx, 2)}) == _lib.FFN_ERR_ALIGN

    def forward(i=idx, wt=w, out=y):
        return lib.ffn_moe_forward(x, i, wt, wg, wu, wd, res, out, 4, 64, 128, 8, 6, _lib.FFN_BF16, 0, ws, 1 << 27, None)

    def forward_q4(i=idx, wt=w, out=y):
        m = [_lib.Q4Weight((20 + n) << 28, (24 + n) << 28) for n in range(3)]
        return lib.ffn_moe_forward_q4(x, i, wt, *m, res, out, 4, 64, 128, 8, 6, ws, 1 << 27, None)
    for f in (forward, forward_q4):
        assert f(i=at(idx, 24), wt=at(w, 24), out=x) == _lib.FFN_ERR_ALIAS
        assert f(i=at(idx, 2)) == _lib.FFN_ERR_ALIGN and f(wt=at(w, 1)) == _lib.FFN_ERR_ALIGN


def test_q4_scales_of_another_16_bit_type_are_refused():
    """bf16 scales have other bits than fp16's and would be read as those."""
    import torch
    from transformer_ffn_rmsnorm_gb300 import ffn
    qs = torch.zeros(3, 32, 64, dtype=torch.uint8)
    sc = torch.ones(3, 32, 4)
    for dtype in (torch.bfloat16, torch.float32):
        with pytest.raises(TypeError):
            ffn._moe_q4_weight("w_gate", (qs, sc.to(dtype)), 3, 32, 128, -1)
    for good in (sc.half(), sc.half().view(torch.int16), sc.half().view(torch.uint16)):
        ffn._moe_q4_weight("w_gate", (qs, good), 3, 32, 128, -1)
    with pytest.raises(ValueError):
        ffn._moe_q4_weight("w_gate", (qs, sc.half()[:2]), 3, 32, 128, -1)


def test_rows_too_long_for_a_bounded_wait_are_refused(lib):
    """A unit of the products reads whole rows of weights within the kernels'
    limit of a second a wait: up to 2^24 values."""
    out = ctypes.c_size_t(0)

    def need16(d, ffn):
        return lib.ffn_moe_workspace_bytes(1, d, ffn, 1, 1, _lib.FFN_BF16, 0, ctypes.byref(out))

    def need4(d, ffn):
        return lib.ffn_moe_q4_workspace_bytes(1, d, ffn, 1, 1, ctypes.byref(out))
    top = 1 << 24
    for need in (need16, need4):
        assert need(top, 64) == _lib.FFN_OK and need(64, top) == _lib.FFN_OK
        assert need(top + 32, 64) == _lib.FFN_ERR_SHAPE and need(64, top + 32) == _lib.FFN_ERR_SHAPE
        assert need(1 << 30, 32) == _lib.FFN_ERR_SHAPE
