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
