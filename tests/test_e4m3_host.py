"""Refusals of the e4m3 and sorting entry points and of their Python wrappers (CPU
only: every one is found before anything is launched)."""

import ctypes

import pytest

from transformer_ffn_rmsnorm_gb300 import _lib

OK, NULL, SHAPE, DTYPE, ALIGN = (_lib.FFN_OK, _lib.FFN_ERR_NULL, _lib.FFN_ERR_SHAPE, _lib.FFN_ERR_DTYPE,
                                 _lib.FFN_ERR_ALIGN)
WORKSPACE, ALIAS, FLAGS = _lib.FFN_ERR_WORKSPACE, _lib.FFN_ERR_ALIAS, _lib.FFN_ERR_FLAGS


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


P = [ctypes.c_void_p((i + 1) << 30) for i in range(10)]   # never dereferenced


def off(p, n):
    return ctypes.c_void_p(p.value + n)


def weight(c, s):
    return _lib.E4m3Weight(c.value if c else None, s.value if s else None)


def test_quantize_refusals(lib):
    def call(x=P[0], q=P[1], s=P[2], batch=1, rows=4, d=64, block_rows=1, group=128, dtype=_lib.FFN_BF16, flags=0):
        return lib.ffn_quantize_e4m3(x, q, s, batch, rows, d, block_rows, group, dtype, flags, None)
    for name in ("x", "q", "s"):
        assert call(**{name: None}) == NULL
    assert call(dtype=_lib.FFN_E4M3) == DTYPE and call(dtype=9) == DTYPE
    assert call(flags=2) == FLAGS and call(flags=1) == FLAGS     # (only blocks are transposed)
    for bad in ({"rows": -1}, {"batch": -1}, {"d": 0}, {"block_rows": 2}, {"block_rows": 64}, {"group": 0},
                {"group": 16}, {"block_rows": 128, "group": 64}, {"block_rows": 128, "d": 72}, {"d": 1 << 30},
                {"block_rows": 128, "flags": 1, "rows": 8}, {"rows": 1 << 31}, {"rows": 1 << 25, "d": 1 << 13},
                {"batch": 1 << 20, "rows": 1 << 20}):
        assert call(**bad) == SHAPE, bad
    for name, p, n in (("x", P[0], 8), ("q", P[1], 8), ("s", P[2], 2)):
        assert call(**{name: off(p, n)}) == ALIGN
    assert call(q=P[0]) == ALIAS and call(s=off(P[0], 16)) == ALIAS and call(s=off(P[1], 240)) == ALIAS
    assert call(rows=0) == OK and call(batch=0, x=None, q=None, s=None) == OK


def test_linear_refusals(lib):
    def call(x=P[0], xs=P[1], c=P[2], s=P[3], offsets=P[4], res=P[5], y=P[6], rows=4, inn=64, out=128, experts=3,
             dtype=_lib.FFN_BF16):
        return lib.ffn_linear_e4m3(x, xs, weight(c, s), offsets, res, y, rows, inn, out, experts, dtype, None)
    for name in ("x", "xs", "c", "s", "y", "offsets"):
        assert call(**{name: None}) == NULL, name
    assert call(dtype=_lib.FFN_E4M3) == DTYPE
    for bad in ({"rows": -1}, {"inn": 0}, {"inn": 24}, {"out": 4}, {"out": 100}, {"experts": 0}, {"experts": 1025},
                {"inn": 1 << 25}, {"out": 1 << 25}, {"experts": 1024, "out": 1 << 21}, {"rows": 1 << 31},
                {"rows": 1 << 29, "out": 4096}):
        assert call(**bad) == SHAPE, bad
    assert call(offsets=None, experts=1, rows=0) == OK
    for name, p in (("x", P[0]), ("c", P[2]), ("res", P[5]), ("y", P[6])):
        assert call(**{name: off(p, 8)}) == ALIGN, name
    for name, p in (("xs", P[1]), ("s", P[3]), ("offsets", P[4])):
        assert call(**{name: off(p, 2)}) == ALIGN, name
    for bad in (P[0], P[1], P[2], P[3], P[4], off(P[2], 64 * 128 * 3 - 16), off(P[5], 16)):
        assert call(y=bad) == ALIAS
    assert call(rows=0) == OK


def test_gateup_refusals(lib):
    def call(x=P[0], xs=P[1], c=P[2], s=P[3], c2=P[4], s2=P[5], offsets=P[6], q=P[7], qs=P[8], rows=4, d=64, ffn=128,
             experts=3):
        return lib.ffn_gateup_e4m3(x, xs, weight(c, s), weight(c2, s2), offsets, q, qs, rows, d, ffn, experts, None)
    for name in ("x", "xs", "c", "s", "c2", "s2", "q", "qs", "offsets"):
        assert call(**{name: None}) == NULL, name
    for bad in ({"rows": -1}, {"d": 8}, {"ffn": 12}, {"experts": 1025}):
        assert call(**bad) == SHAPE, bad
    for name, p, n in (("q", P[7], 4), ("qs", P[8], 2), ("c2", P[4], 4), ("s2", P[5], 2)):
        assert call(**{name: off(p, n)}) == ALIGN, name
    for bad in (P[0], P[1], P[2], P[4], P[5], P[6]):
        assert call(q=bad) == ALIAS and call(qs=bad) == ALIAS
    assert call(qs=off(P[7], 16)) == ALIAS
    assert call(rows=0) == OK


def test_sort_refusals(lib):
    def need(rows=20000, experts=8, k=2):
        out = ctypes.c_size_t(0)
        return lib.ffn_moe_sort_workspace_bytes(rows, experts, k, ctypes.byref(out)), out.value

    def call(x=P[0], sc=P[1], idx=P[2], xs=P[3], xsc=P[4], pos=P[5], offs=P[6], rows=20000, d=64, ns=1, experts=8, k=2,
             dtype=_lib.FFN_E4M3, ws=P[7], nb=1 << 21):
        return lib.ffn_moe_sort(x, sc, idx, xs, xsc, pos, offs, rows, d, ns, experts, k, dtype, ws, nb, None)
    assert need()[0] == OK and need()[1] > 0 and need(rows=1) == (OK, 0) and need(rows=0) == (OK, 0)
    last = 0
    for rows in (1, 128, 129, 1000, 100000, 262144, 262145, 300000, 1 << 24, 1 << 28):
        st, n = need(rows=rows, experts=1024)
        assert st == OK and last <= n <= 1 << 21
        last = n
    for name in ("x", "idx", "xs", "pos", "offs", "sc", "xsc"):
        assert call(**{name: None}) == NULL, name
    assert call(dtype=4) == DTYPE and call(dtype=-1) == DTYPE
    for bad in ({"rows": -1}, {"d": 0}, {"d": 72}, {"d": 4, "dtype": 1}, {"experts": 0}, {"experts": 1025}, {"k": 0},
                {"k": 33}, {"rows": 1 << 30}, {"ns": -1}, {"ns": 0}, {"ns": 65}, {"d": 1 << 31}):
        assert call(**bad) == SHAPE, bad
    assert call(ws=None) == WORKSPACE and call(nb=need()[1] - 1) == WORKSPACE
    for name, p in (("x", P[0]), ("xs", P[3]), ("ws", P[7])):
        assert call(**{name: off(p, 8)}) == ALIGN, name
    for name, p in (("sc", P[1]), ("idx", P[2]), ("xsc", P[4]), ("pos", P[5]), ("offs", P[6])):
        assert call(**{name: off(p, 2)}) == ALIGN, name
    for bad in ({"xs": P[0]}, {"pos": P[2]}, {"offs": off(P[5], 16)}, {"xsc": P[1]}, {"ws": P[3]},
                {"ws": off(P[2], 16)}):
        assert call(**bad) == ALIAS, bad


def test_unsort_refusals(lib):
    def fwd(ys=P[0], pos=P[1], w=P[2], res=P[3], y=P[4], rows=4, d=64, k=2, dtype=_lib.FFN_BF16):
        return lib.ffn_moe_unsort(ys, pos, w, res, y, rows, d, k, dtype, None)

    def bwd(dy=P[0], ys=P[1], pos=P[2], w=P[3], dys=P[4], dw=P[5], rows=4, d=64, k=2, dtype=_lib.FFN_BF16):
        return lib.ffn_moe_unsort_backward(dy, ys, pos, w, dys, dw, rows, d, k, dtype, None)
    for name in ("ys", "pos", "y"):
        assert fwd(**{name: None}) == NULL
    for name in ("dy", "ys", "pos", "w", "dys", "dw"):
        assert bwd(**{name: None}) == NULL
    for f in (fwd, bwd):
        assert f(dtype=_lib.FFN_E4M3) == DTYPE
        for bad in ({"rows": -1}, {"d": 0}, {"d": 4}, {"k": 0}, {"k": 33}, {"rows": 1 << 30}):
            assert f(**bad) == SHAPE, bad
        assert f(rows=0) == OK
        assert f(ys=off(P[0], 8)) == ALIGN and f(pos=off(P[1], 2)) == ALIGN and f(w=off(P[2], 2)) == ALIGN
    assert fwd(y=P[0]) == ALIAS and fwd(y=off(P[3], 16)) == ALIAS and fwd(y=P[1]) == ALIAS and fwd(y=P[2]) == ALIAS
    assert bwd(dys=P[0]) == ALIAS and bwd(dys=off(P[1], 16)) == ALIAS and bwd(dw=P[3]) == ALIAS
    assert bwd(dw=off(P[4], 16)) == ALIAS and bwd(dw=P[1]) == ALIAS


def test_wrappers_refuse_what_the_library_cannot_see():
    """Host tensors, other types and shapes never reach the library."""
    import torch
    from transformer_ffn_rmsnorm_gb300 import ffn
    x = torch.zeros(4, 64)
    q, s = x.to(torch.float8_e4m3fn), torch.zeros(4, 1)
    w = (torch.zeros(8, 64).to(torch.float8_e4m3fn), torch.zeros(1, 1))
    idx = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: ffn.ffn_quantize_e4m3(x), lambda: ffn.ffn_linear_e4m3(q, s, w),
                 lambda: ffn.ffn_gateup_e4m3(q, s, w, w), lambda: ffn.ffn_moe_sort(x, idx, 4),
                 lambda: ffn.ffn_moe_unsort(x, idx), lambda: ffn.ffn_moe_unsort_backward(x, x, idx, s)):
        with pytest.raises(ValueError):
            call()
