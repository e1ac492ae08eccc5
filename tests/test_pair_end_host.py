"""Refusals of ffn_selftest_pair_end (CPU only: nothing is launched)."""

import ctypes

from transformer_ffn_rmsnorm_gb300 import _lib


def test_pair_end_refusals():
    lib = _lib.load()
    src, wrong = ctypes.c_void_p(1 << 30), ctypes.c_void_p(2 << 30)   # never dereferenced

    def call(even, odd, src=src, wrong=wrong):
        return lib.ffn_selftest_pair_end(src, wrong, even, odd, None)
    assert call(4, 4, src=None) == _lib.FFN_ERR_NULL and call(4, 4, wrong=None) == _lib.FFN_ERR_NULL
    for even, odd in ((-1, 3), (3, -1), (5, 0), (0, 5), (3, 7), (9, 7), (65, 64), (64, 68)):
        assert call(even, odd) == _lib.FFN_ERR_SHAPE, (even, odd)
    assert call(4, 4, src=ctypes.c_void_p((1 << 30) + 8)) == _lib.FFN_ERR_ALIGN
    assert call(4, 4, wrong=ctypes.c_void_p((2 << 30) + 2)) == _lib.FFN_ERR_ALIGN
    assert call(4, 4, wrong=ctypes.c_void_p((1 << 30) + 8192 * 4 - 4)) == _lib.FFN_ERR_ALIAS
