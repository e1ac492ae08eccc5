"""Where the pointers of ffn_quantize_e4m3 and ffn_gateup_e4m3 may lie: as rows of a batch do (CPU only: what is
accepted is told by the next refusal, an overlap, so that nothing is ever launched)."""

import ctypes

import pytest

from transformer_ffn_rmsnorm_gb300 import _lib

ALIGN, ALIAS = _lib.FFN_ERR_ALIGN, _lib.FFN_ERR_ALIAS
P = [(i + 1) << 30 for i in range(10)]   # never dereferenced


def weight(c, s):
    return _lib.E4m3Weight(c, s)


@pytest.mark.parametrize("dtype,size", [(_lib.FFN_F32, 4), (_lib.FFN_F16, 2), (_lib.FFN_BF16, 2)])
@pytest.mark.parametrize("d", [1, 7, 16, 96, 128, 130, 132, 136, 264, 1000, 1002, 4096])
def test_quantize_rows_of_a_batch(dtype, size, d):
    lib = _lib.load()

    def call(x, q, s=P[0]):   # the scales overlap x
        return lib.ffn_quantize_e4m3(x, q, s, 1, 3, d, 1, 128, dtype, 0, None)
    for row in range(1, 9):
        assert call(P[0] + row * d * size, P[1] + row * d, P[0] + row * d * size // 4 * 4) == ALIAS, row
    vectors = d * size % 16 == 0
    assert call(P[0] + size, P[1]) == (ALIGN if vectors else ALIAS)
    assert call(P[0], P[1] + 1) == (ALIGN if vectors else ALIAS)
    if d % 16 == 0:
        assert call(P[0] + 8, P[1]) == ALIGN and call(P[0], P[1] + 8) == ALIGN
    assert call(P[0] + 1, P[1]) == ALIGN


@pytest.mark.parametrize("flags", [0, _lib.FFN_QUANT_TRANSPOSE])
def test_quantize_blocks(flags):
    lib = _lib.load()

    def call(x, q):
        return lib.ffn_quantize_e4m3(x, q, x, 1, 32, 48, 128, 128, _lib.FFN_BF16, flags, None)
    assert call(P[0], P[1]) == ALIAS and call(P[0] + 48 * 2, P[1] + 48) == ALIAS
    assert call(P[0] + 8, P[1]) == ALIGN and call(P[0], P[1] + 8) == ALIGN


@pytest.mark.parametrize("ffn", [8, 128, 264, 1000])
def test_gateup_rows_of_a_batch(ffn):
    lib = _lib.load()

    def call(q):
        return lib.ffn_gateup_e4m3(P[0], P[1], weight(P[2], P[3]), weight(P[4], P[5]), P[6], q, P[1], 3, 64, ffn, 2,
                                   None)   # the scales overlap x's
    for row in range(1, 5):
        assert call(P[7] + row * ffn) == ALIAS, row
    assert call(P[7] + 8) == ALIAS
    assert call(P[7] + 4) == ALIGN and call(P[7] + 1) == ALIGN
