"""Arguments of the paged cache's calls that are refused before anything is launched (no GPU)."""
import types

import numpy as np
import pytest

import vector_compression_b200 as tq


def test_attention_with_a_closed_quantizer():
    """The cache's handle keeps the address of the keys' sketch, which closing the quantizer frees."""
    kp = tq.TQParams(128, 3, tq.MODE_MSE, tq.ROT_HADAMARD, signs=np.ones(128, np.int8))
    pg = types.SimpleNamespace(kp=kp, _c=None)
    kp.close()
    with pytest.raises(ValueError, match="closed"):
        tq.tq_paged_attention(pg, None, None, 0, None, None, 1.0)


def test_norm_rope_refuses_outputs_whose_rows_overlap():
    """Each stride may be long enough and rows still meet: token t's head h and token t + i's head h - j."""
    lib, rope, fake = tq._lib.lib(), tq.TQRope(64), 0x10000  # never dereferenced
    for n, heads, ot, oh in ((4, 4, 128, 128), (4, 4, 64, 64), (8, 3, 64, 128), (3, 8, 128, 64), (2, 5, 1000, 250),
                             (2, 5, 1000, 249), (7, 3, 100, 550), (2, 65536, 64 * 65536 - 1, 64),
                             (1 << 30, 2, 64, 64 * ((1 << 30) - 1) + 63)):
        overlap = n < 100 and heads < 100 and any(
            abs(i * ot + j * oh) < 64 for i in range(-n + 1, n) for j in range(heads) if (i, j) != (0, 0))
        assert overlap or max(n, heads) > 100, (n, heads, ot, oh)
        got = lib.tq_qk_norm_rope(rope.handle, 0, n, 64, heads, fake, 64, 64, 0, None, 0, 0, fake, None, None, 0.0,
                                  fake, ot, oh, None, 0, 0, None)
        assert got == 1, (n, heads, ot, oh)
