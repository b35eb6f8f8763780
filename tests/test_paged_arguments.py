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
