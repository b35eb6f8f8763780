"""Append to pages from parts of the encoders' rows, bit for bit against the plain model."""
import numpy as np
import pytest
import torch

import vector_compression_b200 as tq
from tests.paged_ref import Model
from tests.parity import u32
from tests.test_gpu_paged import SHAPES, i32, ints, quantizers, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hkv", [1, 3])
@pytest.mark.parametrize("shape", SHAPES)
def test_a_prompt_in_chunks(shape, hkv):
    """A chunk's rows begin where the last one's ended, at any token of the prompt's."""
    d, bits, vbits, m, r16, layers, _, page = shape
    kp, vp, _, _ = quantizers(d, bits, m, vbits, r16)
    pg, model = tq.TQPaged(kp, vp, layers, hkv, page), Model(kp, vp, layers, hkv, page)
    rng = np.random.default_rng(d + hkv)
    n, n_pages = 2 * page + 21, 5
    pool = rng.integers(0, 1 << 32, (n_pages, model.page_words), dtype=np.uint64).astype(np.uint32)
    tables = np.array([[3, 0, 4]], np.int32)
    ref, keys, vals = rows(rng, n, hkv, model)
    got = i32(pool)
    codes = [x.view(n * hkv, -1) for x in (keys[0], keys[1], vals[0])]
    ends = [0, 1, 2, 5, 38, 39, n - 3, n]
    for a, b in zip(ends, ends[1:]):
        r = slice(a * hkv, b * hkv)
        tq.tq_paged_append(pg, got, 0, (codes[0][r], codes[1][r], keys[2][r], keys[3][r]), (codes[2][r], vals[1][r]),
                           ints([a]), ints(tables), cu=ints([0, b - a]))
    model.append(pool, 0, *ref, [0, n], [0], tables)
    assert np.array_equal(u32(got), pool)
    tq.tq_sync_check()


def test_key_words_that_begin_inside_a_granule_are_refused():
    kp, vp, _, _ = quantizers(128, 3)  # 8 code words and 4 sign words: granules of 4
    pg, model = tq.TQPaged(kp, vp, 1, 1, 32), Model(kp, vp, 1, 1, 32)
    _, keys, vals = rows(np.random.default_rng(1), 2, 1, model)
    pool, tables = pg.new_pool(1), ints([[0]])
    for i in (0, 1):
        part = [keys[0].reshape(-1)[:8], keys[1].reshape(-1)[:4], keys[2][:1], keys[3][:1]]
        part[i] = keys[i].reshape(-1)[1:1 + part[i].numel()]
        with pytest.raises(tq.TQError):
            tq.tq_paged_append(pg, pool, 0, part, (vals[0].reshape(-1)[:12], vals[1][:1]), ints([0]), tables)
    assert bool((pool == 0).all())
