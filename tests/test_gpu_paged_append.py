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


@pytest.mark.parametrize("B,most", [(33, 3), (64, 90), (1025, 2), (2100, 40)])
def test_more_sequences_than_a_warp_holds(B, most):
    """With cu, a token's sequence is searched among more than 32: empty ones at both ends and between, tokens of no
    sequence before and behind."""
    kp, vp, _, _ = quantizers(64, 2, 32)
    pg, model = tq.TQPaged(kp, vp, 1, 1, 32), Model(kp, vp, 1, 1, 32)
    rng = np.random.default_rng(B)
    new = rng.integers(0, most + 1, B) * rng.integers(0, 2, B)
    new[[0, 1, -2, -1]] = 0
    new[[2, 31, 32, B // 2]] = most  # at the borders of the search's steps
    cu = 5 + np.concatenate([[0], np.cumsum(new)])
    n, width = int(cu[-1]) + 4, -(-(most + 40) // 32)
    start = rng.integers(0, 40, B)
    tables = rng.permutation(B * width).reshape(B, width).astype(np.int32)
    pool = rng.integers(0, 1 << 32, (B * width, model.page_words), dtype=np.uint64).astype(np.uint32)
    ref, keys, vals = rows(rng, n, 1, model)
    got = i32(pool)
    tq.tq_paged_append(pg, got, 0, keys, vals, ints(start), ints(tables), cu=ints(cu))
    model.append(pool, 0, *ref, cu, start, tables)
    assert np.array_equal(u32(got), pool)
    tq.tq_sync_check()
