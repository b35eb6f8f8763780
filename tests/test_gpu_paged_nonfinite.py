"""Norms of tokens that are not finite: what they do to their own KV head's outputs does not depend on which kernel a
shape takes, and nothing else notices."""
import numpy as np
import pytest
import torch

import vector_compression_b200 as tq
from tests.paged_ref import Model
from tests.test_gpu_paged import DEV, i32, ints, quantizers, random_cache

pytestmark = pytest.mark.gpu

SHAPES = [
    # d, bits, vbits, m, r16, G: the tensor-core kernel's shapes (each value width, one and two tiles of heads) ...
    (128, 3, 3, 128, False, 4), (128, 3, 1, 64, True, 7), (64, 2, 4, 64, False, 8), (64, 4, 2, 64, False, 2),
    (192, 3, 4, 256, False, 6),
    # ... and others
    (128, 5, 3, 128, False, 4), (64, 3, 4, 32, True, 3),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES)
def test_norms_that_are_not_finite(shape, dtype):
    d, bits, vbits, m, r16, G = shape
    kp, vp, _, _ = quantizers(d, bits, m, vbits, r16)
    hkv, page = 2, 64
    pg, model = tq.TQPaged(kp, vp, 1, hkv, page), Model(kp, vp, 1, hkv, page)
    rng = np.random.default_rng(d + G)
    lens = [330, 77, 1, 200]
    pool, tables = random_cache(rng, model, lens, 6, 0)
    q = torch.from_numpy(rng.standard_normal((4, hkv * G, d))).to(DEV).to(dtype)

    def call(pool):
        return tq.tq_paged_attention(pg, q, i32(pool), 0, ints(lens), ints(tables), d ** -0.5, want_lse=True)

    clean, clean_lse = call(pool)
    assert bool(torch.isfinite(clean).all()) and bool(torch.isfinite(clean_lse).all())
    # first and last token, inside a group and at its end, beside a slot without a token
    for b, t, h in ((0, 0, 1), (0, 329, 0), (0, 127, 0), (1, 76, 1), (2, 0, 0), (3, 150, 1)):
        mine = torch.zeros(4, hkv * G, dtype=torch.bool, device=DEV)
        mine[b, h * G:(h + 1) * G] = True
        for part in ("vn", "kn", "kr"):
            for bad in (np.nan, np.inf) if part == "vn" else (np.nan,):
                p = pool.copy()
                rec = model.record(p, tables[b, t // page], 0, h, t % page // 32)
                if part == "kr" and r16:
                    rec[model.kr:model.v].view(np.float16)[t % 32] = bad
                else:
                    rec.view(np.float32)[dict(vn=model.vn, kn=model.kn, kr=model.kr)[part] + t % 32] = bad
                got, lse = call(p)
                assert bool(torch.isnan(got[mine]).all()), (b, t, h, part, bad)
                assert torch.equal(got[~mine], clean[~mine]) and torch.equal(lse[~mine], clean_lse[~mine])
                # the softmax does not know of the values
                assert torch.equal(lse, clean_lse) if part == "vn" else bool(torch.isnan(lse[mine]).all())
    tq.tq_sync_check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("shape", SHAPES)
def test_scores_of_minus_infinity_take_no_part(shape, dtype):
    """Tokens with an infinite key norm: where the sign makes their score -inf, they count as if they were not there,
    at a sequence's start and where nothing else is left too."""
    d, bits, vbits, m, r16, G = shape
    kp, vp, _, _ = quantizers(d, bits, m, vbits, r16)
    pg, model = tq.TQPaged(kp, vp, 1, 1, 32), Model(kp, vp, 1, 1, 32)
    rng = np.random.default_rng(d + G + 1)
    pool, tables = random_cache(rng, model, [200, 40], 7, 0)
    # one query for all heads, and all of the keys' codes and signs alike: the same sign of score everywhere
    q = torch.from_numpy(np.repeat(rng.standard_normal((2, 1, d)), G, 1)).to(DEV).to(dtype)
    for b in range(2):
        for t in range(224):
            if 0 <= tables[b, t // 32]:
                rec = model.record(pool, tables[b, t // 32], 0, 0, 0)
                for w in range(model.nk):
                    rec[model.key_place(t % 32, w)] = 0x5a3c96f0 * (w + 1) & 0xffffffff

    def call(pool, lens, t, scale):
        return tq.tq_paged_attention(pg, q, i32(pool), 0, ints(lens), ints(t), scale, want_lse=True)

    scale = 0.1
    if float(call(pool, [200, 40], tables, scale)[1][0, 0]) > float(call(pool, [200, 40], tables, -scale)[1][0, 0]):
        scale = -scale  # scores below zero in sequence 0
    inf = pool.copy()
    for t in range(32):  # the first page of sequence 0
        model.record(inf, tables[0, 0], 0, 0, 0).view(np.float32)[model.kn + t] = np.inf
    holes = tables.copy()
    holes[0, 0] = -1
    got, want = call(inf, [200, 40], tables, scale), call(pool, [200, 40], holes, scale)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out, lse = call(inf, [32, 40], tables, scale)  # nothing else
    assert bool((out[0] == 0).all()) and bool(torch.isneginf(lse[0]).all())
    assert torch.equal(out[1], want[0][1])
    tq.tq_sync_check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [1e-30, 3e-32, 9e-33, 2e-34, 1e-40, 0.0])
def test_value_norms_near_the_smallest_numbers(size, dtype):
    """Weights are divided by their largest: of ones below 1e-31 nothing has to be left, but nothing else may come.
    Beside them in one batch, ordinary norms with one tiny group, and with a tiny tail of the softmax."""
    kp, vp, kq, vq = quantizers(128, 3)
    pg, model = tq.TQPaged(kp, vp, 1, 1, 32), Model(kp, vp, 1, 1, 32)
    rng = np.random.default_rng(33)
    lens = [300, 300, 300]
    pool, tables = random_cache(rng, model, lens, 10, 0)
    for b, t0, t1 in ((0, 0, 300), (1, 128, 256)):
        for t in range(t0, t1):
            f = model.record(pool, tables[b, t // 32], 0, 0, 0).view(np.float32)
            f[model.vn + t % 32] *= np.float32(size)
    q = torch.from_numpy(rng.standard_normal((3, 4, 128))).to(DEV).to(dtype)
    q[2] *= 30
    got, lse = tq.tq_paged_attention(pg, q, i32(pool), 0, ints(lens), ints(tables), 0.088, want_lse=True)
    out, want, spread, delta = model.attention(pool, 0, kq, vq, q.double().cpu().numpy(), lens, tables, 0.088)
    # as tests/test_gpu_paged.py, and what is taken to 0: weights of 1e-31 (the softmax's sum is 1 or more), or all
    eps = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
    tol = eps * abs(out) + ((2 * delta + 2.0 ** -15) * spread)[..., None] + np.minimum(spread, 300 * 1e-31)[..., None]
    assert np.all(abs(got.double().cpu().numpy() - out) <= tol)
    assert np.all(abs(lse.double().cpu().numpy() - want) <= delta + 8 * 2.0 ** -24 * abs(want) + 2.0 ** -22)
