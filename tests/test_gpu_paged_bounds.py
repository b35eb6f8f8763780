"""Paged attention within the bounds that its roundings give (tests/paged_bounds.py): every shape of the two kernels,
every type, and what fp32 outputs are worth."""
import math

import numpy as np
import pytest
import torch

import vector_compression_b200 as tq
from tests import paged_bounds as pb
from tests.paged_ref import Model
from tests.test_gpu_paged import ATTENTION, DEV, EPS, i32, ints, quantizers, random_cache

pytestmark = pytest.mark.gpu


def on_tensor_cores(d_pad, m, key_bits):
    return key_bits <= 3 and (d_pad, m) in ((64, 64), (128, 64), (128, 128), (256, 256))


def check(got, lse, model, kq, vq, pool, tables, q, lens, scale, dtype, layer):
    got, lse, q = (x.detach().double().cpu().numpy() for x in (got, lse, q))
    G = q.shape[1] // model.hkv
    fixed = on_tensor_cores(model.dp, model.sw * 32, model.kk)
    steps = (pb.FINE if dtype == torch.float32 else pb.COARSE) if fixed else None
    worst = [0.0, 0.0]
    for b, n in enumerate(lens):
        for h in range(model.hkv):
            if n == 0:
                continue
            w = slice(h * G, (h + 1) * G)
            toks = [model.read(model.record(pool, tables[b, t // model.page], layer, h, t % model.page // 32), t % 32)
                    for t in range(n)]
            K, V = (np.asarray(z.centroids)[np.array([t[i] for t in toks])] for z, i in ((kq, 0), (vq, 4)))
            S = 2.0 * np.array([t[1] for t in toks]) - 1
            kn, kr, vn = (np.array([t[i] for t in toks]) for i in (2, 3, 5))
            qr = kq.rot.apply(q[b, w])
            out, want, e_out, e_lse = pb.head_bounds(qr, qr @ kq.S.T, K, S, kn, kr, V, vn, scale, kq.kappa,
                                                     vq.rot.apply_t, EPS[dtype], steps, fixed, serial=not fixed)
            worst[0] = max(worst[0], (np.linalg.norm(got[b, w] - out, axis=-1) / e_out).max())
            worst[1] = max(worst[1], (abs(lse[b, w] - want) / e_lse).max())
    print(f"of the bounds: output {worst[0]:.2f}, lse {worst[1]:.2f}")
    assert max(worst) <= 1, worst


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("case", ATTENTION)
def test_attention_within_its_roundings(case, dtype):
    d, bits, vbits, m, r16, hkv, G, page, lens = case
    kp, vp, kq, vq = quantizers(d, bits, m, vbits, r16)
    pg, model = tq.TQPaged(kp, vp, 1, hkv, page), Model(kp, vp, 1, hkv, page)
    rng = np.random.default_rng(sum(lens) + G)
    pool, tables = random_cache(rng, model, lens, max(-(-max(lens) // page), 1), 0)
    q = torch.from_numpy(rng.standard_normal((len(lens), hkv * G, d))).to(DEV).to(dtype)
    scale = 1 / math.sqrt(d)
    got, lse = tq.tq_paged_attention(pg, q, i32(pool), 0, ints(lens), ints(tables), scale, want_lse=True)
    tq.tq_sync_check()
    check(got, lse, model, kq, vq, pool, tables, q, lens, scale, dtype, 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("sharp", [0.02, 0.4])
def test_long_contexts_within_their_roundings(sharp, dtype):
    """Many groups a segment and many parts a head; all tokens alike, and a few that have nearly all of the weight."""
    kp, vp, kq, vq = quantizers(128, 3)
    pg, model = tq.TQPaged(kp, vp, 1, 1, 64), Model(kp, vp, 1, 1, 64)
    rng = np.random.default_rng(21)
    lens = [6000, 1500]
    pool, tables = random_cache(rng, model, lens, 94, 0)
    q = torch.from_numpy(rng.standard_normal((2, 6, 128))).to(DEV).to(dtype)
    got, lse = tq.tq_paged_attention(pg, q, i32(pool), 0, ints(lens), ints(tables), sharp, want_lse=True)
    check(got, lse, model, kq, vq, pool, tables, q, lens, sharp, dtype, 0)
