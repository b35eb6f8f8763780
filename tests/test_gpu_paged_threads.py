"""Calls of several host threads at once, on streams of their own."""
import threading

import numpy as np
import pytest
import torch

import vector_compression_b200 as tq
from tests.paged_ref import Model
from tests.test_gpu_paged import DEV, i32, ints, quantizers, random_cache

pytestmark = pytest.mark.gpu


def test_two_shapes_of_the_kernel_for_any_shape_at_once():
    """One function serves both sizes of shared memory (73 KB and 1.5 KB of queries)."""
    sides = []
    for G, m in ((16, 1024), (3, 32)):
        kp, vp, _, _ = quantizers(128 if m > 32 else 64, 3, m)
        pg, model = tq.TQPaged(kp, vp, 1, 1, 32), Model(kp, vp, 1, 1, 32)
        rng = np.random.default_rng(G)
        pool, tables = random_cache(rng, model, [40, 3], 2, 0)
        q = torch.from_numpy(rng.standard_normal((2, G, kp.d))).to(DEV).float()
        args = (pg, q, i32(pool), 0, ints([40, 3]), ints(tables), 0.1)
        sides.append((args, tq.tq_paged_attention(*args)))
    torch.cuda.synchronize()
    failed = []

    def loop(args, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(3000):
                    got = tq.tq_paged_attention(*args)
                torch.cuda.current_stream().synchronize()
                assert torch.equal(got, want)
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=loop, args=s) for s in sides * 2]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    tq.tq_sync_check()
