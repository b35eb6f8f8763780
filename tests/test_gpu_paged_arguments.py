"""Arguments of the paged cache's and the norm + rotation's calls: what is refused, and what is not."""
import pytest
import torch

import vector_compression_b200 as tq
from tests.test_gpu_paged import DEV, ints, quantizers

pytestmark = pytest.mark.gpu


def test_a_workspace_whose_bytes_do_not_lie_together_is_refused():
    kp, vp, _, _ = quantizers(128, 3)
    pg = tq.TQPaged(kp, vp, 1, 2, 32)
    pool, tables, lens = pg.new_pool(3), ints([[0, 1]]), ints([10])
    q = torch.ones(1, 4, 128, device=DEV)
    need = tq.tq_paged_attention_workspace_size(pg, 1, 4)
    also = tq.tq_paged_compact_workspace_size(3)
    byte = lambda n: torch.empty(n, dtype=torch.uint8, device=DEV)  # noqa: E731
    for n, call in ((need, lambda ws: tq.tq_paged_attention(pg, q, pool, 0, lens, tables, 1.0, ws=ws)),
                    (also, lambda ws: tq.tq_paged_compact(pg, pool, tables, lens, ws=ws))):
        for ws in (byte(1).expand(n), byte(2 * n)[::2], byte(2 * n).view(2, n).t()):
            with pytest.raises(ValueError):
                call(ws)
        call(byte(n))
        call(byte(4 * n + 512).view(2, -1)[1, : (n + 3) // 4 * 4].view(torch.int32))  # any type, part of another
    tq.tq_sync_check()
