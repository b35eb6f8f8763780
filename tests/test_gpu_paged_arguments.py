"""Arguments of the paged cache's and the norm + rotation's calls: what is refused, and what is not."""
import pytest
import torch

import vector_compression_b200 as tq
from tests.test_gpu_paged import DEV, ints, quantizers
from tests.test_gpu_rope import check

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


def test_norm_rope_into_rows_between_one_another():
    """Heads of one token between those of others, with nothing shared: written as anywhere else."""
    rope, pos = tq.TQRope(64), torch.arange(5, device=DEV)
    q = torch.randn(5, 2, 64, device=DEV)
    for ot, oh in ((128, 64), (64, 320), (128, 5 * 64), (130, 65), (128, 3 * 64 + 128)):
        buf = torch.full((5 * ot + 2 * oh + 64,), 7.0, device=DEV)
        out = buf.as_strided((5, 2, 64), (ot, oh, 1))
        tq.tq_qk_norm_rope(rope, q, None, pos, q_out=out)
        # by the formula: rows at odd elements are not read and multiplied in the same order as others
        check(out, q, None, range(5), 64, 10000.0, False, "plain")
    for ot, oh in ((64, 64), (64, 128), (128, 100), (100, 350)):
        buf = torch.full((5 * ot + 2 * oh + 64,), 7.0, device=DEV)
        with pytest.raises(tq.TQError):
            tq.tq_qk_norm_rope(rope, q, None, pos, q_out=buf.as_strided((5, 2, 64), (ot, oh, 1)))
        assert bool((buf == 7).all())


def test_sizes_beyond_32_bits_are_refused():
    """Not taken modulo 2^32: heads of 2^32 + 64 elements are no heads of 64."""
    q = torch.empty(1, 1, (1 << 32) + 64, dtype=torch.float16, device=DEV)
    with pytest.raises(ValueError, match="too large"):
        tq.tq_qk_norm_rope(None, q, None)
    q = torch.ones(1, 1, 64, device=DEV)
    with pytest.raises(ValueError, match="too large"):
        tq.tq_qk_norm_rope(None, q.expand(1, (1 << 32) + 1, 64), None, q_out=q.expand(1, (1 << 32) + 1, 64))
    kp, vp, _, _ = quantizers(64, 3)
    pg = tq.TQPaged(kp, vp, 1, 1, 32)
    pool, tables, lens = pg.new_pool(1), ints([[0]]), ints([1])
    with pytest.raises(ValueError, match="too large"):
        tq.tq_paged_attention(pg, q.expand(1, (1 << 32) + 1, 64), pool, 0, lens, tables, 1.0)
    with pytest.raises(ValueError, match="too large"):
        tq.tq_paged_fork(pg, pool, tables, lens, *[ints([0]).expand((1 << 32) + 1)] * 3)
    assert bool((q == 1).all()) and bool((pool == 0).all())


def test_the_sizes_of_a_cache():
    """Of handles that are otherwise right: the largest sizes are taken, the next ones refused."""
    kp, vp, _, _ = quantizers(128, 3)
    for layers, hkv, page in ((4096, 1, 32), (1, 1024, 32), (1, 1, 65536), (1, 1, 96)):
        pg = tq.TQPaged(kp, vp, layers, hkv, page)
        assert pg.page_words == layers * hkv * page // 32 * pg.block_words
    for layers, hkv, page in ((0, 1, 32), (-1, 1, 32), (1, 0, 32), (1, 1, 31), (1, 1, 0), (1, 1, 48), (4097, 1, 32),
                              (1, 1025, 32), (1, 1, 65536 + 32)):
        with pytest.raises(tq.TQError):
            tq.TQPaged(kp, vp, layers, hkv, page)
