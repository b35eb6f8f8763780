"""Value norms that are not finite in the contiguous cache: their KV head's outputs are NaN, whichever kernel a shape
takes, and the other heads' are what they were."""
import pytest
import torch

import vector_compression_b200 as tq
from tests.test_gpu_paged import DEV, quantizers

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [
    # d, bits, vbits, m, G: the tensor-core kernel's shapes, and the other's
    (128, 3, 3, 128, 4), (128, 2, 4, 64, 7), (192, 4, 2, 256, 8), (128, 5, 3, 128, 4), (64, 3, 3, 64, 2),
])
@pytest.mark.parametrize("seq", [1, 77, 3000])
def test_value_norms_that_are_not_finite(shape, seq):
    d, bits, vbits, m, G = shape
    kp, vp, _, _ = quantizers(d, bits, m, vbits)
    hkv, cap = 3, -(-seq // 32) * 32 + 32
    g = torch.Generator(device=DEV).manual_seed(d + seq)
    x = torch.randn(2, hkv, seq, d, device=DEV, generator=g).half()
    kc = tq.tq_encode_prod(kp, x[0], seg_len=seq, seg_cap=cap)
    codes, norms = tq.tq_encode_mse(vp, x[1], layout=tq.LAYOUT_BLOCK32, seg_len=seq, seg_cap=cap)
    q = torch.randn(1, 1, hkv * G, d, device=DEV, generator=g)

    def call(n):
        return tq.tq_decode_attention(kp, vp, q, kc, (codes, n), seq, cap, d ** -0.5)[0, 0].view(hkv, G, d)

    clean = call(norms)
    assert bool(torch.isfinite(clean).all())
    for h, t in ((0, 0), (1, seq - 1), (2, seq // 2)):
        for bad in (float("nan"), float("inf")):
            n = norms.clone()
            n.view(hkv, cap)[h, t] = bad
            got = call(n)
            assert bool(torch.isnan(got[h]).all()), (h, t, bad)
            rest = [i for i in range(hkv) if i != h]
            assert torch.equal(got[rest], clean[rest])
    n = norms.clone()
    n.view(hkv, cap)[:, seq:] = float("nan")  # places without a token
    assert torch.equal(call(n), clean)
    tq.tq_sync_check()
