"""Checks of the paged cache's and the rotary positions' entry points that need
no GPU: what is refused before anything is launched."""
import ctypes as C

import numpy as np
import pytest
import torch

import vector_compression_b200 as tq
from vector_compression_b200 import _lib as L

FAKE = C.c_void_p(0x10000)  # aligned, never dereferenced


def test_rope_create_refusals():
    lib = L.lib()
    h = C.c_void_p()
    ok = dict(rot=128, pairs=0, base=1e4, kind=0, factor=1.0, orig=1.0, low=1.0, high=2.0)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.tq_rope_create(a["rot"], a["pairs"], a["base"], a["kind"], a["factor"], a["orig"], a["low"],
                                  a["high"], C.byref(h))

    for kind in range(4):
        assert call(kind=kind) == 0
        assert lib.tq_rope_destroy(h) == 0
    assert lib.tq_rope_destroy(None) == 0
    nan, inf = float("nan"), float("inf")
    for bad in (dict(rot=0), dict(rot=3), dict(rot=258), dict(rot=-2), dict(base=1.0), dict(base=nan), dict(base=inf),
                dict(kind=4), dict(kind=-1), dict(kind=1, factor=0.5), dict(kind=1, factor=nan),
                dict(kind=2, orig=0.0), dict(kind=2, low=2.0), dict(kind=2, low=0.0), dict(kind=3, high=inf),
                dict(kind=3, factor=inf), dict(kind=3, low=nan)):
        assert call(**bad) == 1, bad
        assert not h.value
    assert lib.tq_rope_create(128, 0, 1e4, 0, 1.0, 0.0, 0.0, 0.0, None) == 1
    # the plain form does not read the others
    assert call(factor=nan, orig=nan, low=nan, high=nan) == 0
    lib.tq_rope_destroy(h)


def test_norm_rope_refusals():
    lib = L.lib()
    rope = tq.TQRope(64)

    def call(r=rope.handle, dt=0, n=4, d=64, Hq=2, q=FAKE, qt=128, qh=64, Hkv=0, pos=FAKE, eps=0.0, out=FAKE, ot=128,
             oh=64, wq=None):
        return lib.tq_qk_norm_rope(r, dt, n, d, Hq, q, qt, qh, Hkv, None, 0, 0, pos, wq, None, eps, out, ot, oh,
                                   None, 0, 0, None)

    for bad in (dict(dt=3), dict(dt=-1), dict(n=-1), dict(d=0), dict(d=32), dict(d=4097), dict(Hq=-1), dict(q=None),
                dict(out=None), dict(pos=None), dict(pos=C.c_void_p(0x10004)), dict(eps=-1.0), dict(eps=float("nan")),
                dict(q=C.c_void_p(0x10002)), dict(ot=63), dict(oh=63), dict(qt=-1), dict(qh=-64), dict(Hkv=1),
                dict(wq=C.c_void_p(0x10002))):
        assert call(**bad) == 1, bad
    assert call(n=0) == 0
    assert call(Hq=0) == 0


def test_paged_null_and_bad_arguments():
    lib = L.lib()
    h, bw, pw, sz = C.c_void_p(), C.c_int(), C.c_int64(), C.c_size_t()
    mse = tq.TQParams(128, 3, tq.MODE_MSE, tq.ROT_HADAMARD, signs=np.ones(128, np.int8))
    for layers, hkv, page in ((0, 1, 32), (1, 0, 32), (1, 1, 31), (1, 1, 0), (1, 1, 48), (4097, 1, 32), (1, 1025, 32),
                              (1, 1, 1 << 17)):
        assert lib.tq_paged_create(mse.handle, mse.handle, layers, hkv, page, C.byref(h)) == 1
    # keys need a Q_prod handle
    assert lib.tq_paged_create(mse.handle, mse.handle, 1, 1, 32, C.byref(h)) == 1
    assert lib.tq_paged_create(None, mse.handle, 1, 1, 32, C.byref(h)) == 1
    assert lib.tq_paged_create(mse.handle, mse.handle, 1, 1, 32, None) == 1
    assert lib.tq_paged_destroy(None) == 0
    assert lib.tq_paged_info(None, C.byref(bw), C.byref(pw)) == 1
    assert lib.tq_paged_append(None, FAKE, 1, 0, *[FAKE] * 6, 1, 1, None, FAKE, FAKE, 1, 1, None) == 1
    assert lib.tq_paged_attention_workspace_size(None, 1, 1, C.byref(sz)) == 1
    assert lib.tq_paged_attention(None, FAKE, 0, 128, 1, 1, FAKE, 1, 0, FAKE, FAKE, 1, 1, 1.0, FAKE, None, FAKE, 0,
                                  None) == 1
    assert lib.tq_paged_fork(None, FAKE, 1, FAKE, 1, 1, FAKE, 1, FAKE, FAKE, FAKE, 1, None) == 1
    assert lib.tq_paged_compact(None, FAKE, 1, FAKE, FAKE, 1, 1, FAKE, 1, FAKE, FAKE, 0, None) == 1
    for n in (0, -1, 1 << 31):
        assert lib.tq_paged_compact_workspace_size(n, C.byref(sz)) == 1
    assert lib.tq_paged_compact_workspace_size(1000, None) == 1
    assert lib.tq_paged_compact_workspace_size(1000, C.byref(sz)) == 0 and sz.value >= 3 * 4000


def test_the_binding_wants_cuda_tensors():
    q, pos = torch.zeros(2, 4, 64), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        tq.tq_qk_norm_rope(tq.TQRope(64), q, None, pos)
    with pytest.raises(ValueError):
        tq.tq_qk_norm_rope(tq.TQRope(64), q[0], None, pos)
    with pytest.raises(ValueError):
        tq.tq_qk_norm_rope(tq.TQRope(64), q.double(), None, pos)


def test_a_closed_rotation_is_not_no_rotation():
    rope = tq.TQRope(64)
    rope.close()
    with pytest.raises(ValueError):
        rope.handle
    rope.close()
