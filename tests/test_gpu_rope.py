"""tq_qk_norm_rope against the formula in 64 bits.

Tolerance per element: half a step of the output type, and for the fp32
arithmetic c 2^-24 (|a| + |b|) of a pair's inputs after the norm.  c counts the
roundings: the sum of d squares (at most d / lanes / vector + log2 lanes <= 40
steps, halved by the root), the reciprocal root (2 units), norm and weight
products (2), sine and cosine (2 units each, and 2 pi 2^-25 turns for the
angle's rounding to 32 and then 24 bits: < 8), the products and their sum (3):
below 48."""
import math

import numpy as np
import pytest
import torch

import vector_compression_b200 as tq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
SCALINGS = {
    "plain": dict(),
    "linear": dict(scaling=tq.ROPE_LINEAR, factor=4.0),
    "bands": dict(scaling=tq.ROPE_BANDS, factor=8.0, orig_len=8192, low=1.0, high=4.0),
    "yarn": dict(scaling=tq.ROPE_YARN, factor=16.0, orig_len=4096, low=1.0, high=32.0),
}


def frequencies(rot, base, name):
    i = np.arange(rot // 2)
    f = np.float64(base) ** (-2.0 * i / rot)
    s = SCALINGS[name]
    if name == "linear":
        return f / s["factor"], 1.0
    if name == "bands":
        keep = [min(1.0, max(0.0, (s["orig_len"] * x / (2 * math.pi) - s["low"]) / (s["high"] - s["low"]))) for x in f]
        return np.array([x * k + x / s["factor"] * (1 - k) for x, k in zip(f, keep)]), 1.0
    if name == "yarn":
        border = lambda t: rot * math.log(s["orig_len"] / (t * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(border(s["high"])), 0), min(math.ceil(border(s["low"])), rot - 1)
        slow = np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
        return f * (1 - slow) + f / s["factor"] * slow, 0.1 * math.log(s["factor"]) + 1
    return f, 1.0


def reference(x, w, pos, rot, base, pairs, name, eps, dtype):
    """(y, tolerance) in 64 bits."""
    x = x.detach().cpu().double().numpy()
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w.cpu().double().numpy()
    y, size = x.copy(), np.abs(x)
    if rot:
        f, mscale = frequencies(rot, base, name)
        # the turns as exact fractions of whole numbers: pos f / (2 pi) mod 1 in extended precision
        turn = np.array([[float((int(p) * np.longdouble(v) / (2 * np.longdouble(np.pi))) % 1) for v in f] for p in pos])
        co, si = np.cos(2 * np.pi * turn)[:, None], np.sin(2 * np.pi * turn)[:, None]
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, rot // 2), slice(rot // 2, rot))
        u, v = x[..., a], x[..., b]
        y[..., a], y[..., b] = (u * co - v * si) * mscale, (v * co + u * si) * mscale
        size[..., a] = size[..., b] = (np.abs(u) + np.abs(v)) * mscale
    return y, EPS[dtype] * np.abs(y) + 48 * 2.0 ** -24 * size + 1e-30


def check(got, x, w, pos, rot, base, pairs, name, eps=1e-6):
    want, tol = reference(x, w, pos, rot, base, pairs, name, eps, x.dtype)
    err = np.abs(got.detach().cpu().double().numpy() - want)
    if x.dtype == torch.float16:
        tol = tol + 2.0 ** -25  # half a step of a subnormal
    assert np.all(err <= tol), (err / tol).max()


def make(n, heads, d, dtype, seed, packed=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if packed:
        return torch.randn(n, heads + 5, d, device=DEV, generator=g).to(dtype)[:, 2:2 + heads]
    return torch.randn(n, heads, d, device=DEV, generator=g).to(dtype)


CASES = [
    # n, Hq, Hkv, d, rot, pairs, norm, scaling, packed
    (1, 32, 8, 128, 128, False, True, "bands", False),
    (37, 8, 2, 128, 128, False, False, "plain", True),
    (5, 7, 1, 80, 80, False, True, "linear", False),
    (6, 4, 4, 80, 40, False, True, "plain", True),
    (9, 3, 1, 96, 96, True, False, "yarn", True),
    (3, 2, 1, 192, 64, True, True, "yarn", False),
    (4, 2, 2, 256, 256, False, True, "plain", False),
    (4, 1, 1, 256, 128, True, False, "bands", False),
    (2, 3, 1, 7, 6, False, True, "plain", False),
    (2, 1, 1, 33, 10, True, True, "linear", True),
    (3, 2, 1, 1000, 200, False, True, "plain", False),
    (300, 40, 8, 64, 64, False, True, "plain", True),
    (2, 5, 0, 128, 0, False, True, "plain", False),
    (2, 1, 1, 1, 0, False, True, "plain", False),
    (3, 2, 2, 4096, 256, True, True, "plain", False),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("case", CASES)
def test_against_the_formula(case, dtype):
    n, Hq, Hkv, d, rot, pairs, norm, name, packed = case
    base = 10000.0
    q = make(n, Hq, d, dtype, 1, packed)
    k = make(n, Hkv, d, dtype, 2, packed) if Hkv else None
    w = [(1 + 0.3 * make(1, 1, d, torch.float32, s)[0, 0]).to(dtype) if norm else None for s in (3, 4)]
    pos = torch.randint(0, 1 << 17, (n,), generator=torch.Generator().manual_seed(5)).to(DEV)
    rope = tq.TQRope(rot, base, interleaved=pairs, **SCALINGS[name]) if rot else None
    qo, ko = tq.tq_qk_norm_rope(rope, q, k, pos if rot else None, w[0], w[1] if Hkv else None)
    check(qo, q, w[0], pos.cpu().numpy(), rot, base, pairs, name)
    if Hkv:
        check(ko, k, w[1], pos.cpu().numpy(), rot, base, pairs, name)
    else:
        assert ko is None


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", [
    # so many rows that a group of lanes takes several heads, of both sides, the last groups fewer
    (6001, 13, 6, 128, 128, False, True, "plain", True),
    (9000, 9, 2, 96, 48, True, False, "bands", False),
    (12345, 7, 0, 64, 64, False, True, "linear", True),
])
def test_many_rows(case, dtype):
    test_against_the_formula(case, dtype)


@pytest.mark.parametrize("pos", [0, 1, (1 << 20) - 1, 1 << 31, (1 << 40) + 12345, -1, -(1 << 33)])
def test_far_and_negative_positions(pos):
    q = make(1, 2, 128, torch.float32, 7)
    p = torch.tensor([pos], device=DEV)
    qo, _ = tq.tq_qk_norm_rope(tq.TQRope(128, 500000.0), q, None, p)
    # 64-bit extended precision carries the angle of 2^40 to 2^-24 of a turn at most; beyond 2^33 that is the
    # reference's own limit, so its share is added
    want, tol = reference(q, None, [pos], 128, 500000.0, False, "plain", 0.0, torch.float32)
    tol = tol + abs(pos) * 2.0 ** -53 * 2 * np.pi * np.abs(q.cpu().numpy()).max()
    assert np.all(np.abs(qo.cpu().double().numpy() - want) <= tol)


def test_in_place_and_layouts_that_other_tests_do_not_use():
    for dtype in (torch.float16, torch.float32):
        rope = tq.TQRope(128, 10000.0)
        pos = torch.arange(6, device=DEV) + 100
        x = make(6, 5, 128, dtype, 11)
        keep = x.clone()
        tq.tq_qk_norm_rope(rope, x[:, :4], x[:, 4:], pos, q_out=x[:, :4], k_out=x[:, 4:])
        check(x, keep, None, pos.cpu().numpy(), 128, 10000.0, False, "plain")
        # heads outside tokens, and rows that begin at odd elements of a larger buffer that keeps its other values
        base = torch.full((4 * 6 * 128 + 64,), 7.0, dtype=dtype, device=DEV)
        src = make(4, 6, 128, dtype, 12)
        out = base[1:1 + 4 * 6 * 128].view(4, 6, 128).transpose(0, 1)
        tq.tq_qk_norm_rope(rope, src.transpose(0, 1), None, pos, q_out=out)
        check(out, src.transpose(0, 1), None, pos.cpu().numpy(), 128, 10000.0, False, "plain")
        assert base[0] == 7 and bool((base[1 + 4 * 6 * 128:] == 7).all())
        # one head for all tokens (stride 0)
        one = make(1, 1, 128, dtype, 13).expand(6, 1, 128)
        got, _ = tq.tq_qk_norm_rope(rope, one, None, pos)
        check(got, one, None, pos.cpu().numpy(), 128, 10000.0, False, "plain")


def test_norm_of_one_side_only_and_a_zero_row():
    q, k = make(3, 2, 128, torch.bfloat16, 21), make(3, 2, 128, torch.bfloat16, 22)
    k[1] = 0
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    qo, ko = tq.tq_qk_norm_rope(None, q, k, None, None, w, eps=1e-5)
    assert torch.equal(qo, q)
    check(ko, k, w, [0] * 3, 0, 1e4, False, "plain", eps=1e-5)
    assert bool((ko[1] == 0).all())


def test_nothing_to_do_and_refusals():
    rope = tq.TQRope(64)
    empty = torch.empty(0, 4, 64, device=DEV)
    qo, _ = tq.tq_qk_norm_rope(rope, empty, None, torch.empty(0, dtype=torch.int64, device=DEV))
    assert qo.shape == (0, 4, 64)
    q, pos = make(2, 2, 64, torch.float32, 31), torch.zeros(2, dtype=torch.int64, device=DEV)
    with pytest.raises(ValueError):
        tq.tq_qk_norm_rope(rope, q, None, pos.int())
    with pytest.raises(ValueError):
        tq.tq_qk_norm_rope(rope, q, make(2, 2, 32, torch.float32, 1), pos)
    with pytest.raises(ValueError):
        tq.tq_qk_norm_rope(rope, q, q.half(), pos)
    with pytest.raises(ValueError):
        tq.tq_qk_norm_rope(rope, q, None, pos, wq=torch.ones(64))
    with pytest.raises(ValueError):
        tq.tq_qk_norm_rope(rope, q.transpose(1, 2), None, pos)
    with pytest.raises(tq.TQError):
        tq.tq_qk_norm_rope(tq.TQRope(128), q, None, pos)
    with pytest.raises(tq.TQError):
        tq.tq_qk_norm_rope(rope, q, None, pos, wq=torch.ones(64, device=DEV), eps=-1.0)
    with pytest.raises(tq.TQError):  # all tokens into one row
        tq.tq_qk_norm_rope(rope, q, None, pos, q_out=torch.empty(1, 2, 64, device=DEV).expand(2, 2, 64))


def test_another_stream_and_a_captured_call():
    rope = tq.TQRope(128, 10000.0)
    q, pos = make(4, 8, 128, torch.float16, 41), torch.arange(4, device=DEV)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tq.tq_qk_norm_rope(rope, q, None, pos, q_out=out)
    side.synchronize()
    check(out, q, None, [0, 1, 2, 3], 128, 10000.0, False, "plain")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tq.tq_qk_norm_rope(rope, q, None, pos, q_out=out)
    pos += 1000
    g.replay()
    torch.cuda.synchronize()
    check(out, q, None, [1000, 1001, 1002, 1003], 128, 10000.0, False, "plain")
