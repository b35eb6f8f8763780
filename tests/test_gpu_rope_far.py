"""Rotations at far positions against frequencies of 60 digits.

Tolerance per element: that of tests/test_gpu_rope.py, 48 2^-24 of the pair's
inputs, and the angle's: pos 2^-63 of a turn (the frequency's fixed point is off
by less than 2 of 2^-64) times 2 pi and the pair's inputs.  Frequencies that are
made in double are off by up to 2^-57 of a turn a position, 64 times that."""
import math
from decimal import Decimal as D
from decimal import getcontext

import numpy as np
import pytest
import torch

import vector_compression_b200 as tq
from tests.test_gpu_rope import DEV, SCALINGS

pytestmark = pytest.mark.gpu
PI = D("3.14159265358979323846264338327950288419716939937510582097494459")


def turns_per_position(rot, base, name):
    """f_i / (2 pi), and the factor on the rotated part."""
    getcontext().prec = 60
    s, out, mscale = SCALINGS[name], [], 1.0
    for i in range(rot // 2):
        f = (D(base).ln() * D(-2 * i) / D(rot)).exp()
        keep = D(1)
        if name == "linear":
            keep = D(0)
        if name == "bands":
            keep = (D(s["orig_len"]) * f / (2 * PI) - D(s["low"])) / (D(s["high"]) - D(s["low"]))
        if name == "yarn":
            border = lambda t: rot * math.log(s["orig_len"] / (t * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
            lo, hi = max(math.floor(border(s["high"])), 0), min(math.ceil(border(s["low"])), rot - 1)
            keep = 1 - D(i - lo) / D(hi - lo)
            mscale = 0.1 * math.log(s["factor"]) + 1
        keep = min(D(1), max(D(0), keep))
        f = f * keep + f / D(s.get("factor", 1.0)) * (1 - keep)
        out.append(f / (2 * PI))
    return out, mscale


@pytest.mark.parametrize("name", list(SCALINGS))
@pytest.mark.parametrize("rot,base", [(128, 500000.0), (64, 10000.0), (256, 1000000.0)])
def test_far_positions(rot, base, name):
    pos = [(1 << 40) + 12345, -(1 << 44) - 1, (1 << 46) + 7, 131071, (1 << 36) - 5]
    q = torch.randn(len(pos), 3, rot, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    got, _ = tq.tq_qk_norm_rope(tq.TQRope(rot, base, **SCALINGS[name]), q, None, torch.tensor(pos, device=DEV))
    f, mscale = turns_per_position(rot, base, name)
    turn = np.array([[float((p * x) % 1) for x in f] for p in pos])[:, None]
    x = q.double().cpu().numpy()
    u, v, co, si = x[..., : rot // 2], x[..., rot // 2:], np.cos(2 * np.pi * turn), np.sin(2 * np.pi * turn)
    want = np.concatenate([u * co - v * si, v * co + u * si], -1) * mscale
    size = np.tile((abs(u) + abs(v)) * mscale, 2)
    tol = 2.0 ** -24 * abs(want) + (48 * 2.0 ** -24 + 2 * np.pi * 2.0 ** -63 * abs(np.array(pos, float))[:, None, None]) * size
    err = abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), (err / tol).max((1, 2))
