"""The bounds of tests/paged_bounds.py hold for the arithmetic that they describe and for none that drops a digit:
the kernel's roundings, redone in numpy."""
import numpy as np
import pytest

from oracle import tq_oracle as o
from tests import paged_bounds as pb


def place_values(x, digits):
    """x as the kernel's images hold it: place values of 24 bits (three bytes), or without the last byte."""
    j = 2.0 ** (np.arange(x.shape[1]) % 4)
    inv = pb.Q_MAX / np.maximum(abs(x).max(-1, keepdims=True), 1e-30)
    v = np.rint(x * inv / j)
    if digits == 2:
        v = v - ((v + 128) % 256 - 128)
    return v * j / inv


def attention(qr, u, K, S, kn, kr, V, vn, scale, kappa, steps, half):
    s = scale * kn * (qr @ K.T + kappa * kr * (u @ S.T))
    top = s.max(-1, keepdims=True)
    p = np.exp(s - top)
    tot = p.sum(-1, keepdims=True)
    w, levels = p * vn, abs(V).max()
    step = levels / (steps[1] + half)
    L = np.where(V > 0, np.rint(V / step - half) + half, -(np.rint(-V / step - half) + half)) * step
    out = np.zeros((len(qr), K.shape[1]))
    for i in range(0, len(kn), 128):
        big = w[:, i:i + 128].max(-1, keepdims=True)
        out += np.rint(w[:, i:i + 128] / big * steps[0]) * big / steps[0] @ L[i:i + 128]
    return out / tot, (top + np.log(tot))[:, 0]


@pytest.mark.parametrize("d,bits,n", [(128, 3, 130), (128, 4, 700), (64, 2, 500), (256, 3, 300), (64, 4, 40)])
def test_bounds_hold_and_a_lost_digit_breaks_them(d, bits, n):
    rng = np.random.default_rng(d + n)
    ck, cv = (np.asarray(o.Quantizer(d, b, prod=False, draws=dict(signs=np.ones(d))).centroids) for b in (bits - 1, bits))
    G, kappa, scale = 4, np.sqrt(np.pi / 2) / d, d ** -0.5
    qr = rng.standard_normal((G, d))
    u = qr @ rng.standard_normal((d, d)).T
    K, V = ck[rng.integers(0, len(ck), (n, d))], cv[rng.integers(0, len(cv), (n, d))]
    S = 2.0 * rng.integers(0, 2, (n, d)) - 1
    kn, vn, kr = rng.uniform(4, 16, n), rng.uniform(4, 16, n), rng.uniform(0.3, 0.4, n)
    args, same = (K, S, kn, kr, V, vn, scale, kappa), lambda x: x
    half = 0.5 if bits == 4 else 0.0

    def off(digits, steps, held):
        out, lse, e_out, e_lse = pb.head_bounds(qr, u, *args, same, 2.0 ** -24, held, True)
        got, l = attention(place_values(qr, digits), place_values(u, digits), *args, steps, half)
        return (np.linalg.norm(got - out, axis=-1) / e_out).max(), (abs(l - lse) / e_lse).max()

    for steps in (pb.FINE, pb.COARSE):
        eo, el = off(3, steps, steps)
        assert eo < 1 and el < 1
    assert off(2, pb.FINE, pb.FINE)[1] > 1      # two bytes of q' and u instead of three: lse shows it
    assert off(3, pb.COARSE, pb.FINE)[0] > 1    # 16-bit weights and levels where fp32 is due: the output shows it
