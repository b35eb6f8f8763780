"""What the paged attention may be off by, from the roundings that it makes.

A bound that adds the largest error of every term (as tests/paged_ref.py's
delta) is hundreds of times what a correct kernel does.  The roundings are
independent, so here their squares add, and six standard deviations are
allowed.

Score of a token, in units of scale n (n its key norm), per query head:
  - fixed point: entry j of q' is off by at most half of 2^(j mod 4) s, s =
    max|q'| / (127 2^16), uniformly: variance s^2 4^(j mod 4) / 12 times C_j^2;
    the entries of u in the same way, times (kappa rho)^2;
  - fp32: the rotation adds log2(d_pad) times, u's sums and the score's last
    steps round a dozen times values of the size of rms(q') (the products with
    0/1 bits times a level's coefficient are that size): 4 2^-24 rms(q').  Where
    the d_pad + m terms are added one by one (serial), each addition rounds a
    sum that grows to |q'| |C| and kappa rho |u|, by 0.3 2^-24 of it on average,
    and sqrt(d_pad + m) / 2 of them add up.
lse: the scores' errors weighted with p, and fp32's steps of the largest score
and of lse (4 each), the power of two's 2^-22.
Output, 2-norm over a head, R = sqrt(sum p^2 |v|^2) (about |out| for random codes):
  - the scores' errors: p changes by p (delta_t - mean delta);
  - weights and levels: half a step of `weight_steps` of the group's largest
    weight (128 tokens), half a step of `level_steps` of the largest level, both
    uniform; zero steps: fp32;
  - fp32: the power of two 2^-22, sums, join and rotation 12 2^-24;
  - the output's rounding, half a step of its type."""
import numpy as np

Q_MAX = 127.0 * 2 ** 16
FINE, COARSE = (8388607.0, 8388607.0), (65535.0, 32767.0)


def score_sigma(qr, u, K, kn, kr, scale, kappa, fixed, serial):
    """Standard deviation of each score [heads, tokens]."""
    dp, m = qr.shape[1], u.shape[1]
    var = (4 * 2.0 ** -24) ** 2 * (qr ** 2).mean(-1)[:, None] * np.ones(len(kn))
    if fixed:
        sq, su = (np.maximum(abs(x).max(-1, keepdims=True), 1e-30) / Q_MAX for x in (qr, u))
        var = var + sq ** 2 * (4.0 ** (np.arange(dp) % 4) / 12 * K ** 2).sum(-1)
        var = var + (kappa * kr) ** 2 * su ** 2 * (4.0 ** (np.arange(m) % 4)).sum() / 12
    if serial:
        size = np.linalg.norm(qr, axis=-1)[:, None] * np.linalg.norm(K, axis=-1) + kappa * kr * np.linalg.norm(u, axis=-1)[:, None]
        var = var + (0.15 * 2.0 ** -24 * np.sqrt(dp + m) * size) ** 2
    return abs(scale) * kn * np.sqrt(var)


def head_bounds(qr, u, K, S, kn, kr, V, vn, scale, kappa, rotate_back, eps, steps, fixed, serial=False):
    """(out, lse, most |out error|, most lse error) per query head of one KV head over its tokens, in 64 bits.  K, V:
    key and value levels [tokens, d_pad], S: +-1 [tokens, m]; steps: (weight_steps, level_steps) or None."""
    s = scale * kn * (qr @ K.T + kappa * kr * (u @ S.T))
    top = s.max(-1, keepdims=True)
    p = np.exp(s - top)
    tot = p.sum(-1, keepdims=True)
    p = p / tot
    out = rotate_back(p @ (V * vn[:, None]))
    lse = (top + np.log(tot))[:, 0]
    sigma = score_sigma(qr, u, K, kn, kr, scale, kappa, fixed, serial)
    mean = np.sqrt((p ** 2 * sigma ** 2).sum(-1))
    e_lse = 6 * mean + 4 * 2.0 ** -24 * (abs(lse) + abs(top[:, 0])) + 2.0 ** -22
    size = vn * np.linalg.norm(V, axis=-1)
    R = np.sqrt((p ** 2 * size ** 2).sum(-1))
    n = np.linalg.norm(out, axis=-1)
    e_out = 6 * np.sqrt((p ** 2 * sigma ** 2 * size ** 2).sum(-1)) + n * 6 * mean
    e_out = e_out + (2.0 ** -22 + 12 * 2.0 ** -24) * (R + n) + eps * n
    if steps:
        w = p * vn
        groups = np.array([w[:, i:i + 128].max(-1) ** 2 * w[:, i:i + 128].shape[1] for i in range(0, w.shape[1], 128)]).sum(0)
        weights = np.sqrt(groups / 12) / steps[0] * np.sqrt((V ** 2).sum(-1).mean())
        levels = np.sqrt((w ** 2).sum(-1) * V.shape[1] / 12) * abs(V).max() / steps[1]
        e_out = e_out + 6 * np.sqrt(weights ** 2 + levels ** 2)
    return out, lse, e_out, e_lse
