"""The paged compressed cache against a plain numpy model (tests/paged_ref.py):
append and page operations bit for bit, attention in 64 bits.

Attention's tolerance: the output type's half step; the change of the weights
by a score error of at most delta (bounded from the terms: every term rounds at
most d_pad + m times in fp32), 2 delta of the sum of p ||value||; and 2^-15 of
that sum for levels and weights held in 16 bits.  The lse is off by delta and a
few of its own steps."""
import math

import numpy as np
import pytest
import torch

import synth
import vector_compression_b200 as tq
from oracle import tq_oracle as o
from tests.paged_ref import Model
from tests.parity import u32

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def quantizers(d, bits, m=None, vbits=None, r16=False, seed=3):
    dp = synth.next_pow2(d)
    m = m or dp
    kd, vd = synth.method_draws(d, m, seed, stream=1), synth.method_draws(d, m, seed, stream=2)
    kp = tq.TQParams(d, bits, tq.MODE_PROD | (tq.STORE_RNORM_F16 if r16 else 0), m=m, signs=kd["signs"], S=kd["S"])
    vp = tq.TQParams(d, vbits or bits, tq.MODE_MSE, signs=vd["signs"])
    return kp, vp, o.Quantizer(d, bits, prod=True, draws=kd), o.Quantizer(d, vbits or bits, prod=False, draws=vd)


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int32)).to(DEV)


def ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def rows(rng, n, hkv, model):
    """Random encoded tokens: (kwords, kn, kr, vidx, vn) for the model and the binding's tensors."""
    kw = rng.integers(0, 1 << 32, (n, hkv, model.nk), dtype=np.uint64).astype(np.uint32)
    kn, vn = (rng.uniform(0.5, 2.0, (n, hkv)).astype(np.float32) for _ in range(2))
    kr = rng.uniform(0.1, 0.6, (n, hkv)).astype(np.float16 if model.r16 else np.float32)
    vi = rng.integers(0, 1 << model.kv, (n, hkv, model.dp))
    vc = o.pack_row(vi.reshape(n * hkv, -1), model.kv)
    keys = (i32(kw[..., : model.kw]), i32(kw[..., model.kw:]), torch.from_numpy(kn.reshape(-1)).to(DEV),
            torch.from_numpy(kr.reshape(-1)).to(DEV))
    bits = kr.view(np.uint16) if model.r16 else kr.view(np.uint32)
    return (kw, kn.view(np.uint32), bits, vi, vn.view(np.uint32)), keys, (i32(vc), torch.from_numpy(vn.reshape(-1)).to(DEV))


SHAPES = [
    # d, bits, vbits, m, r16, layers, hkv, page
    (128, 3, 3, 128, False, 2, 2, 64),
    (128, 3, 3, 64, True, 1, 3, 32),
    (64, 2, 1, 32, False, 1, 2, 96),
    (192, 4, 4, 256, False, 1, 1, 32),
    (32, 2, 2, 32, True, 3, 1, 256),
    (256, 5, 2, 96, False, 1, 2, 64),
]


@pytest.mark.parametrize("shape", SHAPES)
def test_append_bit_for_bit(shape):
    d, bits, vbits, m, r16, layers, hkv, page = shape
    kp, vp, _, _ = quantizers(d, bits, m, vbits, r16)
    pg = tq.TQPaged(kp, vp, layers, hkv, page)
    model = Model(kp, vp, layers, hkv, page)
    assert (pg.block_words, pg.page_words) == (model.words, model.page_words)
    rng = np.random.default_rng(d + bits)
    width, B = 3, 7
    n_pages = B * width + 2
    pool = rng.integers(0, 1 << 32, (n_pages, model.page_words), dtype=np.uint64).astype(np.uint32)
    tables = rng.permutation(n_pages)[: B * width].reshape(B, width).astype(np.int32)
    tables[2, 0], tables[3, 1] = -1, n_pages  # holes
    # empty, one token, over block and page ends, into holes, before 0, past the table
    new = [0, 1, 40, 2 * page, 33, 20, 5]
    start = [3, 31, 20, 1, -10, width * page - 9, page - 2]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    tail = 3  # rows that belong to no sequence
    ref, keys, vals = rows(rng, cu[-1] + tail, hkv, model)
    got = i32(pool)
    layer = layers - 1
    tq.tq_paged_append(pg, got, layer, keys, vals, ints(start), ints(tables), cu=ints(cu))
    model.append(pool, layer, *ref, cu, start, tables)
    assert np.array_equal(u32(got), pool)
    # one token per sequence, and a table that is a part of a wider one
    ref, keys, vals = rows(rng, B, hkv, model)
    start = [0, 31, 32, page, page - 1, width * page - 1, width * page]
    wide = torch.full((B, width + 4), 1 << 30, dtype=torch.int32, device=DEV)
    wide[:, :width] = ints(tables)
    tq.tq_paged_append(pg, got, 0, keys, vals, ints(start), wide[:, :width])
    model.append(pool, 0, *ref, np.arange(B + 1), start, tables)
    assert np.array_equal(u32(got), pool)
    tq.tq_sync_check()


def random_cache(rng, model, lens, width, layer, spare=2):
    """A pool of noise (NaN norms in stale slots) with encoded tokens in the first lens[b] slots of each row."""
    B = len(lens)
    need = [-(-n // model.page) for n in lens]
    n_pages = sum(need) + spare
    pool = rng.integers(0, 1 << 32, (n_pages, model.page_words), dtype=np.uint64).astype(np.uint32)
    ids = rng.permutation(n_pages)
    tables = np.full((B, width), -1, np.int32)
    at = 0
    for b in range(B):
        tables[b, : need[b]] = ids[at:at + need[b]]
        at += need[b]
        for t in range(need[b] * model.page):
            for h in range(model.hkv):
                rec = model.record(pool, tables[b, t // model.page], layer, h, t % model.page // 32)
                f, tau = rec.view(np.float32), t % 32
                live = t < lens[b]
                f[model.kn + tau] = rng.uniform(0.5, 2.0) * 8 if live else np.nan
                f[model.vn + tau] = rng.uniform(0.5, 2.0) * 8 if live else np.nan
                if model.r16:
                    rec[model.kr:model.v].view(np.float16)[tau] = 0.3 + 0.1 * rng.uniform() if live else np.nan
                else:
                    f[model.kr + tau] = 0.3 + 0.1 * rng.uniform() if live else np.nan
    return pool, tables


def check_attention(got, lse, ref, dtype):
    out, want_lse, spread, delta = ref
    got, lse = got.detach().double().cpu().numpy(), lse.double().cpu().numpy()
    tol = EPS[dtype] * np.abs(out) + ((2 * delta + 2.0 ** -15) * spread)[..., None]
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    err = np.abs(got - out)
    assert np.all(err <= tol), (err / np.maximum(tol, 1e-300)).max()
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(lse), empty) and np.all(got[empty] == 0)
    e = np.abs(lse[~empty] - want_lse[~empty])
    assert np.all(e <= (delta + 8 * 2.0 ** -24 * np.abs(want_lse) + 2.0 ** -22)[~empty]), e.max()


ATTENTION = [
    # d, bits, vbits, m, r16, hkv, G, page, lens
    (128, 3, 3, 128, False, 2, 4, 64, [0, 1, 31, 32, 33, 200, 700]),
    (128, 3, 3, 128, False, 1, 1, 32, [129]),
    (128, 3, 3, 128, True, 1, 8, 96, [1, 0, 500]),
    (128, 3, 3, 64, False, 2, 5, 32, [63, 64, 65]),
    (128, 2, 1, 128, False, 1, 2, 32, [257, 10]),
    (128, 4, 4, 128, False, 1, 3, 64, [300, 5]),
    (128, 3, 2, 64, True, 1, 7, 64, [400]),
    (64, 3, 3, 64, False, 2, 4, 32, [100, 290]),
    (64, 2, 4, 64, False, 1, 8, 32, [513]),
    (64, 4, 2, 32, False, 1, 2, 32, [90]),
    (192, 3, 3, 256, False, 1, 4, 32, [333, 2]),
    (256, 4, 4, 256, True, 1, 8, 64, [260]),
    (256, 2, 2, 128, False, 1, 1, 32, [70]),
    (100, 3, 3, 128, False, 1, 6, 32, [150]),
    (32, 3, 3, 32, False, 2, 2, 32, [0, 77]),
    (128, 5, 3, 128, False, 1, 4, 32, [100]),
    (128, 3, 3, 128, False, 1, 16, 32, [140, 3]),
    (128, 3, 3, 512, False, 1, 9, 32, [64]),
    (192, 3, 3, 256, False, 1, 6, 32, [129, 128]),
    (64, 2, 2, 64, True, 2, 12, 32, [127, 200]),
    (128, 2, 3, 64, False, 1, 11, 64, [256, 31]),
    (256, 2, 1, 256, False, 1, 3, 32, [1, 161]),
    (64, 4, 1, 64, False, 1, 5, 96, [97]),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("case", ATTENTION)
def test_attention_against_64_bits(case, dtype):
    d, bits, vbits, m, r16, hkv, G, page, lens = case
    kp, vp, kq, vq = quantizers(d, bits, m, vbits, r16)
    layers = 2
    pg, model = tq.TQPaged(kp, vp, layers, hkv, page), Model(kp, vp, layers, hkv, page)
    rng = np.random.default_rng(sum(lens) + G)
    width = max(-(-max(lens) // page), 1) + 1
    pool, tables = random_cache(rng, model, lens, width, 1)
    q = torch.from_numpy(rng.standard_normal((len(lens), hkv * G, d))).to(DEV).to(dtype)
    scale = 1 / math.sqrt(d)
    got, lse = tq.tq_paged_attention(pg, q, i32(pool), 1, ints(lens), ints(tables), scale, want_lse=True)
    tq.tq_sync_check()
    ref = model.attention(pool, 1, kq, vq, q.double().cpu().numpy(), lens, tables, scale)
    check_attention(got, lse, ref, dtype)


def test_attention_holes_shared_pages_and_odd_lengths():
    kp, vp, kq, vq = quantizers(128, 3)
    pg, model = tq.TQPaged(kp, vp, 1, 2, 64), Model(kp, vp, 1, 2, 64)
    rng = np.random.default_rng(8)
    lens = [300, 300, 130, 64, 40]
    pool, tables = random_cache(rng, model, lens, 6, 0)
    tables[0, 1], tables[0, 4] = -1, len(pool)     # holes, the last page among them
    tables[1, :2] = tables[0, [0, 2]]              # shared pages
    tables[3, 0] = -5                              # nothing left of this one
    asked = [300, 1000000, 130, 64, -3]            # longer than the table, negative
    seen = [300, 6 * 64, 130, 64, 0]
    tables[1, 5:] = -1
    # slots behind row 1's 300 tokens hold NaN norms: give the part that is asked for real ones
    for t in range(300, 5 * 64):
        for h in range(2):
            rec = model.record(pool, tables[1, t // 64], 0, h, t % 64 // 32).view(np.float32)
            rec[[model.kn + t % 32, model.kr + t % 32, model.vn + t % 32]] = (3.0, 0.3, 2.0)
    q = torch.from_numpy(rng.standard_normal((5, 8, 128))).to(DEV).half()
    big = torch.zeros(5, 11, 128, dtype=torch.float16, device=DEV)  # queries inside a fused projection
    big[:, :8] = q
    got, lse = tq.tq_paged_attention(pg, big[:, :8], i32(pool), 0, ints(asked), ints(tables), 0.1, want_lse=True)
    ref = model.attention(pool, 0, kq, vq, q.double().cpu().numpy(), seen, tables, 0.1)
    assert np.isneginf(ref[1][3]).all() and np.isneginf(ref[1][4]).all()
    check_attention(got, lse, ref, torch.float16)


def test_attention_many_short_and_one_long_sequence():
    """More sequences than fit a CTA's share, and one that many CTAs share."""
    kp, vp, kq, vq = quantizers(128, 3)
    pg, model = tq.TQPaged(kp, vp, 1, 1, 32), Model(kp, vp, 1, 1, 32)
    rng = np.random.default_rng(9)
    lens = [int(x) for x in rng.integers(0, 40, 150)] + [3000]
    pool, tables = random_cache(rng, model, lens, 100, 0)
    q = torch.from_numpy(rng.standard_normal((151, 4, 128))).to(DEV).bfloat16()
    got, lse = tq.tq_paged_attention(pg, q, i32(pool), 0, ints(lens), ints(tables), 0.09, want_lse=True)
    ref = model.attention(pool, 0, kq, vq, q.double().cpu().numpy(), lens, tables, 0.09)
    check_attention(got, lse, ref, torch.bfloat16)
    again = tq.tq_paged_attention(pg, q, i32(pool), 0, ints(lens), ints(tables), 0.09)
    assert torch.equal(got, again)  # the parts are joined in a fixed order


def test_attention_extreme_scores_and_not_finite_queries():
    kp, vp, kq, vq = quantizers(128, 3)
    pg, model = tq.TQPaged(kp, vp, 1, 1, 32), Model(kp, vp, 1, 1, 32)
    rng = np.random.default_rng(10)
    pool, tables = random_cache(rng, model, [500, 500, 500, 500], 16, 0)
    q = torch.from_numpy(rng.standard_normal((4, 4, 128))).to(DEV).float()
    q[0] = 0                       # every token weighs the same
    q[1] *= 100                    # one token has it all
    q[2, 1, 5], q[2, 2, 7] = float("nan"), float("inf")
    q[3] *= 1e-30
    got, lse = tq.tq_paged_attention(pg, q, i32(pool), 0, ints([500] * 4), ints(tables), 0.09, want_lse=True)
    clean = q.double().cpu().numpy()
    clean[2, 1:3] = 0
    ref = model.attention(pool, 0, kq, vq, clean, [500] * 4, tables, 0.09)
    keep = np.ones((4, 4), bool)
    keep[2, 1:3] = False
    k = torch.from_numpy(keep)
    check_attention(got.cpu()[k][None], lse.cpu()[k][None], [x[keep][None] for x in ref], torch.float32)
    assert bool(torch.isnan(got[2, 1:3]).all()) and bool(torch.isnan(lse[2, 1:3]).all())


def test_attention_more_sequences_than_a_warp_counts():
    """Beyond 1024 sequences the shares come from the prefix sums, with empty sequences at both ends and between."""
    kp, vp, kq, vq = quantizers(64, 3)
    pg, model = tq.TQPaged(kp, vp, 1, 1, 32), Model(kp, vp, 1, 1, 32)
    rng = np.random.default_rng(13)
    lens = [int(x) for x in rng.integers(0, 9, 1400) * rng.integers(0, 2, 1400)]
    lens[0] = lens[-1] = 0
    lens[700] = 1500
    pool, tables = random_cache(rng, model, lens, 48, 0)
    q = torch.from_numpy(rng.standard_normal((1400, 2, 64))).to(DEV).half()
    got, lse = tq.tq_paged_attention(pg, q, i32(pool), 0, ints(lens), ints(tables), 0.125, want_lse=True)
    ref = model.attention(pool, 0, kq, vq, q.double().cpu().numpy(), lens, tables, 0.125)
    check_attention(got, lse, ref, torch.float16)
    tq.tq_sync_check()
    none = tq.tq_paged_attention(pg, q, i32(pool), 0, torch.zeros(1400, dtype=torch.int32, device=DEV), ints(tables), 0.125)
    assert bool((none == 0).all())


def test_pages_beyond_32_bit_offsets():
    """Everything that a small pool does, at the far end of one of more than 2^31 words, bit for bit."""
    d, hkv, page = 128, 8, 64
    kp, vp, _, _ = quantizers(d, 3)
    pg = tq.TQPaged(kp, vp, 1, hkv, page)
    far_pages = 2 ** 31 // pg.page_words + 40
    far = torch.empty((far_pages, pg.page_words), dtype=torch.int32, device=DEV)
    near = pg.new_pool(40)
    g = torch.Generator(device=DEV).manual_seed(3)
    lens, B = [200, 75], 2
    x = torch.randn(sum(lens), hkv, d, device=DEV, generator=g).half()
    keys, vals = tq.tq_encode_prod(kp, x), tq.tq_encode_mse(vp, x)
    q = torch.randn(3, 4 * hkv, d, device=DEV, generator=g).half()
    near_t = ints([[30, 3, 17, 9], [8, 21, -1, -1], [-1] * 4])
    shift = far_pages - 40
    far_t = torch.where(near_t >= 0, near_t + shift, near_t)
    out = []
    for pool, t, off in ((near, near_t, 0), (far, far_t, shift)):
        n = ints(lens + [0])
        tq.tq_paged_append(pg, pool, 0, keys, vals, ints([0, 0]), t[:2], cu=ints([0, 200, 275]))
        tq.tq_paged_fork(pg, pool, t, n, ints([0]), ints([2]), ints([25 + off]))
        a = tq.tq_paged_attention(pg, q, pool, 0, n, t, 0.09, want_lse=True)
        n[1] = 0
        b = tq.tq_paged_attention(pg, q, pool, 0, n, t, 0.09, want_lse=True)
        used = tq.tq_paged_compact(pg, pool, t, n)
        assert used.item() == 5 and int(t.max()) == 4
        c = tq.tq_paged_attention(pg, q, pool, 0, n, t, 0.09, want_lse=True)
        assert torch.equal(b[0], c[0]) and torch.equal(b[1], c[1])
        out.append((*a, *b))
    for u, v in zip(*out):
        assert torch.equal(u, v)
    tq.tq_sync_check()


def test_calls_on_a_stream_that_is_not_current():
    """Outputs and workspaces that a call makes belong to the stream it runs on."""
    kp, vp, _, _ = quantizers(128, 3)
    pg = tq.TQPaged(kp, vp, 1, 2, 32)
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn(90, 2, 128, device=DEV, generator=g).half()
    keys, vals = tq.tq_encode_prod(kp, x), tq.tq_encode_mse(vp, x)
    t, n, q = ints([[4, 2, 0]]), ints([90]), torch.randn(1, 8, 128, device=DEV, generator=g).half()
    pool = pg.new_pool(6)
    tq.tq_paged_append(pg, pool, 0, keys, vals, ints([0]), t, cu=ints([0, 90]))
    want = tq.tq_paged_attention(pg, q, pool, 0, n, t, 0.09, want_lse=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = pg.new_pool(6)
    side.wait_stream(torch.cuda.current_stream())
    tq.tq_paged_append(pg, other, 0, keys, vals, ints([0]), t, cu=ints([0, 90]), stream=side)
    got = []
    for _ in range(4):
        got.append(tq.tq_paged_attention(pg, q, other, 0, n, t, 0.09, want_lse=True, stream=side))
        torch.empty(1 << 22, dtype=torch.uint8, device=DEV).fill_(255)  # what the current stream takes meanwhile
    t2 = t.clone()
    side.wait_stream(torch.cuda.current_stream())
    used = tq.tq_paged_compact(pg, other, t2, n, stream=side)
    after = tq.tq_paged_attention(pg, q, other, 0, n, t2, 0.09, want_lse=True, stream=side)
    side.synchronize()
    assert used.item() == 3 and sorted(t2[0].tolist()) == [0, 1, 2]
    for o, l in got + [after]:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


def test_fork():
    kp, vp, _, _ = quantizers(64, 3)
    for page, layers in ((32, 1), (96, 3)):
        pg, model = tq.TQPaged(kp, vp, layers, 2, page), Model(kp, vp, layers, 2, page)
        rng = np.random.default_rng(page)
        B, width, n_pages = 12, 4, 60
        pool = rng.integers(0, 1 << 32, (n_pages, model.page_words), dtype=np.uint64).astype(np.uint32)
        tables = rng.permutation(n_pages)[: B * width].reshape(B, width).astype(np.int32)
        free = [p for p in range(n_pages) if p not in tables]
        lens = np.array([5, page, page + 1, 4 * page, 4 * page + 7, 0, 2 * page + 31, 2 * page + 40] + [9] * 4, np.int32)
        tables[7, 2] = -1  # the last page of 7 is a hole (page 96)
        parents = [0, 1, 2, 6, 99, 7, 2]
        children = [8, 9, 10, 11, 3, 4, -1]
        fresh = [free[0], free[1], free[2], n_pages + 5, free[3], free[4], free[5]]
        t, n, p = ints(tables), ints(lens), i32(pool)
        tq.tq_paged_fork(pg, p, t, n, ints(parents), ints(children), ints(fresh))
        for par, ch, fr in zip(parents, children, fresh):
            if not (0 <= par < B and 0 <= ch < B):
                continue
            m = min(int(lens[par]), width * page)
            full, rest = divmod(m, page)
            row = np.full(width, -1, np.int32)
            row[:full] = tables[par, :full]
            src = tables[par, full] if rest else -1
            if rest and 0 <= src < n_pages and 0 <= fr < n_pages:
                row[full] = fr
                for seg in range(layers * 2):
                    at = seg * model.nb * model.words
                    used = -(-rest // 32) * model.words
                    pool[fr, at:at + used] = pool[src, at:at + used]
            tables[ch], lens[ch] = row, m
        assert np.array_equal(t.cpu().numpy(), tables)
        assert np.array_equal(n.cpu().numpy(), lens)
        assert np.array_equal(u32(p), pool)
        tq.tq_paged_fork(pg, p, t, n, ints([]), ints([]), ints([]))  # none
        assert np.array_equal(u32(p), pool)


def compact_model(pool, tables, lens, page):
    n_pages = len(pool)
    live = np.arange(tables.shape[1])[None] * page < np.clip(lens, 0, tables.shape[1] * page)[:, None]
    ok = live & (tables >= 0) & (tables < n_pages)
    used = np.zeros(n_pages, bool)
    used[tables[ok]] = True
    n = int(used.sum())
    src = [p for p in range(n, n_pages) if used[p]]
    dst = [p for p in range(n) if not used[p]]
    to = np.arange(n_pages)
    to[src] = dst
    pool[dst] = pool[src]
    return np.where(ok, to[np.where(ok, tables, 0)], -1).astype(np.int32), n


# the last two: more pages, and more table entries, than one block plans
@pytest.mark.parametrize("n_pages,B,width", [(1, 1, 1), (31, 3, 5), (64, 8, 9), (1000, 40, 11), (20000, 300, 30),
                                             (140000, 50, 40), (900, 1100, 30)])
def test_compact(n_pages, B, width):
    kp, vp, _, _ = quantizers(32, 2)
    page = 32
    pg, model = tq.TQPaged(kp, vp, 1, 1, page), Model(kp, vp, 1, 1, page)
    for trial in range(4):
        rng = np.random.default_rng(n_pages + trial)
        pool = rng.integers(0, 1 << 32, (n_pages, model.page_words), dtype=np.uint64).astype(np.uint32)
        # pages drawn with repeats (shared ones) and holes of both kinds
        tables = rng.integers(-2, n_pages + 2, (B, width)).astype(np.int32)
        lens = rng.integers(-5, (width + 1) * page, B).astype(np.int32)
        if trial == 1:
            lens[:] = 0
        if trial == 2:  # everything in place already
            tables[:] = np.minimum(np.arange(B * width).reshape(B, width), n_pages - 1)
            lens[:] = width * page
        t, p = ints(tables), i32(pool)
        want, n = compact_model(pool, tables, lens, page)
        out = torch.full_like(t, 77)
        used = tq.tq_paged_compact(pg, p, t, ints(lens), tables_out=out if trial % 2 else None)
        assert used.item() == n
        assert np.array_equal((out if trial % 2 else t).cpu().numpy(), want)
        assert np.array_equal(u32(p), pool)
    # no sequences at all
    used = tq.tq_paged_compact(pg, p, ints(np.zeros((0, 3))), ints([]))
    assert used.item() == 0 and np.array_equal(u32(p), pool)


def test_run_together():
    """Prompts and steps through norm and rotation, the encoders, append, fork, attention, an ended sequence and
    compaction: the paged attention agrees with the contiguous one over the same tokens, and does not change
    when pages move."""
    d, hkv, G, page, layers = 128, 2, 4, 32, 2
    kp, vp, _, _ = quantizers(d, 3)
    pg = tq.TQPaged(kp, vp, layers, hkv, page)
    rope = tq.TQRope(d, 10000.0)
    g = torch.Generator(device=DEV).manual_seed(1)
    wk = (1 + 0.1 * torch.randn(d, device=DEV, generator=g)).half()
    B, width = 4, 8
    pool = pg.new_pool(40)
    tables = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    tables[0, :5], tables[1, :3], tables[3, :4] = ints([30, 2, 39, 11, 7]), ints([1, 0, 33]), ints([5, 20, 21, 22])
    lens = [70, 33, 0, 100]
    toks = {b: ([], []) for b in range(B)}  # what a contiguous cache would hold

    def feed(counts, starts):
        n = sum(counts)
        x = torch.randn(n, (G + 2) * hkv, d, device=DEV, generator=g).half()
        pos = torch.cat([torch.arange(s, s + c) for s, c in zip(starts, counts)]).to(DEV)
        q, k = tq.tq_qk_norm_rope(rope, x[:, : G * hkv], x[:, G * hkv:(G + 1) * hkv], pos, wk, wk)
        v = x[:, (G + 1) * hkv:].contiguous()
        keys, vals = tq.tq_encode_prod(kp, k), tq.tq_encode_mse(vp, v)
        cu = ints(np.concatenate([[0], np.cumsum(counts)]))
        tq.tq_paged_append(pg, pool, 1, keys, vals, ints(starts), tables, cu=cu)
        at = 0
        for b, c in enumerate(counts):
            toks[b][0].extend(k[at:at + c])
            toks[b][1].extend(v[at:at + c])
            at += c
        return q

    def attend(q, lens):
        got, lse = tq.tq_paged_attention(pg, q, pool, 1, ints(lens), tables, 0.088, want_lse=True)
        for b, n in enumerate(lens):
            if n == 0:
                assert bool((got[b] == 0).all())
                continue
            cap = -(-n // 32) * 32
            K, V = (torch.stack(t).transpose(0, 1).contiguous() for t in toks[b])
            kc = tq.tq_encode_prod(kp, K, seg_len=n, seg_cap=cap)
            vc = tq.tq_encode_mse(vp, V, layout=tq.LAYOUT_BLOCK32, seg_len=n, seg_cap=cap)
            want = tq.tq_decode_attention(kp, vp, q[b].float().view(1, 1, -1, d), kc, vc, n, cap, 0.088)[0, 0]
            err = (got[b].float() - want).norm(dim=-1) / want.norm(dim=-1)
            # half a step of fp16 (relative to each element, so to the norm) and the 1e-3 of the contiguous one
            assert float(err.max()) <= 2.0 ** -11 + 1e-3
        return got, lse

    feed(lens, [0, 0, 0, 0])
    # sequence 2 begins as a copy of 0; 1 takes page 34 when it grows past a page
    n = ints(lens)
    tq.tq_paged_fork(pg, pool, tables, n, ints([0]), ints([2]), ints([38]))
    toks[2] = (list(toks[0][0]), list(toks[0][1]))
    lens = n.tolist()
    assert lens == [70, 33, 70, 100]
    assert tables[2].tolist() == [30, 2, 38, -1, -1, -1, -1, -1]
    q = feed([1, 1, 1, 1], lens)
    lens = [x + 1 for x in lens]
    attend(q, lens)
    # 3 ends, the others move together
    lens[3], toks[3] = 0, ([], [])
    before, blse = attend(q, lens)
    used = tq.tq_paged_compact(pg, pool, tables, ints(lens))
    assert used.item() == 3 + 2 + 1 and int(tables.max()) == 5
    after, alse = attend(q, lens)
    assert torch.equal(before, after) and torch.equal(blse, alse)
    # the freed pages serve again
    tables[3, :2] = ints([6, 7])
    q = feed([0, 0, 0, 50], [0, 0, 0, 0])
    lens[3] = 50
    attend(torch.randn(B, G * hkv, d, device=DEV, generator=g).half(), lens)
    tq.tq_sync_check()


def test_captured_step_follows_lengths_and_tables():
    """One graph of append and attention, replayed as sequences grow and change, on another stream; two graphs with
    workspaces of their own run at once."""
    kp, vp, kq, vq = quantizers(128, 3)
    pg, model = tq.TQPaged(kp, vp, 1, 1, 32), Model(kp, vp, 1, 1, 32)
    rng = np.random.default_rng(12)
    pool, tables = random_cache(rng, model, [128, 128], 4, 0)
    sides = []
    for i in range(2):
        p, t = i32(pool), ints(tables)
        lens = ints([0, 0])
        q = torch.from_numpy(rng.standard_normal((2, 4, 128))).to(DEV).float()
        ref, keys, vals = rows(rng, 2, 1, model)
        ws = torch.empty(tq.tq_paged_attention_workspace_size(pg, 2, 4), dtype=torch.uint8, device=DEV)
        out, lse = torch.empty_like(q), torch.empty(2, 4, device=DEV)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            tq.tq_paged_append(pg, p, 0, keys, vals, lens, t)
            lens += 1
            tq.tq_paged_attention(pg, q, p, 0, lens, t, 0.09, out=out, lse=lse, ws=ws)
        sides.append((g, p, t, lens, q, ref, out, lse, stream, ws))
    model_pools = [pool.copy(), pool.copy()]
    for n in (0, 40, 97):
        for g, p, t, lens, q, ref, out, lse, stream, ws in sides:
            lens.copy_(ints([n, 5]))
        torch.cuda.synchronize()
        for g, *_, stream, ws in sides:
            with torch.cuda.stream(stream):
                g.replay()
        torch.cuda.synchronize()
        for (g, p, t, lens, q, ref, out, lse, stream, ws), mp in zip(sides, model_pools):
            model.append(mp, 0, *ref, [0, 1, 2], [n, 5], tables)
            assert np.array_equal(u32(p), mp)
            want = model.attention(mp, 0, kq, vq, q.double().cpu().numpy(), [n + 1, 6], tables, 0.09)
            check_attention(out, lse, want, torch.float32)


def test_refusals():
    kp, vp, _, _ = quantizers(128, 3)
    vp64 = quantizers(64, 3)[1]
    with pytest.raises(tq.TQError):
        tq.TQPaged(kp, vp64, 1, 1, 32)
    with pytest.raises(tq.TQError):
        tq.TQPaged(kp, kp, 1, 1, 32)
    with pytest.raises(tq.TQError):
        tq.TQPaged(kp, vp, 1, 1, 40)
    pg = tq.TQPaged(kp, vp, 2, 2, 32)
    pool, tables, lens = pg.new_pool(3), ints([[0, 1]]), ints([10])
    q = torch.zeros(1, 4, 128, device=DEV)
    call = lambda **kw: tq.tq_paged_attention(**{**dict(pg=pg, q=q, pool=pool, layer=0, lens=lens, tables=tables,  # noqa: E731
                                                        scale=1.0), **kw})
    call()
    for bad in (dict(layer=2), dict(layer=-1), dict(q=q[:, :3]), dict(q=torch.zeros(1, 34, 128, device=DEV)),
                dict(ws=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(tq.TQError):
            call(**bad)
    for bad in (dict(q=q[..., :64]), dict(pool=pool[:, :-4]), dict(pool=pool.float()), dict(lens=lens.long()),
                dict(tables=tables.long()), dict(tables=ints([[0, 1], [0, 1]])), dict(lens=lens.cpu()),
                dict(out=torch.zeros(1, 4, 128, device=DEV).half()), dict(lse=torch.zeros(1, 3, device=DEV))):
        with pytest.raises(ValueError):
            call(**bad)
    none = tq.tq_paged_attention(pg, q[:0], pool, 0, lens[:0], tables[:0], 1.0)
    assert none.shape == (0, 4, 128)
    model = Model(kp, vp, 2, 2, 32)
    _, keys, vals = rows(np.random.default_rng(0), 1, 2, model)
    with pytest.raises(tq.TQError):
        tq.tq_paged_append(pg, pool, 2, keys, vals, lens, tables)
    with pytest.raises(ValueError):
        tq.tq_paged_append(pg, pool, 0, keys, vals, ints([1, 2]), ints([[0, 1], [0, 1]]))
    with pytest.raises(ValueError):
        tq.tq_paged_append(pg, pool, 0, keys[:3] + (keys[3].half(),), vals, lens, tables)
    with pytest.raises(ValueError):
        tq.tq_paged_append(pg, pool, 0, keys, (vals[0][:1], vals[1]), lens, tables)
    with pytest.raises(ValueError):
        tq.tq_paged_fork(pg, pool, tables, lens, ints([0]), ints([0, 1]), ints([2]))
    with pytest.raises(tq.TQError):
        tq.tq_paged_compact(pg, pool, tables, lens, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        tq.tq_paged_compact(pg, pool, tables, lens, tables_out=ints([[0, 1, 2]]))
    assert bool((pool == 0).all())
