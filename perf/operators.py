"""The paged-cache operators, measured: per-head norm + rotary positions, append to pages, attention over pages, and
page fork / compaction.  Each has its plain form in elementary torch operations; with `own` the same call is made
of the framework (vector_compression_b200)."""
import math
import random

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SM = "cuda"


# ----------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of one sequence deep in its context: latency
        dict(name="rope one token", op="rope", n=1, hq=32, hkv=8, d=128, rot=128, layout="half", dtype="bf16",
             norm=True, scaling="bands", base=500000.0, pos=131072, packed=False),
        # a long prompt before its keys are encoded: the heads of a fused projection, no norm
        dict(name="rope prompt", op="rope", n=16384, hq=32, hkv=8, d=128, rot=128, layout="half", dtype="f16",
             norm=False, scaling="none", base=500000.0, pos=131072, packed=True),
        # odd count, interleaved pairs over part of the head, fp32, norms
        dict(name="rope partial", op="rope", n=1777, hq=16, hkv=2, d=192, rot=64, layout="pairs", dtype="f32",
             norm=True, scaling="yarn", base=10000.0, pos=65536, packed=True),
        # one token of each of 64 sequences into the pages (a decode step's write)
        dict(name="append step", op="append", b=64, lo=1, hi=1, salt=1, hkv=8, d=128, m=128, bits=3, r16=False,
             page=64, ctx=2048, layers=1),
        # prompts of different lengths into the pages
        dict(name="append prompts", op="append", b=12, lo=1, hi=4096, salt=2, hkv=8, d=128, m=128, bits=3, r16=False,
             page=64, ctx=64, layers=2),
        # one short sequence: latency
        dict(name="attention short", op="attend", b=1, lo=129, hi=129, salt=0, hq=32, hkv=8, d=128, m=128, bits=3,
             r16=False, page=32, layers=1, dtype="bf16"),
        # a ragged batch, eight query heads per KV head
        dict(name="attention ragged", op="attend", b=48, lo=0, hi=6000, salt=3, hq=16, hkv=2, d=128, m=128, bits=3,
             r16=False, page=64, layers=2, dtype="bf16"),
        # long contexts
        dict(name="attention long", op="attend", b=8, lo=30000, hi=32768, salt=4, hq=32, hkv=8, d=128, m=128, bits=3,
             r16=False, page=64, layers=1, dtype="f16"),
        # four samples of one prompt begin
        dict(name="fork few", op="fork", b=8, n=3, page=64, hkv=8, layers=4, ctx=1000, salt=5),
        # wide sampling over a 32-layer cache
        dict(name="fork many", op="fork", b=288, n=256, page=32, hkv=8, layers=32, ctx=300, salt=6),
        # a small pool after two sequences ended
        dict(name="compact small", op="compact", b=8, page=32, hkv=2, layers=1, ctx=400, salt=7, spare=3),
        # a large pool, half of it given up
        dict(name="compact large", op="compact", b=128, page=64, hkv=8, layers=2, ctx=1800, salt=8, spare=50),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "append", "attend", "attend", "attend", "fork", "compact"])
    if op == "rope":
        d = rng.choice([64, 80, 96, 128, 192, 256])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 7, 8])
        dtype = rng.choice(["f32", "f16", "bf16"])
        top = 16384 * 40 * 128 // ((hq + hkv) * d * (2 if dtype == "f32" else 1))
        return dict(op=op, n=_log(rng, 1, top), hq=hq, hkv=hkv, d=d,
                    rot=rng.choice([d, d, d // 2]), layout=rng.choice(["half", "pairs"]), dtype=dtype,
                    norm=rng.random() < 0.6, scaling=rng.choice(["none", "linear", "bands", "yarn"]),
                    base=rng.choice([10000.0, 500000.0, 1000000.0]), pos=_log(rng, 1000, 1000000),
                    packed=rng.random() < 0.6)
    if op == "append":
        d = rng.choice([64, 128, 128, 192])
        b = _log(rng, 1, 128)
        step = rng.random() < 0.4
        hi = 1 if step else _log(rng, 2, max(2, 16000 // b))
        return dict(op=op, b=b, lo=1, hi=hi, salt=rng.randrange(1 << 20), hkv=rng.choice([1, 2, 8]), d=d,
                    m=_pad(d) // rng.choice([1, 1, 2]), bits=rng.choice([2, 3, 3, 4]), r16=rng.random() < 0.3,
                    page=rng.choice([32, 64, 96, 256]), ctx=_log(rng, 1, 2000), layers=rng.choice([1, 2]))
    if op == "attend":
        d = rng.choice([64, 128, 128, 192])
        hkv = rng.choice([1, 2, 4, 8])
        b = _log(rng, 1, 128)
        top = max(40, 1500000 * 128 // (_pad(d) * b * hkv))
        hi = _log(rng, 1, min(top, 60000))
        return dict(op=op, b=b, lo=rng.choice([0, hi // 2, hi]), hi=hi, salt=rng.randrange(1 << 20),
                    hq=hkv * rng.choice([1, 2, 4, 5, 8]), hkv=hkv, d=d, m=_pad(d), bits=rng.choice([2, 3, 3, 4]),
                    r16=rng.random() < 0.3, page=rng.choice([32, 64, 96, 256]), layers=rng.choice([1, 2]),
                    dtype=rng.choice(["f16", "bf16"]))
    layers, hkv, page = rng.choice([1, 4, 16]), rng.choice([2, 8]), rng.choice([32, 64, 128])
    b = _log(rng, 4, 200)
    ctx = _log(rng, 40, max(41, min(4000, 4 * 32 * 16 * 8 * 200 * 700 // (32 * 8) // (b * layers * hkv))))
    if op == "fork":
        return dict(op=op, b=b, n=rng.randint(1, b - 1), page=page, hkv=hkv, layers=layers, ctx=ctx,
                    salt=rng.randrange(1 << 20))
    return dict(op=op, b=b, page=page, hkv=hkv, layers=layers, ctx=ctx, salt=rng.randrange(1 << 20),
                spare=rng.randint(0, 60))


def _pad(d):
    p = 32
    while p < d:
        p *= 2
    return p


def _lens(c):
    """Tokens of each sequence: a property of the case, not of the seed."""
    r = random.Random(c["salt"])
    lens = [r.randint(c["lo"], c["hi"]) for _ in range(c["b"])]
    if c["op"] == "attend" and c["b"] > 4 and c["lo"] == 0:
        lens[1], lens[2] = 0, 1
    return lens


# ----------------------------------------------------------------------------------------------- the quantizer

def _codebook(d, k):
    """Lloyd-Max levels and borders of (1 - x^2)^((d - 3) / 2) on [-1, 1] in 64 bits."""
    x = np.linspace(-1, 1, 400001)
    x = (x[1:] + x[:-1]) / 2
    w = np.exp((d - 3) / 2 * np.log1p(-x * x))
    c0 = np.concatenate([[0], np.cumsum(w)])
    c1 = np.concatenate([[0], np.cumsum(w * x)])
    e = np.linspace(-1, 1, 400001)
    n = 1 << k
    c = np.sqrt(1 / d) * np.linspace(-1.6, 1.6, n) if n > 2 else np.sqrt(1 / d) * np.array([-0.8, 0.8])
    for _ in range(2000):
        b = np.concatenate([[-1], (c[1:] + c[:-1]) / 2, [1]])
        new = np.diff(np.interp(b, e, c1)) / np.diff(np.interp(b, e, c0))
        new = (new - new[::-1]) / 2
        done = np.max(np.abs(new - c)) < 1e-13
        c = new
        if done:
            break
    return c, (c[1:] + c[:-1]) / 2


_tables = {}


def _quantizer(c):
    """What the two quantizers of a cache are made from: signs of both rotations, the sketch, levels, sizes."""
    key = (c["d"], c["m"], c["bits"])
    if key not in _tables:
        rng = np.random.default_rng(c["d"] * 1000 + c["m"])
        dp, k = _pad(c["d"]), c["bits"]
        h = np.ones((1, 1))
        while len(h) < dp:
            h = np.block([[h, h], [h, -h]])
        _tables[key] = dict(
            dp=dp, kk=k - 1, kv=k, sw=c["m"] // 32, h=h,
            dk=rng.choice([-1, 1], dp).astype(np.int8), dv=rng.choice([-1, 1], dp).astype(np.int8),
            s=rng.standard_normal((c["m"], dp)).astype(np.float16).astype(np.float32),
            ck=_codebook(dp, k - 1), cv=_codebook(dp, k), kappa=math.sqrt(math.pi / 2) / c["m"])
    return _tables[key]


def _record(c):
    """Where the parts of one 32-token block record begin, in 32-bit words."""
    z = _quantizer(c)
    nk = z["kk"] * z["dp"] // 32 + z["sw"]
    gr = 4 if nk % 4 == 0 else 2 if nk % 2 == 0 else 1
    kn = 32 * nk
    v = kn + 32 + (16 if c["r16"] else 32)
    vn = v + z["kv"] * z["dp"]
    return dict(nk=nk, gr=gr, kn=kn, kr=kn + 32, v=v, vn=vn, words=vn + 32)


def _i32(x):
    """The low 32 bits of int64 values, as int32."""
    return (((x + (1 << 31)) & 0xFFFFFFFF) - (1 << 31)).to(torch.int32)


def _encode(c, rows, side, g):
    """Level numbers, signs, norms and residual norms of fp32 rows [..., d] (keys with a sketch, values without)."""
    z = _quantizer(c)
    x = torch.nn.functional.pad(rows, (0, z["dp"] - c["d"]))
    h = torch.tensor(z["h"], dtype=torch.float32, device=SM)
    n = x.square().sum(-1).sqrt()
    y = (x * torch.tensor(z["dk" if side == "k" else "dv"], device=SM).float()) @ h / math.sqrt(z["dp"])
    y = y / n.clamp(min=1e-30)[..., None]
    lev, brd = z["ck" if side == "k" else "cv"]
    idx = torch.bucketize(y, torch.tensor(brd, dtype=torch.float32, device=SM))
    if side == "v":
        return idx.to(torch.uint8), n
    r = y - torch.tensor(lev, dtype=torch.float32, device=SM)[idx]
    sig = (r @ torch.tensor(z["s"], device=SM).T) >= 0
    rho = r.square().sum(-1).sqrt()
    return idx.to(torch.uint8), sig, n, rho.half() if c["r16"] else rho


def _planes(bits):
    """0/1 values [..., 32 n] to words [..., n]: bit i of word w is value 32 w + i."""
    b = bits.reshape(*bits.shape[:-1], -1, 32).to(torch.int64) << torch.arange(32, device=SM)
    return _i32(b.sum(-1))


def _code_words(idx, k):
    return torch.cat([_planes((idx >> p) & 1) for p in range(k)], -1)


def _value_fields(idx, t, kv):
    """The bits that level numbers idx [..., dp] of a token at place t [...] of its block put into the block's
    kv value words of each coordinate, and the mask of them: two int64 [..., kv, dp]."""
    idx, t = idx.to(torch.int64), t[..., None]
    s, i = t & 3, t >> 2
    zero = torch.zeros_like(idx)
    if kv == 1:
        val, msk = [idx << t], [(zero + 1) << t]
    elif kv in (2, 3):
        at = 4 * i + 2 * (s & 1)
        val = [torch.where(s >> 1 == h, (idx & 3) << at, zero) for h in (0, 1)]
        msk = [torch.where(s >> 1 == h, (zero + 3) << at, zero) for h in (0, 1)]
        if kv == 3:
            at = (t + 2) & 31
            val.append((idx >> 2) << at)
            msk.append((zero + 1) << at)
    else:
        nib = torch.where(idx >= 8, idx - 8, 15 - idx)  # bit 3: below zero; bits 0..2: which magnitude
        val = [torch.where(s == h, nib << (4 * i), zero) for h in range(4)]
        msk = [torch.where(s == h, (zero + 15) << (4 * i), zero) for h in range(4)]
    return torch.stack(val, -2), torch.stack(msk, -2)


def _rows(c, n, g):
    """Keys or values of n tokens: normal, a few channels of a head much larger, 16-bit as a model gives them."""
    x = torch.randn(n, c["hkv"], c["d"], device=SM, generator=g)
    x[..., torch.randint(0, c["d"], (4,), device=SM, generator=g)] *= 8.0
    return x.half().float()


def _tables_for(lens, page, width, n_pages, g):
    """A page table: every sequence's pages in a random order, -1 behind them."""
    need = torch.tensor([-(-x // page) for x in lens], device=SM)
    valid = torch.arange(width, device=SM)[None] < need[:, None]
    ids = torch.randperm(n_pages, device=SM, generator=g)[: int(need.sum())].to(torch.int32)
    t = torch.full((len(lens), width), -1, dtype=torch.int32, device=SM)
    t[valid] = ids
    return t


# ----------------------------------------------------------------------------------------------- rotary positions

def _frequencies(c):
    """Angle per position of each pair (64 bits) and the factor on the rotated part."""
    r, f = c["rot"], c["base"] ** (-np.arange(0, c["rot"], 2) / c["rot"])
    if c["scaling"] == "linear":
        return f / 4.0, 1.0
    if c["scaling"] == "bands":  # long wavelengths slower by 8, short ones kept, a ramp between
        turns = 8192 * f / (2 * math.pi)
        s = np.clip((turns - 1.0) / (4.0 - 1.0), 0, 1)
        return f * (s + (1 - s) / 8.0), 1.0
    if c["scaling"] == "yarn":
        at = lambda beta: r * math.log(4096 / (beta * 2 * math.pi)) / (2 * math.log(c["base"]))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), r - 1)
        ramp = np.clip((np.arange(r // 2) - lo) / max(hi - lo, 1e-3), 0, 1)
        return f * (1 - ramp) + f / 16.0 * ramp, 0.1 * math.log(16.0) + 1.0
    return f, 1.0


def _prepare_rope(c, g):
    n, d, dt = c["n"], c["d"], DT[c["dtype"]]
    if c["packed"]:  # q, k and v of a token side by side, as one projection leaves them
        qkv = torch.randn(n, c["hq"] + 2 * c["hkv"], d, device=SM, generator=g).to(dt)
        q, k = qkv[:, : c["hq"]], qkv[:, c["hq"]: c["hq"] + c["hkv"]]
    else:
        q = torch.randn(n, c["hq"], d, device=SM, generator=g).to(dt)
        k = torch.randn(n, c["hkv"], d, device=SM, generator=g).to(dt)
    start = torch.randint(0, c["pos"], (1,), device=SM, generator=g)
    st = dict(c=c, q=q, k=k, pos=start + torch.arange(n, device=SM), wq=None, wk=None)
    if c["norm"]:
        st["wq"] = (1 + 0.2 * torch.randn(d, device=SM, generator=g)).to(dt)
        st["wk"] = (1 + 0.2 * torch.randn(d, device=SM, generator=g)).to(dt)
    f, st["mscale"] = _frequencies(c)
    st["f"] = torch.tensor(f, device=SM)
    if own:
        st["rope"] = _rope(c)
    return st


def _rope(c, _handles={}):
    """The rotation's handle, kept as _paged's are."""
    key = tuple(c[k] for k in ("rot", "base", "layout", "scaling"))
    if key not in _handles:
        import vector_compression_b200 as tq

        kind, more = dict(none=(tq.ROPE_PLAIN, {}), linear=(tq.ROPE_LINEAR, dict(factor=4.0)),
                          bands=(tq.ROPE_BANDS, dict(factor=8.0, orig_len=8192, low=1.0, high=4.0)),
                          yarn=(tq.ROPE_YARN, dict(factor=16.0, orig_len=4096, low=1.0, high=32.0)))[c["scaling"]]
        _handles[key] = tq.TQRope(c["rot"], c["base"], interleaved=c["layout"] == "pairs", scaling=kind, **more)
    return _handles[key]


def _rope_plain(x, w, s):
    c = s["c"]
    x, r = x.float(), s["c"]["rot"]
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    a = s["pos"].double()[:, None] * s["f"][None]
    co, si = (a.cos() * s["mscale"]).float()[:, None], (a.sin() * s["mscale"]).float()[:, None]
    if c["layout"] == "half":
        u, v = x[..., : r // 2], x[..., r // 2: r]
        y = torch.cat([u * co - v * si, v * co + u * si], -1)
    else:
        u, v = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([u * co - v * si, v * co + u * si], -1).flatten(-2)
    return torch.cat([y, x[..., r:]], -1).to(DT[c["dtype"]])


def _run_rope(s):
    if own:
        import vector_compression_b200 as tq

        return tq.tq_qk_norm_rope(s["rope"], s["q"], s["k"], s["pos"], s["wq"], s["wk"], eps=1e-6)
    return _rope_plain(s["q"], s["wq"], s), _rope_plain(s["k"], s["wk"], s)


def _exact_rope(s):
    c, out = s["c"], []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x, r = x.double(), c["rot"]
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / c["d"] + 1e-6).sqrt() * w.double()
        turn = torch.polar(torch.full((), s["mscale"], dtype=torch.float64, device=SM), s["pos"].double()[:, None] * s["f"])
        z = torch.complex(x[..., : r // 2], x[..., r // 2: r]) if c["layout"] == "half" else \
            torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous())
        z = z * turn[:, None]
        y = x.clone()
        if c["layout"] == "half":
            y[..., : r // 2], y[..., r // 2: r] = z.real, z.imag
        else:
            y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
        out.append(y)
    return tuple(out)


# ----------------------------------------------------------------------------------------------- append

def _paged(c, _handles={}):
    """The cache's handle.  It says nothing of the inputs: a program makes its quantizers (whose codebooks take
    milliseconds) when it starts, and so this keeps one of each kind, as _tables does for the plain form."""
    key = tuple(c[k] for k in ("d", "m", "bits", "r16", "layers", "hkv", "page"))
    if key not in _handles:
        import vector_compression_b200 as tq

        z = _quantizer(c)
        mode = tq.MODE_PROD | (tq.STORE_RNORM_F16 if c["r16"] else 0)
        kp = tq.TQParams(c["d"], c["bits"], mode, tq.ROT_HADAMARD, m=c["m"], signs=z["dk"], S=z["s"])
        vp = tq.TQParams(c["d"], c["bits"], tq.MODE_MSE, tq.ROT_HADAMARD, signs=z["dv"])
        _handles[key] = tq.TQPaged(kp, vp, layers=c["layers"], hkv=c["hkv"], page=c["page"])
    return _handles[key]


def _prepare_append(c, g):
    z, rec, lens, page = _quantizer(c), _record(c), _lens(c), c["page"]
    b, n = c["b"], sum(lens)
    start = torch.randint(0, c["ctx"] + 1, (b,), device=SM, generator=g).to(torch.int32)
    width = -(-(c["ctx"] + max(lens)) // page)
    n_pages = b * width + 3
    pool = torch.randint(-2 ** 31, 2 ** 31, (n_pages, c["layers"] * c["hkv"] * page // 32 * rec["words"]),
                         device=SM, generator=g, dtype=torch.int32)
    k = _encode(c, _rows(c, n, g), "k", g)
    v = _encode(c, _rows(c, n, g), "v", g)
    st = dict(c=c, pool=pool, layer=c["layers"] - 1, start=start, n_pages=n_pages,
              tables=_tables_for([width * page] * b, page, width, n_pages, g),
              cu=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=SM),
              kcodes=_code_words(k[0], z["kk"]).flatten(0, 1), ksigns=_planes(k[1]).flatten(0, 1),
              kn=k[2].flatten(), kr=k[3].flatten(), vcodes=_code_words(v[0], z["kv"]).flatten(0, 1), vn=v[1].flatten())
    if own:
        st["pg"] = _paged(c)
    return st


def _run_append(s):
    c = s["c"]
    if own:
        import vector_compression_b200 as tq

        tq.tq_paged_append(s["pg"], s["pool"], s["layer"], (s["kcodes"], s["ksigns"], s["kn"], s["kr"]),
                           (s["vcodes"], s["vn"]), s["start"], s["tables"], cu=s["cu"] if c["hi"] > 1 else None)
        return s["pool"]
    z, rec, hkv, page = _quantizer(c), _record(c), c["hkv"], c["page"]
    n = s["kn"].numel() // hkv
    tok = torch.arange(n, device=SM)
    b = torch.bucketize(tok, s["cu"][1:].long(), right=True)
    p = s["start"].long()[b] + tok - s["cu"].long()[b]
    t = p % 32
    pg = s["tables"][b, p // page].long()
    blk = (((pg * c["layers"] + s["layer"])[:, None] * hkv + torch.arange(hkv, device=SM)) * (page // 32)
           + ((p % page) // 32)[:, None]) * rec["words"]  # [n, hkv]: the record's first word
    flat = s["pool"].view(-1)
    w = torch.arange(rec["nk"], device=SM)
    at = blk[..., None] + w // rec["gr"] * (32 * rec["gr"]) + t[:, None, None] * rec["gr"] + w % rec["gr"]
    flat[at] = torch.cat([s["kcodes"], s["ksigns"]], -1).view(n, hkv, -1)
    flat[blk + rec["kn"] + t[:, None]] = s["kn"].view(torch.int32).view(n, hkv)
    flat[blk + rec["vn"] + t[:, None]] = s["vn"].view(torch.int32).view(n, hkv)
    if c["r16"]:
        s["pool"].view(torch.float16).view(-1)[2 * (blk + rec["kr"]) + t[:, None]] = s["kr"].view(n, hkv)
    else:
        flat[blk + rec["kr"] + t[:, None]] = s["kr"].view(torch.int32).view(n, hkv)
    bits = (s["vcodes"].view(n, hkv, z["kv"], -1, 1) >> torch.arange(32, device=SM, dtype=torch.int32)) & 1
    idx = (bits.flatten(-2) << torch.arange(z["kv"], device=SM, dtype=torch.int32)[:, None]).sum(-2)
    val, msk = _value_fields(idx, t[:, None], z["kv"])
    at = (blk[..., None] + rec["v"] + torch.arange(z["kv"] * z["dp"], device=SM)).flatten()
    # a token owns its fields of a word: taking out what they held and adding the new leaves the others alone
    flat.index_add_(0, at, _i32(val).flatten() - (flat[at] & _i32(msk).flatten()))
    return s["pool"]


# ----------------------------------------------------------------------------------------------- attention

def _prepare_attend(c, g, raw=False):
    z, rec, lens, page, hkv = _quantizer(c), _record(c), _lens(c), c["page"], c["hkv"]
    width = max(1, -(-max(lens) // page)) + 1
    n_pages = sum(-(-x // page) for x in lens) + 5
    tables = _tables_for(lens, page, width, n_pages, g)
    words = rec["words"]
    pool = torch.randint(-2 ** 31, 2 ** 31, (n_pages, c["layers"], hkv, page // 32, words), device=SM, generator=g,
                         dtype=torch.int32)
    lens_t = torch.tensor(lens, dtype=torch.int32, device=SM)
    layer = c["layers"] - 1
    # pages are filled in the order of the sequences; slots behind a sequence's end keep what they held
    order = torch.cat([tables[i, : -(-x // page)] for i, x in enumerate(lens)]).long()
    full = order.numel() * page
    k = _encode(c, _rows(c, full, g), "k", g)
    v = _encode(c, _rows(c, full, g), "v", g)
    st = dict(c=c, lens=lens_t, tables=tables, layer=layer, scale=1 / math.sqrt(c["d"]),
              q=torch.randn(c["b"], c["hq"], c["d"], device=SM, generator=g).to(DT[c["dtype"]]))
    if raw:
        return st, k, v, order
    off = torch.cat([torch.arange(-(-x // page) * page, device=SM) < x for x in lens])  # valid slots
    kw = torch.cat([_code_words(k[0], z["kk"]), _planes(k[1])], -1)  # [tok, hkv, nk]
    val, msk = _value_fields(v[0].transpose(0, 1).reshape(hkv, full // 32, 32, z["dp"]),
                             torch.arange(32, device=SM), z["kv"])
    vwords = _i32(val.sum(-3))  # [hkv, blocks, kv, dp]
    del val, msk
    new = torch.empty(full // 32, hkv, words, dtype=torch.int32, device=SM)
    new[..., : rec["kn"]] = kw.reshape(-1, 32, hkv, rec["nk"] // rec["gr"], rec["gr"]).permute(0, 2, 3, 1, 4).flatten(2)
    by = lambda x: x.reshape(-1, 32, hkv).transpose(1, 2).contiguous()  # noqa: E731
    off32 = off.view(-1, 1, 32)
    nan = lambda x: by(x).masked_fill(~off32, float("nan"))  # noqa: E731  stale slots hold anything
    new[..., rec["kn"]: rec["kr"]] = nan(k[2]).view(torch.int32)
    new[..., rec["kr"]: rec["v"]] = nan(k[3]).view(torch.int32)
    new[..., rec["v"]: rec["vn"]] = vwords.transpose(0, 1).flatten(2)
    new[..., rec["vn"]:] = nan(v[1]).view(torch.int32)
    pool[order, layer] = new.view(-1, page // 32, hkv, words).transpose(1, 2)
    st["pool"] = pool.view(n_pages, -1)
    if own:
        st["pg"] = _paged(c)
    return st


def _run_attend(s):
    c = s["c"]
    if own:
        import vector_compression_b200 as tq

        return tq.tq_paged_attention(s["pg"], s["q"], s["pool"], s["layer"], s["lens"], s["tables"], s["scale"],
                                     want_lse=True)
    z, rec, hkv, page, b = _quantizer(c), _record(c), c["hkv"], c["page"], c["b"]
    nb, dp, width = page // 32, z["dp"], s["tables"].shape[1]
    pool = s["pool"].view(-1, c["layers"], hkv, nb, rec["words"])
    r = pool[s["tables"].clamp(min=0).long(), s["layer"]]  # [b, width, hkv, nb, words]
    r = r.transpose(1, 2).reshape(b, hkv, width * nb, rec["words"])
    kw = r[..., : rec["kn"]].reshape(b, hkv, -1, rec["nk"] // rec["gr"], 32, rec["gr"]).transpose(3, 4)
    kw = kw.reshape(b, hkv, -1, rec["nk"])  # [b, hkv, tokens, words]
    kcw = z["kk"] * dp // 32
    bit = torch.arange(32, device=SM, dtype=torch.int32)
    codes = ((kw[..., :kcw, None] >> bit) & 1).reshape(b, hkv, -1, z["kk"], dp)
    idx = codes[..., 0, :]
    idx = idx + 2 * codes[..., 1, :] if z["kk"] > 1 else idx
    idx = idx + 4 * codes[..., 2, :] if z["kk"] > 2 else idx
    keys = torch.tensor(z["ck"][0], dtype=torch.float32, device=SM)[idx]
    sig = (2 * ((kw[..., kcw:, None] >> bit) & 1) - 1).flatten(-2).float()
    kn = r[..., rec["kn"]: rec["kr"]].contiguous().view(torch.float32).reshape(b, hkv, 1, -1)
    kr = r[..., rec["kr"]: rec["v"]].contiguous()
    kr = (kr.view(torch.float16) if c["r16"] else kr.view(torch.float32)).float().reshape(b, hkv, 1, -1)
    h = torch.tensor(z["h"], dtype=torch.float32, device=SM) / math.sqrt(dp)
    q = torch.nn.functional.pad(s["q"].float(), (0, dp - c["d"])) * torch.tensor(z["dk"], device=SM).float() @ h
    u = q @ torch.tensor(z["s"], device=SM).T
    q, u = q.reshape(b, hkv, -1, dp), u.reshape(b, hkv, -1, c["m"])
    sc = kn * (q @ keys.transpose(-1, -2) + z["kappa"] * kr * (u @ sig.transpose(-1, -2))) * s["scale"]
    del keys, sig, idx, codes
    there = (torch.arange(width * page, device=SM)[None] < s["lens"][:, None]) & \
        (s["tables"] >= 0).repeat_interleave(page, 1)
    there = there[:, None, None]
    sc = torch.where(there, sc, -math.inf)
    top = sc.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (sc - top).exp()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1).reshape(b, -1)
    vw = r[..., rec["v"]: rec["vn"]].reshape(b, hkv, -1, 1, z["kv"], dp)
    t = bit.view(32, 1)
    if z["kv"] == 4:
        nib = (vw.expand(-1, -1, -1, 32, -1, -1).gather(-2, (t & 3).long().view(1, 1, 1, 32, 1, 1).expand(
            b, hkv, vw.shape[2], 32, 1, dp)).squeeze(-2) >> (4 * (t >> 2))) & 15
        idx = torch.where(nib >= 8, 15 - nib, nib + 8)
    elif z["kv"] == 1:
        idx = (vw[..., 0, :] >> t) & 1
    else:
        idx = (torch.where((t & 2) > 0, vw[..., 1, :], vw[..., 0, :]) >> (4 * (t >> 2) + 2 * (t & 1))) & 3
        idx = idx + 4 * ((vw[..., 2, :] >> ((t + 2) & 31)) & 1) if z["kv"] == 3 else idx
    vals = torch.tensor(z["cv"][0], dtype=torch.float32, device=SM)[idx].reshape(b, hkv, -1, dp)
    vn = r[..., rec["vn"]:].contiguous().view(torch.float32).reshape(b, hkv, 1, -1)
    o = torch.where(there, p * vn, 0.0) @ vals / total.clamp(min=1e-30)
    o = (o @ h * torch.tensor(z["dv"], device=SM).float())[..., : c["d"]]
    return o.reshape(b, c["hq"], c["d"]).to(DT[c["dtype"]]), lse


def _exact_attend(c, g):
    s, k, v, order = _prepare_attend(c, g, raw=True)
    z, lens, page, grp = _quantizer(c), _lens(c), c["page"], c["hq"] // c["hkv"]
    f8 = lambda x: torch.tensor(x, dtype=torch.float64, device=SM)  # noqa: E731
    hk, hv = f8(z["h"] * z["dk"]) / math.sqrt(z["dp"]), f8(z["h"] * z["dv"]) / math.sqrt(z["dp"])
    out = torch.zeros(c["b"], c["hq"], c["d"], dtype=torch.float64, device=SM)
    lse = torch.full((c["b"], c["hq"]), -math.inf, dtype=torch.float64, device=SM)
    at = 0
    for i, x in enumerate(lens):
        if x:
            a = slice(at, at + x)
            q = s["q"][i].double() @ hk[:, : c["d"]].T
            for j in range(c["hkv"]):
                qj = q[j * grp: (j + 1) * grp]
                key = f8(z["ck"][0])[k[0][a, j].long()]
                est = qj @ key.T + z["kappa"] * k[3][a, j].double() * ((qj @ f8(z["s"]).T) @ (2.0 * k[1][a, j].double() - 1).T)
                w = est * k[2][a, j].double() * s["scale"]
                lse[i, j * grp: (j + 1) * grp] = torch.logsumexp(w, -1)
                val = f8(z["cv"][0])[v[0][a, j].long()] * v[1][a, j].double()[:, None]
                out[i, j * grp: (j + 1) * grp] = torch.softmax(w, -1) @ val @ hv[:, : c["d"]]
        at += -(-x // page) * page
    return out, lse


# ----------------------------------------------------------------------------------------------- pages

_PAGES = dict(d=128, m=128, bits=3, r16=False)


def _page_lens(c):
    r = random.Random(c["salt"])
    return [r.randint(1, c["ctx"]) for _ in range(c["b"])]


def _prepare_pages(c, g):
    c = dict(c, **_PAGES)
    rec, page, lens = _record(c), c["page"], _page_lens(c)
    fork = c["op"] == "fork"
    width = -(-c["ctx"] // page)
    words = c["layers"] * c["hkv"] * page // 32 * rec["words"]
    need = sum(-(-x // page) for x in lens)
    n_pages = need + (c["n"] + 2 if fork else need * c["spare"] // 100 + 4)
    tables = _tables_for(lens, page, width, n_pages, g)
    pool = torch.randint(-2 ** 31, 2 ** 31, (n_pages, words), device=SM, generator=g, dtype=torch.int32)
    st = dict(c=c, pool=pool, tables=tables, lens=torch.tensor(lens, dtype=torch.int32, device=SM))
    if fork:
        # the first sequences stay, the last n rows are taken over by samples of them
        keep = c["b"] - c["n"]
        st["parents"] = torch.randint(0, keep, (c["n"],), device=SM, generator=g).to(torch.int32)
        st["children"] = (keep + torch.randperm(c["n"], device=SM, generator=g)).to(torch.int32)
        used = torch.zeros(n_pages, dtype=torch.bool, device=SM)
        used[tables[tables >= 0].long()] = True
        st["fresh"] = torch.nonzero(~used).flatten()[: c["n"]].to(torch.int32)
    else:
        # a third of the sequences ended; two rows begin with the pages of another (a shared prompt)
        st["lens"][1::3] = 0
        if page < lens[0] and page < lens[3]:
            tables[3, 0] = tables[0, 0]
        st["tables_out"] = torch.empty_like(tables)
        st["n_used"] = torch.zeros(1, dtype=torch.int32, device=SM)
    if own:
        st["pg"] = _paged(c)
    return st


def _run_fork(s):
    c = s["c"]
    if own:
        import vector_compression_b200 as tq

        tq.tq_paged_fork(s["pg"], s["pool"], s["tables"], s["lens"], s["parents"], s["children"], s["fresh"])
        return s["pool"], s["tables"], s["lens"]
    page, blk = c["page"], _record(c)["words"]
    par, ch = s["parents"].long(), s["children"].long()
    n = s["lens"][par]
    rows = s["tables"][par]
    i = torch.arange(rows.shape[1], device=SM)[None]
    rows = torch.where(i < ((n + page - 1) // page)[:, None], rows, -1)
    tail = (n % page != 0)
    last = (n // page).long()[:, None].clamp(max=rows.shape[1] - 1)
    src = rows.gather(1, last).squeeze(1)
    fresh = torch.where(tail, s["fresh"], src)
    # blocks of the tail page that hold tokens: of every layer and head its first ones
    used = ((n % page + 31) // 32)[:, None]
    v = s["pool"].view(-1, c["layers"] * c["hkv"], page // 32, blk)
    which = (torch.arange(page // 32, device=SM)[None] < used) & tail[:, None]
    a, b = torch.nonzero(which, as_tuple=True)
    v[fresh[a].long(), :, b] = v[src[a].long(), :, b]
    rows = torch.where((i == last) & tail[:, None], s["fresh"][:, None], rows)
    s["tables"][ch] = rows
    s["lens"][ch] = n
    return s["pool"], s["tables"], s["lens"]


def _run_compact(s):
    c = s["c"]
    if own:
        import vector_compression_b200 as tq

        tq.tq_paged_compact(s["pg"], s["pool"], s["tables"], s["lens"], tables_out=s["tables_out"], n_used=s["n_used"])
        return s["pool"], s["tables_out"], s["n_used"]
    t, n_pages = s["tables"], s["pool"].shape[0]
    live = torch.arange(t.shape[1], device=SM)[None] < ((s["lens"] + c["page"] - 1) // c["page"])[:, None]
    used = torch.zeros(n_pages, dtype=torch.bool, device=SM)
    used[t[live].long()] = True
    n_used = used.sum()
    ids = torch.arange(n_pages, device=SM)
    src = torch.nonzero(used & (ids >= n_used)).flatten()
    dst = torch.nonzero(~used & (ids < n_used)).flatten()
    s["pool"][dst] = s["pool"][src]
    to = ids.to(torch.int32)
    to[src] = dst.to(torch.int32)
    out = torch.where(live, to[t.clamp(min=0).long()], -1)
    return s["pool"], out, n_used.to(torch.int32).view(1)


# ----------------------------------------------------------------------------------------------- the module's functions

def prepare(case, seed):
    g = torch.Generator(device=SM)
    g.manual_seed(seed)
    op = case["op"]
    return (_prepare_rope if op == "rope" else _prepare_append if op == "append" else
            _prepare_attend if op == "attend" else _prepare_pages)(case, g)


def run(state):
    op = state["c"]["op"]
    return dict(rope=_run_rope, append=_run_append, attend=_run_attend, fork=_run_fork, compact=_run_compact)[op](state)


def exact(case, seed):
    g = torch.Generator(device=SM)
    g.manual_seed(seed)
    if case["op"] == "rope":
        return _exact_rope(_prepare_rope(case, g))
    if case["op"] == "attend":
        return _exact_attend(case, g)
    return None


def work(case):
    c, op = case, case["op"]
    if op == "rope":
        size = 4 if c["dtype"] == "f32" else 2
        rows = c["n"] * (c["hq"] + c["hkv"])
        return dict(bytes=2 * rows * c["d"] * size + 8 * c["n"],
                    flops=rows * (3 * c["rot"] + (4 * c["d"] if c["norm"] else 0)))
    if op == "append":
        z, rec, n = _quantizer(c), _record(c), sum(_lens(c))
        row = 4 * (rec["nk"] + z["kv"] * z["dp"] // 32 + 2) + (2 if c["r16"] else 4)
        # a block's value words hold 32 tokens: each block that gains tokens is written whole, and read where it had some
        blocks = sum(-(-x // 32) for x in _lens(c)) * c["hkv"]
        return dict(bytes=2 * n * c["hkv"] * row + blocks * 4 * z["kv"] * z["dp"] * (2 if c["hi"] == 1 else 0), flops=0)
    if op == "attend":
        z, rec, n = _quantizer(c), _record(c), sum(_lens(c))
        grp = c["hq"] // c["hkv"]
        return dict(bytes=n * c["hkv"] * rec["words"] // 8 + c["b"] * c["hq"] * (4 * c["d"] + 4),
                    flops=2 * n * c["hkv"] * grp * (2 * z["dp"] + c["m"]) + 2 * c["b"] * c["hq"] * z["dp"] * c["m"])
    c = dict(c, **_PAGES)
    lens, words = _page_lens(c), _record(c)["words"]
    unit = 4 * c["layers"] * c["hkv"] * words  # one 32-token block of every layer and head
    table = 8 * c["b"] * -(-c["ctx"] // c["page"])
    if op == "fork":
        keep = lens[: c["b"] - c["n"]]
        return dict(bytes=2 * unit * c["n"] * sum(-(-(x % c["page"]) // 32) for x in keep) / len(keep) + table, flops=0)
    need = sum(-(-x // c["page"]) for x in lens)
    kept = sum(-(-x // c["page"]) for i, x in enumerate(lens) if i % 3 != 1)
    n_pages = need + need * c["spare"] // 100 + 4
    moved = kept * (n_pages - kept) / n_pages  # a live page lies behind the border with this chance
    return dict(bytes=2 * moved * unit * (c["page"] // 32) + table, flops=0)
