"""Plain numpy model of the paged compressed cache: a page pool as uint32
words laid out as include/tq.h says (tq_paged_create), written and read a
token at a time, and attention over it in 64 bits."""
import numpy as np


class Model:
    def __init__(self, kp, vp, layers, hkv, page):
        self.layers, self.hkv, self.page, self.nb = layers, hkv, page, page // 32
        self.dp, self.kk, self.kv = kp.d_pad, kp.k, vp.k
        self.kw, self.sw = kp.code_words, kp.sign_words
        self.nk = self.kw + self.sw
        self.g = next(g for g in (4, 2, 1) if self.nk % g == 0)
        self.r16 = kp.rnorm_dtype == "float16"
        self.kn = 32 * self.nk
        self.kr = self.kn + 32
        self.v = self.kr + (16 if self.r16 else 32)
        self.vn = self.v + self.kv * self.dp
        self.words = self.vn + 32
        self.page_words = layers * hkv * self.nb * self.words

    def record(self, pool, page, layer, h, blk):
        at = ((layer * self.hkv + h) * self.nb + blk) * self.words
        return pool[page, at:at + self.words]

    def key_place(self, t, w):
        return (w // self.g) * 32 * self.g + t * self.g + w % self.g

    def value_place(self, t):
        """(word, bit) of each index bit of token t (k = 4: of its stored nibble)."""
        s, i = t % 4, t // 4
        if self.kv == 1:
            return [(0, t)]
        if self.kv == 4:
            return [(s, 4 * i + p) for p in range(4)]
        at = 4 * i + 2 * (s % 2)
        return [(s // 2, at), (s // 2, at + 1), (2, (t + 2) % 32)][: self.kv]

    @staticmethod
    def nibble(idx):
        return np.where(idx >= 8, idx - 8, 15 - idx)

    def write(self, rec, t, kwords, kn, kr, vidx, vn):
        """Token t of a record: key words, norms (bit patterns) and value indices [dp]."""
        for w in range(self.nk):
            rec[self.key_place(t, w)] = kwords[w]
        rec[self.kn + t], rec[self.vn + t] = kn, vn
        if self.r16:
            rec[self.kr:self.v].view(np.uint16)[t] = kr
        else:
            rec[self.kr + t] = kr
        code = self.nibble(vidx) if self.kv == 4 else vidx
        for p, (word, bit) in enumerate(self.value_place(t)):
            w = rec[self.v + word * self.dp: self.v + (word + 1) * self.dp]
            w[:] = (w & ~np.uint32(1 << bit)) | (((code >> p) & 1).astype(np.uint32) << np.uint32(bit))

    def read(self, rec, t):
        """(key indices [dp], signs [m], norm, residual norm, value indices [dp], norm) of token t."""
        kw = np.array([rec[self.key_place(t, w)] for w in range(self.nk)], np.uint32)
        bits = (kw[:, None] >> np.arange(32, dtype=np.uint32)) & 1
        planes = bits[: self.kw].reshape(self.kk, self.dp)
        kidx = sum(planes[p].astype(int) << p for p in range(self.kk))
        v = rec[self.v:self.vn].reshape(self.kv, self.dp)
        code = sum(((v[word] >> np.uint32(bit)) & 1).astype(int) << p
                   for p, (word, bit) in enumerate(self.value_place(t)))
        vidx = np.where(code >= 8, 15 - code, code + 8) if self.kv == 4 else code
        f = rec.view(np.float32)
        kr = float(rec[self.kr:self.v].view(np.float16)[t]) if self.r16 else float(f[self.kr + t])
        return kidx, bits[self.kw:].reshape(-1), float(f[self.kn + t]), kr, vidx, float(f[self.vn + t])

    def append(self, pool, layer, kwords, kn, kr, vidx, vn, cu, start, tables):
        """Rows [n_tok, hkv, ...]; what the call does to the pool, in place."""
        n_pages = pool.shape[0]
        for b in range(len(start)):
            for i in range(cu[b], cu[b + 1]):
                pos = int(start[b]) + i - int(cu[b])
                if not 0 <= pos < tables.shape[1] * self.page:
                    continue
                pg = tables[b, pos // self.page]
                if not 0 <= pg < n_pages:
                    continue
                for h in range(self.hkv):
                    rec = self.record(pool, pg, layer, h, pos % self.page // 32)
                    self.write(rec, pos % 32, kwords[i, h], kn[i, h], kr[i, h], vidx[i, h], vn[i, h])

    def attention(self, pool, layer, kq, vq, q, lens, tables, scale):
        """(out [B, Hq, d], lse [B, Hq], spread [B, Hq], delta [B, Hq]) in 64 bits.  spread: sum of p ||value||,
        delta: a bound of the error that fp32 sums of the score's terms make."""
        B, Hq, d = q.shape
        G = Hq // self.hkv
        out, lse = np.zeros((B, Hq, d)), np.full((B, Hq), -np.inf)
        spread, delta = np.zeros((B, Hq)), np.zeros((B, Hq))
        m = self.sw * 32
        kappa = np.sqrt(np.pi / 2) / m
        ck, cv = np.asarray(kq.centroids, np.float64), np.asarray(vq.centroids, np.float64)
        for b in range(B):
            n = min(max(int(lens[b]), 0), tables.shape[1] * self.page)
            for h in range(self.hkv):
                toks = [self.read(self.record(pool, tables[b, t // self.page], layer, h, t % self.page // 32), t % 32)
                        for t in range(n) if 0 <= tables[b, t // self.page] < pool.shape[0]]
                if not toks:
                    continue
                K = ck[np.array([t[0] for t in toks])]
                S = 2.0 * np.array([t[1] for t in toks]) - 1
                kn, kr, vn = (np.array([t[i] for t in toks]) for i in (2, 3, 5))
                V = cv[np.array([t[4] for t in toks])] * vn[:, None]
                qr = kq.rot.apply(q[b, h * G:(h + 1) * G])
                u = qr @ kq.S.T
                s = scale * kn * (qr @ K.T + kappa * kr * (u @ S.T))
                mag = abs(scale) * kn * (abs(qr) @ abs(K.T) + kappa * kr * abs(u).sum(-1)[:, None])
                top = s.max(-1, keepdims=True)
                p = np.exp(s - top)
                tot = p.sum(-1, keepdims=True)
                w = slice(h * G, (h + 1) * G)
                out[b, w] = vq.rot.apply_t(p / tot @ V)
                lse[b, w] = (top + np.log(tot))[:, 0]
                spread[b, w] = (p / tot) @ np.linalg.norm(V, axis=1)
                delta[b, w] = mag.max(-1) * (self.dp + m) * 2.0 ** -24
        return out, lse, spread, delta
