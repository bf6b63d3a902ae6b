"""A plain model of the paged 4-bit cache, in numpy and 64 bits, for the tests: pools, page tables and every
kvc_page_* operator written from their definitions in include/kvc.h, one stream and one page at a time."""
import numpy as np

MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
NO_PAGES, BAD_PAGE, TABLE_FULL, BAD_INDEX = 0x10, 0x20, 0x40, 0x4


def e4m3_values():
    """The 256 e4m3 bytes' values (0x7f and 0xff are NaN)."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e > 0, np.exp2(e - 7.0) * (1 + m / 8), m / 512.0)
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >= 128, -v, v)


E4M3 = e4m3_values()


def quantise(x, ts):
    """Rows [..., D] (float64 holding the inputs) -> codes [..., D/2], scale bytes [..., D/16]. The tensor scale, six
    times it and a group's step are fp32 numbers; the quotients by them are exact."""
    ts = np.float32(ts)
    x = np.asarray(x, np.float64)
    g = x.reshape(x.shape[:-1] + (-1, 16))
    a = np.abs(g)
    with np.errstate(invalid="ignore"):
        amax = np.where(np.isnan(a), 0.0, a).max(-1)
        want = np.clip(amax / np.float64(np.float32(6) * ts), 2.0 ** -9, 448.0)
        pos = E4M3[:127]  # ascending, 0 .. 448
        hi = np.clip(np.searchsorted(pos, want), 1, 126)
        lo = hi - 1
        dl, dh = want - pos[lo], pos[hi] - want
        sb = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
        y = a / (E4M3[sb].astype(np.float32) * ts).astype(np.float64)[..., None]
        code = np.zeros(g.shape, np.uint8)
        for k, border in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
            code += ((y > border) if k % 2 == 0 else (y >= border)).astype(np.uint8)
        code += np.where(np.signbit(g) & (code > 0), 8, 0).astype(np.uint8)  # what rounds to zero has no sign
    code = code.reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), sb


def values(codes, sb, ts):
    c = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[:-1] + (-1,))
    v = np.where(c >= 8, -MAGS[c & 7], MAGS[c & 7])
    return v * np.repeat((E4M3[sb].astype(np.float32) * np.float32(ts)).astype(np.float64), 16, -1)


class RefPool:
    def __init__(self, npages, D, page, k_scale=1.0, v_scale=1.0, rng=None):
        self.D, self.page, self.npages, self.ts = D, page, npages, (k_scale, v_scale)
        self.data = np.zeros((npages, page // 16, 18 * D), np.uint8)
        if rng is not None:
            self.data[:] = rng.integers(0, 127, self.data.shape)  # any byte below NaN is a scale
        self.refs = np.zeros(npages, np.int32)
        self.free = np.arange(npages - 1, -1, -1, dtype=np.int32)
        self.nfree = npages
        self.status = 0

    def piece(self, p, tok, piece):
        """View of one token's codes or scales in page p (0 K codes, 1 K scales, 2 V codes, 3 V scales)."""
        D = self.D
        off = (0, 8 * D, 9 * D, 17 * D)[piece]
        w = D // 16 if piece & 1 else D // 2
        i = tok % self.page
        return self.data[p, i // 16, off + (i % 16) * w: off + (i % 16 + 1) * w]

    def token(self, p, tok):
        return [self.piece(p, tok, k).copy() for k in range(4)]

    def put(self, p, tok, parts):
        for k in range(4):
            self.piece(p, tok, k)[:] = parts[k]

    def give_back(self, before):
        for p in np.flatnonzero((before > 0) & (self.refs == 0)):
            self.free[self.nfree] = p
            self.nfree += 1


class RefPages:
    def __init__(self, L, B, Hkv, maxp):
        self.shape, self.maxp = (L, B, Hkv), maxp
        self.table = np.full((L, B, Hkv, maxp), -1, np.int32)
        self.len = np.zeros((L, B, Hkv), np.int32)

    def streams(self):
        return np.ndindex(*self.shape)


def npg(n, page):
    return -(-n // page)


def extend(pool, t, add):
    L, B, Hkv = t.shape
    P = pool.page
    start = np.full(t.shape, -1, np.int32)
    ok, plan, total = {}, {}, 0
    for s in t.streams():
        n, a = int(t.len[s]), int(add[s[1]])
        if a < 0:
            pool.status |= BAD_INDEX
            continue
        if n + a > t.maxp * P:
            pool.status |= TABLE_FULL
            continue
        ok[s] = (n, a)
    for s, (n, a) in ok.items():
        copy = False
        if a > 0 and n % P:
            p = t.table[s][n // P]
            if pool.refs[p] > 1:
                w = [b for b in range(B) if (s[0], b, s[2]) in ok and add[b] > 0
                     and t.len[s[0], b, s[2]] % P and t.table[s[0], b, s[2]][t.len[s[0], b, s[2]] // P] == p]
                copy = not (len(w) >= pool.refs[p] and w[0] == s[1])
        plan[s] = (copy, npg(n + a, P) - npg(n, P) if a > 0 else 0)
        total += copy + plan[s][1]
    if total > pool.nfree:
        pool.status |= NO_PAGES
        return start
    for s in sorted(plan):
        n, a = ok[s]
        copy, fresh = plan[s]
        if copy:
            pool.nfree -= 1
            p, old = pool.free[pool.nfree], t.table[s][n // P]
            pool.data[p] = pool.data[old]
            pool.refs[p] = 1
            pool.refs[old] -= 1
            t.table[s][n // P] = p
        for j in range(fresh):
            pool.nfree -= 1
            t.table[s][npg(n, P) + j] = pool.free[pool.nfree]
            pool.refs[pool.free[pool.nfree]] = 1
        start[s] = n
        t.len[s] = n + a
    return start


def free(pool, t, drop):
    before = pool.refs.copy()
    for s in t.streams():
        n, d = int(t.len[s]), int(drop[s[1]])
        if d < 0:
            pool.status |= BAD_INDEX
            continue
        left = max(n - d, 0)
        for i in range(npg(left, pool.page), npg(n, pool.page)):
            pool.refs[t.table[s][i]] -= 1
            t.table[s][i] = -1
        t.len[s] = left
    pool.give_back(before)


def fork(pool, t, parent):
    L, B, Hkv = t.shape
    out = RefPages(L, len(parent), Hkv, t.maxp)
    before = pool.refs.copy()
    for s in t.streams():
        kids = sum(int(p) == s[1] for p in parent)
        for i in range(npg(int(t.len[s]), pool.page)):
            pool.refs[t.table[s][i]] += kids - 1
    for c in out.streams():
        p = int(parent[c[1]])
        if 0 <= p < B:
            n = t.len[c[0], p, c[2]]
            out.len[c] = n
            e = npg(int(n), pool.page)
            out.table[c][:e] = t.table[c[0], p, c[2]][:e]
        elif p != -1:
            pool.status |= BAD_INDEX
    pool.give_back(before)
    return out


def compact(pool, t, lists):
    """lists: {stream: kept indices or None for a list that is bad}"""
    P = pool.page
    before = pool.refs.copy()
    plan, total = [], 0
    for s in t.streams():
        idx, n = lists[s], int(t.len[s])
        if idx is None:
            pool.status |= BAD_INDEX
            continue
        m = len(idx)
        k0 = next((k for k in range(m) if idx[k] != k), m)
        pages = range(k0 // P, npg(m, P)) if k0 < m else range(0)
        shared = [i for i in pages if before[t.table[s][i]] > 1]
        plan.append((s, idx, n, m, k0, shared))
        total += len(shared)
    if total > pool.nfree:
        pool.status |= NO_PAGES
        return
    old_data = pool.data.copy()
    src = RefPool.__new__(RefPool)
    src.D, src.page, src.data = pool.D, P, old_data
    for s, idx, n, m, k0, shared in plan:
        old = t.table[s].copy()
        new = old.copy()
        for i in shared:
            pool.nfree -= 1
            new[i] = pool.free[pool.nfree]
            pool.refs[new[i]] = 1
            pool.refs[old[i]] -= 1
        first = k0 // P * P if k0 // P in shared else k0
        if k0 < m:
            for k in range(first, m):
                pool.put(new[k // P], k, src.token(old[idx[k] // P], int(idx[k])))
        for i in range(npg(m, P), npg(n, P)):
            pool.refs[old[i]] -= 1
            new[i] = -1
        t.table[s][:] = new
        t.len[s] = m
    pool.give_back(before)


def store(pool, t, k, v, start, n=None):
    """k, v [B, T, Hkv, D] float64; one layer."""
    L, B, Hkv = t.shape
    for j, x in enumerate((k, v)):
        codes, sb = quantise(x, pool.ts[j])
        for _, b, h in t.streams():
            for i in range(x.shape[1] if n is None else int(n[b])):
                tok = int(start[0, b, h]) + i
                p = t.table[0, b, h][tok // pool.page]
                pool.piece(p, tok, 2 * j)[:] = codes[b, i, h]
                pool.piece(p, tok, 2 * j + 1)[:] = sb[b, i, h]


def rows(pool, t, s, j):
    """K (j = 0) or V (1) of stream s: [len, D] float64."""
    n = int(t.len[s])
    if n == 0:
        return np.zeros((0, pool.D))
    pg = t.table[s][:npg(n, pool.page)]
    blk = pool.data[pg].reshape(-1, 18 * pool.D)
    at = 9 * pool.D * j
    c = blk[:, at:at + 8 * pool.D].reshape(-1, pool.D // 2)
    sb = blk[:, at + 8 * pool.D:at + 9 * pool.D].reshape(-1, pool.D // 16)
    return values(c[:n], sb[:n], pool.ts[j])


def attend_rows(q, K, V, scale):
    """Query rows q [r, D] over all of K, V [n, D], n >= 1: out, lse, and what tolerances() needs."""
    s = scale * q @ K.T
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m)
    tot = p.sum(-1, keepdims=True)
    return dict(out=p @ V / tot, lse=(m + np.log(tot))[:, 0], mass=p @ np.abs(V) / tot,
                logit=(abs(scale) * np.abs(q) @ np.abs(K).T).max(-1), vmax=np.abs(V).max(0) + 0 * q)


def attend(pool, t, q, scale, n_q=None, layer=0):
    """attend_rows' results for every query [B, T, Hq, .]: q [B, T, Hq, D] float64."""
    B, T, Hq, D = q.shape
    Hkv = t.shape[2]
    G = Hq // Hkv
    r = dict(out=np.zeros(q.shape), lse=np.full(q.shape[:3], -np.inf), mass=np.zeros(q.shape),
             logit=np.zeros(q.shape[:3]), vmax=np.zeros(q.shape))
    for b in range(B):
        nq = T if n_q is None else min(max(int(n_q[b]), 0), T)
        for h in range(Hkv):
            K, V = rows(pool, t, (layer, b, h), 0), rows(pool, t, (layer, b, h), 1)
            for i in range(nq):
                seen = len(K) - nq + i + 1
                if seen < 1:
                    continue
                one = attend_rows(q[b, i, h * G:(h + 1) * G], K[:seen], V[:seen], scale)
                for name, x in one.items():
                    r[name][b, i, h * G:(h + 1) * G] = x
    return r


def tolerances(dtype, n, D, r):
    """Bounds on |kernel - definition| of out and lse, from the arithmetic alone.
    A logit: products of fp16 factors are exact in fp32 (codes times scales exactly, queries to 2^-11, or 2^-22 in two
    terms; bf16 queries exactly, but for parts below 2^-22 of the row's largest); D additions of relative error 2^-23
    each: ds = (D + 8) 2^-23 max_j scale sum |q k|, plus 2^-21 for the base-2 exponential and its argument's rounding.
    A probability: relative 2 ds, and one rounding to fp16 (2^-11; 2^-22 in two terms); below fp16's normal range,
    which begins 2^-24 under the largest probability, that rounding is absolute, 2^-35 of the largest. Sums of n
    terms: n 2^-23 of the terms' magnitudes, numerator and denominator. The output's own rounding: bf16 2^-8, fp32
    2^-24."""
    f32 = dtype == "f32"
    lse = np.where(np.isfinite(r["lse"]), r["lse"], 0)
    ds = (D + 8) * 2.0 ** -23 * r["logit"] * (2 if f32 else 1) + 2.0 ** -21 + np.abs(lse) * 2.0 ** -22
    rel = 2 * ds + (2.0 ** -21 if f32 else 2.0 ** -11) + 2 * n * 2.0 ** -23
    tol = (2.0 ** -24 if f32 else 2.0 ** -8) * np.abs(r["out"]) * 1.01 + rel[..., None] * (r["mass"] + np.abs(r["out"]))
    return tol + n * 2.0 ** -35 * r["vmax"] + 1e-30, ds + n * 2.0 ** -23 + 2.0 ** -22
