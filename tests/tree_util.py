"""A plain model, in numpy and 64 bits, of the operators for windows and drafted trees over the paged cache, written from
their definitions in include/kvc.h one sequence, one query and one page at a time."""
import numpy as np

import page_util as R


def drafts(n_q, b, T):
    return T if n_q is None else min(max(int(n_q[b]), 0), T)


def malformed(parent, n):
    return any(not -1 <= int(parent[i]) < i for i in range(n))


def chain(parent, i):
    """i and its ancestors, from i up."""
    out = [i]
    while parent[out[-1]] >= 0:
        out.append(int(parent[out[-1]]))
    return out


def tree_mask(parent, n_q=None, window=0):
    """-> mask words [B, T, W] int32, depth [B, T], status"""
    B, T = parent.shape
    mask, depth, status = np.zeros((B, T, (T + 31) // 32), np.uint32), np.zeros((B, T), np.int32), 0
    for b in range(B):
        n = drafts(n_q, b, T)
        if malformed(parent[b], n):
            status |= R.BAD_INDEX
            continue
        for i in range(n):
            up = chain(parent[b], i)
            depth[b, i] = len(up) - 1
            for j in up[:window] if window else up:
                mask[b, i, j // 32] |= np.uint32(1 << (j % 32))
    return mask.view(np.int32), depth, status


def tree_verify(parent, draft, target, n_q=None):
    """-> path [B, T], n_path [B], next [B], status"""
    B, T = parent.shape
    path, n_path, nxt, status = np.full((B, T), -1, np.int32), np.zeros(B, np.int32), np.full(B, -1, np.int32), 0
    for b in range(B):
        n = drafts(n_q, b, T)
        if malformed(parent[b], n):
            status |= R.BAD_INDEX
            continue
        if n == 0:
            continue
        kept = [0]
        while True:
            kids = [c for c in range(n) if parent[b, c] == kept[-1] and draft[b, c] == target[b, kept[-1]]]
            if not kids:
                break
            kept.append(kids[0])
        path[b, :len(kept)] = kept
        n_path[b], nxt[b] = len(kept), target[b, kept[-1]]
    return path, n_path, nxt, status


def seen_tokens(n, nq, i, window=0, sinks=0, mask=None, depth=None):
    """The tokens of a stream of n that query i of nq sees; mask: words of row i, depth: of all the queries."""
    base = n - nq
    pos = base + (i if depth is None else min(max(int(depth[i]), 0), nq - 1))
    near = lambda j: window == 0 or j < sinks or j > pos - window
    out = [j for j in range(min(max(base, 0), n)) if near(j)]
    for j in range(max(base, 0), n):
        u = j - base
        if (near(j) and u <= i) if mask is None else int(np.uint32(mask[u // 32])) >> (u % 32) & 1:
            out.append(j)
    return np.array(out, np.int64)


def attend(pool, t, q, scale, n_q=None, window=0, sinks=0, mask=None, depth=None, bad=()):
    """page_util.attend's results under a mask; tokens of the (sequence, head, entry)s in `bad` take no part."""
    B, T, Hq, D = q.shape
    Hkv = t.shape[2]
    G = Hq // Hkv
    r = dict(out=np.zeros(q.shape), lse=np.full(q.shape[:3], -np.inf), mass=np.zeros(q.shape),
             logit=np.zeros(q.shape[:3]), vmax=np.zeros(q.shape))
    for b in range(B):
        nq = drafts(n_q, b, T)
        for h in range(Hkv):
            K, V = R.rows(pool, t, (0, b, h), 0), R.rows(pool, t, (0, b, h), 1)
            for i in range(nq):
                seen = seen_tokens(len(K), nq, i, window, sinks, None if mask is None else mask[b, i],
                                   None if depth is None else depth[b])
                seen = np.array([j for j in seen if (b, h, j // pool.page) not in bad], np.int64) if bad else seen
                if len(seen) == 0:
                    continue
                one = R.attend_rows(q[b, i, h * G:(h + 1) * G], K[seen], V[seen], scale)
                for name, x in one.items():
                    r[name][b, i, h * G:(h + 1) * G] = x
    return r


def slide(pool, t, window, sinks=0):
    """-> gone [L, B, Hkv]"""
    P = pool.page
    before = pool.refs.copy()
    gone = np.zeros(t.shape, np.int32)
    for s in t.streams():
        n = int(t.len[s])
        row = list(t.table[s][:R.npg(n, P)])
        out = [i for i in range(R.npg(sinks, P), len(row)) if (i + 1) * P <= n + 1 - window]
        for i in out:
            pool.refs[row[i]] -= 1
        left = [p for i, p in enumerate(row) if i not in out]
        t.table[s][:] = left + [-1] * (t.maxp - len(left))
        t.len[s] = n - len(out) * P
        gone[s] = len(out) * P
    pool.give_back(before)
    return gone


def accept_lists(t, path, n_path, n_q=None, T=None):
    """{stream: kept list, None for a bad one}, as page_util.compact takes them"""
    T = path.shape[1]
    out = {}
    for s in t.streams():
        b, n = s[1], int(t.len[s])
        nq, k = drafts(n_q, b, T), int(n_path[b])
        p = [int(v) for v in path[b, :max(k, 0)]]
        ok = 0 <= k <= nq <= n and all(0 <= v < nq for v in p) and all(x < y for x, y in zip(p, p[1:]))
        out[s] = list(range(n - nq)) + [n - nq + v for v in p] if ok else None
    return out


def random_trees(rng, B, T, n_q=None):
    parent = np.full((B, T), -7, np.int32)  # behind the last draft lies anything
    for b in range(B):
        for i in range(drafts(n_q, b, T)):
            parent[b, i] = -1 if i == 0 else i - 1 - min(int(rng.geometric(0.4)) - 1, i - 1 + int(rng.random() < 0.1))
    return parent
