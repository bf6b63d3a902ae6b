"""Operators over the paged 4-bit cache for windowed and speculative decoding, as cases to be measured: each in a
plain form (elementary torch operations, fp32) and, where `own` is true, as the calls a program makes of libkvc.

A pool holds npages pages of `page` tokens of one KV head; a page is a run of 16-token blocks
  [K codes 16 x D/2][K scales 16 x D/16][V codes 16 x D/2][V scales 16 x D/16]   (18 D bytes)
with two e2m1 codes a byte (even channel in the low nibble) and an e4m3 scale per 16 channels;
a code stands for k_scale (or v_scale) * scale * e2m1. Each (layer, sequence, KV head) has a row of
page numbers and a length.

Operators (case["op"]):
  window  attention of T new queries per sequence that see the first `sinks` tokens and, of the others, those
          less than `window` positions back (causal at the cache's end); output and log-sum-exp
  tree    attention of a tree of T drafted tokens per sequence: a draft sees the cached tokens (with window > 0
          as above, its position being the cache's end plus its depth), itself and its ancestors
  slide   room for the step's tokens, then the whole pages between the sinks and the window given back
  accept  room for T drafts, the path of drafts that the model's picks confirm, its rows moved to the drafts'
          front and the rest dropped, then the pages behind the window given back
"""
import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # the smallest call: the tiny model's one sequence, fp32 (latency)
        dict(name="window tiny f32", op="window", B=1, Hkv=2, G=2, D=64, N=224, T=1, window=64, sinks=4, page=16,
             dtype="f32", ragged=0),
        # a decode step of one layer of an 8B model, 16 sequences, every head with its own length
        dict(name="window step", op="window", B=16, Hkv=8, G=4, D=128, N=4096, T=1, window=1024, sinks=4, page=64,
             dtype="bf16", ragged=1),
        # long traces: a window of 8192 out of 32k tokens, 5 query heads per KV head
        dict(name="window long", op="window", B=8, Hkv=8, G=5, D=128, N=32768, T=1, window=8192, sinks=4, page=64,
             dtype="bf16", ragged=0),
        # a prompt's chunk of 1024 tokens behind 7168 cached ones
        dict(name="window prompt", op="window", B=2, Hkv=8, G=4, D=128, N=8192, T=1024, window=2048, sinks=4, page=64,
             dtype="bf16", ragged=0),
        # a few drafts of the tiny model, fp32 (latency)
        dict(name="tree tiny f32", op="tree", B=1, Hkv=2, G=2, D=64, N=224, T=7, window=0, sinks=0, page=16,
             dtype="f32", ragged=0),
        # 27 drafts for each of 16 sequences of an 8B model
        dict(name="tree batch", op="tree", B=16, Hkv=8, G=4, D=128, N=4096, T=27, window=0, sinks=0, page=64,
             dtype="bf16", ragged=1),
        # wide trees, 7 query heads per KV head
        dict(name="tree wide", op="tree", B=8, Hkv=4, G=7, D=128, N=8192, T=64, window=0, sinks=0, page=64,
             dtype="bf16", ragged=0),
        # 16 drafts behind 32k tokens
        dict(name="tree long", op="tree", B=8, Hkv=8, G=5, D=128, N=32768, T=16, window=0, sinks=0, page=64,
             dtype="bf16", ragged=0),
        # a small server's step
        dict(name="slide small", op="slide", L=2, B=4, Hkv=2, D=64, window=64, sinks=4, grow=5, page=16),
        # a decode step of every layer of a 36-layer model, 8 sequences
        dict(name="slide 36 layers", op="slide", L=36, B=8, Hkv=8, D=128, window=1024, sinks=4, grow=1, page=64),
        # seven drafts of a small model
        dict(name="accept small", op="accept", L=2, B=4, Hkv=2, D=64, T=7, window=200, sinks=4, page=16),
        # trees of 64 drafts of a 36-layer model, 8 sequences
        dict(name="accept 36 layers", op="accept", L=36, B=8, Hkv=8, D=128, T=64, window=2000, sinks=4, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window", "window", "tree", "tree", "tree", "slide", "accept"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8, 8])
    page = rng.choice([16, 32, 64, 64, 128, 256])
    if op in ("window", "tree"):
        B, G = _log(rng, 1, 16), rng.randint(1, 8)
        T = rng.choice([1, 1, _log(rng, 2, 512)]) if op == "window" else _log(rng, 1, 128)
        most = min(32768, (1 << 29) // (B * Hkv * G * T), (2 << 20) // (B * Hkv))  # within the largest listed cases
        N = _log(rng, 1, max(2, most))
        window = _log(rng, 1, max(2, N + N // 4)) if op == "window" else rng.choice([0, 0, _log(rng, 1, max(2, N))])
        return dict(op=op, B=B, Hkv=Hkv, G=G, D=D, N=N, T=T, window=window,
                    sinks=rng.choice([0, 1, 4, _log(rng, 2, 100)]) if window else 0, page=page,
                    dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]), ragged=rng.randint(0, 1))
    L, B = _log(rng, 1, 32), _log(rng, 1, 8)
    window, sinks = _log(rng, 8, 1500), rng.choice([0, 1, 4, _log(rng, 2, 100)])
    if op == "slide":
        return dict(op=op, L=L, B=B, Hkv=Hkv, D=D, window=window, sinks=sinks, grow=_log(rng, 1, 200), page=page)
    return dict(op=op, L=L, B=B, Hkv=Hkv, D=D, T=_log(rng, 1, 64), window=window, sinks=sinks, page=page)


def _pages(n, page):
    return -(-n // page)


def _lengths(case, rows):
    """The streams' lengths, fixed by the case: N for all, or spread over N/4..N; those of the page operators
    lie around the window."""
    if case["op"] in ("slide", "accept"):
        w = case["window"]
        return np.random.RandomState(w + rows).randint(max(1, w // 2), w + 2 * case["page"] + 1, rows)
    N = case["N"]
    if not case["ragged"]:
        return np.full(rows, N)
    return np.random.RandomState(N + rows).randint(max(1, N // 4), N + 1, rows)


def _most(case):
    """The most tokens that a stream of the page operators reaches: what a slide leaves behind the sinks' pages, and
    the step's room."""
    p, room = case["page"], case["grow"] if case["op"] == "slide" else case["T"]
    return _pages(case["sinks"], p) * p + case["window"] + 3 * p + room


def _parents(case, seed):
    """Trees of T nodes, one per sequence: node 0 is the root, every other node's parent is one of the nodes before
    it, mostly a recent one, so that depths differ."""
    r = np.random.RandomState(seed % (1 << 31))
    B, T = case["B"], case["T"]
    out = np.full((B, T), -1, np.int32)
    for i in range(1, T):
        out[:, i] = i - np.minimum(r.geometric(0.25, B), i)
    return out


def work(case):
    D = case["D"]
    row = 2 * (D // 2 + D // 16)  # a token's K and V in 4 bits, with their scales
    S = case.get("L", 1) * case["B"] * case["Hkv"]
    if case["op"] in ("window", "tree"):
        n, T, G, w, k = _lengths(case, S).astype(np.float64), case["T"], case["G"], case["window"], case["sinks"]
        es = 2 if case["dtype"] == "bf16" else 4
        if case["op"] == "window":
            pos = n[:, None] - T + np.arange(T)
            lo = np.clip(pos - w + 1, 0, None)
            pairs = np.clip(pos + 1 - lo, 0, None) + np.clip(np.minimum(np.minimum(k, pos + 1), lo), 0, None)
            first = np.clip(n - T - w + 1, 0, None)  # the first query's window
            read = np.minimum(n, n - first + np.minimum(k, first))
        else:
            dep = _depths(_parents(case, 0))
            base = np.clip(n - T, 0, None)
            read = n if not w else np.minimum(n, np.minimum(base, w - 1) + np.minimum(k, base) + T)
            pairs = (read - np.minimum(n, T))[:, None] * np.ones(T) + dep.mean(0) + 1
        return dict(bytes=float(read.sum()) * row + S * T * G * (2 * D * es + 4) + 8.0 * S,
                    flops=4.0 * D * G * float(pairs.sum()))
    grow = case["grow"] if case["op"] == "slide" else case["T"]
    entries = S * _pages(_most(case), case["page"])
    # lengths in and out, the tables' entries of streams that lose a page in and out, the pages taken and given back
    share = min(1.0, grow / case["page"])
    moved = S * min(case["T"], 8) * 2.0 * row if case["op"] == "accept" else 0.0
    return dict(bytes=8.0 * S + 8.0 * entries * share + 16.0 * S * grow / case["page"] + moved, flops=float(S))


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _rows(shape, g, dtype=torch.float32):
    """K or V rows as a model makes them: N(0,1) with a scale per channel, 4 channels heavy-tailed."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= 0.5 + 1.5 * torch.rand(shape[-1], generator=g, device="cuda")
    at = torch.randperm(shape[-1], generator=g, device="cuda")[:4]
    x[..., at] *= 2.0
    return x.to(dtype)


def _quantise(x, tensor_scale):
    """Rows [..., D] to codes [..., D/2] and scales [..., D/16], both uint8."""
    x = x.float().unflatten(-1, (-1, 16))
    want = (x.abs().amax(-1) / (6.0 * tensor_scale)).clamp(2.0 ** -9, 448.0)
    sc = want.to(torch.float8_e4m3fn)
    y = x / (sc.float() * tensor_scale)[..., None]
    a = y.abs()
    code = torch.zeros_like(x, dtype=torch.uint8)
    for border in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
        code += a > border
    code += (y < 0).to(torch.uint8) * 8
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), sc.view(torch.uint8)


def _pool(npages, page, D, g, scales):
    """A pool's arrays: bytes of quantised rows in every page, no page in use yet."""
    data = torch.zeros((npages, page // 16, 18 * D), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (page * D))
    for a in range(0, npages, step):
        b = min(npages, a + step)
        parts = []
        for s in scales:
            codes, sc = _quantise(_rows((b - a, page // 16, 16, D), g), s)
            parts += [codes.flatten(2), sc.flatten(2)]
        data[a:b] = torch.cat(parts, -1)
    return data.view(npages, -1)


def _tables(S, maxp, npages, used, g):
    """Page tables of S streams with used[s] pages each, scattered over the pool; refs, free list, count."""
    order = torch.randperm(npages, generator=g, device="cuda")
    used = torch.as_tensor(used, device="cuda")
    first = torch.cumsum(used, 0) - used
    i = torch.arange(maxp, device="cuda")
    at = (first[:, None] + i).clamp(max=npages - 1)
    table = torch.where(i < used[:, None], order[at], -1).to(torch.int32)
    total = int(used.sum())
    refs = torch.zeros(npages, dtype=torch.int32, device="cuda")
    refs[order[:total]] = 1
    free = torch.full((npages,), -1, dtype=torch.int32, device="cuda")
    free[:npages - total] = order[total:].flip(0).to(torch.int32)
    nfree = torch.tensor([npages - total], dtype=torch.int32, device="cuda")
    return table, refs, free, nfree


def _int(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def prepare(case, seed):
    g = _gen(seed)
    op, page, D = case["op"], case["page"], case["D"]
    L, B, Hkv = case.get("L", 1), case["B"], case["Hkv"]
    S = L * B * Hkv
    st = dict(case=dict(case), k_scale=1.0, v_scale=0.5)
    n = _lengths(case, S)
    attends = op in ("window", "tree")
    maxp = _pages(case["N"] if attends else _most(case), page)
    used = -(-n // page)
    npages = int(used.sum()) if attends else S * maxp
    npages += 3 + npages // 16
    st["data"] = _pool(npages, page, D, g, (st["k_scale"], st["v_scale"]))
    table, refs, free, nfree = _tables(S, maxp, npages, used, g)
    st.update(table=table.view(L, B, Hkv, maxp), refs=refs, free=free, nfree=nfree, len=_int(n).view(L, B, Hkv))
    if attends:
        G, T = case["G"], case["T"]
        st["q"] = torch.randn((B, T, Hkv * G, D), generator=g, device="cuda").to(DTYPES[case["dtype"]])
    if op in ("tree", "accept"):
        parent = _parents(case, seed)
        st["parent"] = _int(parent)
    if op == "accept":
        # drafts, and the model's pick behind each: two times in three the token of one of its children
        T, r = case["T"], np.random.RandomState((seed + 1) % (1 << 31))
        draft = r.randint(0, 1000, (B, T))
        target = r.randint(1000, 2000, (B, T))
        for b in range(B):
            for i in range(1, T):
                if r.rand() < 0.67:
                    target[b, parent[b, i]] = draft[b, i]
        st["draft"], st["target"] = _int(draft), _int(target)
    if own:  # what a program keeps between calls: the handles over these arrays, workspaces and outputs
        from decoding_kv_cache_gb300 import kvc
        new = lambda shape, dt=torch.int32: torch.empty(shape, dtype=dt, device="cuda")
        st["pool"] = kvc.Pool(st["data"], st["refs"], st["free"], st["nfree"], D, page, st["k_scale"], st["v_scale"])
        st["pages"] = kvc.Pages(st["table"], st["len"])
        st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if attends:
            st["out"], st["lse"] = torch.empty_like(st["q"]), new((B, T, Hkv * G), torch.float32)
            nb = kvc.kvc_page_attend_masked_workspace_size(st["pool"], st["pages"], Hkv * G, T, case["window"],
                                                           case["sinks"])
        else:
            nb = kvc.kvc_page_workspace_size(st["pool"], st["pages"])
        if op == "tree":
            st["mask"], st["depth"] = new((B, T, (T + 31) // 32)), new((B, T))
        if op == "accept":
            st["path"], st["n_path"], st["next"] = new((B, T)), new((B,)), new((B,))
        st["ws"] = new((max(nb, 256),), torch.uint8)
    return st


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(st):
    return globals()["_run_" + st["case"]["op"]](st)


def _values(codes, scales, tensor_scale):
    """What the codes stand for, fp32."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    return lut[c] * (scales.view(torch.float8_e4m3fn).float() * tensor_scale).repeat_interleave(16, -1)


def _parts(st):
    """Views of the pool's rows: K codes, K scales, V codes, V scales, each [npages * page/16, 16, .]."""
    D = st["case"]["D"]
    blk = st["data"].view(-1, 18 * D)
    out, at = [], 0
    for w in (D // 2, D // 16, D // 2, D // 16):
        out.append(blk[:, at:at + 16 * w].unflatten(1, (16, w)))
        at += 16 * w
    return out


def _where(table, page, tok):
    """Block and row of tokens `tok` [S, n] in the streams' pages."""
    p = torch.gather(table, 1, tok // page).long()
    return p * (page // 16) + (tok % page) // 16, tok % 16


def _attend(st, seen):
    """Attention of the queries over the tokens that seen [S, T, N] marks."""
    c = st["case"]
    B, Hkv, G, D, T = c["B"], c["Hkv"], c["G"], c["D"], c["T"]
    S, n = B * Hkv, st["len"].view(-1)
    tok = torch.arange(c["N"], device="cuda").expand(S, -1)
    at = _where(st["table"].view(S, -1).clamp(min=0), c["page"], tok)
    kc, ks, vc, vs = (x[at] for x in _parts(st))
    k, v = _values(kc, ks, st["k_scale"]), _values(vc, vs, st["v_scale"])
    v = torch.where((tok < n[:, None])[..., None], v, 0.0)
    q = st["q"].float().view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(S, T * G, D)
    s = torch.matmul(q, k.transpose(1, 2)) * (1.0 / math.sqrt(D))
    s = torch.where(seen[:, :, None], s.view(S, T, G, -1), -torch.inf).view(S, T * G, -1)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), 0.0, m))
    tot = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(tot > 0, tot, 1.0)
    lse = torch.where(tot > 0, m + torch.log(tot), -torch.inf)[..., 0]
    o = o.view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hkv * G, D)
    return o.to(st["q"].dtype), lse.view(B, Hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, Hkv * G).contiguous()


def _run_window(st):
    c = st["case"]
    if own:
        from decoding_kv_cache_gb300 import kvc
        kvc.kvc_page_attend_masked(st["pool"], st["pages"], st["q"], st["out"], window=c["window"], sinks=c["sinks"],
                                   lse=st["lse"], status=st["status"], workspace=st["ws"])
        return st["out"], st["lse"]
    pos = st["len"].view(-1, 1, 1) - c["T"] + torch.arange(c["T"], device="cuda")[:, None]
    j = torch.arange(c["N"], device="cuda")
    return _attend(st, (j <= pos) & ((j > pos - c["window"]) | (j < c["sinks"])))


def _ancestors(parent):
    """[B, T, T]: node j is i or one of its ancestors. Each squaring of the relation doubles its reach."""
    B, T = parent.shape
    i = torch.arange(T, device=parent.device)
    a = ((parent[..., None] == i) | (i[:, None] == i)).float()
    for _ in range(max(1, (T - 1).bit_length())):
        a = (torch.matmul(a, a) > 0).float()
    return a > 0


def _run_tree(st):
    c = st["case"]
    if own:
        from decoding_kv_cache_gb300 import kvc
        kvc.kvc_tree_mask(st["parent"], st["mask"], st["depth"], window=c["window"], status=st["status"])
        kvc.kvc_page_attend_masked(st["pool"], st["pages"], st["q"], st["out"], window=c["window"], sinks=c["sinks"],
                                   mask=st["mask"], depth=st["depth"], lse=st["lse"], status=st["status"],
                                   workspace=st["ws"])
        return st["out"], st["lse"]
    B, Hkv, T, w = c["B"], c["Hkv"], c["T"], c["window"]
    anc = _ancestors(st["parent"])
    depth = anc.sum(-1) - 1
    if w:
        anc = anc & (depth[:, :, None] - depth[:, None] < w)
    base = (st["len"].view(B, Hkv, 1, 1) - T).long()
    j = torch.arange(c["N"], device="cuda")
    u = j - base  # [B, Hkv, 1, N] a token's place among the drafts
    pos = base + depth.view(B, 1, T, 1)
    cached = (u < 0) & ((j > pos - w) | (j < c["sinks"]) if w else torch.ones_like(pos, dtype=torch.bool))
    new = torch.gather(anc[:, None].expand(B, Hkv, T, T), 3, u.clamp(0, T - 1).expand(B, Hkv, T, -1))
    return _attend(st, (cached | (new & (u >= 0) & (u < T))).view(B * Hkv, T, -1))


def _pool_state(st):
    """What the page operators leave: tables, lengths, counts, the free list, and the pages' bytes."""
    return dict(table=st["table"], len=st["len"], refs=st["refs"], free=st["free"], nfree=st["nfree"], data=st["data"])


def _count(st, pages, by):
    """refs[p] += by for every entry of pages >= 0."""
    p = pages.reshape(-1)
    st["refs"].index_add_(0, p.clamp(min=0).long(), torch.where(p >= 0, by, 0).to(torch.int32))


def _give_back(st, had):
    """Pages counted down to zero join the free list in the order of their numbers."""
    gone = torch.nonzero((had > 0) & (st["refs"] == 0)).view(-1).to(torch.int32)
    at = st["nfree"].long() + torch.arange(gone.numel(), device="cuda")
    st["free"][at] = gone
    st["nfree"] += gone.numel()


def _extend(st, a):
    """Room for `a` tokens behind every stream; no page is shared here. Pages go from the free list's end, in stream
    order."""
    page, table, n = st["case"]["page"], st["table"], st["len"]
    i = torch.arange(table.shape[-1], device="cuda")
    fresh = (i >= ((n + page - 1) // page)[..., None]) & (i < ((n + a + page - 1) // page)[..., None])
    rank = torch.cumsum(fresh.reshape(-1).long(), 0).view(fresh.shape) - 1
    new = torch.where(fresh, st["free"][(st["nfree"].long() - 1 - rank).clamp(min=0)], -1)
    _count(st, new, 1)
    table.copy_(torch.where(fresh, new, table))
    st["nfree"] -= fresh.sum().to(torch.int32)
    n += a


def _drop_pages(st, out):
    """The table's entries that `out` marks are given up; their places are cleared."""
    had = st["refs"].clone()
    _count(st, torch.where(out, st["table"], -1), -1)
    st["table"].masked_fill_(out, -1)
    _give_back(st, had)


def _slide(st):
    """The whole pages behind the sinks' and before the window's first go, the pages behind them move up."""
    c, page, table, n = st["case"], st["case"]["page"], st["table"], st["len"]
    i = torch.arange(table.shape[-1], device="cuda")
    first = _pages(c["sinks"], page)
    last = (n + 1 - c["window"]).clamp(min=0) // page
    m = (last - first).clamp(min=0)  # pages that go
    _drop_pages(st, (i >= first) & (i < last[..., None]))
    src = torch.where(i < first, i, i + m[..., None])
    moved = torch.gather(table, 3, src.clamp(max=table.shape[-1] - 1).long())
    table.copy_(torch.where(src < table.shape[-1], moved, -1))
    n -= m * page


def _run_slide(st):
    c = st["case"]
    if own:
        from decoding_kv_cache_gb300 import kvc
        kvc.kvc_page_extend(st["pool"], st["pages"], add_all=c["grow"], status=st["status"], workspace=st["ws"])
        kvc.kvc_page_slide(st["pool"], st["pages"], window=c["window"], sinks=c["sinks"], status=st["status"],
                           workspace=st["ws"])
        return _pool_state(st)
    _extend(st, c["grow"])
    _slide(st)
    return _pool_state(st)


def _run_accept(st):
    c = st["case"]
    if own:
        from decoding_kv_cache_gb300 import kvc
        kvc.kvc_page_extend(st["pool"], st["pages"], add_all=c["T"], status=st["status"], workspace=st["ws"])
        kvc.kvc_tree_verify(st["parent"], st["draft"], st["target"], st["path"], st["n_path"], next=st["next"],
                            status=st["status"])
        kvc.kvc_page_accept(st["pool"], st["pages"], st["path"], st["n_path"], status=st["status"], workspace=st["ws"])
        kvc.kvc_page_slide(st["pool"], st["pages"], window=c["window"], sinks=c["sinks"], status=st["status"],
                           workspace=st["ws"])
        return dict(_pool_state(st), path=st["path"], n_path=st["n_path"], next=st["next"])
    L, B, Hkv, T, page = c["L"], c["B"], c["Hkv"], c["T"], c["page"]
    _extend(st, T)
    # the walk: from the root on, the lowest child whose token is what the model picked
    parent, draft, target = st["parent"].long(), st["draft"], st["target"]
    i = torch.arange(T, device="cuda")
    fits = (i > 0) & (draft == torch.gather(target, 1, parent.clamp(min=0)))
    at = torch.zeros((B, 1), dtype=torch.long, device="cuda")
    alive = torch.ones((B, 1), dtype=torch.bool, device="cuda")
    path = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
    for k in range(T):
        path[:, k:k + 1] = torch.where(alive, at, -1).to(torch.int32)
        kids = fits & (parent == at) & alive
        alive = kids.any(1, keepdim=True)
        at = torch.where(alive, kids.long().argmax(1, keepdim=True), at)
    n_path = (path >= 0).sum(1).to(torch.int32)
    nxt = torch.gather(target, 1, at)[:, 0]
    # the path's rows to the drafts' front, every layer and head
    S = L * B * Hkv
    table = st["table"].view(S, -1)
    of = torch.arange(B, device="cuda").view(1, B, 1).expand(L, B, Hkv).reshape(S)
    base = st["len"].view(S, 1).long() - T
    s, k = torch.nonzero(path[of] >= 0, as_tuple=True)
    src, dst = base[s, 0] + path[of][s, k].long(), base[s, 0] + k
    b = page // 16
    for x in _parts(st):
        rows = x[table[s, src // page].long() * b + src % page // 16, src % 16]
        x[table[s, dst // page].long() * b + dst % page // 16, dst % 16] = rows
    left = st["len"] - T + n_path[of].view(L, B, Hkv)
    j = torch.arange(table.shape[-1], device="cuda")
    _drop_pages(st, (j >= ((left + page - 1) // page)[..., None]) & (j < ((st["len"] + page - 1) // page)[..., None]))
    st["len"].copy_(left)
    _slide(st)
    return dict(_pool_state(st), path=path, n_path=n_path, next=nxt)


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _depths(parent):
    d = np.zeros(parent.shape, np.int64)
    for i in range(parent.shape[1]):
        p = parent[:, i]
        d[:, i] = np.where(p < 0, 0, d[np.arange(len(p)), np.maximum(p, 0)] + 1)
    return d


def exact(case, seed):
    if case["op"] not in ("window", "tree"):
        return None  # whole numbers and bytes
    st = prepare(case, seed)
    B, Hkv, D, T, G, page = (case[x] for x in ("B", "Hkv", "D", "T", "G", "page"))
    w, k = case["window"], case["sinks"]
    q = st["q"].double()
    o = torch.zeros((B, T, Hkv * G, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, Hkv * G), -math.inf, dtype=torch.float64, device="cuda")
    mags = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    blocks = st["data"].view(-1, page // 16, 18 * D)
    if case["op"] == "tree":
        parent = _parents(case, seed)
        depth = _depths(parent)
        up = np.zeros((B, T, T), bool)
        for i in range(T):
            for b in range(B):
                if parent[b, i] >= 0:
                    up[b, i] = up[b, parent[b, i]]
                up[b, i, i] = True
    for b in range(B):
        for h in range(Hkv):
            n = int(st["len"][0, b, h])
            raw = blocks[st["table"][0, b, h, :_pages(n, page)].long()].reshape(-1, 18 * D)
            kv = []
            for half, ts in ((0, st["k_scale"]), (9 * D, st["v_scale"])):
                c = raw[:, half:half + 8 * D].reshape(-1, D // 2).long()
                sb = raw[:, half + 8 * D:half + 9 * D].reshape(-1, D // 16).long()
                ex, ma = (sb >> 3) & 15, sb & 7
                sc = torch.where(ex > 0, torch.exp2(ex.double() - 7) * (1 + ma.double() / 8), ma.double() / 512)
                x = torch.empty((c.shape[0], D), dtype=torch.float64, device="cuda")
                for par, code in ((0, c % 16), (1, c // 16)):
                    x[:, par::2] = torch.where(code >= 8, -mags[code % 8], mags[code % 8])
                kv.append((x.view(-1, D // 16, 16) * (sc * ts)[..., None]).view(-1, D)[:n])
            base = n - T
            j = torch.arange(n, device="cuda")[None]
            if case["op"] == "window":
                pos = base + torch.arange(T, device="cuda")[:, None]
                seen = (j <= pos) & ((j < k) | (pos - j < w))
            else:
                dep = torch.from_numpy(depth[b]).cuda()[:, None]
                seen = (j < base).expand(T, n)
                if w:
                    seen = seen & ((j < k) | (base + dep - j < w))
                seen = seen.clone()
                for u in range(max(0, -base), T):
                    see = torch.from_numpy(up[b, :, u]).cuda()
                    seen[:, base + u] = see & (dep[:, 0] - int(depth[b, u]) < w) if w else see
            step = max(1, (1 << 28) // (8 * G * max(n, 1)))
            for t in range(0, T, step):
                s = torch.einsum("tgd,nd->tgn", q[b, t:t + step, h * G:(h + 1) * G], kv[0]) / math.sqrt(D)
                s = s.masked_fill(~seen[t:t + step, None], -math.inf)
                z = torch.logsumexp(s, -1)
                lse[b, t:t + step, h * G:(h + 1) * G] = z
                p = torch.exp(s - torch.where(torch.isinf(z), 0.0, z)[..., None])
                o[b, t:t + step, h * G:(h + 1) * G] = torch.einsum("tgn,nd->tgd", p, kv[1])
    return o, lse
