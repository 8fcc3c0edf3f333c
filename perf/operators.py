"""Measured cases of the shared-prefix tree attention and of the paged cache's page
operators: their inputs, their plain forms in elementary torch operations, and
the calls of librd that compute the same.

  attend   tree attention of a batch whose groups of requests share a long
           prefix (the same leading pages of the cache)
  resize   rows of the cache grow and shrink: pages taken and given back
  fork     requests branch: full pages shared, the last partial page copied
  copy     pages of the pools copied by a list of (source, destination)
  compact  live pages moved to the lowest ids, tables rewritten
"""
import math

import numpy as np
import torch

own = False                     # run() calls librd instead of the plain forms

DEV = "cuda"

# ------------------------------------------------------------------------ cases
def _attend(name, B, W, L, Hq, Hkv, D, page, groups, prefix, suffix):
    return dict(name=name, op="attend", B=B, W=W, L=L, Hq=Hq, Hkv=Hkv, D=D, page=page,
                groups=groups, prefix=prefix, suffix=suffix)


def _pages(name, op, rows, pages, page, Hkv, D, layers, n, ctx):
    return dict(name=name, op=op, rows=rows, pages=pages, page=page, Hkv=Hkv, D=D, layers=layers,
                n=n, ctx=ctx)


def listed():
    return [
        # eight chats behind one system prompt, one token each: a call of latency
        _attend("attend token b8", 8, 1, 1, 32, 8, 128, 64, 1, 2048, 128),
        # four answers to one prompt, five beams of four tokens each
        _attend("attend tree 7b b4", 4, 5, 4, 32, 32, 128, 64, 1, 2048, 64),
        # a serving batch of drafts behind three prompts of a ragged number of pages
        _attend("attend tree 8b b16", 16, 8, 5, 32, 8, 128, 64, 3, 4032, 700),
        # small heads in groups of five, an odd batch, groups of two or three
        _attend("attend d64 b13", 13, 4, 4, 40, 8, 64, 64, 5, 1088, 333),
        # the large batch of drafts, every request behind one long prompt
        _attend("attend tree 13b b64", 64, 8, 6, 40, 40, 128, 256, 1, 8192, 300),
        # the scheduler's step of a small and of a large batch (tables only)
        _pages("resize r16", "resize", 16, 4096, 64, 8, 128, 1, 0, 4096),
        _pages("resize r1000", "resize", 1000, 65536, 64, 8, 128, 1, 0, 3000),
        # a few requests branch once; a batch branches through all layers of a cache
        _pages("fork n5", "fork", 32, 1024, 64, 8, 128, 1, 5, 1000),
        _pages("fork n200", "fork", 512, 2500, 64, 8, 128, 6, 200, 500),
        # copies on write of a few pages, and of a hundred pages of every layer
        _pages("copy n12", "copy", 1, 512, 64, 8, 128, 1, 12, 0),
        _pages("copy n300", "copy", 1, 1200, 64, 8, 128, 8, 300, 0),
        # a fragmented pool of several layers after many requests have left
        _pages("compact p2000", "compact", 100, 2000, 64, 8, 128, 4, 0, 1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "resize", "fork", "copy", "compact"])
    if op == "attend":
        Hkv = rng.choice([1, 2, 4, 8, 16, 32])
        G = rng.choice([1, 2, 3, 4, 5, 8])
        if Hkv * G > 40:
            G = 1
        B = _log(rng, 1, 64)
        W, L = rng.choice([(1, 1), (2, 3), (4, 4), (5, 4), (8, 5), (8, 6)])
        page = rng.choice([64, 128, 256])
        return dict(op=op, B=B, W=W, L=L, Hq=Hkv * G, Hkv=Hkv, D=rng.choice([64, 128, 128]),
                    page=page, groups=rng.randint(1, max(1, B // 2)), prefix=_log(rng, 64, 8192) // page * page,
                    suffix=_log(rng, 1, 1000))
    page, Hkv, D = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    if op == "resize":
        rows = _log(rng, 1, 1000)
        return dict(op=op, rows=rows, pages=rows * 64 + rng.randint(0, 999), page=page, Hkv=Hkv, D=D,
                    layers=1, n=0, ctx=_log(rng, 60, 3000))
    layers = rng.randint(1, 6)
    if op == "copy":
        n = _log(rng, 1, 250)
        return dict(op=op, rows=1, pages=2 * n + rng.randint(1, 500), page=page, Hkv=Hkv, D=D, layers=layers,
                    n=n, ctx=0)
    if op == "fork":
        n = _log(rng, 1, 200)
        return dict(op=op, rows=2 * n + rng.randint(0, 9), pages=n * 10 + rng.randint(10, 99), page=page, Hkv=Hkv,
                    D=D, layers=layers, n=n, ctx=_log(rng, 30, 500))
    pages = _log(rng, 50, 2000)
    return dict(op=op, rows=max(1, pages // 20), pages=pages, page=page, Hkv=Hkv, D=D, layers=layers, n=0,
                ctx=_log(rng, 60, 1000))


# ----------------------------------------------------------------------- inputs
def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device=DEV)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)


def _trees(rng, B, W, L, P):
    """Packed lengths and ancestor bits of B random draft tries: each beam copies
    its predecessor down to a random depth, then goes on alone."""
    lens = np.zeros(B, np.int64)
    anc = np.zeros((B, P, P), bool)
    for b in range(B):
        path = []
        for w in range(W):
            keep = 0 if w == 0 else int(rng.integers(1, L + 1))
            path = path[:keep]
            while len(path) < L:
                k = int(lens[b])
                lens[b] += 1
                path.append(k)
                anc[b, k, path] = True
    return lens, anc


def _attend_layout(c, rng):
    """Lengths, groups and tables: each group's requests name the same leading
    pages, and own the rest; page ids are shuffled over the pool."""
    B, page = c["B"], c["page"]
    cuts = np.sort(rng.choice(np.arange(1, B), c["groups"] - 1, replace=False)) if c["groups"] > 1 else np.zeros(0)
    offsets = np.concatenate([[0], cuts, [B]]).astype(np.int64)
    longest = c["prefix"] // page
    pre = np.array([longest if g == 0 else int(rng.integers(longest // 2, longest + 1))
                    for g in range(c["groups"])], np.int64)
    group = np.repeat(np.arange(c["groups"]), np.diff(offsets))
    ctx = pre[group] * page + rng.integers(0, c["suffix"] + 1, B)
    if B > 2:                                  # one request has nothing of its own
        b = int(rng.integers(0, B))
        ctx[b] = pre[group[b]] * page
    need = -(-ctx // page)
    total = int(pre.sum() + (need - pre[group]).sum())
    ids = rng.permutation(total + 3)[:total]
    shared = np.split(ids[:int(pre.sum())], np.cumsum(pre)[:-1])
    table = np.full((B, max(1, int(need.max()))), -1, np.int64)
    at = int(pre.sum())
    for b in range(B):
        k, n = int(pre[group[b]]), int(need[b])
        table[b, :k] = shared[group[b]]
        table[b, k:n] = ids[at:at + n - k]
        at += n - k
    return offsets, pre, ctx, table, total + 3


def _prepare_attend(c, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    B, P, Hq, Hkv, D = c["B"], c["W"] * c["L"], c["Hq"], c["Hkv"], c["D"]
    lens, anc = _trees(rng, B, c["W"], c["L"], P)
    words = np.zeros((B, P, (P + 31) // 32 * 32), bool)
    words[:, :, :P] = anc
    mask = np.packbits(words.reshape(B, P, -1, 32), axis=-1, bitorder="little").view(np.uint32)[..., 0]
    offsets, pre, ctx, table, pages = _attend_layout(c, rng)
    return dict(op="attend", page=c["page"], max_ctx=int(ctx.max()),
                q=_randn(gen, B, P, Hq, D), k_new=_randn(gen, B, P, Hkv, D), v_new=_randn(gen, B, P, Hkv, D),
                k_pool=_randn(gen, pages, c["page"], Hkv, D), v_pool=_randn(gen, pages, c["page"], Hkv, D),
                table=_i32(table), ctx=_i32(ctx), offsets=_i32(offsets), prefix_pages=_i32(pre),
                lens=_i32(lens), mask=_i32(mask.view(np.int32)), anc=torch.as_tensor(anc, device=DEV))


def _cache(c, rng, rows_held):
    """Tables of a cache in use: row r holds rows_held[r] pages of a shuffled pool
    (fewer where the pool ends)."""
    ids = rng.permutation(c["pages"])
    ends = np.minimum(np.cumsum(rows_held), c["pages"])
    held = np.diff(np.concatenate([[0], ends]))
    width = 8 + 2 * (c["ctx"] // c["page"])
    table = np.full((c["rows"], width), -1, np.int64)
    refs = np.zeros(c["pages"], np.int64)
    at = 0
    for r in range(c["rows"]):
        k = min(int(held[r]), width)
        table[r, :k] = ids[at:at + k]
        refs[ids[at:at + k]] = 1
        held[r] = k
        at += k
    return table, held, refs


def _prepare_pages(c, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rows, page = c["rows"], c["page"]
    s = dict(op=c["op"], page=page)
    most = max(1, -(-c["ctx"] // page))
    ctx = rng.integers(1, max(2, c["ctx"] + 1), rows)
    if c["op"] == "resize":
        # three rows of four run on, some by a page; the others' requests have ended
        held = -(-ctx // page)
        table, held, refs = _cache(c, rng, np.minimum(held, max(1, c["pages"] // (2 * rows))))
        grow = np.maximum(0, held * page - rng.integers(0, page, rows)) + rng.integers(0, page, rows)
        kind = rng.integers(0, 8, rows)
        s["new_lens"] = _i32(np.where(kind < 2, 0, np.where(kind == 2, -1, grow)))
        tables = [table, held, refs]
    elif c["op"] == "fork":
        # the first rows are in use, the others empty; every child is an empty row
        live = max(1, rows - c["n"])
        held = np.where(np.arange(rows) < live, -(-ctx // page), 0)
        table, held, refs = _cache(c, rng, np.minimum(held, max(1, (c["pages"] - c["n"]) // live)))
        ctx = np.where(np.arange(rows) < live, np.minimum(ctx, held * page), 0)
        n = min(c["n"], rows - live)
        s["parent"] = _i32(rng.integers(0, live, n))
        s["child"] = _i32(live + rng.permutation(rows - live)[:n])
        tables = [table, held, refs, ctx]
    elif c["op"] == "copy":
        ids = rng.permutation(c["pages"])
        s["src"], s["dst"] = _i32(ids[:c["n"]]), _i32(ids[c["n"]:2 * c["n"]])
        tables = []
    else:
        # rows hold half of the pool, at random places; some pages are held twice
        held = rng.integers(1, most + 1, rows)
        table, held, refs = _cache(c, rng, np.minimum(held, max(1, c["pages"] // (2 * rows))))
        twin = np.flatnonzero(held[:-1] * held[1:])[::3]
        table[twin + 1, 0], old = table[twin, 0], table[twin + 1, 0]
        np.subtract.at(refs, old, 1)
        np.add.at(refs, table[twin, 0], 1)
        tables = [table, held, refs]
    if tables:
        # the tables as they were before the step, and the ones that it changes,
        # each set in one buffer
        flat = np.concatenate([t.reshape(-1) for t in tables])
        s["before"], s["now"] = _i32(flat), _i32(flat)
        at = np.cumsum([0] + [t.size for t in tables])
        names = ("table", "held", "refs", "ctx")
        for k, t in enumerate(tables):
            for set_, tag in (("before", "0"), ("now", "")):
                s[names[k] + tag] = s[set_][int(at[k]):int(at[k + 1])].view(t.shape)
    if c["op"] != "resize":
        for n in ("k_pool", "v_pool"):
            s[n] = _randn(gen, c["layers"], c["pages"], page, c["Hkv"], c["D"])
    return s


def prepare(case, seed):
    return _prepare_attend(case, seed) if case["op"] == "attend" else _prepare_pages(case, seed)


# ------------------------------------------------------------------ plain forms
def _plain_attend(s, dtype=torch.float32):
    B, P, Hq, D = s["q"].shape
    Hkv, page = s["k_new"].shape[2], s["page"]
    G = Hq // Hkv
    rows = s["table"].clamp(min=0).long()
    C = rows.shape[1] * page
    kc, vc = (s[n][rows].reshape(B, C, Hkv, D) for n in ("k_pool", "v_pool"))
    # [B, Hkv, keys, D]: the context, then the packed drafts
    k, v = (torch.cat([a, b], 1).transpose(1, 2).to(dtype) for a, b in ((kc, s["k_new"]), (vc, s["v_new"])))
    q = s["q"].to(dtype).view(B, P, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, P * G, D)
    x = q @ k.transpose(2, 3) / math.sqrt(D)
    seen = torch.cat([(torch.arange(C, device=DEV) < s["ctx"][:, None])[:, None].expand(B, P, C), s["anc"]], 2)
    real = (torch.arange(P, device=DEV) < s["lens"][:, None])[:, :, None]
    seen = (seen & real).repeat_interleave(G, 1)[:, None]
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    o = (e @ v) / e.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.view(B, Hkv, P, G, D).permute(0, 2, 1, 3, 4).reshape(B, P, Hq, D)


def _free_first(refs):
    """Page ids, the free ones first and in ascending order."""
    return torch.argsort((refs != 0).int(), stable=True)


def _plain_resize(s):
    table, held, refs = s["table0"].long(), s["held0"].long(), s["refs0"].long()
    n, j = s["new_lens"].long(), torch.arange(table.shape[1], device=DEV)
    want = torch.where(n < 0, held, (n + s["page"] - 1) // s["page"])
    out = (j >= want[:, None]) & (j < held[:, None])
    refs = refs.index_add(0, table.clamp(min=0).reshape(-1), -out.reshape(-1).long())
    table = torch.where(out, -1, table)
    more = (want - held).clamp(min=0)
    first = torch.cumsum(more, 0) - more
    new = (j >= held[:, None]) & (j < want[:, None])
    take = (first[:, None] + j - held[:, None]).clamp(0, refs.numel() - 1)
    pages = _free_first(refs)[take]
    table = torch.where(new, pages, table)
    refs = refs.index_add(0, pages.reshape(-1), new.reshape(-1).long())
    return [table.int(), want.int(), refs.int()]


def _plain_fork(s):
    table, held, refs, ctx = (s[n + "0"].long() for n in ("table", "held", "refs", "ctx"))
    par, kid, page = s["parent"].long(), s["child"].long(), s["page"]
    j = torch.arange(table.shape[1], device=DEV)
    full, part = ctx[par] // page, ctx[par] % page
    tail = (part > 0).long()
    pages = _free_first(refs)[(torch.cumsum(tail, 0) - tail)]
    last = table[par].gather(1, full[:, None].clamp(max=table.shape[1] - 1))[:, 0].clamp(min=0)
    shared = j < full[:, None]
    row = torch.where(shared, table[par], -1)
    row = torch.where((j == full[:, None]) & (tail[:, None] > 0), pages[:, None], row)
    refs = refs.index_add(0, row.clamp(min=0).reshape(-1), (row >= 0).reshape(-1).long())
    table = table.index_copy(0, kid, row)
    held, ctx = held.index_copy(0, kid, full + tail), ctx.index_copy(0, kid, ctx[par])
    # the used positions of each last page; the others are copied onto themselves
    pos = torch.arange(page, device=DEV)
    to = pages[:, None] * page + pos
    keep = (pos < part[:, None])
    live = keep.any(1)
    to, src = to[live], torch.where(keep, last[:, None] * page + pos, to)[live]
    for n in ("k_pool", "v_pool"):
        flat = s[n].view(s[n].shape[0], -1, s[n].shape[3] * s[n].shape[4])
        flat[:, to] = flat[:, src]
    return [table.int(), held.int(), refs.int(), ctx.int(), _bits(s["k_pool"]), _bits(s["v_pool"])]


def _plain_copy(s):
    for n in ("k_pool", "v_pool"):
        s[n][:, s["dst"].long()] = s[n][:, s["src"].long()]
    return [_bits(s["k_pool"]), _bits(s["v_pool"])]


def _plain_compact(s):
    table, held, refs = s["table0"].long(), s["held0"].long(), s["refs0"].long()
    live = refs > 0
    n, ids = live.sum(), torch.arange(refs.numel(), device=DEV)
    to = torch.nonzero(~live & (ids < n))[:, 0]
    src = torch.nonzero(live & (ids >= n))[:, 0]
    remap = torch.where(live, ids, -1).index_copy(0, src, to)
    refs = refs.index_copy(0, to, refs[src]).index_fill(0, src, 0)
    mine = torch.arange(table.shape[1], device=DEV) < held[:, None]
    table = torch.where(mine, remap[table.clamp(min=0)], table)
    for name in ("k_pool", "v_pool"):
        s[name][:, to] = s[name][:, src]
    return [table.int(), refs.int(), remap.int(), n.int().view(1), _bits(s["k_pool"]), _bits(s["v_pool"])]


def _bits(t):
    return t.view(torch.int16)


# ------------------------------------------------------------- the library's calls
def _own(s):
    import tree_attention_verify_gb300 as rd
    if s["op"] == "attend":
        if "workspace" not in s:
            B, P, Hq, D = s["q"].shape
            size = rd.rd_tree_attention_shared_workspace_size(B, P, Hq, s["k_new"].shape[2], D, s["max_ctx"],
                                                              s["offsets"].numel() - 1, s["q"].device)
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device=s["q"].device)
        return rd.rd_tree_attention_shared(s["q"], s["k_new"], s["v_new"], s["k_pool"], s["v_pool"], s["table"],
                                           s["ctx"], s["offsets"], s["prefix_pages"], s["lens"], s["mask"],
                                           max_ctx=s["max_ctx"], workspace=s["workspace"])
    if s["op"] == "copy":
        rd.rd_copy_pages(s["k_pool"], s["v_pool"], s["src"], s["dst"])
        return [_bits(s["k_pool"]), _bits(s["v_pool"])]
    s["now"].copy_(s["before"])          # the tables as the step finds them
    if s["op"] == "resize":
        rd.rd_resize_pages(s["table"], s["held"], s["refs"], s["new_lens"], s["page"])
        return [s["table"], s["held"], s["refs"]]
    if s["op"] == "fork":
        rd.rd_fork_pages(s["k_pool"], s["v_pool"], s["table"], s["held"], s["refs"], s["ctx"], s["parent"],
                         s["child"])
        return [s["table"], s["held"], s["refs"], s["ctx"], _bits(s["k_pool"]), _bits(s["v_pool"])]
    remap, n_live = rd.rd_compact_pages(s["k_pool"], s["v_pool"], s["table"], s["held"], s["refs"])
    return [s["table"], s["refs"], remap, n_live, _bits(s["k_pool"]), _bits(s["v_pool"])]


def run(state):
    if own:
        return _own(state)
    if state["op"] == "attend":
        return _plain_attend(state).to(torch.bfloat16)
    return dict(resize=_plain_resize, fork=_plain_fork, copy=_plain_copy, compact=_plain_compact)[state["op"]](state)


# ------------------------------------------------------------------------- work
def _rows(c, what):
    """A seed's own counts of what a pass touches (they vary little over seeds)."""
    rng = np.random.default_rng(1)
    if what == "attend":
        lens, anc = _trees(rng, c["B"], c["W"], c["L"], c["W"] * c["L"])
        offsets, pre, ctx, _, _ = _attend_layout(c, rng)
        return lens, anc.sum((1, 2)), offsets, pre, ctx
    return rng


def work(case):
    c = case
    if c["op"] == "attend":
        lens, pairs, offsets, pre, ctx = _rows(c, "attend")
        Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
        group = np.repeat(np.arange(c["groups"]), np.diff(offsets))
        own_rows = (ctx - pre[group] * page).sum() + pre.sum() * page
        return dict(bytes=float(4 * Hkv * D * (own_rows + lens.sum()) + 2 * Hq * D * (lens.sum() + c["B"] * c["W"] * c["L"])),
                    flops=float(4 * Hq * D * ((lens * ctx).sum() + pairs.sum())))
    page_bytes = c["page"] * c["Hkv"] * c["D"] * 2 * 2 * c["layers"]          # K and V, every layer
    if c["op"] == "copy":
        return dict(bytes=float(2 * page_bytes * c["n"] + 8 * c["n"]), flops=0.0)
    held = min(max(1, (c["ctx"] + c["page"]) // (2 * c["page"])), max(1, c["pages"] // (2 * c["rows"])))
    tables = 4 * (2 * c["pages"] + 2 * c["rows"])
    if c["op"] == "resize":
        return dict(bytes=float(tables + 8 * c["rows"] * (1 + held // 4)), flops=0.0)
    if c["op"] == "fork":
        return dict(bytes=float(tables + c["n"] * (page_bytes + 8 * held)), flops=0.0)
    moved = held * c["rows"] * (1 - min(1.0, held * c["rows"] / c["pages"]))
    return dict(bytes=float(tables + 8 * held * c["rows"] + 2 * page_bytes * moved), flops=0.0)


# ------------------------------------------------------------------------ exact
def exact(case, seed):
    """Attention from its definition in 64 bits, request by request; the page
    operators give whole numbers and copies, which have no nearer value."""
    if case["op"] != "attend":
        return None
    s = prepare(case, seed)
    B, P, Hq, D = s["q"].shape
    Hkv, page = s["k_new"].shape[2], s["page"]
    out = torch.zeros(B, P, Hq, D, dtype=torch.float64, device=DEV)
    head = torch.arange(Hq, device=DEV) // (Hq // Hkv)
    for b in range(B):
        n, c = int(s["lens"][b]), int(s["ctx"][b])
        at = torch.arange(c, device=DEV)
        cells = s["table"][b, at // page].long(), at % page
        keys = torch.cat([s["k_pool"][cells], s["k_new"][b, :n]]).double()
        values = torch.cat([s["v_pool"][cells], s["v_new"][b, :n]]).double()
        for h0 in range(0, Hq, 8):
            hs = head[h0:h0 + 8]
            w = torch.einsum("phd,khd->hpk", s["q"][b, :n, h0:h0 + 8].double(), keys[:, hs]) * D ** -0.5
            w[:, :, c:][:, ~s["anc"][b, :n, :n]] = -math.inf
            out[b, :n, h0:h0 + 8] = torch.einsum("hpk,khd->phd", torch.softmax(w, -1), values[:, hs])
    return out
