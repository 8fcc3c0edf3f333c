"""Measured cases of the quantised paged cache (what writes it, reads it back and
attends to it, in 4 and in 8 bits) and of the log probabilities of tokens: their
inputs, their plain forms in elementary torch operations, and the calls of librd
that compute the same.

  attend    tree attention over the quantised pages and the packed drafts
  append    keys and values of prompt tokens quantised into the pages, and read back
  commit    the same for the accepted path of a verification step
  read      whole contexts of the cache read back in 16 bits
  logprobs  log probabilities of given tokens, entropies and top alternatives

A row of the cache is one position of one kv head.  In 8 bits it is D e4m3 codes c
that stand for g c; in 4 bits D / 2 bytes of e2m1 codes (element 2 j in the low
half) and an e4m3 scale s for each block of 16, and c stands for g s c.  g is the
tensor's scale.
"""
import math

import numpy as np
import torch

own = False                     # run() calls librd instead of the plain forms

DEV = "cuda"


# ------------------------------------------------------------------------ cases
def _attend(name, B, W, L, Hq, Hkv, D, page, low, high, bits):
    return dict(name=name, op="attend", B=B, W=W, L=L, Hq=Hq, Hkv=Hkv, D=D, page=page, low=low, high=high,
                bits=bits)


def _cache(name, op, B, tokens, ctx, Hkv, D, page, bits):
    return dict(name=name, op=op, B=B, tokens=tokens, ctx=ctx, Hkv=Hkv, D=D, page=page, bits=bits)


def _logprobs(name, B, W, L, V, top, temperature, dtype):
    return dict(name=name, op="logprobs", B=B, W=W, L=L, V=V, top=top, temperature=temperature, dtype=dtype)


def listed():
    return [
        # eight chats, one token each: a call of latency
        _attend("attend token b8", 8, 1, 1, 32, 8, 128, 64, 1500, 2500, 4),
        # a serving batch of drafts, grouped heads, ragged contexts
        _attend("attend tree 8b b16", 16, 8, 5, 32, 8, 128, 64, 1024, 4096, 4),
        # two long documents in 8 bits, small heads in groups of five
        _attend("attend long d64 b2", 2, 4, 4, 40, 8, 64, 128, 30000, 50001, 8),
        # the large batch of drafts
        _attend("attend tree 13b b64", 64, 8, 6, 40, 40, 128, 256, 8192, 8192, 4),
        # one short prompt
        _cache("append b1", "append", 1, 57, 0, 8, 128, 64, 4),
        # the context half of an in-flight batch, some behind a cached prompt
        _cache("append b32", "append", 32, 512, 700, 8, 128, 64, 4),
        # the accepted paths of the large batch: up to six tokens a request
        _cache("commit b64", "commit", 64, 6, 8192, 40, 128, 64, 4),
        # contexts read back for a call that takes 16 bits
        _cache("read b16", "read", 16, 4096, 0, 8, 128, 64, 4),
        _cache("read 8 bits b8", "read", 8, 8192, 0, 40, 128, 256, 8),
        # four rows of a sampler, in 32 bits
        _logprobs("logprobs rows4", 4, 0, 0, 32000, 0, 0.7, "float32"),
        # the emitted tokens of the large batch, with five alternatives
        _logprobs("logprobs accepted b64", 64, 8, 6, 32000, 5, 1.0, "bfloat16"),
        # every token of prompts scored, with twenty alternatives
        _logprobs("logprobs prompt 4096", 4096, 0, 0, 128256, 20, 1.0, "bfloat16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "commit", "read", "logprobs", "logprobs"])
    if op == "logprobs":
        top, dtype = rng.choice([0, 1, 5, 8, 20, 32]), rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
        V = _log(rng, 300, 150000)
        if rng.random() < 0.3:
            W, L = rng.choice([(2, 3), (4, 4), (5, 4), (8, 5)])
            return dict(op=op, B=_log(rng, 1, 48), W=W, L=L, V=V, top=top, temperature=1.0, dtype="bfloat16")
        rows = _log(rng, 1, 4096)
        if rows * V > 2 ** 28:
            rows = 2 ** 28 // V
        return dict(op=op, B=rows, W=0, L=0, V=V, top=top, temperature=rng.choice([1.0, 0.5, 1.3]), dtype=dtype)
    bits, page, D = rng.choice([4, 4, 8]), rng.choice([64, 128, 256]), rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 32, 40])
    if op == "attend":
        G = rng.choice([1, 2, 3, 4, 5, 8])
        if Hkv * G > 40:
            G = 1
        B, high = _log(rng, 1, 64), _log(rng, 1, 60000)
        while B * high * Hkv * G > 2 ** 23:
            B, high = (B + 1) // 2, (high + 1) // 2
        W, L = rng.choice([(1, 1), (1, 1), (2, 3), (4, 4), (5, 4), (8, 5), (8, 6)])
        return dict(op=op, B=B, W=W, L=L, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, low=rng.randint(0, high), high=high,
                    bits=bits)
    if op == "commit":
        return dict(op=op, B=_log(rng, 1, 64), tokens=rng.randint(1, 6), ctx=_log(rng, 1, 2000), Hkv=Hkv, D=D,
                    page=page, bits=bits)
    B, tokens = _log(rng, 1, 32), _log(rng, 1, 6000)
    while B * tokens * Hkv > 2 ** 20:
        B, tokens = (B + 1) // 2, (tokens + 1) // 2
    return dict(op=op, B=B, tokens=tokens, ctx=_log(rng, 1, 1000) if op == "append" else 0, Hkv=Hkv, D=D, page=page,
                bits=bits)


# ---------------------------------------------------------- the cache's formats
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_MOST = {4: 6.0 * 448.0, 8: 448.0}      # the largest value of a row at scale 1


def _row_bytes(D, bits):
    return D if bits == 8 else D // 2 + D // 16


def _e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _quantise(x, g, bits, dtype=torch.float64):
    """Rows [..., D] -> (e4m3 scales, codes as values): what a row holds."""
    x = x.to(dtype)
    if bits == 8:
        return None, _e4m3((x / g).float()).to(dtype)
    x = x.reshape(*x.shape[:-1], -1, 16)
    s = _e4m3((x.abs().amax(-1, keepdim=True) / (6.0 * g)).float())
    d = s.to(dtype) * g
    y = torch.where(d > 0, x / torch.where(d > 0, d, torch.ones_like(d)), torch.zeros_like(x))
    a = y.abs()
    # to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6; a tie to the even code
    up = ((a > 0.25).to(dtype) + (a >= 0.75) + (a > 1.25) + (a >= 1.75)) * 0.5 + (a > 2.5) + (a >= 3.5) + 2.0 * (a > 5.0)
    return s, torch.copysign(up, y)


def _pack(x, g, bits):
    """Rows [..., D] -> bytes [..., row_bytes]."""
    s, c = _quantise(x, g, bits, torch.float32)
    if bits == 8:
        return c.to(torch.float8_e4m3fn).view(torch.uint8)
    a = c.abs()
    code = torch.where(a <= 2.0, a * 2.0, torch.where(a < 4.0, a + 2.0, a * 0.5 + 4.0)) + 8.0 * torch.signbit(c)
    code = code.to(torch.uint8).flatten(-2)
    return torch.cat([code[..., 0::2] | code[..., 1::2] << 4, s.squeeze(-1).view(torch.uint8)], -1)


def _values(rows, g, D, bits):
    """Bytes [..., row_bytes] -> the values that they stand for [..., D], in 32 bits."""
    if bits == 8:
        return rows.view(torch.float8_e4m3fn).float() * g
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=rows.device)
    codes, s = rows[..., :D // 2], rows[..., D // 2:].contiguous().view(torch.float8_e4m3fn).float()
    c = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).reshape(*rows.shape[:-1], D // 16, 16)
    return (c * s.unsqueeze(-1) * g).flatten(-2)


# ----------------------------------------------------------------------- inputs
def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32, device=DEV)


def _channels(gen, Hkv, D):
    """Keys and values differ in size from channel to channel."""
    return torch.exp(0.5 * torch.randn(Hkv, D, generator=gen, device=DEV))


def _randn(gen, *shape, by=None):
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
    return x if by is None else (x * by).to(torch.bfloat16)


def _trees(rng, B, W, L, P):
    """Packed lengths, ancestor bits and node of (beam, position) of B random draft
    tries: each beam copies its predecessor down to a random depth, then goes on alone."""
    lens = np.zeros(B, np.int64)
    anc = np.zeros((B, P, P), bool)
    node = np.zeros((B, W, L), np.int64)
    for b in range(B):
        path = []
        for w in range(W):
            path = path[:0 if w == 0 else int(rng.integers(1, L + 1))]
            while len(path) < L:
                k = int(lens[b])
                lens[b] += 1
                path.append(k)
                anc[b, k, path] = True
            node[b, w] = path
    return lens, anc, node


def _tables(rng, lens, page):
    """Block table of rows that hold ceil(lens / page) pages of a shuffled pool."""
    need = -(-lens // page)
    ids = rng.permutation(int(need.sum()) + 3)
    table = np.full((len(lens), max(1, int(need.max()))), -1, np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, int(need.sum()) + 3


def _pools(gen, pages, page, Hkv, D, bits, by, fill=True):
    """A pool of quantised rows and the scale it was calibrated to."""
    g = float(np.float32(6.0 * float(by.max()) / _MOST[bits]))      # a scale is a 32-bit number
    pool = torch.zeros(pages, page, Hkv, _row_bytes(D, bits), dtype=torch.uint8, device=DEV)
    step = max(1, 2 ** 26 // (page * Hkv * D))
    for i in range(0, pages if fill else 0, step):
        n = min(step, pages - i)
        pool[i:i + n] = _pack(_randn(gen, n, page, Hkv, D, by=by), g, bits)
    return pool, g


def _context(c, rng):
    """Lengths of the contexts in the cache, and of what the pass adds or reads."""
    B = c["B"]
    if c["op"] == "attend":
        ctx = rng.integers(c["low"], c["high"] + 1, B)
        return ctx, ctx
    ctx = rng.integers(c["ctx"] // 2, c["ctx"] + 1, B) if c["ctx"] else np.zeros(B, np.int64)
    new = np.random.default_rng(c["tokens"]).integers((c["tokens"] + 1) // 2, c["tokens"] + 1, B)
    new[0] = c["tokens"]                     # (the same for every seed: so many rows come out)
    return ctx, ctx + new


def _prepare_cache(c, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    B, Hkv, D, bits, op = c["B"], c["Hkv"], c["D"], c["bits"], c["op"]
    ctx, end = _context(c, rng)
    table, pages = _tables(rng, end, c["page"])
    s = dict(op=op, page=c["page"], D=D, bits=bits, table=_i32(table), ctx=_i32(ctx))
    kby, vby = _channels(gen, Hkv, D), _channels(gen, Hkv, D)
    fill = op in ("attend", "read")
    (s["k_pool"], s["gk"]), (s["v_pool"], s["gv"]) = (_pools(gen, pages, c["page"], Hkv, D, bits, by, fill)
                                                      for by in (kby, vby))
    if op == "attend":
        P = c["W"] * c["L"]
        lens, anc, _ = _trees(rng, B, c["W"], c["L"], P)
        words = np.zeros((B, P, (P + 31) // 32 * 32), bool)
        words[:, :, :P] = anc
        mask = np.packbits(words.reshape(B, P, -1, 32), axis=-1, bitorder="little").view(np.uint32)[..., 0]
        s.update(max_ctx=int(ctx.max()), q=_randn(gen, B, P, c["Hq"], D), k_new=_randn(gen, B, P, Hkv, D, by=kby),
                 v_new=_randn(gen, B, P, Hkv, D, by=vby), lens=_i32(lens), mask=_i32(mask.view(np.int32)),
                 anc=torch.as_tensor(anc, device=DEV))
        return s
    new = end - ctx
    cu = np.concatenate([[0], np.cumsum(new)])
    s.update(total=int(cu[-1]), cu=_i32(cu), offsets=torch.as_tensor(cu, dtype=torch.int64, device=DEV))
    # where each new token lies in the pools (the plain forms' indices)
    b = np.repeat(np.arange(B), new)
    pos = np.arange(int(cu[-1])) - cu[b] + ctx[b]
    s["slot"] = torch.as_tensor(table[b, pos // c["page"]] * c["page"] + pos % c["page"], device=DEV)
    s["new"] = _i32(new)
    if op == "append":
        s["k_new"], s["v_new"] = (_randn(gen, s["total"], Hkv, D, by=by) for by in (kby, vby))
    elif op == "commit":
        W, L = 8, c["tokens"]
        _, _, node = _trees(rng, B, W, L, W * L)
        best = rng.integers(0, W, B)
        s["k_new"], s["v_new"] = (_randn(gen, B, W * L, Hkv, D, by=by) for by in (kby, vby))
        s.update(unpacker=_i32(node), best=_i32(best), accepted=_i32(new - 1))
        i = np.arange(int(cu[-1])) - cu[b]
        s["source"] = torch.as_tensor(b * W * L + node[b, best[b], i], device=DEV)
    return s


def _prepare_logprobs(c, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    B, W, L, V, dtype = c["B"], c["W"], c["L"], c["V"], getattr(torch, c["dtype"])
    s = dict(op="logprobs", top=min(c["top"], V), temperature=c["temperature"], tree=W > 0)
    shape = (B, W * L, V) if W else (B, V)
    x = torch.empty(shape, dtype=dtype, device=DEV)
    flat = x.view(-1, V)
    step = max(1, 2 ** 27 // V)
    for i in range(0, flat.shape[0], step):
        part = flat[i:i + step]
        part.copy_(2.0 * torch.randn(part.shape, generator=gen, device=DEV))
    # a model's likely next token stands out, in most rows
    likely = torch.randint(0, V, (flat.shape[0],), generator=gen, device=DEV)
    flat[torch.arange(flat.shape[0], device=DEV), likely] = (
        12.0 + 3.0 * torch.randn(flat.shape[0], generator=gen, device=DEV)).to(dtype)
    s["logits"] = x
    other = torch.randint(0, V, (flat.shape[0],), generator=gen, device=DEV)
    token = torch.where(torch.rand(flat.shape[0], generator=gen, device=DEV) < 0.7, likely, other).int()
    if not W:
        s["tokens"] = token
        return s
    _, _, node = _trees(rng, B, W, L, W * L)
    best, n = rng.integers(0, W, B), rng.integers(0, L, B)
    row = np.arange(B)[:, None] * W * L + node[np.arange(B), best]
    live = np.arange(L)[None] <= n[:, None]
    s.update(unpacker=_i32(node), best=_i32(best), accepted=_i32(n), row=torch.as_tensor(row, device=DEV),
             live=torch.as_tensor(live, device=DEV))
    s["tokens"] = torch.where(s["live"], token[s["row"]], -1).int()
    return s


def prepare(case, seed):
    return _prepare_logprobs(case, seed) if case["op"] == "logprobs" else _prepare_cache(case, seed)


# ------------------------------------------------------------------ plain forms
def _plain_attend(s):
    B, P, Hq, D = s["q"].shape
    Hkv, page = s["k_new"].shape[2], s["page"]
    G, C = Hq // Hkv, s["table"].shape[1] * page
    out = torch.empty_like(s["q"])
    step = max(1, 2 ** 29 // (C * Hkv * max(D, P * G)))
    for b0 in range(0, B, step):
        b = slice(b0, b0 + step)
        rows, n = s["table"][b].clamp(min=0).long(), s["table"][b].shape[0]
        k, v = (torch.cat([_values(pool[rows].view(n, C, Hkv, -1), g, D, s["bits"]), new[b].float()], 1).transpose(1, 2)
                for pool, g, new in ((s["k_pool"], s["gk"], s["k_new"]), (s["v_pool"], s["gv"], s["v_new"])))
        q = s["q"][b].float().view(n, P, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(n, Hkv, P * G, D)
        x = q @ k.transpose(2, 3) / math.sqrt(D)
        seen = torch.cat([(torch.arange(C, device=DEV) < s["ctx"][b, None])[:, None].expand(n, P, C), s["anc"][b]], 2)
        real = (torch.arange(P, device=DEV) < s["lens"][b, None])[:, :, None]
        seen = (seen & real).repeat_interleave(G, 1)[:, None]
        x = x.masked_fill(~seen, -math.inf)
        top = x.amax(-1, keepdim=True)
        e = torch.exp(x - torch.where(top > -math.inf, top, torch.zeros_like(top)))
        o = (e @ v) / e.sum(-1, keepdim=True).clamp(min=1e-30)
        out[b] = o.view(n, Hkv, P, G, D).permute(0, 2, 1, 3, 4).reshape(n, P, Hq, D).to(out.dtype)
    return out


def _plain_write(s):
    """Each new row quantised (in 64 bits: values next to a border), stored, and read back."""
    out = []
    for name in ("k", "v"):
        x, pool, g = s[name + "_new"], s[name + "_pool"], s["g" + name]
        if s["op"] == "commit":
            x = x.flatten(0, 1)[s["source"]]
        rows = _pack_exactly(x, g, s["bits"])
        flat = pool.view(-1, *pool.shape[2:])
        flat[s["slot"]] = rows
        out.append(_values(flat[s["slot"]], g, s["D"], s["bits"]).to(torch.bfloat16))
    return out + [s["ctx"] + s["new"]]


def _pack_exactly(x, g, bits):
    scale, c = _quantise(x, g, bits, torch.float64)
    if bits == 8:
        return c.float().to(torch.float8_e4m3fn).view(torch.uint8)
    a = c.abs()
    code = torch.where(a <= 2.0, a * 2.0, torch.where(a < 4.0, a + 2.0, a * 0.5 + 4.0)) + 8.0 * torch.signbit(c)
    code = code.to(torch.uint8).flatten(-2)
    return torch.cat([code[..., 0::2] | code[..., 1::2] << 4, scale.squeeze(-1).view(torch.uint8)], -1)


def _plain_read(s):
    return [_values(pool.view(-1, *pool.shape[2:])[s["slot"]], g, s["D"], s["bits"]).to(torch.bfloat16)
            for pool, g in ((s["k_pool"], s["gk"]), (s["v_pool"], s["gv"]))]


def _plain_logprobs(s):
    x, V, k = s["logits"].view(-1, s["logits"].shape[-1]), s["logits"].shape[-1], s["top"]
    rows, tokens = (s["row"].flatten() if s["tree"] else torch.arange(x.shape[0], device=DEV)), s["tokens"].flatten()
    n = rows.numel()
    logp, ent = (torch.zeros(n, device=DEV) for _ in range(2))
    top = torch.full((n, k), -1, dtype=torch.int32, device=DEV)
    top_logp = torch.zeros(n, k, device=DEV)
    step = max(1, 2 ** 28 // V)
    for i in range(0, n, step):
        part, t = x[rows[i:i + step]].float(), tokens[i:i + step].long()
        live = t >= 0
        z = (part - part.amax(1, keepdim=True)) / s["temperature"]
        e = torch.exp(z)
        total = e.sum(1)
        lse = torch.log(total)
        logp[i:i + step] = torch.where(live, z.gather(1, t.clamp(min=0)[:, None])[:, 0] - lse, 0.0)
        ent[i:i + step] = torch.where(live, lse - (e * z).sum(1) / total, 0.0)
        if k:
            # values as whole numbers of the same order, the lower index first among equals
            bits = (part + 0.0).view(torch.int32).long()
            key = torch.where(bits >= 0, bits, -2 ** 31 - bits - 1) * 2 ** 32 + (V - torch.arange(V, device=DEV))
            ids = V - (key.topk(k, 1).values % 2 ** 32)
            top[i:i + step] = torch.where(live[:, None], ids, -1).int()
            top_logp[i:i + step] = torch.where(live[:, None], z.gather(1, ids) - lse[:, None], 0.0)
    shape = s["tokens"].shape
    return [logp.view(shape), ent.view(shape)] + ([top.view(*shape, k), top_logp.view(*shape, k)] if k else [])


# ------------------------------------------------------------- the library's calls
def _own(s):
    import tree_attention_verify_gb300 as rd
    if s["op"] == "attend":
        if "workspace" not in s:
            B, P, Hq, D = s["q"].shape
            size = rd.rd_tree_attention_quant_workspace_size(B, P, Hq, s["k_new"].shape[2], D, s["max_ctx"],
                                                             s["q"].device)
            s["workspace"] = torch.empty(max(16, size), dtype=torch.uint8, device=s["q"].device)
        return rd.rd_tree_attention_quant(s["q"], s["k_new"], s["v_new"], s["k_pool"], s["v_pool"], s["gk"], s["gv"],
                                          s["table"], s["ctx"], s["lens"], s["mask"], max_ctx=s["max_ctx"],
                                          workspace=s["workspace"])
    if s["op"] == "logprobs":
        if s["tree"]:
            out = rd.rd_accepted_logprobs(s["logits"], s["unpacker"], s["best"], s["accepted"], s["tokens"],
                                          top=s["top"], temperature=s["temperature"])
        else:
            out = rd.rd_token_logprobs(s["logits"], s["tokens"], top=s["top"], temperature=s["temperature"])
        return [out["logprob"], out["entropy"]] + ([out["top_tokens"], out["top_logprobs"]] if s["top"] else [])
    more = []
    if s["op"] == "append":
        more = [rd.rd_append_quant(s["k_new"], s["v_new"], s["cu"], s["k_pool"], s["v_pool"], s["gk"], s["gv"],
                                   s["table"], s["ctx"])]
    elif s["op"] == "commit":
        more = [rd.rd_commit_accepted_quant(s["k_new"], s["v_new"], s["unpacker"], s["best"], s["accepted"],
                                            s["k_pool"], s["v_pool"], s["gk"], s["gv"], s["table"], s["ctx"])]
    k, v = rd.rd_read_quant(s["k_pool"], s["v_pool"], s["gk"], s["gv"], s["table"], s["offsets"], total=s["total"],
                            starts=s["ctx"])
    return [k, v] + more


def run(state):
    if own:
        return _own(state)
    return dict(attend=_plain_attend, append=_plain_write, commit=_plain_write, read=_plain_read,
                logprobs=_plain_logprobs)[state["op"]](state)


# ------------------------------------------------------------------------- work
def work(case):
    """A seed's own counts of what a pass touches (they vary little over seeds)."""
    c, rng = case, np.random.default_rng(1)
    if c["op"] == "logprobs":
        W, L, V, k = c["W"], c["L"], c["V"], min(c["top"], c["V"])
        rows, out = (c["B"] * (L + 1) / 2, c["B"] * L) if W else (c["B"], c["B"])
        size = 4 if c["dtype"] == "float32" else 2
        return dict(bytes=float(rows * V * size + out * (12 + 8 * k)), flops=float(4 * rows * V))
    ctx, end = _context(c, rng)
    Hkv, D, row = c["Hkv"], c["D"], _row_bytes(c["D"], c["bits"])
    if c["op"] == "attend":
        P, Hq = c["W"] * c["L"], c["Hq"]
        lens, anc, _ = _trees(rng, c["B"], c["W"], c["L"], P)
        return dict(bytes=float(2 * Hkv * row * ctx.sum() + 4 * Hkv * D * lens.sum() + 2 * Hq * D * (lens.sum() + c["B"] * P)),
                    flops=float(4 * Hq * D * ((lens * ctx).sum() + anc.sum())))
    n = int((end - ctx).sum())
    # written and read back: 16 bits in, the row out, the row in, 16 bits out; or the last two
    moved = (4 * D + row * 2 if c["op"] != "read" else 2 * D + row) * 2 * Hkv * n
    return dict(bytes=float(moved), flops=float((6 if c["op"] != "read" else 2) * 2 * Hkv * D * n))


# ------------------------------------------------------------------------ exact
def _decode(rows, D, bits):
    """The values of rows at tensor scale 1, from the formats' bits, in 64 bits."""
    def e4m3(b):
        b = b.long()
        e, m = (b >> 3) & 15, (b & 7).double()
        v = torch.where(e > 0, (8 + m) * torch.pow(2.0, (e - 10).double()), m * 2.0 ** -9)
        return torch.where(b > 127, -v, v)
    if bits == 8:
        return e4m3(rows)
    b = rows[..., :D // 2].long()
    n = torch.stack([b % 16, b // 16], -1).flatten(-2)
    e, m = (n >> 1) & 3, (n & 1).double()
    v = torch.where(e > 0, (2 + m) * torch.pow(2.0, (e - 2).double()), m / 2)
    return torch.where(n > 7, -v, v) * e4m3(rows[..., D // 2:]).repeat_interleave(16, -1)


def _exact_row(x, g, bits):
    """What a row of values is read back as: nearest representable values, in 64 bits."""
    x = x.double()
    positive = [(8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9 for e in range(16) for m in range(8)][:127]

    def nearest(y, grid):
        # the grid's points in ascending order stand at even and odd places: ties to even
        grid = torch.tensor(grid, dtype=torch.float64, device=y.device)
        mid = (grid[1:] + grid[:-1]) / 2
        a = y.abs().contiguous()
        low, high = torch.searchsorted(mid, a, right=False), torch.searchsorted(mid, a, right=True)
        i = torch.where(low % 2 == 0, low, high)
        return torch.copysign(grid[i], y)
    if bits == 8:
        return nearest(x / g, positive) * g
    blocks = x.unflatten(-1, (-1, 16))
    s = nearest(blocks.abs().amax(-1, keepdim=True) / 6.0 / g, positive)
    c = nearest(blocks / (s * g).clamp(min=1e-300), _E2M1)
    return (c * s * g).flatten(-2)


def exact(case, seed):
    """Each operator from its definition in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(s)
    if case["op"] == "logprobs":
        return _exact_logprobs(s)
    if case["op"] == "read":
        return [torch.cat([_decode(part, s["D"], s["bits"]) * g for part in pool.flatten(0, 1)[s["slot"]].split(8192)])
                for pool, g in ((s["k_pool"], s["gk"]), (s["v_pool"], s["gv"]))]
    out = []
    for name in ("k", "v"):
        x = s[name + "_new"]
        if case["op"] == "commit":
            x = x.view(-1, *x.shape[2:])[s["source"]]
        out.append(torch.cat([_exact_row(part, s["g" + name], s["bits"]) for part in x.split(8192)]))
    return out + [(s["ctx"] + s["new"])]


def _exact_attend(s):
    B, P, Hq, D = s["q"].shape
    Hkv, page = s["k_new"].shape[2], s["page"]
    out = torch.zeros(B, P, Hq, D, dtype=torch.float64, device=DEV)
    G = Hq // Hkv
    for b in range(B):
        n, c = int(s["lens"][b]), int(s["ctx"][b])
        at = torch.arange(c, device=DEV)
        cells = s["table"][b, at // page].long(), at % page
        for h in range(0, Hkv, 8):
            keys, values = (torch.cat([_decode(pool[cells][:, h:h + 8], D, s["bits"]) * g, new[b, :n, h:h + 8].double()])
                            for pool, g, new in ((s["k_pool"], s["gk"], s["k_new"]), (s["v_pool"], s["gv"], s["v_new"])))
            q = s["q"][b, :n, h * G:(h + 8) * G].double().unflatten(1, (-1, G))
            w = torch.einsum("phgd,khd->hgpk", q, keys) * D ** -0.5
            w[..., c:][:, :, ~s["anc"][b, :n, :n]] = -math.inf
            out[b, :n, h * G:(h + 8) * G] = torch.einsum("hgpk,khd->phgd", torch.softmax(w, -1), values).flatten(1, 2)
    return out


def _exact_logprobs(s):
    x, V, k = s["logits"].flatten(0, -2), s["logits"].shape[-1], s["top"]
    tokens = s["tokens"].flatten().long()
    rows = s["row"].flatten() if s["tree"] else torch.arange(len(tokens), device=DEV)
    n = len(tokens)
    logp, ent = (torch.zeros(n, dtype=torch.float64, device=DEV) for _ in range(2))
    ids = torch.full((n, k), -1, dtype=torch.int32, device=DEV)
    values = torch.zeros(n, k, dtype=torch.float64, device=DEV)
    live = torch.nonzero(tokens >= 0)[:, 0]
    for r in live.split(max(1, 2 ** 26 // V)):
        lp = torch.log_softmax(x[rows[r]].double() / s["temperature"], 1)
        logp[r] = lp.gather(1, tokens[r, None])[:, 0]
        ent[r] = -(lp.exp() * lp).sum(1)
        if k:
            order = torch.sort(x[rows[r]], dim=1, descending=True, stable=True).indices[:, :k]
            ids[r], values[r] = order.int(), lp.gather(1, order)
    shape = s["tokens"].shape
    return [logp.view(shape), ent.view(shape)] + ([ids.view(*shape, k), values.view(*shape, k)] if k else [])
