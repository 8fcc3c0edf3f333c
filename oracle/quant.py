"""Plain 64-bit numpy implementation of the quantised paged cache (formats, writing,
reading back, attention) and of the log probabilities of tokens.  One row, one
request, one entry at a time; nothing here is shared with the kernels."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
# the 127 finite magnitudes of e4m3, code by code
E4M3 = np.array([(8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9 for e in range(16) for m in range(8)][:127])


def row_bytes(D, bits):
    return D if bits == 8 else D // 2 + D // 16


def nearest_code(x, grid):
    """Code of the magnitude nearest to |x| (ties to the even code, saturating), and the
    distance of |x| from the nearest border between two codes, relative to that border."""
    a = np.abs(np.asarray(x, np.float64))
    mid = (grid[1:] + grid[:-1]) / 2
    low = np.searchsorted(mid, a, side="left")
    high = np.searchsorted(mid, a, side="right")
    code = np.where(low % 2 == 0, low, high)
    near = np.min(np.abs(a[..., None] - mid) / mid, axis=-1)
    return code, np.where(low != high, 0.0, near)


def e4m3_value(byte):
    byte = np.asarray(byte, np.int64)
    mag = np.append(E4M3, np.nan)[byte & 127]
    return np.where(byte & 128, -mag, mag)


def encode_row(x, g, bits):
    """Bytes of the row of values x [D], and its smallest distance from a border
    (relative; in 4 bits, exact ties do not count)."""
    x = np.asarray(x, np.float64)
    if bits == 8:
        code, near = nearest_code(x / g, E4M3)
        return (code + 128 * np.signbit(x)).astype(np.uint8), near.min()
    codes, scales, least = [], [], np.inf
    for block in x.reshape(-1, 16):
        s, near = nearest_code(min(448.0, np.abs(block).max() / (6 * g)), E4M3)
        d = E4M3[s] * g
        scales.append(int(s))
        if d == 0:
            codes += [0] * 16
            least = min(least, float(near))
            continue
        c, n = nearest_code(block / d, E2M1)
        # a tie that the numbers reach exactly is decided by the rule, not by rounding
        codes += list(c + 8 * np.signbit(block))
        least = min(least, float(near) if near > 0 else np.inf, float(np.where(n > 0, n, np.inf).min()))
    codes = np.array(codes, np.int64)
    return np.concatenate([codes[0::2] | codes[1::2] << 4, scales]).astype(np.uint8), least


def decode(rows, g, D, bits):
    """Bytes [..., row_bytes] -> values [..., D]."""
    rows = np.asarray(rows)
    if bits == 8:
        return g * e4m3_value(rows)
    b = rows[..., :D // 2].astype(np.int64)
    n = np.stack([b & 15, b >> 4], -1).reshape(*rows.shape[:-1], D)
    v = np.where(n & 8, -E2M1[n & 7], E2M1[n & 7])
    return g * v * np.repeat(e4m3_value(rows[..., D // 2:]), 16, axis=-1)


def cell(table, b, pos, page_size):
    return int(table[b][pos // page_size]), pos % page_size


def attention(q, k_new, v_new, k_ctx, v_ctx, lens, mask, scale=None):
    """q [B, P, Hq, D], k_new/v_new [B, P, Hkv, D], k_ctx/v_ctx a list of [C_b, Hkv, D],
    mask words [B, P, NW].  Returns (o, sum p |v| over the context, over the drafts)."""
    B, P, Hq, D = q.shape
    Hkv = k_new.shape[2]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    o, a_ctx, a_new = (np.zeros((B, P, Hq, D)) for _ in range(3))
    for b in range(B):
        C = k_ctx[b].shape[0]
        for p in range(int(lens[b])):
            seen = [j for j in range(int(lens[b])) if mask[b, p, j // 32] >> (j % 32) & 1]
            for h in range(Hq):
                k = np.concatenate([k_ctx[b][:, h // G], k_new[b, seen, h // G]])
                v = np.concatenate([v_ctx[b][:, h // G], v_new[b, seen, h // G]])
                if len(k) == 0:
                    continue
                x = scale * (k @ q[b, p, h])
                w = np.exp(x - x.max())
                w /= w.sum()
                o[b, p, h] = w @ v
                a_ctx[b, p, h] = w[:C] @ np.abs(v[:C])
                a_new[b, p, h] = w[C:] @ np.abs(v[C:])
    return o, a_ctx, a_new


def logprobs(x, token, temperature=1.0, top=0):
    """(log p(token), entropy, top ids, their log p, sum p |log p|) of one row of logits."""
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        z = (x - x.max()) / temperature
        lp = z - np.log(np.exp(z).sum())
        h = np.where(np.exp(lp) > 0, np.exp(lp) * lp, 0.0 * np.exp(lp))
    ids = np.lexsort((np.arange(len(x)), -x))[:top]
    return lp[token], -h.sum(), ids, lp[ids], np.abs(h).sum()
