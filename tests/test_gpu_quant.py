"""The quantised paged cache on the GPU against 64-bit numpy: what is written byte by byte,
what is read back, the attention over it, and runs of all of them together."""
import numpy as np
import pytest
import torch

from oracle import quant as oq

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
NAN16 = 0x7fc1                                # a bf16 NaN, where nothing may be read


def _rd():
    import tree_attention_verify_gb300 as rd
    return rd


def _d(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _bf(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).to(DEV)


def _f64(t):
    return t.double().cpu().numpy()


def _status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _tables(rng, rows, pages, spare=3):
    """Block table of rows that hold pages[r] pages of a shuffled pool; -1 behind them."""
    total = int(np.sum(pages))
    ids = rng.permutation(total + spare)
    table = np.full((rows, max(1, int(np.max(pages)) if rows else 1)), -1, np.int32)
    at = 0
    for r in range(rows):
        table[r, :pages[r]] = ids[at:at + pages[r]]
        at += int(pages[r])
    return table, total + spare


def _random_rows(rng, shape, D, bits, amp=1.0):
    """Random codes with scales that real data has (an amax of a few units)."""
    rows = rng.integers(0, 256, (*shape, oq.row_bytes(D, bits))).astype(np.uint8)
    if bits == 8:
        # |value| <= 3.75: codes up to e4m3 0x47, either sign
        return ((rows & 0x80) | (rows & 0x7f) % 0x48).astype(np.uint8)
    near = np.abs(oq.E4M3 - amp * 0.4).argmin()
    rows[..., D // 2:] = rng.integers(near - 8, near + 5, (*shape, D // 16))
    return rows


# ------------------------------------------------------------------------ writing
def _same_bytes(got, x, g, bits):
    """Every row of bytes is the definition's (or, where a quotient lies within the 32-bit
    quotient's error, 2^-21, of a border, decodes to a neighbour: then the next code)."""
    for r in np.ndindex(got.shape[:-1]):
        want, least = oq.encode_row(x[r], g, bits)
        if least > 2.0 ** -21:
            np.testing.assert_array_equal(got[r], want, err_msg=str(r))
        else:
            assert (np.abs(got[r].astype(int) - want.astype(int)) > 0).sum() <= 10


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hkv,D,page,lens,ctx", [
    (8, 128, 64, [57], [0]), (1, 64, 64, [1, 0, 130], [63, 5, 64]), (3, 128, 128, [0, 200, 1], [0, 100, 1]),
    (5, 64, 256, [40, 40], [250, 0]), (40, 128, 64, [7, 9], [60, 0]), (2, 64, 16, [33], [3])])
def test_append(bits, Hkv, D, page, lens, ctx):
    rd, rng = _rd(), np.random.default_rng(Hkv * D + bits)
    lens, ctx = np.array(lens), np.array(ctx, np.int32)
    table, n = _tables(rng, len(lens), -(-(ctx + lens) // page))
    extra = 3                                 # tokens behind the last sequence: not written
    T = int(lens.sum()) + extra
    k, v = (_bf(rng.standard_normal((T, Hkv, D)) * np.exp(rng.standard_normal((1, Hkv, D)))) for _ in range(2))
    gk, gv = 0.5 ** 9, 0.0031
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rb = oq.row_bytes(D, bits)
    old = rng.integers(0, 256, (2, n, page, Hkv, rb)).astype(np.uint8)
    kp, vp, st = _d(old[0]), _d(old[1]), _status()
    new = rd.rd_append_quant(k, v, _d(cu), kp, vp, gk, gv, _d(table), _d(ctx), dev_status=st)
    assert int(st) == 0
    np.testing.assert_array_equal(new.cpu().numpy(), ctx + lens)
    touched = np.zeros((n, page), bool)
    for t, pool, g in ((k, kp, gk), (v, vp, np.float32(gv).astype(float))):
        pool, x = pool.cpu().numpy(), _f64(t)
        for b in range(len(lens)):
            for i in range(int(lens[b])):
                at = oq.cell(table, b, int(ctx[b]) + i, page)
                touched[at] = True
                _same_bytes(pool[at], x[cu[b] + i], float(np.float32(g)), bits)
    for pool, was in ((kp, old[0]), (vp, old[1])):       # nothing else changes
        np.testing.assert_array_equal(pool.cpu().numpy()[~touched], was[~touched])


def test_append_special_values():
    """Zeros (of either sign), the smallest and largest numbers, infinities, ties."""
    rd = _rd()
    x = np.zeros((1, 5, 64), np.float32)
    x[0, 0, :16] = -0.0
    x[0, 1] = 1e-38
    x[0, 2, :8] = [np.inf, -np.inf, 1, -3e38, 3e38, 0, 2.0 ** -133, -1]
    x[0, 3, :16] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -6, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5]
    x[0, 4, 16:20] = [448 * 6, 448 * 5, -448 * 2.5, 7]
    k = _bf(x)
    for bits in (4, 8):
        pool, st = torch.zeros(1, 64, 5, oq.row_bytes(64, bits), dtype=torch.uint8, device=DEV), _status()
        vp = torch.zeros_like(pool)
        rd.rd_append_quant(k, k, _d(np.array([0, 1], np.int32)), pool, vp, 1.0, 1.0, _d(np.zeros((1, 1), np.int32)),
                           _d(np.zeros(1, np.int32)), dev_status=st)
        rows, xs = pool.cpu().numpy()[0, 0], _f64(k)[0]
        for h in (0, 1, 3, 4):
            np.testing.assert_array_equal(rows[h], oq.encode_row(xs[h], 1.0, bits)[0], err_msg=f"{bits} {h}")
        y = oq.decode(rows[2], 1.0, 64, bits)
        most = 448 * 6 if bits == 4 else 448
        np.testing.assert_array_equal(y[[0, 1, 3, 4, 5, 6]], [most, -most, -most, most, 0, 0])
        assert int(st) == 0 and torch.equal(pool, vp)


def test_append_and_commit_flag_what_they_skip():
    rd, rng = _rd(), np.random.default_rng(3)
    Hkv, D, page = 2, 64, 64
    k = _bf(rng.standard_normal((30, Hkv, D)))
    table = np.array([[0, 1], [2, 9], [3, 4]], np.int32)          # page 9 does not exist
    cu, ctx = np.array([0, 10, 20, 30], np.int32), np.array([60, 60, 125], np.int32)
    kp, vp = (torch.full((5, page, Hkv, 36), 7, dtype=torch.uint8, device=DEV) for _ in range(2))
    st = _status()
    new = rd.rd_append_quant(k, k, _d(cu), kp, vp, 1.0, 1.0, _d(table), _d(ctx), dev_status=st)
    assert int(st) == rd.DEV_BAD_INDEX | rd.DEV_BAD_LENGTH        # and row 2 ends behind its two pages
    np.testing.assert_array_equal(new.cpu().numpy(), ctx + 10)
    wrote = (kp.cpu().numpy() != 7).any(-1).any(-1)
    want = np.zeros((5, page), bool)
    want[0, 60:] = want[1, :6] = want[2, 60:] = want[4, 61:] = True
    np.testing.assert_array_equal(wrote, want)
    # whole requests that are refused
    for bad_cu, bad_ctx in (([0, 10, 5, 30], [0, 0, 0]), ([0, 10, 20, 31], [0, 0, 0]), ([0, 10, 20, 30], [0, -1, 2 ** 31 - 10]),
                            ([-3, 10, 20, 30], [0, 0, 0])):
        kp.fill_(7)
        st.zero_()
        c, x = np.array(bad_cu, np.int64), np.array(bad_ctx, np.int64)
        fine = [c[b] >= 0 and c[b] <= c[b + 1] <= 30 and x[b] >= 0 and x[b] + c[b + 1] - c[b] < 2 ** 31 for b in range(3)]
        new = rd.rd_append_quant(k, k, _d(c.astype(np.int32)), kp, vp, 1.0, 1.0, _d(np.arange(6).reshape(3, 2).astype(np.int32)),
                                 _d(x.astype(np.int32)), dev_status=st)
        assert int(st) & rd.DEV_BAD_LENGTH
        np.testing.assert_array_equal(new.cpu().numpy(), [x[b] + (c[b + 1] - c[b] if fine[b] else 0) for b in range(3)])
        wrote = (kp.cpu().numpy() != 7).any(-1).any(-1).reshape(-1)[:5 * page]
        for b in range(2):
            assert wrote[128 * b:128 * (b + 1)].sum() == (c[b + 1] - c[b] if fine[b] else 0)


@pytest.mark.parametrize("bits,Hkv,D,page", [(4, 8, 128, 64), (8, 3, 64, 128), (4, 1, 64, 64)])
def test_commit(bits, Hkv, D, page):
    rd, rng = _rd(), np.random.default_rng(bits + Hkv)
    B, W, L, P = 6, 3, 4, 9
    ctx = rng.integers(0, 200, B).astype(np.int32)
    table, n = _tables(rng, B, -(-(ctx + L) // page))
    kn, vn = (_bf(rng.standard_normal((B, P, Hkv, D))) for _ in range(2))
    unp = rng.integers(0, P, (B, W, L)).astype(np.int32)
    best, acc = rng.integers(0, W, B).astype(np.int32), rng.integers(0, L, B).astype(np.int32)
    best[4], acc[5] = W, L                                         # two requests with wrong inputs
    unp[3, best[3], 0] = P
    old = rng.integers(0, 256, (2, n, page, Hkv, oq.row_bytes(D, bits))).astype(np.uint8)
    kp, vp, st = _d(old[0]), _d(old[1]), _status()
    new = rd.rd_commit_accepted_quant(kn, vn, _d(unp), _d(best), _d(acc), kp, vp, 0.25, 0.5, _d(table), _d(ctx),
                                      dev_status=st)
    assert int(st) == rd.DEV_BAD_INDEX
    np.testing.assert_array_equal(new.cpu().numpy(), ctx + np.where(np.arange(B) < 4, acc + 1, 0))
    want = old.copy()
    for b in range(4):
        for i in range(acc[b] + 1):
            node = unp[b, best[b], i]
            if node < P:
                for w, t, g in ((want[0], kn, 0.25), (want[1], vn, 0.5)):
                    for h in range(Hkv):
                        w[oq.cell(table, b, int(ctx[b]) + i, page)][h] = oq.encode_row(_f64(t[b, node, h]), g, bits)[0]
    np.testing.assert_array_equal(kp.cpu().numpy(), want[0])
    np.testing.assert_array_equal(vp.cpu().numpy(), want[1])


# ------------------------------------------------------------------------ reading
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hkv,D,page,lens", [(8, 128, 64, [100, 1, 0, 64]), (1, 64, 64, [3]), (5, 64, 16, [50, 7]),
                                             (3, 128, 256, [300])])
def test_read(bits, Hkv, D, page, lens):
    rd, rng = _rd(), np.random.default_rng(D + bits)
    lens = np.array(lens)
    starts = rng.integers(0, 70, len(lens)).astype(np.int32)
    table, n = _tables(rng, len(lens), -(-(lens + starts) // page))
    rows = _random_rows(rng, (2, n, page, Hkv), D, bits)
    off = np.concatenate([[2], 2 + np.cumsum(lens)]).astype(np.int64)
    total = int(off[-1]) + 3
    gk, gv = 0.125, float(np.float32(0.0173))
    for st0 in (starts, None):
        k, v = (torch.full((total, Hkv, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        st = _status()
        got = rd.rd_read_quant(_d(rows[0]), _d(rows[1]), gk, gv, _d(table), _d(off), total=total,
                               starts=None if st0 is None else _d(st0), k_out=k, v_out=v, dev_status=st)
        assert got[0] is k and got[1] is v and int(st) == 0
        for out, pool, g in ((k, rows[0], gk), (v, rows[1], gv)):
            want = np.full((total, Hkv, D), 7.0)
            for b in range(len(lens)):
                for i in range(lens[b]):
                    at = oq.cell(table, b, i + (0 if st0 is None else int(st0[b])), page)
                    want[off[b] + i] = oq.decode(pool[at], g, D, bits)
            # one rounding to bf16 (half a step, 2^-8), one of the product to 32 bits before it
            np.testing.assert_allclose(_f64(out), want, rtol=2.0 ** -8 + 2.0 ** -23, atol=0)
            if g == 0.125:                    # every value times a power of two has few bits: exact
                np.testing.assert_array_equal(_f64(out), want)


def test_read_flags_what_it_cannot_read():
    rd = _rd()
    pool = torch.full((2, 64, 1, 64), 0x38, dtype=torch.uint8, device=DEV)        # e4m3 1.0
    table = _d(np.array([[0, 5], [1, 1]], np.int32))
    for off, starts, want, bits in (([0, 70, 80], None, [1] * 64 + [0] * 6 + [1] * 10, rd.DEV_BAD_INDEX),
                                    ([0, 2, 10], [0, 125], [1] * 5 + [0] * 5, rd.DEV_BAD_LENGTH),
                                    ([0, 2, 4], [-1, 0], [0, 0, 1, 1], rd.DEV_BAD_LENGTH)):
        st, total = _status(), off[-1]
        k, v = rd.rd_read_quant(pool, pool, 1.0, 2.0, table, _d(np.array(off, np.int64)), total=total,
                                starts=None if starts is None else _d(np.array(starts, np.int32)), dev_status=st)
        assert int(st) == bits
        np.testing.assert_array_equal(_f64(k)[:, 0, 0], want)
        np.testing.assert_array_equal(_f64(v)[:, 0, 5], 2.0 * np.array(want))
    st = _status()                            # offsets past the output: nothing outside is touched
    k = torch.full((6, 1, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    rd.rd_read_quant(pool, pool, 1.0, 1.0, table, _d(np.array([0, 4, 9], np.int64)), total=6, k_out=k, v_out=k.clone(),
                     dev_status=st)
    assert int(st) == rd.DEV_BAD_LENGTH
    np.testing.assert_array_equal(_f64(k)[:4, 0, 0], 1.0)


# ---------------------------------------------------------------------- attention
def make(B, P, Hq, Hkv, D, page, bits, lens, ctx, seed=0, mask="tree", amp=1.0):
    rng = np.random.default_rng(seed)
    lens, ctx = np.array(lens, np.int32), np.array(ctx, np.int32)
    table, n = _tables(rng, B, -(-ctx // page))
    rows = _random_rows(rng, (2, n, page, Hkv), D, bits)
    gk, gv = float(np.float32(0.7)), float(np.float32(1.3))
    q, kn, vn = (rng.standard_normal((B, P, h, D)) for h in (Hq, Hkv, Hkv))
    q *= amp
    seen = rng.random((B, P, P)) < 0.4 if mask == "random" else np.tril(rng.random((B, P, P)) < 0.5)
    if mask != "none":
        seen |= np.eye(P, dtype=bool)
    else:
        seen[:] = False
    words = np.zeros((B, P, -(-P // 32) * 32), bool)
    words[:, :, :P] = seen
    words[:, :, P:] = True                    # bits of no node
    mask = np.packbits(words.reshape(B, P, -1, 32), axis=-1, bitorder="little").view(np.uint32)[..., 0]
    s = dict(q=_bf(q), kn=_bf(kn), vn=_bf(vn), kp=_d(rows[0]), vp=_d(rows[1]), gk=gk, gv=gv, table=_d(table), ctx=_d(ctx),
             lens=_d(lens), mask=_d(mask.view(np.int32)), max_ctx=int(ctx.max()) if B else 0, page=page, bits=bits,
             np=(table, ctx, lens, mask, rows))
    for b in range(B):                        # behind the last node, and behind the context: anything
        for t in (s["q"], s["kn"], s["vn"]):
            t[b, int(max(0, lens[b])):] = float("nan")
        if ctx[b] % page:
            for t in (s["kp"], s["vp"]):
                t[int(table[b, ctx[b] // page]), int(ctx[b] % page):] = 0xff
    return s


def call(s, st=None, **kw):
    args = {**dict(max_ctx=s["max_ctx"], dev_status=st), **kw}
    return _rd().rd_tree_attention_quant(s["q"], s["kn"], s["vn"], s["kp"], s["vp"], s["gk"], s["gv"], s["table"], s["ctx"],
                                         s["lens"], s["mask"], **args)


def reference(s, scale=None):
    table, ctx, lens, mask, _ = s["np"]
    D = s["q"].shape[3]
    ctxs = []
    for pool, g in ((s["kp"], s["gk"]), (s["vp"], s["gv"])):
        pool = pool.cpu().numpy()
        ctxs.append([oq.decode(np.concatenate([pool[p] for p in table[b, :-(-int(ctx[b]) // s["page"])]]
                                              or [pool[0][:0]])[:int(ctx[b])], g, D, s["bits"]) for b in range(len(lens))])
    clean = [np.nan_to_num(_f64(t)) for t in (s["q"], s["kn"], s["vn"])]
    return (*oq.attention(*clean, *ctxs, lens, mask, scale), ctxs, clean)


def check(o, s, scale=None):
    """The tolerance, from the roundings that there are: the output's to bf16 (half a step,
    2^-8 of it); each context weight's to f16 (2^-11) and each draft weight's to bf16 (2^-8), relative to
    the weighted mean of |v| over those keys; 32-bit sums of D products in the scores (which move a
    weight by the error itself), of n weights and of n products, and the hardware's 2^x (2^-21).
    A context weight that is less than 2^-21 of the row's largest is a subnormal 16-bit number: the
    largest stands at 2^7 or above, half a subnormal step is 2^-25, so it is off by 2^-32 of the largest at
    most, and the output by 2^-32 of the sum of |v| over the context."""
    want, a_ctx, a_new, (kc, vc), (q, kn, _) = reference(s, scale)
    D, P = q.shape[3], q.shape[1]
    G = q.shape[2] // kn.shape[2]
    f = D ** -0.5 if scale is None else scale
    n = P + s["max_ctx"]
    most = np.zeros(q.shape[:3])              # the largest sum |q k| of a row
    sums = np.zeros(q.shape)                  # sum of |v| over the context
    for b in range(len(kc)):
        for h in range(q.shape[2]):
            k = np.abs(np.concatenate([kc[b][:, h // G], kn[b, :, h // G]]))
            most[b, :, h] = f * (np.abs(q[b, :, h]) @ k.T).max(1)
            sums[b, :, h] = np.abs(vc[b][:, h // G]).sum(0)
    eps = 2 * (D + 8) * 2.0 ** -24 * most[..., None] + 2 * n * 2.0 ** -24 + 2.0 ** -20
    tol = np.abs(want) * 2.0 ** -8 + a_ctx * (2.0 ** -11 + eps) + a_new * (2.0 ** -8 + eps) + sums * 2.0 ** -32 + 1e-30
    got = _f64(o)
    assert np.isfinite(got).all()
    worst = np.unravel_index(np.argmax(np.abs(got - want) - tol), got.shape)
    assert (np.abs(got - want) <= tol).all(), (worst, got[worst], want[worst], tol[worst])


CASES = {
    # B, P, Hq, Hkv, D, page, bits, lens, ctx
    "one token": (1, 1, 1, 1, 64, 64, 4, [1], [1]),
    "no context": (2, 3, 2, 2, 128, 64, 4, [3, 1], [0, 0]),
    "tokens": (8, 1, 32, 8, 128, 64, 4, [1] * 8, [100, 1, 0, 64, 63, 65, 200, 128]),
    "tokens 8 bits": (4, 1, 32, 8, 128, 64, 8, [1] * 4, [100, 1, 257, 64]),
    "padded": (5, 7, 4, 4, 128, 64, 4, [7, 0, 3, 1, 5], [130, 50, 0, 64, 31]),
    "rows 9": (2, 9, 4, 4, 128, 128, 4, [9, 8], [150, 300]),
    "rows 24": (2, 24, 8, 8, 128, 64, 4, [24, 17], [70, 400]),
    "rows 48": (3, 48, 4, 4, 128, 256, 4, [48, 33, 40], [500, 90, 256]),
    "grouped": (3, 40, 16, 4, 128, 64, 4, [40, 13, 21], [333, 64, 150]),
    "grouped 8 bits": (2, 20, 20, 4, 64, 64, 8, [20, 11], [333, 90]),
    "one kv head": (2, 5, 8, 1, 128, 64, 4, [5, 4], [700, 255]),
    "one kv head 8 bits": (2, 5, 8, 1, 64, 64, 8, [5, 4], [700, 257]),
    "two kv heads": (2, 6, 6, 2, 128, 64, 4, [6, 2], [300, 129]),
    "three kv heads": (2, 6, 3, 3, 128, 64, 4, [6, 2], [300, 129]),
    "three kv heads d64": (2, 6, 6, 3, 64, 64, 4, [6, 2], [300, 129]),
    "three kv heads 8 bits": (2, 6, 3, 3, 128, 64, 8, [6, 2], [300, 129]),
    "six kv heads d64": (2, 6, 6, 6, 64, 64, 4, [6, 2], [300, 129]),
    "d64": (3, 16, 8, 8, 64, 64, 4, [16, 9, 1], [200, 31, 32]),
    "d64 8 bits": (3, 16, 8, 8, 64, 64, 8, [16, 9, 1], [200, 31, 32]),
    "two kv heads 8 bits": (2, 6, 6, 2, 128, 192, 8, [6, 2], [300, 129]),
    "many nodes": (1, 256, 4, 4, 64, 64, 4, [256], [100]),
    "many rows": (1, 130, 32, 4, 64, 64, 8, [130], [65]),
    "long": (1, 3, 4, 4, 128, 64, 4, [3], [9000]),
    "long 8 bits": (1, 3, 4, 4, 64, 128, 8, [3], [9000]),
    "many requests": (500, 1, 4, 4, 64, 64, 4, [1] * 500, [int(i * 37 % 190) for i in range(500)]),
}


@pytest.mark.parametrize("name", CASES)
def test_attention(name):
    s, st = make(*CASES[name]), _status()
    o = call(s, st)
    assert int(st) == 0
    check(o, s)
    lens = s["np"][2]
    for b in range(len(lens)):
        assert (o[b, int(lens[b]):] == 0).all()
    assert torch.equal(o, call(s))            # the same bits every time


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("mask", ["none", "random"])
def test_masks(mask, bits):
    """Rows whose mask leaves nothing of the drafts (and, without a context, nothing at all)."""
    s = make(3, 20, 8, 4, 128, 64, bits, [20, 17, 20], [100, 0, 1], mask=mask)
    o, st = call(s, _status()), _status()
    check(o, s)
    if mask == "none":
        assert (o[1] == 0).all()


def test_scales_and_query_sizes():
    for amp, scale in ((1e-30, 0.0), (1e30, 1e-31), (300.0, 0.0), (1.0, 3.0), (2.0 ** -126, 1e38)):
        s = make(2, 6, 4, 4, 128, 64, 4, [6, 5], [150, 40], seed=5, amp=amp)
        check(call(s, scale=scale), s, scale or None)
    s = make(1, 4, 4, 4, 64, 64, 4, [4], [90], seed=6)
    s["q"][0, 1] = 0                          # equal weights
    s["q"][0, 2] = 3.0e38
    check(call(s, scale=1e-38), s, 1e-38)


def test_scores_that_keep_rising():
    """The running maximum moves in every chunk, by less and by more than it may lag."""
    for step in (0.02, 0.3):
        s = make(1, 2, 4, 4, 64, 64, 4, [2], [640], seed=7)
        rows = s["kp"]
        table = s["np"][0]
        rows[..., :32] = 0x22                 # every code 1
        for j in range(640):
            byte = int(np.abs(oq.E4M3 - step * (j + 1)).argmin())
            rows[int(table[0, j // 64]), j % 64, :, 32:] = byte
        s["q"][0] = 0.125
        check(call(s), s)


def test_nan_codes_reach_only_who_sees_them():
    s = make(3, 4, 4, 4, 64, 64, 8, [4, 4, 4], [70, 70, 70], seed=8)
    table = s["np"][0]
    s["vp"][int(table[1, 0]), 3, 2, 5] = 0x7f
    o = call(s)
    bad = torch.isnan(o)
    want = torch.zeros_like(bad)
    want[1, :, 2, 5] = True
    assert torch.equal(bad, want)
    s["kp"][int(table[2, 0]), 3, 1, 5] = 0xff
    bad = torch.isnan(call(s))
    want[2, :, 1, :] = True
    assert torch.equal(bad, want)


def test_wrong_requests_are_skipped():
    rd = _rd()
    s = make(6, 4, 4, 4, 64, 64, 4, [4, 4, 4, 4, 4, 4], [70, 70, 70, 70, 70, 70], seed=9)
    def rest(o):
        """The others' rows: each sum may be cut elsewhere, as the batch's work has changed."""
        table, ctx, lens, mask, rows = s["np"]
        lens = np.where(np.arange(6) == 2, 0, lens)
        check(o, {**s, "np": (table, ctx, lens, mask, rows)})

    for what, value, bits in (("ctx", -1, rd.DEV_BAD_LENGTH), ("ctx", 71, rd.DEV_BAD_LENGTH), ("lens", 5, rd.DEV_BAD_LENGTH),
                              ("lens", -1, rd.DEV_BAD_LENGTH), ("ctx", 2 ** 31 - 1, rd.DEV_BAD_LENGTH)):
        t = {**s, what: s[what].clone()}
        t[what][2] = value
        st = _status()
        o = call(t, st)
        assert int(st) == bits
        assert (o[2] == 0).all()
        rest(o)
    t, st = {**s, "ctx": s["ctx"].clone()}, _status()
    t["ctx"][2] = 2 ** 31 - 1
    assert (call(t, st, max_ctx=2 ** 31 - 1)[2] == 0).all() and int(st) == rd.DEV_BAD_LENGTH
    # a page id out of range: page 0 in its place
    for bad in (-1, s["kp"].shape[0], 2 ** 31 - 1):
        t, st = {**s, "table": s["table"].clone()}, _status()
        t["table"][3, 1] = bad
        o = call(t, st)
        assert int(st) == rd.DEV_BAD_INDEX
        t["table"][3, 1] = 0
        assert torch.equal(o, call(t))


def test_empty_calls():
    rd = _rd()
    s = make(2, 4, 4, 4, 64, 64, 4, [4, 2], [70, 3])
    none = {**s, **{k: s[k][:0] for k in ("q", "kn", "vn", "table", "ctx", "lens", "mask")}}
    assert call(none).shape == (0, 4, 4, 64)
    empty = {**s, "kp": s["kp"][:0], "vp": s["vp"][:0]}          # no pages: only requests without a context count
    st = _status()
    assert (call(empty, st) == 0).all() and int(st) == rd.DEV_BAD_LENGTH
    zero, st = {**empty, "ctx": torch.zeros_like(s["ctx"]), "np": (s["np"][0], 0 * s["np"][1], *s["np"][2:])}, _status()
    zero["kp"], zero["vp"] = s["kp"][:0], s["vp"][:0]
    o = call(zero, st)
    assert int(st) == 0
    check(o, {**zero, "kp": s["kp"], "vp": s["vp"]})
    zero = {**s, "lens": torch.zeros_like(s["lens"]), "ctx": torch.full_like(s["ctx"], -7)}      # nothing is asked
    st = _status()
    assert (call(zero, st) == 0).all() and int(st) == 0


def test_graphs_streams_and_workspaces():
    rd = _rd()
    a, b = make(4, 20, 8, 8, 128, 64, 4, [20, 9, 1, 15], [900, 30, 2000, 0]), make(3, 1, 32, 8, 128, 64, 8, [1] * 3, [500, 9, 70])
    want = [call(x) for x in (a, b)]
    size = max(rd.rd_tree_attention_quant_workspace_size(4, 20, 8, 8, 128, 2000, DEV),
               rd.rd_tree_attention_quant_workspace_size(3, 1, 32, 8, 128, 500, DEV))
    ws = torch.full((size,), 0xff, dtype=torch.uint8, device=DEV)
    outs = [torch.empty_like(x) for x in want]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for x, o in zip((a, b), outs):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                call(x, out=o, workspace=ws)
            graphs.append(g)
        for _ in range(3):
            for g, o, w in zip(graphs, outs, want):
                o.fill_(float("nan"))
                g.replay()
                assert torch.equal(o, w)
    # another stream than the current one
    o = call(a, stream=side)
    side.synchronize()
    assert torch.equal(o, want[0])
    # two streams at once, a workspace each
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got += [(call(a, stream=side), want[0]), (call(b, stream=other), want[1])]
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in got)
    with pytest.raises(rd.RdError):
        call(a, workspace=ws[:size // 2])


def test_pages_past_32_bits():
    """A pool of more than 2^32 bytes, its last page read and written."""
    rd = _rd()
    pages, page, Hkv, D = 31000, 256, 8, 128
    kp = torch.zeros(pages, page, Hkv, 72, dtype=torch.uint8, device=DEV)
    vp = torch.zeros_like(kp)
    table = _d(np.array([[pages - 1, 30000]], np.int32))
    k = _bf(np.random.default_rng(1).standard_normal((300, Hkv, D)))
    v = _bf(np.random.default_rng(2).standard_normal((300, Hkv, D)))
    new = rd.rd_append_quant(k, v, _d(np.array([0, 300], np.int32)), kp, vp, 0.25, 0.5, table, _d(np.zeros(1, np.int32)))
    small = torch.stack([kp[pages - 1], kp[30000]]), torch.stack([vp[pages - 1], vp[30000]])
    q = _bf(np.random.default_rng(3).standard_normal((1, 2, 8, D)))
    rest = (_bf(np.zeros((1, 2, Hkv, D))), _bf(np.zeros((1, 2, Hkv, D))))
    tail = (new, _d(np.array([2], np.int32)), _d(np.array([[[1], [3]]], np.int32)))
    o = rd.rd_tree_attention_quant(q, *rest, kp, vp, 0.25, 0.5, table, *tail, max_ctx=300)
    near = rd.rd_tree_attention_quant(q, *rest, *small, 0.25, 0.5, _d(np.array([[0, 1]], np.int32)), *tail, max_ctx=300)
    assert torch.equal(o, near) and o.abs().max() > 0
    off = _d(np.array([0, 300], np.int64))
    far = rd.rd_read_quant(kp, vp, 0.25, 0.5, table, off, total=300)
    here = rd.rd_read_quant(*small, 0.25, 0.5, _d(np.array([[0, 1]], np.int32)), off, total=300)
    assert torch.equal(far[0], here[0]) and torch.equal(far[1], here[1]) and far[0].abs().max() > 0


def test_a_wait_that_runs_out_is_reported():
    rd = _rd()
    s = make(4, 20, 8, 8, 128, 64, 4, [20, 9, 1, 15], [900, 30, 2000, 0])
    want, st = call(s), _status()
    rd.rd_debug_stall_attention(2_000_000)
    try:
        call(s, st)
        torch.cuda.synchronize()
    finally:
        rd.rd_debug_stall_attention(0)
    assert int(st) & rd.DEV_TIMEOUT
    st = _status()
    assert torch.equal(call(s, st), want) and int(st) == 0


def test_page_operators_take_the_pools():
    """Fork, compact and resize move quantised pages as any others: a branch attends as its parent."""
    rd = _rd()
    rng = np.random.default_rng(4)
    Hkv, D, page = 3, 64, 64                  # rows of 108 bytes a position: no multiple of 16
    N, R = 12, 4
    table = _d(np.full((R, 4), -1, np.int32))
    held, refs = (torch.zeros(n, dtype=torch.int32, device=DEV) for n in (R, N))
    lens = _d(np.array([100, 0, 70, 0], np.int32))
    kp, vp = (torch.zeros(N, page, Hkv, 36, dtype=torch.uint8, device=DEV) for _ in range(2))
    rd.rd_resize_pages(table, held, refs, lens, page)
    T = 170
    k, v = (_bf(rng.standard_normal((T, Hkv, D))) for _ in range(2))
    cu = _d(np.array([0, 100, 100, 170, 170], np.int32))
    ctx = rd.rd_append_quant(k, v, cu, kp, vp, 1.0, 1.0, table, torch.zeros_like(lens))
    st = _status()
    rd.rd_fork_pages(kp, vp, table, held, refs, ctx, _d(np.array([0, 2], np.int32)), _d(np.array([1, 3], np.int32)), dev_status=st)
    rd.rd_resize_pages(table, held, refs, _d(np.array([0, -1, -1, -1], np.int32)), page, dev_status=st)
    rd.rd_compact_pages(kp, vp, table, held, refs, dev_status=st)
    assert int(st) == 0 and ctx.tolist() == [100, 100, 70, 70]
    off = _d(np.array([0, 0, 100, 170, 240], np.int64))
    got, _ = rd.rd_read_quant(kp, vp, 1.0, 1.0, table, off, total=240, dev_status=st)
    assert int(st) == 0
    assert torch.equal(got[100:170], got[170:]) and got[:100].abs().max() > 0
    want = np.stack([[oq.decode(oq.encode_row(_f64(k[t, h]), 1.0, 4)[0], 1.0, D, 4) for h in range(Hkv)] for t in range(T)])
    np.testing.assert_array_equal(_f64(got[:170]), want)


@pytest.mark.parametrize("bits", [4, 8])
def test_a_run_of_steps(bits):
    """Prompts appended, then three verification steps: attention over the quantised pages, greedy
    acceptance, log probabilities of what was emitted, commit; each step's attention against the
    plain one over what has been written so far, captured in one graph and replayed."""
    rd, rng = _rd(), np.random.default_rng(bits)
    B, W, L, Hq, Hkv, D, V, page = 3, 3, 4, 4, 4, 64, 97, 64
    P = W * L
    lens = np.array([70, 5, 64])
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    table, n = _tables(rng, B, -(-(lens + 3 * L) // page))
    kp, vp = (torch.full((n, page, Hkv, oq.row_bytes(D, bits)), 0xff, dtype=torch.uint8, device=DEV) for _ in range(2))
    t = _d(table)
    k, v = (_bf(rng.standard_normal((int(cu[-1]), Hkv, D))) for _ in range(2))
    st = _status()
    ctx = rd.rd_append_quant(k, v, _d(cu), kp, vp, 0.5, 0.25, t, torch.zeros(B, dtype=torch.int32, device=DEV), dev_status=st)
    beams = torch.zeros(B, W, L, dtype=torch.int32, device=DEV)
    q, kn, vn = (torch.zeros(B, P, h, D, dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hkv))
    logits = torch.zeros(B, P, V, dtype=torch.bfloat16, device=DEV)

    def step():
        pk = rd.rd_pack_beams(beams, P, dev_status=st)
        o = rd.rd_tree_attention_quant(q, kn, vn, kp, vp, 0.5, 0.25, t, ctx, pk["packed_len"], pk["mask"],
                                       max_ctx=page * table.shape[1], dev_status=st)
        acc = rd.rd_greedy_accept(logits, beams, pk["unpacker"], pk["packed_len"], dev_status=st)
        lp = rd.rd_accepted_logprobs(logits, pk["unpacker"], acc["best_beam"], acc["n_accepted"], acc["out_tokens"], top=3,
                                     dev_status=st)
        new = rd.rd_commit_accepted_quant(kn, vn, pk["unpacker"], acc["best_beam"], acc["n_accepted"], kp, vp, 0.5, 0.25, t,
                                          ctx, dev_status=st)
        return pk, o, acc, lp, new

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        with torch.cuda.stream(side):
            kept = kp.clone(), vp.clone()
            step()                            # (warm-up: what it commits is taken back)
            kp.copy_(kept[0]), vp.copy_(kept[1])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    st.zero_()
    with torch.cuda.graph(graph):
        pk, o, acc, lp, new = step()
    emitted = 0
    for i in range(3):
        beams.copy_(_d(rng.integers(0, 3, (B, W, L)).astype(np.int32)))
        beams[:, :, 0] = 1
        for x in (q, kn, vn):
            x.copy_(_bf(rng.standard_normal(tuple(x.shape))))
        logits.copy_(_bf(rng.standard_normal((B, P, V)) * 2))
        logits[:, :, :3] += 6
        before = ctx.cpu().numpy().copy()
        pools = kp.clone(), vp.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert int(st) == 0
        s = dict(q=q, kn=kn, vn=vn, kp=pools[0], vp=pools[1], gk=0.5, gv=0.25, page=page, bits=bits,
                 max_ctx=int(before.max()),
                 np=(table, before, pk["packed_len"].cpu().numpy(), pk["mask"].cpu().numpy().view(np.uint32), None))
        check(o, s)
        best, a, unp = (x.cpu().numpy() for x in (acc["best_beam"], acc["n_accepted"], pk["unpacker"]))
        for b in range(B):
            for j in range(a[b] + 1):
                node = unp[b, best[b], j]
                at = oq.cell(table, b, int(before[b]) + j, page)
                for pool, x, g in ((kp, kn, 0.5), (vp, vn, 0.25)):
                    for h in range(Hkv):
                        np.testing.assert_array_equal(pool[at][h].cpu().numpy(), oq.encode_row(_f64(x[b, node, h]), g, bits)[0])
                lo, ent, ids, tops, _ = oq.logprobs(_f64(logits[b, node]), int(acc["out_tokens"][b, j]), 1.0, 3)
                assert abs(float(lp["logprob"][b, j]) - lo) < 1e-5 and abs(float(lp["entropy"][b, j]) - ent) < 1e-5
                assert lp["top_tokens"][b, j].tolist() == list(ids)
                emitted += 1
            assert (lp["top_tokens"][b, a[b] + 1:] == -1).all()
        np.testing.assert_array_equal(new.cpu().numpy(), before + a + 1)
        ctx.copy_(new)
    assert emitted > 9


def test_matches_the_bf16_attention():
    """Reading the cache back and calling rd_tree_attention gives the same up to the roundings
    of both (cached values that bf16 holds exactly: scales that are powers of two)."""
    rd = _rd()
    s = make(3, 12, 8, 4, 128, 64, 4, [12, 5, 9], [200, 64, 333], seed=11)
    for t in (s["q"], s["kn"], s["vn"]):
        t.nan_to_num_()
    s["gk"], s["gv"] = 0.5, 2.0
    ctx = s["np"][1]
    off = _d(np.concatenate([[0], np.cumsum(ctx)]).astype(np.int64))
    total = int(ctx.sum())
    k, v = rd.rd_read_quant(s["kp"], s["vp"], s["gk"], s["gv"], s["table"], off, total=total)
    want = rd.rd_tree_attention(s["q"], s["kn"], s["vn"], k, v, off, s["lens"], s["mask"], max_ctx=s["max_ctx"])
    check(call(s), s)
    a = np.abs(_f64(want)) + 4.0              # |v| is below 16: both are within 2^-7 of the weighted means
    assert (np.abs(_f64(call(s)) - _f64(want)) <= a * 2.0 ** -6).all()


MORE = {
    # B, P, Hq, Hkv, D, page, bits, lens, ctx
    "rows 40 8 bits": (2, 40, 4, 4, 128, 64, 8, [40, 33], [500, 130]),
    "rows 33 two heads 8 bits": (2, 33, 2, 2, 128, 64, 8, [33, 32], [260, 129]),
    "chunk ends, four heads": (6, 20, 4, 4, 64, 64, 4, [20, 17, 16, 8, 9, 1], [95, 96, 97, 191, 192, 193]),
    "chunk ends, two heads": (5, 25, 2, 2, 64, 64, 8, [25, 24, 16, 7, 1], [191, 192, 193, 383, 385]),
    "chunk ends, one head": (5, 24, 1, 1, 64, 64, 4, [24, 20, 1, 9, 17], [383, 384, 385, 767, 769]),
    "chunk ends, wide rows": (6, 33, 4, 4, 128, 64, 4, [33, 32, 31, 16, 8, 1], [63, 64, 65, 127, 128, 129]),
    "one token, 64 rows of a head": (2, 1, 64, 1, 128, 64, 4, [1, 1], [700, 1]),
    "five rows of a head, small pages": (3, 5, 15, 3, 64, 64, 8, [5, 4, 5], [65, 640, 0]),
}


@pytest.mark.parametrize("name", MORE)
def test_attention_at_the_ends_of_chunks(name):
    s, st = make(*MORE[name], seed=11), _status()
    o = call(s, st)
    assert int(st) == 0
    check(o, s)
    lens = s["np"][2]
    for b in range(len(lens)):
        assert (o[b, int(lens[b]):] == 0).all()


def _shifted(t):
    """The same tensor 16 bytes behind a 32-byte boundary."""
    flat = torch.empty(t.numel() + 16, dtype=t.dtype, device=DEV)
    at = 8 if flat.data_ptr() % 32 == 0 else 0
    u = flat[at:at + t.numel()].view(t.shape)
    u.copy_(t)
    assert u.data_ptr() % 32 == 16
    return u


@pytest.mark.parametrize("bits", [4, 8])
def test_tensors_on_16_byte_boundaries(bits):
    """Sources and outputs that 32-byte accesses do not fit give the same bytes."""
    rd, rng = _rd(), np.random.default_rng(bits)
    Hkv, D, page, T = 3, 64, 64, 100
    k, v = (_bf(rng.standard_normal((T, Hkv, D))) for _ in range(2))
    cu, ctx, table = _d(np.array([0, 40, T], np.int32)), _d(np.array([30, 0], np.int32)), _d(np.array([[0, 1], [2, 3]], np.int32))
    pools = [[torch.zeros(4, page, Hkv, oq.row_bytes(D, bits), dtype=torch.uint8, device=DEV) for _ in range(2)]
             for _ in range(3)]
    rd.rd_append_quant(k, v, cu, *pools[0], 0.5, 0.25, table, ctx)
    rd.rd_append_quant(_shifted(k), _shifted(v), cu, *pools[1], 0.5, 0.25, table, ctx)
    rd.rd_append_quant(_shifted(k), v, cu, *pools[2], 0.5, 0.25, table, ctx)
    for other in pools[1:]:
        assert all(torch.equal(a, b) for a, b in zip(pools[0], other))
    off = _d(np.array([0, 40, T], np.int64))
    want = rd.rd_read_quant(*pools[0], 0.5, 0.25, table, off, total=T, starts=ctx)
    out = [_shifted(torch.zeros_like(k)), torch.zeros_like(v)]
    rd.rd_read_quant(*pools[0], 0.5, 0.25, table, off, total=T, starts=ctx, k_out=out[0], v_out=out[1])
    assert all(torch.equal(a, b) for a, b in zip(want, out))
    unp, best, acc = _d(np.arange(8, dtype=np.int32).reshape(2, 1, 4)), _d(np.zeros(2, np.int32)), _d(np.array([3, 1], np.int32))
    kn, vn = (_bf(rng.standard_normal((2, 8, Hkv, D))) for _ in range(2))
    rd.rd_commit_accepted_quant(kn, vn, unp, best, acc, *pools[0], 0.5, 0.25, table, ctx)
    rd.rd_commit_accepted_quant(_shifted(kn), _shifted(vn), unp, best, acc, *pools[1], 0.5, 0.25, table, ctx)
    assert all(torch.equal(a, b) for a, b in zip(pools[0], pools[1]))


@pytest.mark.parametrize("case", [(1, 5, 8, 4, 64, 64, 4, [5], [40000]), (1, 24, 4, 4, 128, 64, 4, [24], [30001]),
                                  (2, 3, 4, 2, 128, 128, 8, [3, 1], [20000, 0]), (3, 4, 4, 4, 64, 64, 8, [4, 1, 2], [9000, 1, 9100])])
def test_units_in_many_pieces(case):
    """A few long contexts: every CTA has a piece of the same unit, and the merge joins more than 32."""
    s, st = make(*case, seed=12), _status()
    o = call(s, st)
    assert int(st) == 0
    check(o, s)
    assert torch.equal(o, call(s))


@pytest.mark.parametrize("bits,Hkv,D", [(4, 4, 64), (8, 2, 64)])
def test_contexts_at_the_end_of_31_bits(bits, Hkv, D):
    """The longest context there is: 2^31 - 257 positions on one page that its row of the table names again and again.  Nodes in
    many tiles, so that pieces begin with drafts too.  A warp's share is 2^31 / 152 / 3 positions in steps of 16
    products, each off by 2^-23 of the sum at most (the matrix unit may cut it off), which both the sums of
    weights and of products may drift by: 2 x 295,000 x 2^-23 of the mean |v|, and 0.01 for the rest."""
    rd, rng = _rd(), np.random.default_rng(bits)
    page, C, P = 1 << 16, 2 ** 31 - 257, 40
    width = 1 << 15
    rows = _random_rows(rng, (2, 1, page, Hkv), D, bits)
    kp, vp = _d(rows[0]), _d(rows[1])
    table = torch.zeros(1, width, dtype=torch.int32, device=DEV)
    q, kn, vn = (_bf(rng.standard_normal((1, P, Hkv, D))) for _ in range(3))
    words = np.zeros((1, P, 2), np.int64)
    for i in range(P):
        words[0, i, i // 32] = 1 << i % 32
    mask = _d(words.astype(np.uint32).view(np.int32))
    st = _status()
    o = rd.rd_tree_attention_quant(q, kn, vn, kp, vp, 0.25, 0.5, table, _d(np.array([C], np.int32)),
                                   _d(np.array([P], np.int32)), mask, max_ctx=2 ** 31 - 1, dev_status=st)
    assert int(st) == 0
    times = torch.full((page,), float(C // page), dtype=torch.float64, device=DEV)
    times[:C % page] += 1                     # how often a row of the page is seen
    k, v = (_d(oq.decode(r[0], g, D, bits)) for r, g in ((rows[0], 0.25), (rows[1], 0.5)))
    for h in range(Hkv):
        x = (q[0, :, h].double() @ k[:, h].T) * D ** -0.5
        w = torch.exp(x - x.amax(1, keepdim=True)) * times
        w /= w.sum(1, keepdim=True)           # (a draft's own weight is below 2^-20)
        want, size = w @ v[:, h], w @ v[:, h].abs()
        assert ((o[0, :, h].double() - want).abs() <= want.abs() * 2.0 ** -8 + size * (2 * 295000 * 2.0 ** -23 + 0.01)).all()


@pytest.mark.parametrize("bits,D", [(4, 64), (4, 128), (8, 64), (8, 128)])
def test_factors_that_are_zero(bits, D):
    """Queries and a scale so small that a row's factor is 0 in 32 bits: equal weights, also where the context ends
    inside a tile."""
    for lens, ctx in (([3, 1], [70, 41]), ([2, 3], [9, 128])):
        s = make(2, 3, 4, 4, D, 64, bits, lens, ctx, seed=13, amp=1e-30)
        s["kn"].nan_to_num_()
        check(call(s, scale=1e-30), s, 1e-30)


def _close(o, s, scale):
    """check() without its absolute term, for outputs of any size: 32-bit sums are off by 2^-150 of nothing, outputs below
    2^-126 by half a step of 2^-133."""
    want, a_ctx, a_new, (kc, vc), (q, kn, _) = reference(s, scale)
    D, P = q.shape[3], q.shape[1]
    G = q.shape[2] // kn.shape[2]
    most, sums = np.zeros(q.shape[:3]), np.zeros(q.shape)
    for b in range(len(kc)):
        for h in range(q.shape[2]):
            k = np.abs(np.concatenate([kc[b][:, h // G], kn[b, :, h // G]]))
            most[b, :, h] = scale * (np.abs(q[b, :, h]) @ k.T).max(1)
            sums[b, :, h] = np.abs(vc[b][:, h // G]).sum(0)
    eps = 2 * (D + 8) * 2.0 ** -24 * most[..., None] + 2 * (P + s["max_ctx"]) * 2.0 ** -24 + 2.0 ** -20
    tol = np.maximum(np.abs(want) * 2.0 ** -8, 2.0 ** -134) + a_ctx * (2.0 ** -11 + eps) + a_new * (2.0 ** -8 + eps) + sums * 2.0 ** -32
    got = _f64(o)
    assert np.isfinite(got).all()
    worst = np.unravel_index(np.argmax(np.abs(got - want) - tol), got.shape)
    assert (np.abs(got - want) <= tol).all(), (worst, got[worst], want[worst], tol[worst])


SCALES = [1e-45, 1e-40, 1e-38, 1e-30, 1e30, 6e37]


@pytest.mark.parametrize("bits,D", [(4, 128), (8, 64)])
@pytest.mark.parametrize("gk", SCALES)
def test_key_scales(gk, bits, D):
    """Every scale of the keys: drafts are weighed as ever, and the cached keys too, with queries or a softmax scale
    that bring their scores to a few units or leave them at nothing."""
    gk = float(np.float32(gk))
    for seed, (amp, scale) in enumerate(((1.0, D ** -0.5), (1.0, 0.1 / gk), (0.05 / gk, 1.0))):
        if not (1e-37 < scale < 1e37 and 1e-37 < amp < 1e37 and amp * scale * gk < 3):
            continue                          # not numbers of 32 bits, or scores of thousands
        s = make(2, 5, 4, 4, D, 64, bits, [5, 3], [150, 41], seed=seed, amp=amp)
        size = 1.0 if seed == 0 else min(gk, 2.0 ** 90)           # drafts of the cache's size, as far as they may reach
        s["kn"], s["vn"] = (s["kn"].nan_to_num().float() * size).bfloat16(), s["vn"].nan_to_num()
        s["gk"] = gk
        _close(call(s, scale=scale), s, float(np.float32(scale)))


@pytest.mark.parametrize("bits,D", [(4, 128), (8, 64)])
@pytest.mark.parametrize("gv", SCALES)
def test_value_scales(gv, bits, D):
    """Every scale of the values, in one piece a row and in many, with drafts of the cache's size and with none."""
    gv = float(np.float32(gv))
    for mask, ctx in (("tree", [150, 41]), ("none", [150, 41]), ("tree", [9000, 41])):
        s = make(2, 5, 4, 4, D, 64, bits, [5, 3], ctx, seed=3, mask=mask)
        s["gv"] = gv
        s["vn"] = (s["vn"].nan_to_num().float() * gv).bfloat16()
        _close(call(s, scale=D ** -0.5), s, float(np.float32(D ** -0.5)))


@pytest.mark.parametrize("bits,D", [(4, 64), (4, 128), (8, 64)])
@pytest.mark.parametrize("e", [-149, -140, -127, -126, -100, 0, 90, 110, 124, 126, 127])
def test_append_at_the_ends_of_the_scales(e, bits, D):
    """Powers of two for a scale, where every quotient is exact: the definition's bytes, and read back what they stand
    for in bf16 (infinite behind its largest number)."""
    rd, rng = _rd(), np.random.default_rng(abs(e) + bits)
    T, Hkv, g = 40, 3, 2.0 ** e
    x = rng.standard_normal((T, Hkv, D)) * np.exp2(rng.integers(-12, 13, (T, Hkv, 1)))
    x[3, 1] = 0
    with np.errstate(over="ignore"):
        k = torch.from_numpy(np.clip(x * g * 16, -3.3e38, 3.3e38)).to(torch.bfloat16).to(DEV)
    kp, vp = (torch.zeros(1, 64, Hkv, oq.row_bytes(D, bits), dtype=torch.uint8, device=DEV) for _ in range(2))
    table, ctx, st = _d(np.zeros((1, 1), np.int32)), _d(np.zeros(1, np.int32)), _status()
    rd.rd_append_quant(k, k, _d(np.array([0, T], np.int32)), kp, vp, g, g, table, ctx, dev_status=st)
    assert int(st) == 0 and torch.equal(kp, vp)
    rows, xs = kp.cpu().numpy()[0, :T], _f64(k)
    want = np.stack([[oq.encode_row(xs[t, h], g, bits)[0] for h in range(Hkv)] for t in range(T)])
    np.testing.assert_array_equal(rows, want)
    out, _ = rd.rd_read_quant(kp, vp, g, g, table, _d(np.array([0, T], np.int64)), total=T, dev_status=st)
    np.testing.assert_array_equal(_f64(out), _f64(torch.from_numpy(oq.decode(rows, g, D, bits)).to(torch.bfloat16)))


def _written(x, g, bits):
    """The bytes of rows x [T, Hkv, D], and the values that they were made from."""
    T, Hkv, D = x.shape
    k = _bf(x)
    kp = torch.zeros(-(-T // 64), 64, Hkv, oq.row_bytes(D, bits), dtype=torch.uint8, device=DEV)
    table = torch.arange(kp.shape[0], dtype=torch.int32, device=DEV)[None].contiguous()
    _rd().rd_append_quant(k, k, _d(np.array([0, T], np.int32)), kp, torch.empty_like(kp), g, g, table, _d(np.zeros(1, np.int32)))
    return kp.cpu().numpy().reshape(-1, Hkv, kp.shape[3])[:T], _f64(k)


def _neighbours(rows):
    """Bytes of the definition that differ from these: none may."""
    got, x, g, bits = rows
    want = np.stack([oq.encode_row(r, g, bits)[0] for r in x.reshape(-1, x.shape[-1])]).reshape(got.shape)
    return np.argwhere(got != want)


@pytest.mark.parametrize("bits", [4, 8])
def test_values_beside_borders(bits):
    """Scales calibrated to the largest value are no short numbers, and values in simple ratios to it lie
    beside a border between two codes, nearer than a 32-bit quotient tells."""
    D = 64
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0] if bits == 4 else list((oq.E4M3[1:] + oq.E4M3[:-1])[-60:] / 2)
    most = 6.0 if bits == 4 else 448.0
    for j in range(1, 32):
        amax = (3.0 if bits == 4 else 7.0) * j
        g = float(np.float32(amax / (2688 if bits == 4 else 448)))
        x = np.zeros((8, 1, D))
        x[:, :, 0] = amax
        x[:, :, 1:16] = np.resize(np.array(ties) * amax / most, (8, 1, 15)) * np.where(np.arange(15) % 3 == 1, -1, 1)
        x[:, :, 16:] = np.random.default_rng(j).choice(ties, (8, 1, 48)) * amax / most
        x[4:] *= 2.0 ** -5                    # (in 4 bits: other scales of blocks)
        got, x = _written(x, g, bits)
        assert len(_neighbours((got, x, g, bits))) == 0, j


@pytest.mark.parametrize("bits", [4, 8])
def test_bytes_at_calibrated_scales(bits):
    """Every byte of many rows is the definition's; none is left out for lying beside a border."""
    rng = np.random.default_rng(bits)
    for D, T in ((64, 400), (128, 200)):
        x = rng.standard_normal((T, 4, D)) * np.exp(0.5 * rng.standard_normal((1, 4, D)))
        x[::7, :, ::5] = 0
        x = _f64(_bf(x))
        g = float(np.float32(np.abs(x).max() / (448 if bits == 8 else 2688)))
        for by in (1.0, 0.37, 3.0):           # beside the calibrated one, scales that saturate and that leave range
            got, y = _written(x, float(np.float32(g * by)), bits)
            assert len(_neighbours((got, y, float(np.float32(g * by)), bits))) == 0, (D, by)


@pytest.mark.parametrize("bits", [4, 8])
def test_values_are_rounded_once(bits):
    """Scales at which a product of 32 bits lies midway between two bf16 numbers and the exact one does not, found on
    the CPU; and scales whose values have few bits left (below 2^-126)."""
    rng, D, T = np.random.default_rng(bits), 64, 512
    rows = rng.integers(0, 256, (T, 1, oq.row_bytes(D, bits))).astype(np.uint8)
    if bits == 8:
        rows[(rows & 0x7f) == 0x7f] = 0
    else:
        rows[..., 32:] = rng.integers(1, 0x7f, (T, 1, 4))
    units = oq.decode(rows, 1.0, D, bits)
    scales, some = [3e-39, 7.3e-38, 1e37], np.unique(np.abs(units[units != 0]))
    while len(scales) < 12:                   # v g = (2 n + 1) 2^k / 2 + a little, with n of 8 bits
        v, n = rng.choice(some), 2 * int(rng.integers(128, 256)) + 1
        g = np.float32(n * 2.0 ** -12 / v)
        once, twice = (torch.tensor(float(v) * float(g), dtype=t) for t in (torch.float64, torch.float32))
        if not float(once) == float(twice) and int(twice.view(torch.int32)) & 0xffff == 0x8000:
            scales.append(float(g))
    pool, off = _d(rows.reshape(T // 64, 64, 1, -1)), _d(np.array([0, T], np.int64))
    table = torch.arange(T // 64, dtype=torch.int32, device=DEV)[None].contiguous()
    for g in scales:
        g = float(np.float32(g))
        k, v = _rd().rd_read_quant(pool, pool, g, g, table, off, total=T)
        x = units * g                         # exact in 64 bits
        e = np.maximum(np.frexp(x)[1] - 8, -133).astype(float)
        want = np.rint(x * 2.0 ** -e) * 2.0 ** e               # 8 bits, or multiples of 2^-133; ties to even
        want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
        assert torch.equal(k, v)
        np.testing.assert_array_equal(_f64(k), want, err_msg=str(g))


@pytest.mark.parametrize("cu", [[0, 10, 5, 30], [0, 30, 1, 2, 3, 4, 30], [20, 30, 0, 20], [5, 25, 5, 25, 5, 25], [0, 30, 0, 30],
                                [0, 0, 30, 12, 12, 17], [29, 30] + list(range(300)) * 1])
@pytest.mark.parametrize("bits", [4, 8])
def test_sequences_that_overlap(cu, bits):
    """cu_seqlens that does not ascend is flagged, and every request whose own sequence lies within the tokens has
    all of its rows: none grows by rows that nobody wrote."""
    rd, rng = _rd(), np.random.default_rng(bits)
    T, Hkv, D = 30, 2, 64
    cu = np.array(cu, np.int64)
    B = len(cu) - 1
    k = _bf(rng.standard_normal((T, Hkv, D)))
    ctx = np.arange(B, dtype=np.int32) % 40
    kp, vp = (torch.full((B + 1, 128, Hkv, oq.row_bytes(D, bits)), 0x55, dtype=torch.uint8, device=DEV) for _ in range(2))
    table, st = _d(rng.permutation(B + 1)[:B, None].astype(np.int32)), _status()
    new = rd.rd_append_quant(k, k, _d(cu.astype(np.int32)), kp, vp, 0.25, 0.25, table, _d(ctx), dev_status=st)
    assert int(st) == rd.DEV_BAD_LENGTH and torch.equal(kp, vp)
    fine = (cu[:-1] >= 0) & (cu[:-1] <= cu[1:]) & (cu[1:] <= T)
    np.testing.assert_array_equal(new.cpu().numpy(), ctx + np.where(fine, cu[1:] - cu[:-1], 0))
    rows = np.stack([[oq.encode_row(_f64(k[t, h]), 0.25, bits)[0] for h in range(Hkv)] for t in range(T)])
    want = np.full(kp.shape, 0x55, np.uint8)
    for b in np.flatnonzero(fine):
        n = int(cu[b + 1] - cu[b])
        want[int(table[b, 0]), ctx[b]:ctx[b] + n] = rows[cu[b]:cu[b + 1]]
    np.testing.assert_array_equal(kp.cpu().numpy(), want)


def test_long_sequences_that_overlap():
    """The same with sequences of many tokens, more requests than a CTA has threads, and a page that does not exist."""
    rd, rng = _rd(), np.random.default_rng(0)
    T, Hkv, D, B = 300, 40, 128, 400
    cu = np.sort(rng.integers(0, T + 1, B + 1))
    cu[[0, 1, 2, 3]] = 0, T, 7, 290           # 0 .. T, then a descent, then 7 .. 290
    cu[300], cu[301] = 0, 250
    k = _bf(rng.standard_normal((T, Hkv, D)))
    need = np.where(cu[1:] >= cu[:-1], cu[1:] - cu[:-1], 0)
    table, n = _tables(rng, B, -(-need // 64) + 0)
    table[2, 1] = n + 5
    st = _status()
    kp = torch.zeros(n, 64, Hkv, oq.row_bytes(D, 8), dtype=torch.uint8, device=DEV)
    ctx = _d(np.zeros(B, np.int32))
    new = rd.rd_append_quant(k, k, _d(cu.astype(np.int32)), kp, kp.clone(), 0.25, 0.25, _d(table), ctx, dev_status=st)
    assert int(st) == rd.DEV_BAD_LENGTH | rd.DEV_BAD_INDEX
    np.testing.assert_array_equal(new.cpu().numpy(), need)
    plain = torch.zeros(T, 1, Hkv, oq.row_bytes(D, 8), dtype=torch.uint8, device=DEV)      # one token a page
    rd.rd_append_quant(k, k, _d(np.array([0, T], np.int32)), plain, plain.clone(), 0.25, 0.25,
                       torch.arange(T, dtype=torch.int32, device=DEV)[None].contiguous(), ctx[:1])
    want = torch.zeros_like(kp)
    for b in range(B):
        for i in range(int(need[b])):
            if table[b, i // 64] < n:
                want[int(table[b, i // 64]), i % 64] = plain[int(cu[b]) + i, 0]
    assert torch.equal(kp, want)
