"""rd_token_logprobs and rd_accepted_logprobs against 64-bit numpy."""
import numpy as np
import pytest
import torch

from oracle import quant as oq

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _rd():
    import tree_attention_verify_gb300 as rd
    return rd


def _d(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def check(out, i, x, token, T=1.0, top=0):
    """fp32 sums of V terms over 256 threads or more, each 2^z off by 2^-21 and z by 2^-22 of
    itself; the same for the products of the entropy, relative to sum p |log p|."""
    x = x.double().cpu().numpy()
    lp, h, ids, tops, hs = oq.logprobs(x, token, T, top)
    eps = (len(x) / 256 + 60) * 2.0 ** -24 + 2.0 ** -20
    got = {k: v[i].cpu().numpy() for k, v in out.items()}
    close = lambda a, b: a == b or abs(a - b) <= eps * (1 + hs) + abs(b) * 2.0 ** -21
    assert close(float(got["logprob"]), lp), (got["logprob"], lp)
    assert abs(float(got["entropy"]) - h) <= eps * (1 + 2 * hs), (got["entropy"], h)
    np.testing.assert_array_equal(got["top_tokens"], ids)
    assert all(close(a, b) for a, b in zip(got["top_logprobs"].astype(float), tops))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,V,top", [(1, 1, 1), (3, 2, 2), (5, 40, 32), (2, 997, 0), (7, 1000, 5), (1, 4096, 32),
                                     (3, 16385, 8), (1, 32001, 20), (2, 128256, 20), (700, 2051, 3), (310, 9000, 32)])
def test_rows(dtype, n, V, top):
    rd = _rd()
    gen = torch.Generator(device=DEV).manual_seed(V)
    x = (2.5 * torch.randn(n, V, generator=gen, device=DEV)).to(TYPES[dtype])
    tokens = torch.randint(0, V, (n,), generator=gen, device=DEV, dtype=torch.int32)
    T = 1.0 if n % 2 else 0.6
    st = _status()
    out = rd.rd_token_logprobs(x, tokens, top=top, temperature=T, dev_status=st)
    assert int(st) == 0
    for i in sorted({0, n // 2, n - 1, min(n - 1, 5)}):
        check(out, i, x[i], int(tokens[i]), float(np.float32(T)), top)


@pytest.mark.parametrize("V", [5, 300, 20000, 70001])
def test_equal_logits(V):
    """Every logit alike (the list of candidates overfills), or two values."""
    rd = _rd()
    top = min(V, 32)
    x = torch.zeros(3, V, dtype=torch.bfloat16, device=DEV)
    x[1, 1::2] = -0.0
    x[2, V // 2:] = 3.0
    out = rd.rd_token_logprobs(x, _i32([0, V - 1, 0]), top=top)
    for i, token in enumerate((0, V - 1, 0)):
        check(out, i, x[i], token, 1.0, top)


@pytest.mark.parametrize("V", [3000, 50001, 128256])
@pytest.mark.parametrize("order", ["rising", "falling"])
def test_sorted_logits(V, order):
    """A row that keeps rising passes the threshold all the way."""
    rd = _rd()
    x = torch.linspace(-20, 20, V, device=DEV)
    x = (x if order == "rising" else x.flip(0)).expand(2, V).contiguous()
    for t in (x, x.bfloat16()):
        out = rd.rd_token_logprobs(t, _i32([0, V - 1]), top=32)
        check(out, 0, t[0], 0, 1.0, 32)
        check(out, 1, t[1], V - 1, 1.0, 32)


def test_masked_logits():
    """-inf in all but a few places, as a grammar leaves them."""
    rd = _rd()
    V = 32000
    x = torch.full((4, V), -float("inf"), device=DEV)
    x[0, 31999] = 3.0
    x[1, [5, 700, 30000]] = torch.tensor([-1e4, -1e4 + 1, -1e4], device=DEV)
    x[2, ::7] = torch.randn(len(range(0, V, 7)), device=DEV)
    x[3, 17] = -3e38
    tokens = [31999, 6, 7, 17]
    for t in (x, x.bfloat16()):
        out = rd.rd_token_logprobs(t, _i32(tokens), top=8)
        for i in range(4):
            check(out, i, t[i], tokens[i], 1.0, 8)
    x[:] = -float("inf")
    x[1, 5], x[2, 9] = float("nan"), float("inf")
    out = rd.rd_token_logprobs(x, _i32([0, 5, 9, 3]), top=2)
    for k in ("logprob", "entropy", "top_logprobs"):
        assert torch.isnan(out[k][:3]).all()
    assert out["top_tokens"][0].tolist() == [0, 1] and int(out["top_tokens"][2, 0]) == 9
    assert ((out["top_tokens"] >= 0) & (out["top_tokens"] < V)).all()


def test_far_and_large_logits():
    rd = _rd()
    x = torch.tensor([[1e30, 0.0, -1e30, 5e29], [60000.0, 59999.0, 0.0, -60000.0], [1e-30, 0.0, -1e-30, 0.0],
                      [0.0, 200.0, 100.0, 199.5]], device=DEV)
    for T in (1.0, 1e-3, 1e6):
        out = rd.rd_token_logprobs(x, _i32([0, 1, 2, 3]), top=4, temperature=T)
        for i in range(4):
            check(out, i, x[i], i, float(np.float32(T)), 4)
    # each thread's first logits far below the others
    V = 40000
    y = torch.full((1, V), -500.0, device=DEV)
    y[0, 20000:] = torch.linspace(0, 100, V - 20000, device=DEV)
    check(rd.rd_token_logprobs(y, _i32([V - 1]), top=3), 0, y[0], V - 1, 1.0, 3)


@pytest.mark.parametrize("dtype", TYPES)
def test_unaligned_rows_and_row_indices(dtype):
    """Rows that start anywhere; the same row twice; entries that are skipped; nothing is read outside."""
    rd = _rd()
    V, n_rows = 1001, 6
    flat = torch.full((n_rows * V + 16,), float("nan"), dtype=TYPES[dtype], device=DEV)
    for shift in (0, 1, 3, 7):
        x = flat[shift:shift + n_rows * V].view(n_rows, V)
        x.copy_(torch.randn(n_rows, V, device=DEV) * 3)
        rows, tokens = [5, 0, 0, 3, 2, 6, -1, 1], [7, V - 1, 0, -1, V, 3, 4, -5]
        st = _status()
        out = rd.rd_token_logprobs(x, _i32(tokens), rows=_i32(rows), top=3, dev_status=st)
        assert int(st) == rd.DEV_BAD_TOKEN | rd.DEV_BAD_INDEX
        for i in (0, 1, 2):
            check(out, i, x[rows[i]], tokens[i], 1.0, 3)
        assert (out["logprob"][3:] == 0).all() and (out["entropy"][3:] == 0).all()
        assert (out["top_tokens"][3:] == -1).all() and (out["top_logprobs"][3:] == 0).all()
        flat.fill_(float("nan"))


def test_accepted():
    rd = _rd()
    gen = torch.Generator(device=DEV).manual_seed(0)
    B, W, L, V, top = 6, 3, 4, 5000, 5
    beams = torch.randint(0, 3, (B, W, L), generator=gen, device=DEV, dtype=torch.int32)
    beams[:, :, 0] = 1
    pk = rd.rd_pack_beams(beams)
    P = W * L
    logits = (2 * torch.randn(B, P, V, generator=gen, device=DEV)).bfloat16()
    logits[:, :, :3] += 9
    acc = rd.rd_greedy_accept(logits, beams, pk["unpacker"], pk["packed_len"])
    st = _status()
    out = rd.rd_accepted_logprobs(logits, pk["unpacker"], acc["best_beam"], acc["n_accepted"], acc["out_tokens"], top=top,
                                  dev_status=st)
    assert int(st) == 0
    for b in range(B):
        a = int(acc["n_accepted"][b])
        for i in range(L):
            if i <= a:
                node = int(pk["unpacker"][b, int(acc["best_beam"][b]), i])
                token = int(acc["out_tokens"][b, i])
                check({k: v[b] for k, v in out.items()}, i, logits[b, node], token, 1.0, top)
                assert int(out["top_tokens"][b, i, 0]) == token       # greedy
            else:
                assert out["logprob"][b, i] == 0 and (out["top_tokens"][b, i] == -1).all()
    # wrong beams, lengths and nodes
    best, n, unp = acc["best_beam"].clone(), acc["n_accepted"].clone(), pk["unpacker"].clone()
    best[0], n[1] = W, L
    unp[2, int(best[2]), 0] = P
    got = rd.rd_accepted_logprobs(logits, unp, best, n, acc["out_tokens"], top=top, dev_status=st)
    assert int(st) == rd.DEV_BAD_INDEX
    assert (got["top_tokens"][:2] == -1).all() and (got["top_tokens"][2, 0] == -1).all() and (got["logprob"][:2] == 0).all()
    for k in out:
        assert torch.equal(got[k][3:], out[k][3:])


def test_graph_stream_and_given_outputs():
    rd = _rd()
    x = torch.randn(9, 30000, device=DEV).bfloat16()
    t = _i32(range(9))
    want = rd.rd_token_logprobs(x, t, top=4)
    out = {k: torch.empty_like(v) for k, v in want.items()}
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        assert rd.rd_token_logprobs(x, t, top=4, out=out)["entropy"] is out["entropy"]
    for _ in range(2):
        for v in out.values():
            v.zero_()
        g.replay()
        assert all(torch.equal(out[k], want[k]) for k in want)
    torch.cuda.synchronize()
    got = rd.rd_token_logprobs(x, t, top=4, stream=side)
    side.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    none = rd.rd_token_logprobs(x, t[:0], top=4)
    assert none["top_tokens"].shape == (0, 4)


def test_rows_past_32_bits():
    rd = _rd()
    V, n_rows = 131072, 17000                 # 2^31 logits and some
    x = torch.zeros(n_rows, V, dtype=torch.bfloat16, device=DEV)
    x[-1] = torch.randn(V, device=DEV).bfloat16()
    out = rd.rd_token_logprobs(x, _i32([5]), rows=_i32([n_rows - 1]), top=2)
    check(out, 0, x[-1], 5, 1.0, 2)


@pytest.mark.parametrize("n", [1, 400])
@pytest.mark.parametrize("dtype", TYPES)
def test_candidates_behind_a_low_start(dtype, n):
    """The first part of a row tells nothing of the rest: every later group is a candidate, and the
    list of them overfills (a row alone is shared by several CTAs, 400 are not)."""
    rd = _rd()
    V = 60000
    gen = torch.Generator(device=DEV).manual_seed(n)
    x = torch.full((1, V), -60.0, device=DEV)
    x[0, 20000:] = 3 * torch.randn(V - 20000, generator=gen, device=DEV)
    x = x.to(TYPES[dtype]).expand(n, V).contiguous()
    out = rd.rd_token_logprobs(x, _i32([V - 7] * n), top=32)
    for i in {0, n - 1}:
        check(out, i, x[i], V - 7, 1.0, 32)


def test_numbers_at_the_ends_of_the_range():
    """References and logits near the largest and the lowest numbers of each type, and infinities."""
    rd = _rd()
    V = 9000
    gen = torch.Generator(device=DEV).manual_seed(1)
    noise = torch.randn(V, generator=gen, device=DEV)
    low32, low16 = torch.finfo(torch.bfloat16).min, torch.finfo(torch.float16).min
    for dtype, low, tops in ((torch.float32, -3.4e38, (0.0, 9e29, 2e30, 3.3e38, -9e37, -2e38)),
                             (torch.bfloat16, low32, (0.0, 9e29, 2e30, 3.3e38, -9e37, -2e38)),
                             (torch.float16, low16, (0.0, 65504.0, -60000.0))):
        x = torch.full((len(tops), V), low, dtype=torch.float64, device=DEV)
        for i, top in enumerate(tops):
            x[i, 3::50] = top
            x[i, 7::50] = top + noise[7::50] * (abs(top) * 2.0 ** -6 + 1)
            x[i, 11::50] = -float("inf")
        x = x.clamp(max=torch.finfo(dtype).max).to(dtype)
        tokens = [3, 7, 53, 57, 103, 107][:len(tops)]
        for T in (1.0, 1e3, 1e-2):
            out = rd.rd_token_logprobs(x, _i32(tokens), top=4, temperature=T)
            for i, t in enumerate(tokens):
                far = oq.logprobs(x[i].double().cpu().numpy(), t, float(np.float32(T)), 4)[0] < -2.0 ** 128
                if far:                       # below every 32-bit number: its rounding is -inf
                    assert float(out["logprob"][i]) == -float("inf")
                    # (the rest of the entry against a token that has a logarithm)
                    t = int(out["top_tokens"][i, 0])
                    one = rd.rd_token_logprobs(x[i:i + 1], _i32([t]), top=4, temperature=T)
                    check(one, 0, x[i], t, float(np.float32(T)), 4)
                else:
                    check(out, i, x[i], t, float(np.float32(T)), 4)


@pytest.mark.parametrize("dtype", TYPES)
def test_one_nan_anywhere(dtype):
    rd = _rd()
    V = 40009
    x = torch.randn(6, V, device=DEV).to(TYPES[dtype])
    for i, at in enumerate((0, 5, 16390, 20000, V - 1)):
        x[i, at] = float("nan")
    out = rd.rd_token_logprobs(x, _i32([9] * 6), top=2)
    assert torch.isnan(out["logprob"][:5]).all() and torch.isnan(out["entropy"][:5]).all()
    check(out, 5, x[5], 9, 1.0, 2)


@pytest.mark.parametrize("size", [1e36, 1e28, 1e-28, 2e-38])
def test_very_large_and_small_temperatures(size):
    """Logits of the temperature's size: sums of differences would leave 32 bits."""
    rd = _rd()
    gen = torch.Generator(device=DEV).manual_seed(3)
    x = (3 * torch.randn(2, 50000, generator=gen, device=DEV).double() * size).float()
    T = float(np.float32(size))
    out = rd.rd_token_logprobs(x, _i32([7, 49999]), top=3, temperature=T)
    check(out, 0, x[0], 7, T, 3)
    check(out, 1, x[1], 49999, T, 3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [538, 40000, 128256])
def test_a_token_with_nearly_all_of_the_probability(V, dtype):
    """log p = -log(1 + l) with l the sum of the other weights: as exact, relative to itself, as l.  Each weight
    is off by its exponent's roundings (|z| up to 64, 2 x 2^-24 of it) and the hardware's 2^x (2^-21), the sum by
    a rounding a term of a thread and of the joins."""
    rd = _rd()
    gen = torch.Generator(device=DEV).manual_seed(V)
    x = torch.randn(6, V, generator=gen, device=DEV).clamp(-4, 4)
    for i, (at, top) in enumerate(((0, 14.0), (V - 1, 20.0), (300, 24.0), (V // 2, 31.0), (7, 38.0), (V - 9, 9.0))):
        x[i, at] = top
    x = x.to(TYPES[dtype])
    tokens = x.float().argmax(1).int()
    out = rd.rd_token_logprobs(x, tokens, top=1)
    want = x.double()
    others = torch.exp(want - want.amax(1, keepdim=True))
    others.scatter_(1, tokens.long()[:, None], 0.0)
    want = -torch.log1p(others.sum(1))
    eps = (V / 256 + 60) * 2.0 ** -24 + 64 * 0.7 * 2.0 ** -23 + 2.0 ** -21
    assert ((out["logprob"].double() - want).abs() <= eps * want.abs()).all(), (out["logprob"], want)
    assert torch.equal(out["top_logprobs"][:, 0], out["logprob"])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", range(1, 18))
def test_rows_without_a_whole_group(V, dtype):
    """Rows of a few logits at every offset from 16 bytes: none, one or two groups that lie partly outside, and every
    logit an alternative."""
    rd = _rd()
    n = 200
    gen = torch.Generator(device=DEV).manual_seed(V)
    flat = torch.full((n * V + 16,), float("nan"), dtype=TYPES[dtype], device=DEV)
    for shift in range(8):
        x = flat[shift:shift + n * V].view(n, V)
        x.copy_(3 * torch.randn(n, V, generator=gen, device=DEV))
        tokens = torch.randint(0, V, (n,), generator=gen, device=DEV, dtype=torch.int32)
        out = rd.rd_token_logprobs(x, tokens, top=V)
        order = torch.sort(x.double(), dim=1, descending=True, stable=True).indices
        assert torch.equal(out["top_tokens"].long(), order)
        for i in (0, 1, n // 2, n - 1):
            check(out, i, x[i], int(tokens[i]), 1.0, V)
        flat.fill_(float("nan"))


def _rows_of_many_candidates(V, dtype):
    """Rows whose first part tells nothing of the largest logits, with equal logits where the type is short."""
    up = torch.linspace(-30, 30, V, device=DEV)
    steps = torch.floor(torch.linspace(0, 40, V, device=DEV))
    saw = up + 5 * (torch.arange(V, device=DEV) % 3 == 0)
    late = torch.where(torch.arange(V, device=DEV) < V // 2, -up - 60, up)
    few = torch.where(torch.arange(V, device=DEV) % 2048 < 16, up + 100, up)       # some threads have all of the largest
    return torch.stack([up, steps, saw, late, few, -(up * up)]).to(TYPES[dtype])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [20000, 128256, 1 << 20])
@pytest.mark.parametrize("copies", [1, 40])
def test_many_candidates(V, dtype, copies):
    rd = _rd()
    x = _rows_of_many_candidates(V, dtype)
    rows = torch.arange(len(x), dtype=torch.int32, device=DEV).repeat(copies)      # (one CTA a row where there are many)
    for top in (1, 32):
        out = rd.rd_token_logprobs(x, torch.full_like(rows, 7), rows=rows, top=top)
        for i in range(len(x)):
            want = torch.sort(x[i], descending=True, stable=True).indices[:top]
            for c in {0, copies - 1}:
                assert torch.equal(out["top_tokens"][c * len(x) + i].long(), want), (i, top)
            if V < 1 << 20:
                check(out, i, x[i], 7, 1.0, top)


def test_rising_rows_are_read_a_few_times():
    """2^22 logits that rise: about 500 times the falling row's time, if each pass over them left out a thousand."""
    rd = _rd()
    V = 1 << 22
    up = torch.linspace(-30, 30, V, device=DEV)[None]
    rows, t = (up.contiguous(), up.flip(1).contiguous()), _i32([5])

    def time(x):
        rd.rd_token_logprobs(x, t, top=32)
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(3):
            out = rd.rd_token_logprobs(x, t, top=32)
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b), out

    (rising, out), (falling, other) = time(rows[0]), time(rows[1])
    print(f"rising {rising / 3:.3f} ms, falling {falling / 3:.3f} ms")
    want = torch.sort(rows[0], descending=True, stable=True)
    assert torch.equal(out["top_tokens"].long(), want.indices[:, :32])
    assert rising < 100 * falling


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_differences_beyond_the_range(dtype):
    """Logits of either sign near the largest numbers under a temperature of their size: the differences are no 32-bit
    numbers, their quotients are a few units."""
    rd = _rd()
    gen = torch.Generator(device=DEV).manual_seed(5)
    for V in (3, 700, 40000):
        x = (torch.rand(4, V, generator=gen, device=DEV) * 6.6e38 - 3.3e38).to(dtype) if V > 3 else \
            torch.tensor([[3e38, -3e38, 0.0]] * 4, device=DEV).to(dtype)
        x[1, 1] = -float("inf")
        for T in (3.0e38, 4e37, 1e30, 2.0):
            t = [0, 2, V - 1, 1]
            out = rd.rd_token_logprobs(x, _i32(t), top=3, temperature=T)
            for i in range(4):
                far = oq.logprobs(x[i].double().cpu().numpy(), t[i], float(np.float32(T)), 3)
                if np.isfinite(np.float32(far[0])) and np.isfinite(np.float32(far[3])).all():
                    check(out, i, x[i], t[i], float(np.float32(T)), 3)
