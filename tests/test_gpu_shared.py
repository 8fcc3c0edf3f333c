"""rd_tree_attention_shared (groups of requests with shared leading pages) on the
GPU against the fp64 oracle of the paged tree attention.

Tolerance, per element: the softmax weights enter the second product rounded to
bf16, each off by at most 2^-8 of itself, so the weighted sum is off by at most
2^-8 A, where A is the attention of |v|; the result is rounded to bf16 once,
2^-8 |o|.  Scores and sums are fp32: a score of D <= 128 products errs by at
most 128 * 2^-24 * sum |q k| * scale, which moves a weight by under 2^-12 of itself
for these inputs (sum |q k| * scale < 16), numerator and denominator alike: 2^-11 A."""
import numpy as np
import pytest
import torch

import oracle
import workloads
from workloads import bf16_bits

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
NAN = float("nan")


def _rd():
    import tree_attention_verify_gb300 as rd
    return rd


def make(B, W, L, Hq, Hkv, D, page, offsets, pages, suffix, seed=0, junk=NAN, spare=2):
    """A batch over a shared-prefix cache.  What no request may read (pages nobody
    names, page tails behind a context, rows behind packed_len, table entries
    behind a row's pages) holds `junk` or wild ids."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    P = W * L
    beams = workloads.draft_trees(B, W, L, 50, ("p", 0.4), rng).beams
    pk = oracle.oracle_pack(beams, P)
    gid = np.full(B, -1)
    for g in range(len(pages)):
        gid[offsets[g]:offsets[g + 1]] = g
    skip = np.array([pages[g] * page if g >= 0 else 0 for g in gid])
    own = rng.integers(0, suffix + 1, B)
    own[rng.integers(0, B)] = 0
    ctx = skip + own
    need = -(-ctx // page)
    total = sum(pages) + int((need - skip // page).sum()) + spare
    ids = list(rng.permutation(total))
    shared = [[ids.pop() for _ in range(n)] for n in pages]
    width = max(1, int(need.max())) + 1
    table = rng.integers(-9, total + 9, (B, width)).astype(np.int32)
    k = torch.full((total, page, Hkv, D), junk, dtype=torch.bfloat16, device=DEV)
    v = k.clone()

    def fill(p, n):
        k[p, :n] = torch.randn(n, Hkv, D, generator=gen, device=DEV, dtype=torch.bfloat16)
        v[p, :n] = torch.randn(n, Hkv, D, generator=gen, device=DEV, dtype=torch.bfloat16)
    for s in shared:
        for p in s:
            fill(p, page)
    for b in range(B):
        row = list(shared[gid[b]]) if gid[b] >= 0 else []
        while len(row) < need[b]:
            row.append(ids.pop())
            fill(row[-1], min(page, int(ctx[b]) - (len(row) - 1) * page))
        table[b, :len(row)] = row
    r = dict(dtype=torch.bfloat16, device=DEV, generator=gen)
    q, kn, vn = torch.randn(B, P, Hq, D, **r), torch.randn(B, P, Hkv, D, **r), torch.randn(B, P, Hkv, D, **r)
    for b in range(B):
        n = int(pk["packed_len"][b])
        for t in (q, kn, vn):
            t[b, n:] = junk
    return dict(q=q, k_new=kn, v_new=vn, k_pool=k, v_pool=v, table=table, ctx=ctx.astype(np.int32),
                offsets=np.array(offsets, np.int32), pages=np.array(pages, np.int32),
                lens=pk["packed_len"].astype(np.int32), mask=pk["mask"], max_ctx=int(ctx.max()))


def call(s, st=None, **kw):
    rd = _rd()
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
    return rd.rd_tree_attention_shared(
        s["q"], s["k_new"], s["v_new"], s["k_pool"], s["v_pool"], d(s["table"]), d(s["ctx"]), d(s["offsets"]),
        d(s["pages"]), d(s["lens"]), d(s["mask"].view(np.int32)), max_ctx=s["max_ctx"], dev_status=st, **kw)


def reference(s, scale=0.0):
    def ref(absolute):
        def bits(t):                              # what may not be read is read as zero
            return bf16_bits(torch.nan_to_num(t.abs() if absolute else t))
        v, vn = bits(s["v_pool"]), bits(s["v_new"])
        q, k, kn = (bf16_bits(torch.nan_to_num(s[n])) for n in ("q", "k_pool", "k_new"))
        table = np.where((s["table"] < 0) | (s["table"] >= len(k)), 0, s["table"]).astype(np.int32)
        return oracle.oracle_tree_attention_paged(q, kn, vn, k, v, table, s["ctx"], s["lens"], s["mask"], scale)
    return ref(False), ref(True)


def check(o, s, scale=0.0):
    want, size = reference(s, scale)
    got = o.float().cpu().numpy()
    tol = 2.0 ** -8 * (size + np.abs(want)) + 2.0 ** -11 * size
    err = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), f"{int((err > tol).sum())} of {err.size} off, worst {np.max(err / np.maximum(tol, 1e-30)):.3g}"
    for b, n in enumerate(s["lens"]):
        assert (got[b, n:] == 0).all()


CASES = {
    # one request, one page; one token
    "one": dict(B=1, W=1, L=1, Hq=1, Hkv=1, D=64, page=64, offsets=[0, 1], pages=[1], suffix=0),
    "one token each": dict(B=8, W=1, L=1, Hq=32, Hkv=8, D=128, page=64, offsets=[0, 8], pages=[17], suffix=70),
    "tokens, no own context": dict(B=5, W=1, L=1, Hq=8, Hkv=8, D=128, page=128, offsets=[0, 5], pages=[9], suffix=0),
    "half chunks": dict(B=4, W=4, L=3, Hq=8, Hkv=4, D=128, page=64, offsets=[0, 2, 4], pages=[1, 3], suffix=65),
    "groups of five heads": dict(B=13, W=4, L=4, Hq=20, Hkv=4, D=64, page=64, offsets=[0, 3, 4, 9, 9, 13],
                                 pages=[5, 7, 0, 2, 12], suffix=333),
    "outside any group": dict(B=9, W=3, L=4, Hq=6, Hkv=2, D=128, page=256, offsets=[2, 6, 7], pages=[3, 1], suffix=400),
    "many rows": dict(B=33, W=8, L=6, Hq=16, Hkv=1, D=128, page=64, offsets=[0, 33], pages=[11], suffix=20),
    "whole units": dict(B=40, W=2, L=3, Hq=40, Hkv=40, D=64, page=128, offsets=[0, 20, 40], pages=[4, 7], suffix=130),
    "more requests than the table": dict(B=500, W=1, L=2, Hq=4, Hkv=2, D=128, page=64, offsets=[0, 1, 499, 500],
                                         pages=[2, 5, 1], suffix=90),
    # 64 rows per kv head and one more; 16, 32, 33 and 48 of them
    "64 rows": dict(B=6, W=4, L=4, Hq=8, Hkv=2, D=128, page=64, offsets=[0, 6], pages=[5], suffix=500),
    "66 rows": dict(B=6, W=11, L=1, Hq=12, Hkv=2, D=128, page=64, offsets=[0, 6], pages=[5], suffix=500),
    "64 rows d64": dict(B=3, W=8, L=8, Hq=4, Hkv=4, D=64, page=64, offsets=[0, 3], pages=[3], suffix=700),
    "16 rows": dict(B=5, W=4, L=2, Hq=8, Hkv=4, D=128, page=128, offsets=[1, 5], pages=[2], suffix=300),
    "32 rows d64": dict(B=5, W=4, L=4, Hq=8, Hkv=4, D=64, page=128, offsets=[0, 5], pages=[2], suffix=300),
    "33 rows": dict(B=7, W=11, L=1, Hq=6, Hkv=2, D=64, page=64, offsets=[0, 7], pages=[1], suffix=129),
    "48 rows": dict(B=4, W=8, L=6, Hq=3, Hkv=3, D=128, page=256, offsets=[0, 4], pages=[1], suffix=1000),
    # enough units that the CTAs take them whole off a counter
    "counter": dict(B=50, W=4, L=3, Hq=120, Hkv=40, D=64, page=64, offsets=[0, 20, 50], pages=[2, 1], suffix=100),
    # two requests whose own contexts are long: cut into many pieces
    "long own contexts": dict(B=2, W=2, L=4, Hq=8, Hkv=2, D=128, page=64, offsets=[0, 2], pages=[4], suffix=6000),
    "long own contexts, one token": dict(B=2, W=1, L=1, Hq=8, Hkv=1, D=64, page=64, offsets=[0, 2], pages=[1],
                                         suffix=9000),
    "long": dict(B=3, W=5, L=4, Hq=4, Hkv=2, D=128, page=64, offsets=[0, 3], pages=[129], suffix=200),
    # more requests and groups than the plan keeps in shared memory: in ranges, off the counter
    "1100 requests": dict(B=1100, W=1, L=1, Hq=2, Hkv=1, D=64, page=64, offsets=list(range(0, 82, 2)) + list(range(81, 1101)),
                          pages=[i % 3 for i in range(1060)], suffix=40),
    "1500 requests": dict(B=1500, W=1, L=2, Hq=2, Hkv=1, D=64, page=64, offsets=list(range(0, 800, 2)) + list(range(800, 1501)),
                          pages=[(i + 1) % 2 for i in range(1100)], suffix=50),
    # more than 64 rows per kv head, units enough to be taken whole; more requests than a table of them holds
    "80 rows, whole units": dict(B=80, W=5, L=4, Hq=32, Hkv=8, D=128, page=64, offsets=[0, 30, 80], pages=[3, 1], suffix=100),
    "72 rows, 600 requests": dict(B=600, W=3, L=4, Hq=6, Hkv=1, D=64, page=64, offsets=[0, 600], pages=[2], suffix=70),
    # two and three units of up to 64 rows a kv head, the last one short or empty
    "160 rows": dict(B=6, W=8, L=5, Hq=8, Hkv=2, D=128, page=64, offsets=[0, 4, 6], pages=[5, 2], suffix=300),
    "2 x 33 heads": dict(B=3, W=2, L=1, Hq=66, Hkv=2, D=64, page=64, offsets=[0, 3], pages=[2], suffix=90),
    "192 rows, whole units": dict(B=70, W=8, L=8, Hq=24, Hkv=8, D=64, page=64, offsets=[0, 50], pages=[3], suffix=60),
    "160 rows, long own contexts": dict(B=2, W=8, L=5, Hq=8, Hkv=2, D=64, page=64, offsets=[0, 2], pages=[2], suffix=5000),
    "100 rows, long own contexts": dict(B=2, W=5, L=5, Hq=8, Hkv=2, D=128, page=64, offsets=[0, 2], pages=[2], suffix=5000),
    "128 rows": dict(B=9, W=8, L=4, Hq=8, Hkv=2, D=128, page=64, offsets=[0, 2, 9], pages=[9, 3], suffix=200),
    "120 rows, whole units": dict(B=80, W=5, L=1, Hq=192, Hkv=8, D=64, page=64, offsets=[0, 50], pages=[3], suffix=60),
    "150 rows, 600 requests": dict(B=600, W=5, L=5, Hq=6, Hkv=1, D=64, page=64, offsets=[0, 600], pages=[2], suffix=70),
    # one of many units far longer than the others
    "counter, long own contexts": dict(B=160, W=1, L=3, Hq=8, Hkv=8, D=64, page=64, offsets=[0, 150], pages=[1],
                                       suffix=2500),
    # as many drafts as a request may have; many query heads of one kv head
    "256 drafts": dict(B=2, W=32, L=8, Hq=8, Hkv=2, D=128, page=64, offsets=[0, 2], pages=[3], suffix=200),
    "200 heads of one": dict(B=3, W=1, L=1, Hq=200, Hkv=1, D=128, page=64, offsets=[0, 3], pages=[4], suffix=150),
    "64 heads of one": dict(B=3, W=1, L=1, Hq=64, Hkv=1, D=64, page=64, offsets=[0, 3], pages=[4], suffix=150),
}


@pytest.mark.parametrize("name", list(CASES))
def test_matches_oracle(name):
    s = make(**CASES[name], seed=len(name))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    o = call(s, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    check(o, s)
    again = call(s, st, out=torch.full_like(o, NAN))
    assert torch.equal(o.view(torch.int16), again.view(torch.int16))    # the same bits every time


def test_rows_without_a_visible_key_are_zero():
    s = make(**CASES["half chunks"], seed=4)
    s["pages"][:] = 0
    s["ctx"][:] = 0
    s["mask"] = s["mask"].copy()
    s["mask"][0, 0] = 0                                # node 0 of request 0 sees nothing at all
    s["lens"] = s["lens"].copy()
    s["lens"][2] = 0                                   # request 2 has no nodes
    o = call(s)
    check(o, s)
    assert (o[0, 0] == 0).all() and (o[2] == 0).all()


def test_given_scale_and_infinities():
    s = make(**CASES["outside any group"], seed=6)
    check(call(s, scale=0.31), s, 0.31)
    # an infinite key: its weight is 1 where the score is +inf (the row is NaN, as
    # inf - inf), 0 where it is -inf; other requests are untouched
    k = s["k_pool"].clone()
    page = int(s["table"][8, 0])
    if s["ctx"][8] > 0:
        k[page, 0, 0, 0] = float("inf")
    o = call({**s, "k_pool": k})
    want, _ = reference(s)
    np.testing.assert_allclose(o[:8].float().cpu().numpy(), want[:8], atol=2e-2, rtol=1e-2)


def test_wrong_groups_are_flagged_and_the_outputs_stay():
    rd = _rd()
    s = make(**CASES["groups of five heads"], seed=9)
    bad = [(dict(offsets=np.array([0, 5, 3, 9, 9, 13], np.int32)), rd.DEV_BAD_INDEX),
           (dict(offsets=np.array([-1, 3, 4, 9, 9, 13], np.int32)), rd.DEV_BAD_INDEX),
           (dict(offsets=np.array([0, 3, 4, 9, 9, 14], np.int32)), rd.DEV_BAD_INDEX),
           (dict(pages=np.array([-1, 7, 0, 2, 12], np.int32)), rd.DEV_BAD_LENGTH),
           (dict(pages=np.array([5, 7, 0, 2, 2 ** 31 - 1], np.int32)), rd.DEV_BAD_LENGTH)]
    for kw, flag in bad:
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        o = call({**s, **kw}, st)
        assert st.item() == flag
        check(o, s)


def test_wrong_requests_are_skipped():
    rd = _rd()
    s = make(**CASES["groups of five heads"], seed=10)
    want, _ = reference(s)
    for b, kw in ((0, dict(ctx=5 * 64 - 1)), (9, dict(ctx=-3)), (9, dict(ctx=s["max_ctx"] + 1)), (4, dict(lens=17)),
                  (4, dict(lens=-1))):
        t = {n: s[n].copy() for n in ("ctx", "lens")}
        for n, x in kw.items():
            t[n][b] = x
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        o = call({**s, **t}, st).float().cpu().numpy()
        assert st.item() == rd.DEV_BAD_LENGTH
        assert (o[b] == 0).all()
        rest = np.arange(13) != b
        np.testing.assert_allclose(o[rest], want[rest], atol=2e-2, rtol=1e-2)
    # prefix pages that differ, or are out of range: the first request's are read
    t = s["table"].copy()
    t[12, 3] = (t[12, 3] + 1) % len(s["k_pool"])
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    o = call({**s, "table": t}, st)
    assert st.item() == rd.DEV_BAD_INDEX
    check(o, s)
    t[9:13, 2] = len(s["k_pool"]) + 7
    st.zero_()
    call({**s, "table": t}, st)
    assert st.item() == rd.DEV_BAD_INDEX


@pytest.mark.parametrize("name", ["half chunks", "groups of five heads", "counter", "many rows", "192 rows, whole units",
                                  "1100 requests"])
def test_padded_requests_in_a_group(name):
    """Finished requests stay in their groups: no drafts, no context, no pages.  The
    others' outputs and the status do not depend on them, a group's first among them."""
    s = make(**CASES[name], seed=13)
    for n in ("ctx", "lens", "table"):
        s[n] = s[n].copy()
    o = s["offsets"]
    for b in {int(o[0]), int(o[1]) - 1, int(o[-2])}:
        s["ctx"][b] = s["lens"][b] = 0
        s["table"][b] = -1
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = call(s, st)
    assert st.item() == 0
    check(out, s)
    s["lens"][:] = 0                                   # and nobody has any
    assert not call(s, st).any() and st.item() == 0


def test_equals_the_paged_call_without_groups():
    rd = _rd()
    s = make(**CASES["half chunks"], seed=11)
    s["offsets"], s["pages"] = np.zeros(1, np.int32), np.zeros(0, np.int32)
    for n in ("q", "k_new", "v_new", "k_pool", "v_pool"):
        s[n] = torch.nan_to_num(s[n])
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
    a = call(s)
    b = rd.rd_tree_attention_paged(s["q"], s["k_new"], s["v_new"], s["k_pool"], s["v_pool"], d(s["table"]),
                                   d(s["ctx"]), d(s["lens"]), d(s["mask"].view(np.int32)), max_ctx=s["max_ctx"])
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_graphs_streams_and_one_workspace():
    rd = _rd()
    s = make(**CASES["outside any group"], seed=12)
    B, P, Hq, D = s["q"].shape
    ws = torch.empty(rd.rd_tree_attention_shared_workspace_size(B, P, Hq, 2, D, s["max_ctx"], 2, DEV),
                     dtype=torch.uint8, device=DEV)
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
    args = [s["q"], s["k_new"], s["v_new"], s["k_pool"], s["v_pool"], d(s["table"]), d(s["ctx"]), d(s["offsets"]),
            d(s["pages"]), d(s["lens"]), d(s["mask"].view(np.int32))]
    want = rd.rd_tree_attention_shared(*args, max_ctx=s["max_ctx"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = rd.rd_tree_attention_shared(*args, max_ctx=s["max_ctx"], stream=side)
    side.synchronize()
    assert torch.equal(want, other)
    outs, graphs = [torch.empty_like(want) for _ in range(2)], []
    for o in outs:                                     # two graphs that share a workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            rd.rd_tree_attention_shared(*args, max_ctx=s["max_ctx"], out=o, workspace=ws)
        graphs.append(g)
    q2 = s["q"].flip(2).contiguous()
    for q in (s["q"].clone(), q2):
        s["q"].copy_(q)
        ws.fill_(255)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o in outs:
            check(o, s)


@pytest.mark.parametrize("pair", [("one token each", "many rows"), ("counter", "48 rows"), ("whole units", "whole units")])
def test_two_streams_at_once(pair):
    """Calls that overlap in time, each with a workspace of its own."""
    rd = _rd()
    runs = []
    for i, name in enumerate(pair):
        s = make(**CASES[name], seed=20 + i)
        d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
        args = [s["q"], s["k_new"], s["v_new"], s["k_pool"], s["v_pool"], d(s["table"]), d(s["ctx"]), d(s["offsets"]),
                d(s["pages"]), d(s["lens"]), d(s["mask"].view(np.int32))]
        alone = rd.rd_tree_attention_shared(*args, max_ctx=s["max_ctx"])
        runs.append((args, s, alone, torch.cuda.Stream(), torch.zeros(1, dtype=torch.int32, device=DEV)))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(12):
        for i, (args, s, _, stream, st) in enumerate(runs):
            outs[i].append(rd.rd_tree_attention_shared(*args, max_ctx=s["max_ctx"], dev_status=st, stream=stream))
    torch.cuda.synchronize()
    for i, (_, s, alone, _, st) in enumerate(runs):
        assert st.item() == 0
        check(alone, s)
        assert all(torch.equal(alone.view(torch.int16), o.view(torch.int16)) for o in outs[i])


@pytest.mark.parametrize("name", ["one token each", "66 rows", "counter"])
def test_pages_past_32_bits(name):
    """Pools whose last pages begin behind 2^32 elements."""
    s = make(**CASES[name], seed=30)
    n, page, Hkv, D = s["k_pool"].shape
    total = 2 ** 32 // (page * Hkv * D) + 1 + n        # 8.6 GB each
    first = total - n
    big = {}
    for p in ("k_pool", "v_pool"):
        big[p] = torch.empty((total, page, Hkv, D), dtype=torch.bfloat16, device=DEV)
        big[p][:first].fill_(NAN)
        big[p][first:].copy_(s[p])
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    o = call({**s, **big, "table": s["table"] + first}, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    check(o, s)


def test_refuses_before_a_launch():
    rd = _rd()
    s = make(**CASES["one"], seed=1)
    with pytest.raises(rd.RdError):
        call(s, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(rd.RdError):                    # pages of 32 positions
        call({**s, "k_pool": s["k_pool"].view(-1, 32, 1, 64), "v_pool": s["v_pool"].view(-1, 32, 1, 64)})
    with pytest.raises(ValueError):
        call({**s, "offsets": np.zeros(3, np.int32)})
    with pytest.raises(ValueError):
        call({**s, "ctx": np.zeros(2, np.int32)})
    with pytest.raises(TypeError):
        call({**s, "pages": np.zeros(1, np.int64)})
    with pytest.raises(ValueError):
        call(s, out=torch.empty(1, 1, 2, 64, dtype=torch.bfloat16, device=DEV))


@pytest.mark.parametrize("name", ["one token each", "many rows", "48 rows", "counter"])
def test_a_wait_that_runs_out_is_reported(name):
    rd = _rd()
    s = make(**CASES[name], seed=2)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    B, P, Hq, D = s["q"].shape
    size = rd.rd_tree_attention_shared_workspace_size(B, P, Hq, s["k_new"].shape[2], D, s["max_ctx"], len(s["pages"]), DEV)
    for fill in (0, 255, 7):                           # tables that the kernels then leave as they are
        ws = torch.full((size,), fill, dtype=torch.uint8, device=DEV)
        rd.rd_debug_stall_attention(2_000_000)
        try:
            call(s, st, workspace=ws)
            torch.cuda.synchronize()
        finally:
            rd.rd_debug_stall_attention(0)
        assert st.item() & rd.DEV_TIMEOUT
        st.zero_()
        check(call(s, st, workspace=ws), s)
        assert st.item() == 0


def test_a_run_of_steps_over_one_cache():
    """Serving steps as they are used together: prompts are reserved and branch,
    the branches are verified over the shared pages, accepted drafts committed,
    finished rows freed and the pool compacted; each step's attention against the
    oracle on the cache as it then stands."""
    rd = _rd()
    rng = np.random.default_rng(5)
    gen = torch.Generator(device=DEV).manual_seed(5)
    R, N, page, width, Hq, Hkv, D, W, L, V = 8, 96, 64, 16, 8, 2, 128, 3, 4, 64
    P = W * L
    i32 = dict(dtype=torch.int32, device=DEV)
    k_pool, v_pool = (torch.randn(N, page, Hkv, D, generator=gen, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    table, held, refs, ctx = (torch.full((R, width), -1, **i32), torch.zeros(R, **i32), torch.zeros(N, **i32),
                              torch.zeros(R, **i32))
    st = torch.zeros(1, **i32)
    prompts = {0: 5 * page + 17, 4: 2 * page}          # rows 0 and 4 hold prompts, 1-3 and 5-7 branch off
    lens = torch.tensor([prompts.get(r, 0) for r in range(R)], **i32)
    rd.rd_resize_pages(table, held, refs, lens, page, dev_status=st)
    ctx.copy_(lens)
    par, kid = torch.tensor([0, 0, 0, 4, 4, 4], **i32), torch.tensor([1, 2, 3, 5, 6, 7], **i32)
    rd.rd_fork_pages(k_pool, v_pool, table, held, refs, ctx, par, kid, dev_status=st)
    offsets, pages = torch.tensor([0, 4, 8], **i32), torch.tensor([5, 2], **i32)
    for step in range(4):
        rd.rd_resize_pages(table, held, refs, torch.where(ctx > 0, ctx + L, ctx), page, dev_status=st)
        beams = torch.from_numpy(workloads.draft_trees(R, W, L, V, ("p", 0.4), rng).beams).to(DEV)
        pk = rd.rd_pack_beams(beams, P, dev_status=st)
        q = torch.randn(R, P, Hq, D, generator=gen, device=DEV, dtype=torch.bfloat16)
        kn, vn = (torch.randn(R, P, Hkv, D, generator=gen, device=DEV, dtype=torch.bfloat16) for _ in range(2))
        o = rd.rd_tree_attention_shared(q, kn, vn, k_pool, v_pool, table, ctx, offsets, pages, pk["packed_len"],
                                        pk["mask"], max_ctx=width * page, dev_status=st)
        check(o, dict(q=q, k_new=kn, v_new=vn, k_pool=k_pool, v_pool=v_pool, table=table.cpu().numpy(),
                      ctx=ctx.cpu().numpy(), lens=pk["packed_len"].cpu().numpy(),
                      mask=pk["mask"].cpu().numpy().view(np.uint32)))
        best, acc = (torch.from_numpy(rng.integers(0, n, R).astype(np.int32)).to(DEV) for n in (W, L))
        ctx = rd.rd_commit_accepted(kn, vn, pk["unpacker"], best, acc, k_pool, v_pool, table, ctx, dev_status=st)
        rd.rd_resize_pages(table, held, refs, ctx, page, dev_status=st)          # what was reserved too much
        if step == 1:                                  # row 6's answer has ended; row 2 branches into it
            lens = torch.where(torch.arange(R, device=DEV) == 6, 0, -1).to(torch.int32)
            rd.rd_resize_pages(table, held, refs, lens, page, dev_status=st)
            rd.rd_fork_pages(k_pool, v_pool, table, held, refs, ctx, torch.tensor([5], **i32),
                             torch.tensor([6], **i32), dev_status=st)
        if step == 2:
            _, n_live = rd.rd_compact_pages(k_pool, v_pool, table, held, refs, dev_status=st)
            assert n_live.item() == int((refs > 0).sum()) and (refs[n_live.item():] == 0).all()
    assert st.item() == 0


def test_contexts_at_the_end_of_31_bits_are_refused():
    """A context whose last chunk would end behind 2^31 positions (its row names one
    page over and over) is flagged and its rows are zeros; the others are as ever."""
    rd = _rd()
    s = make(**CASES["half chunks"], seed=41)
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
    page, width = s["k_pool"].shape[1], 2 ** 25
    table = torch.zeros((len(s["ctx"]), width), dtype=torch.int32, device=DEV)
    table[:, :s["table"].shape[1]] = d(s["table"])
    want, size = reference(s)
    for ctx in (2 ** 31 - 1, 2 ** 31 - 256):
        t = s["ctx"].copy()
        t[1] = ctx
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        o = rd.rd_tree_attention_shared(s["q"], s["k_new"], s["v_new"], s["k_pool"], s["v_pool"], table, d(t),
                                        d(s["offsets"]), d(s["pages"]), d(s["lens"]), d(s["mask"].view(np.int32)),
                                        max_ctx=2 ** 31 - 1, dev_status=st).float().cpu().numpy()
        assert st.item() == rd.DEV_BAD_LENGTH and (o[1] == 0).all()
        rest = np.arange(len(t)) != 1
        assert (np.abs(o - want)[rest] <= (2.0 ** -8 * (size + np.abs(want)) + 2.0 ** -11 * size)[rest]).all()
    assert width * page == 2 ** 31


@pytest.mark.parametrize("where", ["prefix", "own"])
@pytest.mark.parametrize("name", ["outside any group", "66 rows", "counter", "many rows", "80 rows, whole units"])
def test_infinite_key_and_value(name, where):
    """An infinite element of a key that a whole group shares, or of one request's own:
    scores of +inf make their rows NaN (inf - inf), scores of -inf give the key no
    weight, and nobody else is touched.  An infinite element of a value makes that
    element of the rows that see it infinite or NaN (a tile of at most 64 rows of the
    kernel for many rows gives each row two lanes, with weights of zero where the other
    lane's positions are: zero times infinity), and no other element.  In ranges with a
    merge, in two units a head, off the counter, and in the kernel for many rows."""
    s = make(**CASES[name], seed=40)
    page, Hkv = s["k_pool"].shape[1:3]
    B, _, Hq, _ = s["q"].shape
    if where == "prefix":
        g = int(np.argmax(s["pages"]))
        seen = np.arange(s["offsets"][g], s["offsets"][g + 1])
        at, pos = int(s["table"][seen[0], s["pages"][g] - 1]), page - 2
    else:
        gid = np.searchsorted(s["offsets"], np.arange(B), side="right") - 1
        skip = np.array([s["pages"][g] * page if 0 <= g < len(s["pages"]) else 0 for g in gid])
        b = int(np.argmax(s["ctx"] - skip))
        assert s["ctx"][b] > skip[b]
        seen, at, pos = np.array([b]), int(s["table"][b, skip[b] // page]), 0
    h, e = Hkv - 1, 3
    heads = np.arange(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
    live = np.arange(s["q"].shape[1])[None] < s["lens"][:, None]
    rows = np.zeros((B, s["q"].shape[1], Hq), bool)            # (request, node, head) that see the element
    rows[np.ix_(seen, np.arange(rows.shape[1]), heads)] = True
    rows &= live[:, :, None]
    assert rows.any() and not rows.all()

    def compare(t, skipped):
        want, size = reference(t)                              # infinities read as the largest finite value
        got = call(t).float().cpu().numpy()
        err, tol = np.abs(got - want), 2.0 ** -8 * (size + np.abs(want)) + 2.0 ** -11 * size
        assert (err <= tol)[~skipped].all()
        return got
    k = s["k_pool"].clone()
    k[at, pos, h, e] = float("inf")
    q = torch.nan_to_num(s["q"]).float().cpu().numpy()[..., e]
    assert (q[rows] != 0).all()
    nan = rows & (q > 0)
    assert nan.any() and (rows & (q < 0)).any()
    got = compare({**s, "k_pool": k}, np.broadcast_to(nan[..., None], s["q"].shape))
    assert np.isnan(got[nan]).all()
    v = s["v_pool"].clone()
    v[at, pos, h, e] = float("inf")
    out = np.zeros(tuple(s["q"].shape), bool)
    out[..., e] = rows
    got = compare({**s, "v_pool": v}, out)
    assert not np.isfinite(got[out]).any() and not np.isneginf(got[out]).any()


@pytest.mark.parametrize("name,max_ctx", [("counter", 50_000_000), ("150 rows, 600 requests", 50_000_000)])
def test_loose_bound_of_the_contexts(name, max_ctx):
    """Many units with a max_ctx far above the contexts: their chunks at that length would
    not count in 31 bits, and nobody counts them."""
    s = make(**CASES[name], seed=42)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    o = call({**s, "max_ctx": max_ctx}, st)
    assert st.item() == 0
    check(o, s)


@pytest.mark.parametrize("B", [1000, 20000])
def test_plan_of_requests_without_rows(B):
    """A group without prefix pages, and one whose requests have finished but for the
    last, take no longer to plan than requests in no group: its first request with rows
    is searched, not walked to (20,000 requests: 1,260 and 1,150 us so, against 240 and
    130 outside of a group)."""
    rd = _rd()
    i32 = dict(dtype=torch.int32, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(B)
    q, kn, vn = (torch.randn(B, 1, 1, 64, generator=gen, device=DEV, dtype=torch.bfloat16) for _ in range(3))
    pool = torch.randn(2, 64, 64, 1, 64, generator=gen, device=DEV, dtype=torch.bfloat16)
    table = (torch.arange(2 * B, **i32) % 64).view(B, 2)
    table[:, 0] = 5
    ctx, mask = torch.full((B,), 70, **i32), torch.ones(B, 1, 1, **i32)
    top = max(pool[1].abs().max().item(), vn.abs().max().item())
    live = torch.ones(B, **i32)
    last = torch.zeros(B, **i32)
    last[-1] = 1

    def run(lens, offsets, pages):
        args = [q, kn, vn, pool[0], pool[1], table, ctx, torch.tensor(offsets, **i32), torch.tensor(pages, **i32), lens, mask]
        o = rd.rd_tree_attention_shared(*args, max_ctx=128)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rd.rd_tree_attention_shared(*args, max_ctx=128)
        times = []
        for _ in range(20):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            graph.replay()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return o.float(), min(times)
    for lens, pages in ((live, 0), (last, 1)):
        want, alone = run(lens, [0, 1, 2], [1, 1])
        got, grouped = run(lens, [0, B], [pages])
        # both within the tolerance above of the formula; A and |o| are at most max |v|
        assert (got - want).abs().max() <= 2 * (2.0 ** -7 + 2.0 ** -11) * top
        assert grouped < 1.6 * alone + 0.01, (grouped, alone)
