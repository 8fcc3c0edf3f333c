"""The paged cache's page operators on the GPU against the plain Python oracle:
tables, reference counts, status bits and the pools' bits, all exactly."""
import numpy as np
import pytest
import torch

from oracle import pages as op

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _rd():
    import tree_attention_verify_gb300 as rd
    return rd


def _d(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _pool(rng, layers, N, ps, Hkv, D):
    return rng.integers(-2 ** 15, 2 ** 15, (layers, N, ps, Hkv, D)).astype(np.int16)


def _bf16(x):
    return _d(x).view(torch.bfloat16)


def _tables(rng, R, N, width, share=0.2):
    """A cache in use: random rows over distinct pages, some pages held twice."""
    table, held, refs = np.full((R, width), -1, np.int32), np.zeros(R, np.int32), np.zeros(N, np.int32)
    ids = list(rng.permutation(N))
    for r in range(R):
        k = int(rng.integers(0, width + 1)) if rng.random() < 0.7 else 0
        k = min(k, len(ids))
        for j in range(k):
            used = np.flatnonzero(refs)
            p = int(rng.choice(used)) if len(used) and rng.random() < share and j == 0 else int(ids.pop())
            table[r, j] = p
            refs[p] += 1
        held[r] = k
    return table, held, refs


@pytest.mark.parametrize("R,N,width,ps", [(1, 1, 1, 64), (1, 40, 9, 64), (13, 100, 7, 128), (200, 2049, 17, 64),
                                          (1500, 40000, 33, 1), (3, 262144, 5, 16), (16384, 3000, 3, 64)])
def test_resize(R, N, width, ps):
    rd = _rd()
    rng = np.random.default_rng(R + N)
    table, held, refs = _tables(rng, R, N, width)
    lens = np.where(rng.random(R) < 0.2, -1, np.where(rng.random(R) < 0.3, 0, rng.integers(0, width * ps + 1, R)))
    lens = lens.astype(np.int32)
    t, h, f, st = _d(table), _d(held), _d(refs), _status()
    for step in range(2):                     # the second call works on what the first left
        want = op.oracle_resize_pages(table, held, refs, lens, ps)
        st.zero_()
        got = rd.rd_resize_pages(t, h, f, _d(lens), ps, dev_status=st)
        assert got is h and st.item() == want[3]
        for a, b in zip((t, h, f), want):
            np.testing.assert_array_equal(a.cpu().numpy(), b)
        table, held, refs = want[:3]
        lens = rng.integers(-1, width * ps + 1, R).astype(np.int32)


def test_resize_flags_what_does_not_fit_and_what_is_wrong():
    rd = _rd()
    table = np.array([[0, 9, -5, -1], [1, 2, -1, -1], [3, -1, -1, -1], [-1, -1, -1, -1], [4, 4, -1, -1]], np.int32)
    held, refs = np.array([3, 2, 9, 0, 2], np.int32), np.array([1, 1, 0, 1, 1, 0, 0, 1], np.int32)
    for lens in ([0, 0, 0, 0, 0], [64, 300, 5, 64, 0], [-1, 128, -1, 257, 256], [192, 128, 0, 256, 256],
                 [192, 192, 3, 64 * 4, 129]):
        lens = np.array(lens, np.int32)
        want = op.oracle_resize_pages(table, held, refs, lens, 64)
        t, h, f, st = _d(table), _d(held), _d(refs), _status()
        rd.rd_resize_pages(t, h, f, _d(lens), 64, dev_status=st)
        assert st.item() == want[3] and want[3] != 0
        for a, b in zip((t, h, f), want):
            np.testing.assert_array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("R,N,width,ps,Hkv,D,layers,n", [
    (2, 3, 2, 64, 1, 64, 1, 1), (9, 50, 5, 64, 3, 128, 2, 4), (40, 300, 6, 128, 2, 64, 3, 25),
    (400, 2500, 6, 64, 1, 64, 1, 180), (30, 60, 4, 16, 1, 8, 5, 20), (60, 400, 6, 128, 4, 64, 3, 40)])
def test_fork(R, N, width, ps, Hkv, D, layers, n):
    rd = _rd()
    rng = np.random.default_rng(R * N)
    table, held, refs = _tables(rng, R, N, width)
    ctx = np.maximum(0, held * ps - rng.integers(0, 2 * ps, R)).astype(np.int32)
    ctx = np.where(rng.random(R) < 0.3, held * ps, ctx).astype(np.int32)
    k, v = _pool(rng, layers, N, ps, Hkv, D), _pool(rng, layers, N, ps, Hkv, D)
    empty, full = np.flatnonzero(held == 0), np.flatnonzero(held > 0)
    kid = rng.choice(empty, n).astype(np.int32)              # some rows twice
    par = np.where(rng.random(n) < 0.15, -1, rng.choice(full if len(full) else empty, n)).astype(np.int32)
    want = op.oracle_fork_pages(k, v, table, held, refs, ctx, par, kid)
    kp, vp, t, h, f, c, st = _bf16(k), _bf16(v), _d(table), _d(held), _d(refs), _d(ctx), _status()
    rd.rd_fork_pages(kp, vp, t, h, f, c, _d(par), _d(kid), dev_status=st)
    assert st.item() == want[6]
    for a, b in zip((kp.view(torch.int16), vp.view(torch.int16), t, h, f, c), want):
        np.testing.assert_array_equal(a.cpu().numpy(), b)


def test_fork_flags_and_skips_what_is_wrong():
    rd = _rd()
    rng = np.random.default_rng(3)
    N, ps = 12, 64
    k, v = _pool(rng, 1, N, ps, 1, 64), _pool(rng, 1, N, ps, 1, 64)
    table, held, refs = np.full((8, 3), -1, np.int32), np.zeros(8, np.int32), np.zeros(N, np.int32)
    table[0, :2], table[1, :3], table[2, :1] = [4, 7], [1, 99, 2], [5]
    held[:3] = [2, 3, 1]
    refs[[4, 7, 1, 2, 5]] = 1
    ctx = np.array([100, 150, 65, -2, 0, 0, 0, 0], np.int32)
    cases = [([0, 0], [3, 3]), ([0, 8, 0], [4, 5, -1]), ([0, 0], [0, 1]), ([2, 3, 0], [5, 6, 7]), ([1, 4], [3, 6]),
             ([0, 3], [3, 5]), ([0] * 5, [3, 4, 5, 6, 7])]
    for par, kid in cases:
        for spare in (N, 2):                 # two spare pages only: the last pairs find none
            full = refs.copy()
            full[np.flatnonzero(refs == 0)[spare:]] = 1
            par_, kid_ = np.array(par, np.int32), np.array(kid, np.int32)
            want = op.oracle_fork_pages(k, v, table, held, full, ctx, par_, kid_)
            kp, vp, t, h, f, c, st = _bf16(k), _bf16(v), _d(table), _d(held), _d(full), _d(ctx), _status()
            rd.rd_fork_pages(kp, vp, t, h, f, c, _d(par_), _d(kid_), dev_status=st)
            assert st.item() == want[6]
            for a, b in zip((kp.view(torch.int16), vp.view(torch.int16), t, h, f, c), want):
                np.testing.assert_array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("N,ps,Hkv,D,layers,n", [(2, 64, 1, 64, 1, 1), (600, 16, 1, 64, 1, 256), (600, 16, 1, 64, 1, 257), (40, 64, 8, 128, 1, 13), (30, 64, 3, 64, 4, 15),
                                                 (700, 1, 1, 8, 2, 300), (64, 256, 2, 128, 2, 31)])
def test_copy(N, ps, Hkv, D, layers, n):
    rd = _rd()
    rng = np.random.default_rng(N + n)
    k, v = _pool(rng, layers, N, ps, Hkv, D), _pool(rng, layers, N, ps, Hkv, D)
    ids = rng.permutation(N)
    src, dst = ids[:n].astype(np.int32), ids[n:2 * n].astype(np.int32)
    src[rng.random(n) < 0.1] = -1
    if n > 3:
        src[1] = src[0] if src[0] >= 0 else ids[0]          # one source twice
    want = op.oracle_copy_pages(k, v, src, dst)
    kp, vp, st = _bf16(k), _bf16(v), _status()
    rd.rd_copy_pages(kp, vp, _d(src), _d(dst), dev_status=st)
    assert st.item() == 0 == want[2]
    np.testing.assert_array_equal(kp.view(torch.int16).cpu().numpy(), want[0])
    np.testing.assert_array_equal(vp.view(torch.int16).cpu().numpy(), want[1])


@pytest.mark.parametrize("seed", range(4))
def test_copy_skips_pairs_that_depend_on_one_another(seed):
    rd = _rd()
    rng = np.random.default_rng(seed)
    N, n = 600, 520 if seed % 2 else 200      # compared by a kernel of its own, or by each copying block
    k, v = _pool(rng, 1, N, 1, 1, 8), _pool(rng, 1, N, 1, 1, 8)
    src, dst = rng.integers(-2, N + 3, n).astype(np.int32), rng.integers(-1, N + 1, n).astype(np.int32)
    want = op.oracle_copy_pages(k, v, src, dst)
    kp, vp, st = _bf16(k), _bf16(v), _status()
    rd.rd_copy_pages(kp, vp, _d(src), _d(dst), dev_status=st)
    assert st.item() == want[2] == rd.DEV_BAD_INDEX
    np.testing.assert_array_equal(kp.view(torch.int16).cpu().numpy(), want[0])
    np.testing.assert_array_equal(vp.view(torch.int16).cpu().numpy(), want[1])


@pytest.mark.parametrize("R,N,width,ps,Hkv,D,layers", [(1, 1, 1, 64, 1, 64, 1), (5, 33, 4, 64, 2, 128, 2),
                                                       (60, 400, 5, 64, 1, 64, 3), (300, 9000, 12, 1, 1, 8, 1)])
def test_compact(R, N, width, ps, Hkv, D, layers):
    rd = _rd()
    rng = np.random.default_rng(R + 7 * N)
    table, held, refs = _tables(rng, R, N, width)
    refs[rng.integers(0, N)] += 1             # a page that somebody holds outside the tables
    k, v = _pool(rng, layers, N, ps, Hkv, D), _pool(rng, layers, N, ps, Hkv, D)
    want = op.oracle_compact_pages(k, v, table, held, refs)
    kp, vp, t, h, f, st = _bf16(k), _bf16(v), _d(table), _d(held), _d(refs), _status()
    remap, n_live = rd.rd_compact_pages(kp, vp, t, h, f, dev_status=st)
    assert st.item() == want[6] == 0 and n_live.item() == want[5]
    for a, b in zip((kp.view(torch.int16), vp.view(torch.int16), t, f, remap), want):
        np.testing.assert_array_equal(a.cpu().numpy(), b)
    again = rd.rd_compact_pages(kp, vp, t, h, f, dev_status=st)[0]     # nothing left to move
    np.testing.assert_array_equal(again.cpu().numpy()[:want[5]], np.arange(want[5]))
    np.testing.assert_array_equal(kp.view(torch.int16).cpu().numpy(), want[0])


@pytest.mark.parametrize("refs", [[0, 0, 0, 0], [1, 2, 3, 1], [0, 0, 0, 1], [1, 0, 0, 0]])
def test_compact_empty_full_and_one_page(refs):
    rd = _rd()
    rng = np.random.default_rng(0)
    k = _pool(rng, 1, 4, 16, 1, 8)
    refs = np.array(refs, np.int32)
    table, held = np.array([[3, 77]], np.int32), np.array([2], np.int32)
    want = op.oracle_compact_pages(k, k, table, held, refs)
    kp, vp, t, h, f, st = _bf16(k), _bf16(k), _d(table), _d(held), _d(refs), _status()
    remap, n_live = rd.rd_compact_pages(kp, vp, t, h, f, dev_status=st)
    assert st.item() == want[6] == rd.DEV_BAD_INDEX and n_live.item() == want[5]
    for a, b in zip((kp.view(torch.int16), vp.view(torch.int16), t, f, remap), want):
        np.testing.assert_array_equal(a.cpu().numpy(), b)


def test_fp8_pools_of_four_dimensions():
    rd = _rd()
    rng = np.random.default_rng(8)
    k = rng.integers(0, 256, (10, 64, 2, 128)).astype(np.uint8)
    kp, vp = _d(k), _d(k[::-1].copy())
    rd.rd_copy_pages(kp, vp, _d(np.array([3, 9], np.int32)), _d(np.array([0, 5], np.int32)))
    k[0], k[5] = k[3], k[9]
    np.testing.assert_array_equal(kp.cpu().numpy(), k)
    kf = kp.view(torch.float8_e4m3fn)
    rd.rd_copy_pages(kf, vp.view(torch.float8_e4m3fn), _d(np.array([1], np.int32)), _d(np.array([2], np.int32)))
    np.testing.assert_array_equal(kp[2].cpu().numpy(), k[1])


def test_captured_step_replays_on_other_tables():
    # reserve, fork and compact in one graph: each replay works on what the
    # tables then hold
    rd = _rd()
    rng = np.random.default_rng(1)
    R, N, width, ps = 20, 200, 6, 64
    k0 = _pool(rng, 1, N, ps, 1, 64)
    kp, vp, st = _bf16(k0), _bf16(k0), _status()
    t, h, f = _d(np.full((R, width), -1, np.int32)), _d(np.zeros(R, np.int32)), _d(np.zeros(N, np.int32))
    c, lens = _d(np.zeros(R, np.int32)), _d(np.zeros(R, np.int32))
    par, kid = _d(np.array([0, 1], np.int32)), _d(np.array([18, 19], np.int32))

    def step():
        rd.rd_resize_pages(t, h, f, lens, ps, dev_status=st)
        rd.rd_fork_pages(kp, vp, t, h, f, c, par, kid, dev_status=st)
        rd.rd_compact_pages(kp, vp, t, h, f, dev_status=st)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    table, held, refs = (x.cpu().numpy() for x in (t, h, f))
    ctx, k, v = c.cpu().numpy(), k0, k0
    k, v = (x.view(torch.int16).cpu().numpy() for x in (kp, vp))
    for i in range(4):
        n = np.where(np.arange(R) < 18, rng.integers(0, width * ps, R), 0).astype(np.int32)
        lens.copy_(_d(n))
        ctx = np.where(np.arange(R) < 18, n, 0).astype(np.int32)
        c.copy_(_d(ctx))
        graph.replay()
        table, held, refs, st1 = op.oracle_resize_pages(table, held, refs, n, ps)
        k, v, table, held, refs, ctx, st2 = op.oracle_fork_pages(k, v, table, held, refs, ctx, par.cpu().numpy(),
                                                                 kid.cpu().numpy())
        k, v, table, refs, _, _, st3 = op.oracle_compact_pages(k, v, table, held, refs)
        assert st.item() == st1 | st2 | st3 == 0
        for a, b in zip((kp.view(torch.int16), vp.view(torch.int16), t, h, f, c), (k, v, table, held, refs, ctx)):
            np.testing.assert_array_equal(a.cpu().numpy(), b)


def test_given_stream_and_workspace():
    rd = _rd()
    rng = np.random.default_rng(2)
    k = _pool(rng, 1, 8, 64, 1, 64)
    kp, vp = _bf16(k), _bf16(k)
    src, dst = _d(np.array([1], np.int32)), _d(np.array([6], np.int32))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    rd.rd_copy_pages(kp, vp, src, dst, stream=s)
    rd.rd_copy_pages(kp, vp, dst, src, stream=s, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    s.synchronize()
    k[0, 6] = k[0, 1]
    np.testing.assert_array_equal(kp.view(torch.int16).cpu().numpy(), k)
    many = torch.full((300,), -1, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        rd.rd_copy_pages(kp, vp, many, many, workspace=torch.empty(2399, dtype=torch.uint8, device=DEV))
    rd.rd_copy_pages(kp, vp, many, many)
    with pytest.raises(rd.RdError):           # pages of 12 bytes: not whole 16-byte units
        rd.rd_copy_pages(torch.zeros(4, 1, 2, 3, dtype=torch.bfloat16, device=DEV),
                         torch.zeros(4, 1, 2, 3, dtype=torch.bfloat16, device=DEV), src, dst)


def test_fork_at_the_limit_of_rows():
    """16,384 rows and pairs: half of the pairs name rows that hold nothing."""
    rd = _rd()
    rng = np.random.default_rng(8)
    R = n = 16384
    N, width, ps = 20000, 2, 16
    table, held, refs = _tables(rng, R, N, width)
    held[R // 2:] = 0
    refs[:] = 0
    for r in range(R):
        table[r, :held[r]] = rng.choice(N // 2, held[r])
        np.add.at(refs, table[r, :held[r]], 1)
    ctx = np.maximum(0, held * ps - rng.integers(0, ps, R)).astype(np.int32)
    k, v = _pool(rng, 1, N, ps, 1, 8), _pool(rng, 1, N, ps, 1, 8)
    par = rng.integers(-1, R // 2, n).astype(np.int32)
    kid = (R // 2 + rng.permutation(n) % (R // 2)).astype(np.int32)
    want = op.oracle_fork_pages(k, v, table, held, refs, ctx, par, kid)
    kp, vp, t, h, f, c, st = _bf16(k), _bf16(v), _d(table), _d(held), _d(refs), _d(ctx), _status()
    rd.rd_fork_pages(kp, vp, t, h, f, c, _d(par), _d(kid), dev_status=st)
    assert st.item() == want[6]
    for a, b in zip((kp.view(torch.int16), vp.view(torch.int16), t, h, f, c), want):
        np.testing.assert_array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("n", [3, 300])
def test_copy_and_fork_past_32_bits(n):
    """Pools whose last pages begin behind 2^32 bytes, and 2^32 elements in the last layer."""
    rd = _rd()
    ps, Hkv, D, layers = 64, 8, 128, 2
    N = 2 ** 31 // (ps * Hkv * D) + 2 * n + 1          # per layer; 8.6 GB a pool
    k = torch.zeros((layers, N, ps, Hkv, D), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    src, dst = torch.arange(N - 2 * n, N - n, device=DEV), torch.arange(N - n, N, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(n)
    for p in (k, v):
        p[:, N - 2 * n:N - n] = torch.randn(layers, n, ps, Hkv, D, generator=gen, device=DEV, dtype=torch.bfloat16)
    st = _status()
    rd.rd_copy_pages(k, v, src.int(), dst.int(), dev_status=st)
    assert st.item() == 0
    for p in (k, v):
        assert torch.equal(p[:, N - n:], p[:, N - 2 * n:N - n])
        assert not p[:, :N - 2 * n].any() and p[:, N - n:].any()
    # n rows of one page each, the lowest free pages being the pool's last
    refs = torch.ones(N, dtype=torch.int32, device=DEV)
    refs[N - n:] = 0
    k[:, N - n:], v[:, N - n:] = 7, 7
    table = torch.full((2 * n, 1), -1, dtype=torch.int32, device=DEV)
    table[:n, 0] = src.int()
    held = torch.zeros(2 * n, dtype=torch.int32, device=DEV)
    held[:n] = 1
    ctx = torch.where(held > 0, 33, 0).int()
    rows = torch.arange(n, device=DEV).int()
    rd.rd_fork_pages(k, v, table, held, refs, ctx, rows, rows + n, dev_status=st)
    assert st.item() == 0 and torch.equal(table[n:, 0], dst.int()) and (refs == 1).all()
    for p in (k, v):
        assert torch.equal(p[:, N - n:, :33], p[:, N - 2 * n:N - n, :33])
        assert (p[:, N - n:, 33:] == 7).all()


@pytest.mark.parametrize("op_name", ["resize", "fork"])
def test_large_and_small_tables_from_many_threads(op_name):
    """Host threads, each with its own stream and tables: one changes tables of 16,384
    rows, the others of 16, many times over.  No call may fail for what another
    thread's needs.  (The C entries are called directly: the threads then spend their
    time in them, at the same time, and not in Python.)"""
    import threading
    rd = _rd()
    i32 = dict(dtype=torch.int32, device=DEV)
    wrong, running, start = [], [True], threading.Barrier(4)

    def work(R, times):
        s = torch.cuda.Stream()
        t, h, f, c = torch.full((R, 1), -1, **i32), torch.zeros(R, **i32), torch.zeros(R, **i32), torch.zeros(R, **i32)
        kp, vp = (torch.zeros(R, 16, 1, 8, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        lens, none, st = torch.full((R,), 5, **i32), torch.full((R,), -1, **i32), _status()
        ws = torch.empty(12 * R, dtype=torch.uint8, device=DEV)
        p = lambda x: x.data_ptr()  # noqa: E731
        if op_name == "resize":
            call, args = rd._lib.rd_resize_pages, (p(t), R, 1, p(h), p(f), R, p(lens), 16, p(st), s.cuda_stream)
        else:
            call, args = rd._lib.rd_fork_pages, (p(kp), p(vp), 1, R, 256, 16, p(t), R, 1, p(h), p(f), p(c), p(none),
                                                 p(none), R, p(ws), ws.nbytes, p(st), s.cuda_stream)
        torch.cuda.synchronize()
        start.wait()
        while running[0]:
            got = [call(*args) for _ in range(50)]
            if any(got):
                wrong.append((R, got))
            times -= 1
            if times == 0:
                running[0] = False
        s.synchronize()
        if st.item() or op_name == "resize" and not ((h == 1).all() and (f == 1).all()):
            wrong.append((R, st.item()))
    threads = [threading.Thread(target=work, args=a) for a in ((16384, 200), (16, -1), (16, -1), (16, -1))]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not wrong, wrong[:2]


@pytest.mark.parametrize("layers", [1, 3])
def test_fork_of_rows_that_name_free_pages(layers):
    """Parents whose rows name pages that nobody holds, the lowest free ones, which the
    same call hands out: flagged, entries copied but not counted, nothing copied from
    them, and the outcome the same every time."""
    rd = _rd()
    rng = np.random.default_rng(layers)
    R, N, width, ps, n = 400, 4000, 9, 64, 180
    table, held, refs = np.full((R, width), -1, np.int32), np.zeros(R, np.int32), np.zeros(N, np.int32)
    held[:n] = rng.integers(1, width + 1, n)
    for r in range(n):
        table[r, :held[r]] = rng.integers(0, 2 * n, held[r])         # half of them among those held
    refs[rng.permutation(2 * n)[:n]] = 3
    ctx = np.maximum(0, held * ps - rng.integers(0, ps, R)).astype(np.int32)
    k, v = _pool(rng, layers, N, ps, 1, 64), _pool(rng, layers, N, ps, 1, 64)
    for pairs in (n, 4):                      # with a copy launch, and without
        par, kid = np.arange(pairs).astype(np.int32), (n + np.arange(pairs)).astype(np.int32)
        want = op.oracle_fork_pages(k, v, table, held, refs, ctx, par, kid)
        for _ in range(5):
            kp, vp, t, h, f, c, st = _bf16(k), _bf16(v), _d(table), _d(held), _d(refs), _d(ctx), _status()
            rd.rd_fork_pages(kp, vp, t, h, f, c, _d(par), _d(kid), dev_status=st)
            assert st.item() == want[6] == rd.DEV_BAD_INDEX
            for a, b in zip((kp.view(torch.int16), vp.view(torch.int16), t, h, f, c), want):
                np.testing.assert_array_equal(a.cpu().numpy(), b)


def test_fork_at_the_limits_of_rows_and_pages():
    """16,384 rows and pairs over 262,144 pages: all that the table kernel holds in
    shared memory.  Every 16th pair is one; the free pages are the last of the pool."""
    rd = _rd()
    R = n = 16384
    N, ps = 262144, 8
    table, held, refs = np.full((R, 2), -1, np.int32), np.zeros(R, np.int32), np.ones(N, np.int32)
    held[:R // 2] = 2
    table[:R // 2] = np.arange(R).reshape(-1, 2)
    refs[N - 3000::3] = 0
    ctx = np.where(held > 0, 13, 0).astype(np.int32)
    par, kid = np.full(n, -1, np.int32), np.zeros(n, np.int32)
    par[::16], kid[::16] = np.arange(n // 16), R // 2 + np.arange(n // 16)
    k = np.broadcast_to(np.arange(N, dtype=np.int32).astype(np.int16)[None, :, None, None, None], (1, N, ps, 1, 8)).copy()
    want = op.oracle_fork_pages(k, k, table, held, refs, ctx, par, kid)
    kp, vp, t, h, f, c, st = _bf16(k), _bf16(k), _d(table), _d(held), _d(refs), _d(ctx), _status()
    rd.rd_fork_pages(kp, vp, t, h, f, c, _d(par), _d(kid), dev_status=st)
    assert st.item() == want[6] == rd.DEV_OVERFLOW          # 1,000 free pages for 1,024 pairs
    for a, b in zip((kp.view(torch.int16), vp.view(torch.int16), t, h, f, c), want):
        np.testing.assert_array_equal(a.cpu().numpy(), b)


def test_resize_of_a_row_that_ends_behind_31_bits():
    """A row of 2^31 - 1 entries (8.6 GB) gives its last ones back: a step of several
    entries a lane may end behind 2^31."""
    rd = _rd()
    width, keep, N = 2 ** 31 - 1, 2 ** 31 - 1 - 900, 64
    t = torch.empty((1, width), dtype=torch.int32, device=DEV)
    t[0, keep - 100:] = torch.arange(1000, device=DEV) % N
    refs, held = torch.full((N,), 1000, dtype=torch.int32, device=DEV), _d(np.array([width], np.int32))
    st = _status()
    rd.rd_resize_pages(t, held, refs, _d(np.array([keep], np.int32)), 1, dev_status=st)
    assert st.item() == 0 and held.item() == keep
    assert (t[0, keep:] == -1).all() and torch.equal(t[0, keep - 100:keep].long(), torch.arange(100, device=DEV) % N)
    given = torch.bincount(torch.arange(100, 1000, device=DEV) % N, minlength=N)
    assert torch.equal(refs.long(), 1000 - given)


@pytest.mark.parametrize("way", ["fork", "copy"])
@pytest.mark.parametrize("cut", [100, 64, 1])
def test_a_row_cut_back_into_a_shared_page_goes_on_in_its_own(way, cut):
    """The two ways in which a row that is cut back into a page that it shares may be
    written on: its branch keeps every position, the row keeps its first ones and
    receives the committed rows behind them."""
    rd = _rd()
    rng = np.random.default_rng(cut)
    i32 = dict(dtype=torch.int32, device=DEV)
    R, N, ps, width, L = 3, 12, 64, 4, 3
    k0 = _pool(rng, 1, N, ps, 2, 64)
    kp, vp, st = _bf16(k0), _bf16(k0[:, ::-1]), _status()
    t, h, f, c = torch.full((R, width), -1, **i32), torch.zeros(R, **i32), torch.zeros(N, **i32), torch.zeros(R, **i32)
    length = 158                              # two full pages and 30 positions
    rd.rd_resize_pages(t, h, f, torch.tensor([length, 0, 0], **i32), ps, dev_status=st)
    c[0] = length
    rd.rd_fork_pages(kp, vp, t, h, f, c, torch.tensor([0], **i32), torch.tensor([1], **i32), dev_status=st)

    def contents(r, n):
        pages = t[r, :-(-n // ps)].long()
        return [x[0, pages].view(torch.int16).reshape(-1, 2, 64)[:n].clone() for x in (kp, vp)]
    branch, row = contents(1, length), contents(0, cut)
    if way == "fork":
        r = 2
        c[0] = cut
        rd.rd_fork_pages(kp, vp, t, h, f, c, torch.tensor([0], **i32), torch.tensor([r], **i32), dev_status=st)
        rd.rd_resize_pages(t, h, f, torch.tensor([0, -1, cut + L], **i32), ps, dev_status=st)
    else:
        r = 0
        last = cut // ps
        old = t[0, last:last + 1].clone()
        rd.rd_resize_pages(t, h, f, torch.tensor([last * ps, -1, -1], **i32), ps, dev_status=st)
        rd.rd_resize_pages(t, h, f, torch.tensor([cut + L, -1, -1], **i32), ps, dev_status=st)
        rd.rd_copy_pages(kp, vp, old, t[0, last:last + 1].clone(), dev_status=st)
        c[0] = cut
    # one beam of L tokens a row, all accepted; only row r's are looked at (the branch
    # has room behind its length, and the third row no pages: flagged and skipped)
    kn, vn = (torch.randn(R, L, 2, 64, device=DEV).bfloat16() for _ in range(2))
    unpacker = torch.arange(L, **i32).expand(R, 1, L).contiguous()
    assert st.item() == 0
    new = rd.rd_commit_accepted(kn, vn, unpacker, torch.zeros(R, **i32), torch.full((R,), L - 1, **i32), kp[0], vp[0],
                                t, c)
    assert new[r].item() == cut + L
    for got, want in zip(contents(1, length), branch):
        assert torch.equal(got, want)
    for got, want, rows in zip(contents(r, cut + L), row, (kn, vn)):
        assert torch.equal(got[:cut], want) and torch.equal(got[cut:], rows[r].view(torch.int16))
