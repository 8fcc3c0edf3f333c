"""Host-side checks of the page operators, without a GPU: the C entries refuse
bad arguments before they touch the device, the binding refuses tensors whose
shapes, types or places disagree."""
import ctypes

import pytest
import torch

import tree_attention_verify_gb300 as rd

N = None
ONE = ctypes.c_void_p(256)


def test_resize_validation():
    f = rd._lib.rd_resize_pages
    assert f(N, 0, 8, N, N, 16, N, 64, N, N) == rd.RD_OK                      # no rows
    for args in ((ONE, -1, 8, ONE, ONE, 16, ONE, 64), (ONE, 4, -8, ONE, ONE, 16, ONE, 64),
                 (ONE, 4, 8, ONE, ONE, -1, ONE, 64), (ONE, 4, 8, ONE, ONE, 16, ONE, 0),
                 (N, 4, 8, ONE, ONE, 16, ONE, 64), (ONE, 4, 8, N, ONE, 16, ONE, 64),
                 (ONE, 4, 8, ONE, N, 16, ONE, 64), (ONE, 4, 8, ONE, ONE, 16, N, 64)):
        assert f(*args, N, N) == rd.RD_ERR_INVALID_ARG, args
    for args in ((ONE, 16385, 8, ONE, ONE, 16, ONE, 64), (ONE, 4, 8, ONE, ONE, 262145, ONE, 64),
                 (ONE, 16384, 1 << 17, ONE, ONE, 16, ONE, 64)):
        assert f(*args, N, N) == rd.RD_ERR_UNSUPPORTED, args


def test_fork_validation():
    f = rd._lib.rd_fork_pages
    good = dict(k=ONE, v=ONE, layers=2, pages=16, bytes=4096, ps=64, table=ONE, R=4, width=8, rows=ONE,
                refs=ONE, ctx=ONE, par=ONE, kid=ONE, n=300, ws=ONE, wsb=3600)

    def call(**kw):
        return f(*{**good, **kw}.values(), N, N)
    assert call(n=0) == rd.RD_OK and call(R=0) == rd.RD_OK
    for kw in (dict(k=N), dict(v=N), dict(layers=0), dict(pages=-1), dict(bytes=0), dict(ps=0), dict(ps=48),
               dict(table=N), dict(R=-1), dict(width=-1), dict(rows=N), dict(refs=N), dict(ctx=N), dict(par=N),
               dict(kid=N), dict(n=-1), dict(ws=N), dict(wsb=3599), dict(k=ctypes.c_void_p(264))):
        assert call(**kw) == rd.RD_ERR_INVALID_ARG, kw
    for kw in (dict(bytes=4104), dict(n=16385, wsb=1 << 20), dict(R=16385), dict(pages=262145)):
        assert call(**kw) == rd.RD_ERR_UNSUPPORTED, kw
    assert rd._lib.rd_fork_pages_workspace_size(300, 2, 4096) == 3600          # 4.9 MB: a list for the copy
    assert rd._lib.rd_fork_pages_workspace_size(3, 2, 4096) == 0               # little data: no workspace


def test_copy_and_compact_validation():
    f = rd._lib.rd_copy_pages
    assert f(N, N, 1, 16, 4096, N, N, 0, N, 0, N, N) == rd.RD_OK
    good = dict(k=ONE, v=ONE, layers=2, pages=16, bytes=4096, src=ONE, dst=ONE, n=257, ws=ONE, wsb=2056)
    for kw in (dict(k=N), dict(v=N), dict(src=N), dict(dst=N), dict(n=-1), dict(ws=N), dict(wsb=2055),
               dict(layers=0), dict(v=ctypes.c_void_p(257))):
        assert f(*{**good, **kw}.values(), N, N) == rd.RD_ERR_INVALID_ARG, kw
    for kw in (dict(bytes=4100), dict(n=262145, wsb=1 << 22)):
        assert f(*{**good, **kw}.values(), N, N) == rd.RD_ERR_UNSUPPORTED, kw
    g = rd._lib.rd_compact_pages
    good = dict(k=ONE, v=ONE, layers=2, pages=16, bytes=4096, table=ONE, R=4, width=8, rows=ONE, refs=ONE,
                remap=ONE, live=ONE, ws=ONE, wsb=80)
    assert rd._lib.rd_compact_pages_workspace_size(16) == 80
    for kw in (dict(k=N), dict(table=N), dict(rows=N), dict(refs=N), dict(remap=N), dict(live=N), dict(ws=N),
               dict(wsb=79), dict(pages=-1)):
        assert g(*{**good, **kw}.values(), N, N) == rd.RD_ERR_INVALID_ARG, kw
    assert g(*{**good, "bytes": 100}.values(), N, N) == rd.RD_ERR_UNSUPPORTED


def _i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_binding_refuses_before_a_launch():
    pool, table = torch.zeros(8, 64, 1, 64, dtype=torch.bfloat16), _i(4, 3)
    # CPU tensors (and with them every call here) are refused by name
    with pytest.raises(ValueError, match="block_table must be a CUDA tensor"):
        rd.rd_resize_pages(table, _i(4), _i(8), _i(4), 64)
    with pytest.raises(ValueError, match="k_pool must be a CUDA tensor"):
        rd.rd_fork_pages(pool, pool, table, _i(4), _i(8), _i(4), _i(2), _i(2))
    with pytest.raises(ValueError, match="k_pool must be a CUDA tensor"):
        rd.rd_copy_pages(pool, pool, _i(2), _i(2))
    with pytest.raises(ValueError, match="k_pool must be a CUDA tensor"):
        rd.rd_compact_pages(pool, pool, table, _i(4), _i(8))
    with pytest.raises(TypeError):
        rd.rd_resize_pages(table.long(), _i(4), _i(8), _i(4), 64)
    with pytest.raises(TypeError):
        rd.rd_copy_pages([1], pool, _i(2), _i(2))
    with pytest.raises(ValueError, match="at least"):
        rd._scratch(torch.zeros(3, dtype=torch.uint8), 16, pool, None)
    with pytest.raises(TypeError):
        rd._need_status(torch.zeros(1), pool)


def test_binding_asks_the_library_how_much_workspace(monkeypatch):
    """Workspaces are as large as the library says, whatever it says."""
    runs = {}
    monkeypatch.setattr(rd, "_fine", lambda *a: True)         # as if the tensors were on a GPU
    monkeypatch.setattr(rd, "_need", lambda *a, **kw: None)
    monkeypatch.setattr(rd, "_run", lambda name, like, *a, stream=None: runs.__setitem__(name, a))
    pool, table = torch.zeros(8, 64, 1, 64, dtype=torch.bfloat16), _i(4, 3)
    for extra in (0, 4096):
        for name in ("rd_fork_pages", "rd_copy_pages", "rd_compact_pages"):
            f = getattr(rd._lib, name + "_workspace_size")
            monkeypatch.setattr(rd._lib, name + "_workspace_size", lambda *a, f=f, extra=extra: f(*a) + extra)
        for n in (2, 256, 257, 300):
            need = rd._lib.rd_copy_pages_workspace_size(n)
            rd.rd_copy_pages(pool, pool, _i(n), _i(n))
            assert runs["rd_copy_pages"][9] >= need and (need > 0 or runs["rd_copy_pages"][9] == 0)
            if need:
                with pytest.raises(ValueError, match="at least"):
                    rd.rd_copy_pages(pool, pool, _i(n), _i(n), workspace=torch.zeros(need - 1, dtype=torch.uint8))
        for pages in (1, 2, 7, 8):
            need = rd._lib.rd_compact_pages_workspace_size(pages)
            args = [pool[:pages].clone(), pool[:pages].clone(), table, _i(4), _i(pages)]
            rd.rd_compact_pages(*args)
            assert runs["rd_compact_pages"][13] >= need
            rd.rd_compact_pages(*args, n_live=_i(1))
            assert runs["rd_compact_pages"][13] >= need
            with pytest.raises(ValueError, match="at least"):
                rd.rd_compact_pages(*args, workspace=torch.zeros(need - 1, dtype=torch.uint8))
        rd.rd_fork_pages(pool, pool, table, _i(4), _i(8), _i(4), _i(300), _i(300))
        assert runs["rd_fork_pages"][16] >= rd._lib.rd_fork_pages_workspace_size(300, 1, 64 * 64 * 2)
