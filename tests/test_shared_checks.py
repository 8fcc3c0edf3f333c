"""Host-side checks of rd_tree_attention_shared, without a GPU: the C entry refuses
bad arguments before it touches the device, the binding refuses tensors that are
not on one."""
import ctypes

import pytest
import torch

import tree_attention_verify_gb300 as rd

N = None
ONE = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(264)
GOOD = dict(B=4, P=8, Hq=8, Hkv=2, D=128, scale=0.0, q=ONE, kn=ONE, vn=ONE, kp=ONE, vp=ONE, pages=64, ps=64,
            table=ONE, width=16, ctx=ONE, max_ctx=1024, n=2, offs=ONE, pre=ONE, lens=ONE, mask=ONE, words=1, o=ONE,
            ws=ONE, wsb=1 << 40)


def call(**kw):
    return rd._lib.rd_tree_attention_shared(*{**GOOD, **kw}.values(), N, N)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(P=0), dict(Hq=7), dict(Hq=0), dict(Hkv=0), dict(pages=-1), dict(ps=0), dict(width=-1),
    dict(max_ctx=-1), dict(words=2), dict(words=0), dict(P=33), dict(wsb=0)]
    + [{k: N} for k in ("q", "kn", "vn", "kp", "vp", "table", "ctx", "offs", "pre", "lens", "mask", "o", "ws")]
    + [{k: ODD} for k in ("q", "kn", "vn", "kp", "vp", "o", "ws")], ids=str)
def test_refuses_bad_arguments(kw):
    assert call(**kw) == rd.RD_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(D=96), dict(D=256), dict(ps=48), dict(P=257, words=9), dict(B=65536), dict(n=65536),
    dict(Hq=65536, Hkv=65536), dict(pages=1 << 25, ps=64),
    dict(B=64, max_ctx=1 << 30),                       # 64 x 2 heads x 2^25 chunks behind the prefix: 2^32
    dict(B=1, P=1, Hq=1, Hkv=1, n=65535, max_ctx=1 << 20)], ids=str)
def test_refuses_what_it_does_not_support(kw):
    assert call(**kw) == rd.RD_ERR_UNSUPPORTED


def test_workspace():
    size = rd._lib.rd_tree_attention_shared_workspace_size
    args = [GOOD[k] for k in ("B", "P", "Hq", "Hkv", "D", "max_ctx", "n")]
    need = size(*args)
    assert need > 0 and call(wsb=need - 1) == rd.RD_ERR_INVALID_ARG
    # holds every row's fp32 sums over the prefix, on each of the paths (few rows with
    # few and many units, many rows), and the groups
    for B, P, G in ((4, 8, 1), (400, 8, 4), (4, 64, 4)):
        a = size(B, P, 4 * G, 4, 128, 1024, 2)
        assert a >= B * P * 4 * G * (128 + 2) * 4
        assert size(B, P, 4 * G, 4, 128, 1024, 900) > a
    # without groups it is the paged call's
    assert size(*args[:-1], 0) == rd._lib.rd_tree_attention_workspace_size(*args[:-1])
    for bad in ((0, 8, 8, 2, 128, 64, 1), (4, 0, 8, 2, 128, 64, 1), (4, 8, 7, 2, 128, 64, 1), (4, 8, 8, 2, 128, -1, 1)):
        assert size(*bad) == 0


def test_nothing_shared_is_the_paged_call():
    assert call(B=0) == rd.RD_OK                       # no requests
    assert call(B=0, n=0, offs=N, pre=N) == rd.RD_OK
    assert call(n=0, q=N) == rd.RD_ERR_INVALID_ARG     # the paged call's own checks
    assert call(n=0, D=96) == rd.RD_ERR_UNSUPPORTED


def test_binding_refuses_before_a_launch():
    bf = torch.zeros(4, 8, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    pool, table = torch.zeros(8, 64, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 3, dtype=torch.int32)
    mask = torch.zeros(4, 8, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        rd.rd_tree_attention_shared(bf, bf, bf, pool, pool, table, i, i[:2], i[:1], i, mask, max_ctx=64)
    with pytest.raises((TypeError, ValueError)):
        rd.rd_tree_attention_shared(None, bf, bf, pool, pool, table, i, i[:2], i[:1], i, mask, max_ctx=64)


@pytest.mark.parametrize("kw", [dict(B=512, P=48, words=2, Hq=40, Hkv=40, max_ctx=1_700_000),
                                dict(B=481, P=64, words=2, Hq=32, Hkv=8, max_ctx=4_000_000)], ids=str)
def test_counts_only_what_it_divides(kw):
    """Many units are taken whole, off a counter or in turn: their chunks are not counted
    and need not fit 31 bits.  (Without a workspace the call ends at that check, before a
    launch.)"""
    assert call(**kw, wsb=0) == rd.RD_ERR_INVALID_ARG


def test_numbers_past_32_bits_are_refused(monkeypatch):
    """ctypes would cut them: 2^32 + 64 positions became 64, and longer requests zero rows."""
    runs = []
    monkeypatch.setattr(rd, "_fine", lambda *a: True)         # as if the tensors were on a GPU
    monkeypatch.setattr(rd, "_need", lambda *a, **kw: None)
    monkeypatch.setattr(rd, "_run", lambda name, like, *a, stream=None: runs.append(a))
    bf = torch.zeros(4, 8, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    pool, table = torch.zeros(8, 64, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 3, dtype=torch.int32)
    mask = torch.zeros(4, 8, 1, dtype=torch.int32)
    for bad in (2 ** 32 + 64, 2 ** 31, -2 ** 31 - 1):
        with pytest.raises(ValueError, match="max_ctx must fit 32 bits"):
            rd.rd_tree_attention_shared_workspace_size(4, 8, 2, 2, 64, bad, 1)
        for kw in ({}, dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8))):
            with pytest.raises(ValueError, match="max_ctx must fit 32 bits"):
                rd.rd_tree_attention_shared(bf, bf, bf, pool, pool, table, i, i[:2], i[:1], i, mask, max_ctx=bad, **kw)
        with pytest.raises(ValueError, match="max_ctx must fit 32 bits"):
            rd.rd_tree_attention_workspace_size(4, 8, 2, 2, 64, bad)
        with pytest.raises(ValueError, match="page_size must fit 32 bits"):
            rd.rd_resize_pages(table, i, torch.zeros(8, dtype=torch.int32), i, bad)
    assert not runs
    rd.rd_resize_pages(table, i, torch.zeros(8, dtype=torch.int32), i, 64)
    assert runs[0][7] == 64
