"""Host-side checks of the quantised cache's calls and of the log probabilities, without a
GPU: the C entries refuse bad arguments before they touch the device, the binding
refuses tensors that are not on one."""
import ctypes

import pytest
import torch

import tree_attention_verify_gb300 as rd

N = None
ONE, ODD = ctypes.c_void_p(256), ctypes.c_void_p(264)
TWO = ctypes.c_void_p(512)
NAN, INF = float("nan"), float("inf")
POOL = dict(ks=1.0, vs=1.0, pages=64, ps=64, table=ONE, width=16)
GOOD = {
    "rd_append_quant": dict(B=4, Hkv=2, D=128, bits=4, k=ONE, v=ONE, T=100, cu=ONE, kp=ONE, vp=ONE, **POOL, ctx=ONE, new=TWO),
    "rd_commit_accepted_quant": dict(B=4, W=2, L=3, P=6, Hkv=2, D=128, bits=4, k=ONE, v=ONE, unp=ONE, best=ONE, acc=ONE,
                                     kp=ONE, vp=ONE, **POOL, ctx=ONE, new=TWO),
    "rd_read_quant": dict(B=4, Hkv=2, D=128, bits=4, kp=ONE, vp=ONE, **POOL, offs=ONE, starts=N, total=10, k=ONE, v=ONE),
    "rd_tree_attention_quant": dict(B=4, P=8, Hq=8, Hkv=2, D=128, bits=4, scale=0.0, q=ONE, kn=ONE, vn=ONE, kp=ONE, vp=ONE,
                                    **POOL, ctx=ONE, max_ctx=1024, lens=ONE, mask=ONE, words=1, o=ONE, ws=ONE, wsb=1 << 40),
    "rd_token_logprobs": dict(x=ONE, dt=0, n_rows=10, V=100, rows=N, tokens=ONE, n=10, T=1.0, top=3, lp=ONE, ent=ONE, ids=ONE,
                              tops=ONE),
    "rd_accepted_logprobs": dict(x=ONE, dt=0, B=4, P=6, V=100, unp=ONE, W=2, L=3, best=ONE, acc=ONE, tokens=ONE, T=1.0, top=3,
                                 lp=ONE, ent=ONE, ids=ONE, tops=ONE),
}


def call(name, **kw):
    assert set(kw) <= set(GOOD[name])
    return getattr(rd._lib, name)(*{**GOOD[name], **kw}.values(), N, N)


COMMON = [dict(ks=0.0), dict(vs=-1.0), dict(ks=NAN), dict(vs=INF), dict(pages=-1), dict(ps=0), dict(width=-1), dict(Hkv=0),
          dict(D=0), dict(B=-1), dict(kp=N), dict(vp=N), dict(kp=ODD), dict(vp=ODD), dict(table=N)]
INVALID = {
    "rd_append_quant": COMMON + [dict(T=-1)] + [{k: N} for k in ("k", "v", "cu", "ctx", "new")] + [dict(k=ODD), dict(v=ODD)],
    "rd_commit_accepted_quant": COMMON + [dict(W=0), dict(L=0), dict(P=0), dict(new=ONE)]
    + [{k: N} for k in ("k", "v", "unp", "best", "acc", "ctx", "new")] + [dict(k=ODD), dict(v=ODD)],
    "rd_read_quant": COMMON + [dict(total=-1)] + [{k: N} for k in ("offs", "k", "v")] + [dict(k=ODD), dict(v=ODD)],
    "rd_tree_attention_quant": COMMON + [dict(P=0), dict(Hq=7), dict(Hq=0), dict(max_ctx=-1), dict(words=2), dict(words=0),
                                         dict(P=33), dict(wsb=0)]
    + [{k: N} for k in ("q", "kn", "vn", "ctx", "lens", "mask", "o", "ws")] + [{k: ODD} for k in ("q", "kn", "vn", "o", "ws")],
    "rd_token_logprobs": [dict(n_rows=-1), dict(n=-1), dict(n=11), dict(V=0), dict(top=-1), dict(top=101), dict(T=0.0),
                          dict(T=-1.0), dict(T=NAN), dict(T=INF), dict(x=ctypes.c_void_p(257)),
                          dict(dt=2, x=ctypes.c_void_p(258))] + [{k: N} for k in ("x", "tokens", "lp", "ent", "ids", "tops")],
    "rd_accepted_logprobs": [dict(B=-1), dict(P=0), dict(W=0), dict(L=0), dict(V=0), dict(top=-1), dict(top=101), dict(T=0.0),
                             dict(x=ctypes.c_void_p(257))]
    + [{k: N} for k in ("x", "unp", "best", "acc", "tokens", "lp", "ent", "ids", "tops")],
}
SHAPES = [dict(D=96), dict(D=256), dict(bits=3), dict(bits=16), dict(Hkv=65536)]
UNSUPPORTED = {
    "rd_append_quant": SHAPES + [dict(T=1 << 31)],
    "rd_commit_accepted_quant": SHAPES + [dict(B=65536), dict(W=64, L=65)],
    "rd_read_quant": SHAPES + [dict(total=1 << 40)],
    "rd_tree_attention_quant": [dict(D=96), dict(bits=2), dict(ps=48), dict(P=257, words=9), dict(B=65536),
                                dict(Hq=65536, Hkv=65536), dict(Hq=65536, Hkv=2)],
    "rd_token_logprobs": [dict(dt=3), dict(top=33), dict(V=(1 << 30) + 1), dict(n=1 << 31, n_rows=1 << 32)],
    "rd_accepted_logprobs": [dict(dt=3), dict(top=33), dict(W=33), dict(P=257), dict(B=2 ** 31 - 1)],
}


@pytest.mark.parametrize("name,kw", [(n, kw) for n in INVALID for kw in INVALID[n]], ids=str)
def test_refuses_bad_arguments(name, kw):
    assert call(name, **kw) == rd.RD_ERR_INVALID_ARG


@pytest.mark.parametrize("name,kw", [(n, kw) for n in UNSUPPORTED for kw in UNSUPPORTED[n]], ids=str)
def test_refuses_what_it_does_not_support(name, kw):
    assert call(name, **kw) == rd.RD_ERR_UNSUPPORTED


def test_calls_without_work():
    for name in ("rd_append_quant", "rd_commit_accepted_quant", "rd_read_quant", "rd_tree_attention_quant", "rd_accepted_logprobs"):
        assert call(name, B=0) == rd.RD_OK
    assert call("rd_read_quant", total=0, k=N, v=N) == rd.RD_OK
    assert call("rd_token_logprobs", n=0) == rd.RD_OK


def test_sizes():
    assert [rd.rd_quant_row_bytes(*x) for x in ((128, 4), (64, 4), (128, 8), (64, 8), (96, 4), (128, 5))] == [72, 36, 128, 64, 0, 0]
    size = rd.rd_tree_attention_quant_workspace_size
    need = size(4, 8, 8, 2, 128, 1024)
    assert need > 0 and need % 16 == 0 and call("rd_tree_attention_quant", wsb=need - 1) == rd.RD_ERR_INVALID_ARG
    assert size(0, 8, 8, 2, 128, 64) == size(4, 0, 8, 2, 128, 64) == size(4, 8, 7, 2, 128, 64) == size(4, 8, 8, 2, 128, -1) == 0
    with pytest.raises(ValueError, match="32 bits"):
        size(4, 8, 8, 2, 128, 2 ** 32 + 64)


def test_binding_refuses_before_a_launch():
    bf = torch.zeros(4, 8, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    pool, table = torch.zeros(8, 64, 2, 36, dtype=torch.uint8), torch.zeros(4, 3, dtype=torch.int32)
    mask = torch.zeros(4, 8, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        rd.rd_tree_attention_quant(bf, bf, bf, pool, pool, 1.0, 1.0, table, i, i, mask, max_ctx=64)
    with pytest.raises(ValueError, match="k must be a CUDA tensor"):
        rd.rd_append_quant(bf[0], bf[0], i, pool, pool, 1.0, 1.0, table, i)
    with pytest.raises(ValueError, match="k_new must be a CUDA tensor"):
        rd.rd_commit_accepted_quant(bf, bf, i, i, i, pool, pool, 1.0, 1.0, table, i)
    with pytest.raises(ValueError, match="k_pool must be a CUDA tensor"):
        rd.rd_read_quant(pool, pool, 1.0, 1.0, table, i, total=3)
    with pytest.raises(ValueError, match="logits must be a CUDA tensor"):
        rd.rd_token_logprobs(torch.zeros(4, 10), i)
    with pytest.raises(TypeError, match="logits must be bfloat16"):
        rd.rd_token_logprobs(torch.zeros(4, 10, dtype=torch.float64), i)
    with pytest.raises(ValueError, match="logits must be a CUDA tensor"):
        rd.rd_accepted_logprobs(torch.zeros(4, 5, 10), table, i, i, table)


def test_binding_checks_shapes(monkeypatch):
    """As if the tensors were on a GPU: shapes that disagree never reach the library."""
    runs = []
    monkeypatch.setattr(rd, "_fine", lambda *a: True)
    monkeypatch.setattr(rd, "_need", lambda *a, **kw: None)
    monkeypatch.setattr(rd, "_run", lambda name, like, *a, stream=None: runs.append(name))
    z = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype)
    bf = lambda *s: z(*s, dtype=torch.bfloat16)
    pool = z(8, 64, 2, 36, dtype=torch.uint8)
    ok = (z(4, 3), z(4))
    rd.rd_append_quant(bf(9, 2, 64), bf(9, 2, 64), z(5), pool, pool, 1.0, 1.0, *ok)
    assert runs == ["rd_append_quant"]
    ctx = z(4)
    with pytest.raises(ValueError, match="alias"):
        rd.rd_append_quant(bf(9, 2, 64), bf(9, 2, 64), z(5), pool, pool, 1.0, 1.0, z(4, 3), ctx, new_ctx_lens=ctx)
    for args in ((bf(9, 2, 128), bf(9, 2, 128), z(5), pool, pool), (bf(9, 3, 64), bf(9, 3, 64), z(5), pool, pool),
                 (bf(9, 2, 64), bf(8, 2, 64), z(5), pool, pool), (bf(9, 2, 64), bf(9, 2, 64), z(4), pool, pool),
                 (bf(9, 2, 64), bf(9, 2, 64), z(5), pool, pool[:4])):
        with pytest.raises(ValueError):
            rd.rd_append_quant(*args, 1.0, 1.0, *ok)
    for kw in (dict(q=bf(4, 8, 4, 128)), dict(kn=bf(4, 8, 3, 64)), dict(vn=bf(4, 7, 2, 64)), dict(table=z(3, 3)), dict(ctx=z(3)),
               dict(lens=z(5)), dict(mask=z(4, 7, 1)), dict(kp=z(8, 64, 2, 40, dtype=torch.uint8))):
        a = {**dict(q=bf(4, 8, 4, 64), kn=bf(4, 8, 2, 64), vn=bf(4, 8, 2, 64), kp=pool, vp=pool, ks=1.0, vs=1.0, table=z(4, 3),
                    ctx=z(4), lens=z(4), mask=z(4, 8, 1)), **kw}
        with pytest.raises(ValueError):
            rd.rd_tree_attention_quant(*a.values(), max_ctx=64)
    for a in ((z(4, 10), z(5)),):
        with pytest.raises((ValueError, TypeError)):
            rd.rd_token_logprobs(*a)
    with pytest.raises(ValueError):
        rd.rd_token_logprobs(bf(4, 10), z(5))
    with pytest.raises(ValueError):
        rd.rd_accepted_logprobs(bf(4, 6, 10), z(4, 2, 3), z(4), z(4), z(4, 2))
    with pytest.raises(ValueError):
        rd.rd_read_quant(pool, pool, 1.0, 1.0, z(4, 3), z(4), total=3)
    assert runs == ["rd_append_quant"]


def test_append_refuses_lengths_in_place():
    assert call("rd_append_quant", ctx=ONE, new=ONE) == rd.RD_ERR_INVALID_ARG


@pytest.mark.parametrize("top", [33, 10 ** 9, -1, 2 ** 31 - 1])
def test_refused_alternatives_take_no_memory(top, monkeypatch):
    """A number of alternatives that the call refuses is refused, before outputs of its size are asked for."""
    asked = []
    monkeypatch.setattr(rd, "_fine", lambda *a: True)
    monkeypatch.setattr(rd, "_need", lambda *a, **kw: None)
    monkeypatch.setattr(rd, "_run", lambda name, like, *a, stream=None: (_ for _ in ()).throw(rd.RdError(name, rd.RD_ERR_UNSUPPORTED)))
    monkeypatch.setattr(rd, "_new", lambda shape, dtype, like, stream: asked.append(shape) or torch.zeros(shape, dtype=dtype))
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(rd.RdError):
        rd.rd_token_logprobs(torch.zeros(4, 10), i32(4), top=top)
    with pytest.raises(rd.RdError):
        rd.rd_accepted_logprobs(torch.zeros(4, 6, 10), i32(4, 2, 3), i32(4), i32(4), i32(4, 3), top=top)
    assert len(asked) == 8 and all(max(s) <= 32 for s in asked)
