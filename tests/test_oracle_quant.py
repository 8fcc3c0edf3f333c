"""Pins of the plain implementation of the quantised cache and of the log probabilities."""
import numpy as np
import pytest
import torch

from oracle import quant


def test_e4m3_is_the_ocp_format():
    codes = np.arange(256, dtype=np.uint8)
    ref = torch.tensor(codes).view(torch.float8_e4m3fn).double().numpy()
    got = quant.e4m3_value(codes)
    np.testing.assert_array_equal(got[~np.isnan(ref)], ref[~np.isnan(ref)])
    assert np.isnan(got[np.isnan(ref)]).all()


def test_nearest_code_rounds_as_torch_does():
    x = torch.randn(4000, dtype=torch.float64) * 3
    want = x.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy() & 127
    np.testing.assert_array_equal(quant.nearest_code(x.float().double().numpy(), quant.E4M3)[0], want)


@pytest.mark.parametrize("x,code", [(0.25, 0), (0.26, 1), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6),
                                    (5.01, 7), (100.0, 7), (-2.5, 4)])
def test_e2m1_ties_go_to_the_even_code(x, code):
    assert quant.nearest_code(x, quant.E2M1)[0] == code


def test_a_row_worked_by_hand():
    x = np.zeros(64)
    x[:4] = [6, -3, 1.2, 0.2]              # scale 1: codes 7, 5 | 8, 2 (1), 0
    x[16:18] = [0.75, -0.125]              # amax 0.75: scale 0.125, codes 6 -> 7, -1 -> 2 | 8
    row, _ = quant.encode_row(x, 1.0, 4)
    assert row.shape == (36,) and row[0] == 7 | (13 << 4) and row[1] == 2 and row[8] == 7 | (10 << 4)
    np.testing.assert_array_equal(quant.decode(row, 1.0, 64, 4)[[0, 1, 2, 3, 16, 17]], [6, -3, 1, 0, 0.75, -0.125])
    row, _ = quant.encode_row(x, 0.5, 8)
    np.testing.assert_array_equal(quant.decode(row, 0.5, 64, 8)[[0, 1, 16, 17]], [6, -3, 0.75, -0.125])


@pytest.mark.parametrize("bits,step", [(4, 1 / 4), (8, 2.0 ** -4)])
def test_decoded_values_are_near(bits, step):
    rng = np.random.default_rng(0)
    for _ in range(20):
        x = rng.standard_normal(128) * rng.choice([0.01, 1, 30])
        g = np.abs(x).max() / (448 if bits == 8 else 2688)
        y = quant.decode(quant.encode_row(x, g, bits)[0], g, 128, bits)
        amax = np.abs(x).reshape(-1, 16).max(1).repeat(16) if bits == 4 else np.abs(x)
        # e4m3: half a step of the value; e2m1: the scale's half step and half a step below the block's largest
        tol = amax * step * (1 + 2.0 ** -4) + g * 2.0 ** -9
        assert (np.abs(x - y) <= tol).all()


def test_attention_is_softmax():
    rng = np.random.default_rng(1)
    B, P, Hq, Hkv, D = 2, 3, 4, 2, 8
    q, kn, vn = rng.standard_normal((B, P, Hq, D)), rng.standard_normal((B, P, Hkv, D)), rng.standard_normal((B, P, Hkv, D))
    kc, vc = ([rng.standard_normal((c, Hkv, D)) for c in (5, 0)] for _ in range(2))
    mask = np.array([[[1], [3], [7]], [[1], [2], [0]]], np.int64)
    lens = [3, 3]
    o, _, _ = quant.attention(q, kn, vn, kc, vc, lens, mask)
    t = torch.tensor
    k = t(np.concatenate([kc[0], kn[0]])).repeat_interleave(2, 1).transpose(0, 1)
    v = t(np.concatenate([vc[0], vn[0]])).repeat_interleave(2, 1).transpose(0, 1)
    see = torch.ones(3, 8, dtype=torch.bool)
    see[:, 5:] = torch.tril(torch.ones(3, 3, dtype=torch.bool))
    want = torch.nn.functional.scaled_dot_product_attention(t(q[0]).transpose(0, 1), k, v, attn_mask=see)
    np.testing.assert_allclose(o[0], want.transpose(0, 1).numpy(), atol=1e-12)
    np.testing.assert_allclose(o[1, 0], np.repeat(vn[1, 0], 2, 0), atol=1e-12)      # one visible key
    assert (o[1, 2] == 0).all()                                                      # none


def test_logprobs():
    x = torch.randn(50, dtype=torch.float64) * 3
    lp = torch.log_softmax(x / 0.7, 0)
    a, h, ids, tops, _ = quant.logprobs(x.numpy(), 7, 0.7, 5)
    assert abs(a - lp[7]) < 1e-12 and abs(h + (lp.exp() * lp).sum()) < 1e-12
    np.testing.assert_array_equal(ids, torch.topk(x, 5).indices.numpy())
    np.testing.assert_allclose(tops, lp[ids.copy()].numpy(), atol=1e-12)
    assert list(quant.logprobs([1.0, 2.0, 2.0, 1.0], 0, 1.0, 3)[2]) == [1, 2, 0]     # equals: the lower id
    a, h, ids, tops, _ = quant.logprobs([0.0, -np.inf, 0.0], 1, 1.0, 3)
    assert a == -np.inf and abs(h - np.log(2)) < 1e-12 and list(ids) == [0, 2, 1] and tops[2] == -np.inf
