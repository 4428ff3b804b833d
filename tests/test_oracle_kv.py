"""Pins of the head norm / cache / attention oracle (CPU)."""
import numpy as np
import pytest
import torch

from kv_util import batch, random_cache, rng
from oracle import e4m3, kv as okv, quant as oq


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_composes(interleaved):
    r = rng(1)
    D, rot, P = 64, 32, 40
    ang = np.arange(P)[:, None] * 0.37 ** np.arange(rot // 2)
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    x = r.standard_normal((3, 2 * D))
    y, _ = okv.norm_rope(x, 1, 1, D, [0, 7, 30], cs, interleaved=interleaved)
    x3 = x.reshape(3, 2, D)
    assert np.allclose(y[0], x3[0]) and np.allclose((y ** 2).sum(-1), (x3 ** 2).sum(-1))
    assert np.array_equal(y[..., rot:], x3[..., rot:])
    again, _ = okv.norm_rope(y[1:2].reshape(1, -1), 1, 1, D, [9], cs, interleaved=interleaved)
    once, _ = okv.norm_rope(x[1:2], 1, 1, D, [16], cs, interleaved=interleaved)
    assert np.allclose(again, once)
    # as complex numbers
    z = x3[1, :, 0:rot:2] + 1j * x3[1, :, 1:rot:2] if interleaved else x3[1, :, :rot // 2] + 1j * x3[1, :, rot // 2:rot]
    z = z * np.exp(1j * ang[7])
    got = y[1, :, 0:rot:2] + 1j * y[1, :, 1:rot:2] if interleaved else y[1, :, :rot // 2] + 1j * y[1, :, rot // 2:rot]
    assert np.allclose(got, z)


def test_norm_has_unit_mean_square_and_padding_rows_are_nan():
    x = rng(2).standard_normal((2, 256)) * 100
    w = np.full(64, 2.0)
    y, _ = okv.norm_rope(x, 3, 1, 64, wq=w, wk=w / 2, eps=0.0)
    assert np.allclose((y[:, :3] ** 2).mean(-1), 4) and np.allclose((y[:, 3] ** 2).mean(-1), 1)
    y, _ = okv.norm_rope(x, 3, 1, 64, [-1, 5], np.ones((5, 16)))
    assert np.isnan(y).all()


@pytest.mark.parametrize("block,D", [(16, 64), (32, 128)])
def test_a_fresh_block_is_one_group_of_the_ue8m0_quant(block, D):
    r = rng(3)
    k, v = (r.standard_normal((block, 2, D)).astype(np.float32) * s for s in (1, 1e-3))
    c = random_cache(r, 1, 2, block, D)
    okv.write(c, k, v, [0, block], [block], np.zeros((1, 1), dtype=np.int32))
    for which, x in ((0, k), (1, v)):
        for h in range(2):
            q = oq.quant_group(x[:, h].reshape(1, -1), block * D, pow2=True)
            assert int(c.exp[which][0, h]) == int(q.ue8m0_byte.reshape(-1)[0])
            got = np.stack([c.get(which, 0, s, h) for s in range(block)])
            assert np.array_equal(got.reshape(-1), q.codes.reshape(-1))


def test_appending_raises_the_exponent_and_rounds_again():
    r = rng(4)
    c = random_cache(r, 1, 1, 16, 64)
    table = np.zeros((1, 1), dtype=np.int32)
    x = r.standard_normal((5, 1, 64)) * np.array([1, 0.1, 30, 2, 1e4])[:, None, None]
    for i in range(5):
        okv.write(c, x[i:i + 1], x[i:i + 1], [0, 1], [i + 1], table)
        top = max(okv.exponent(np.abs(x[j]).max()) for j in range(i + 1))
        assert c.exp[0][0, 0] == c.exp[1][0, 0] == top + 127
        step = 2.0 ** top
        for j in range(i + 1):
            val = c.token(0, 0, j)[0]
            # two roundings at most to the code grid of the largest step: half a
            # code step each, 2^-4 of the value or 2^-10 of the scale
            assert np.all(np.abs(val - x[j, 0]) <= (i + 1) * np.maximum(np.abs(x[j, 0]) * 2.0 ** -4, step * 2.0 ** -10))
            assert np.array_equal(val, c.token(1, 0, j)[0])


def test_exponent_rule_at_its_border_and_for_zero():
    assert okv.exponent(448.0) == 0 and okv.exponent(np.nextafter(448.0, 500)) == 1
    assert okv.exponent(0.0) + 127 == 85 and okv.exponent(448.0 * 2.0 ** -9) == -9


def test_non_finite_values_do_not_set_the_scale():
    x = np.array([np.inf, -np.inf, np.nan, 1.0] + [0.5] * 60).reshape(1, 1, 64)
    c = random_cache(rng(5), 1, 1, 16, 64)
    okv.write(c, x, x, [0, 1], [1], np.zeros((1, 1), dtype=np.int32))
    e = okv.exponent(1.0)
    assert c.exp[0][0, 0] == e + 127
    val = c.token(0, 0, 0)[0]
    assert val[0] == 448 * 2.0 ** e and val[1] == -448 * 2.0 ** e and np.isnan(val[2]) and val[3] == 1.0


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 5), (False, 0)])
def test_attention_equals_a_dense_softmax(causal, window):
    r = rng(6)
    n, lens = [3, 1, 0, 20], [40, 17, 5, 20]
    cu, L, table, blocks = batch(r, n, lens, 16)
    c = random_cache(r, blocks, 2, 16, 64)
    q = r.standard_normal((sum(n), 4, 64))
    out, lse, _, _ = okv.attention(q, c, cu, L, table, 0.2, causal, window)
    kk, vv = okv.read(c, np.concatenate([[0], np.cumsum(lens)]), L, table, sum(lens))
    at = 0
    for b, (a, ln) in enumerate(zip(n, lens)):
        K, V = (torch.from_numpy(x[at:at + ln]).repeat_interleave(2, 1) for x in (kk, vv))
        at += ln
        if a == 0:
            continue
        s = torch.einsum("qhd,khd->hqk", torch.from_numpy(q[cu[b]:cu[b + 1]]), K) * 0.2
        d = torch.arange(ln - a, ln)[:, None] - torch.arange(ln)
        if causal:
            s = s.masked_fill((d < 0) | ((d >= window) if window else (d < 0)), -np.inf)
        ref = torch.einsum("hqk,khd->qhd", s.softmax(-1), V)
        assert np.allclose(out[cu[b]:cu[b + 1]], ref.numpy(), rtol=1e-12, atol=1e-12)
        assert np.allclose(lse[cu[b]:cu[b + 1]], s.logsumexp(-1).T.numpy(), rtol=1e-12)


def test_rows_that_see_nothing_and_blocks_that_do_not_exist():
    r = rng(7)
    c = random_cache(r, 3, 1, 16, 64)
    q = r.standard_normal((4, 1, 64))
    out, lse, _, _ = okv.attention(q, c, [0, 4], [2], np.zeros((1, 1), dtype=np.int32), 1.0)
    assert np.all(out[:2] == 0) and np.all(np.isneginf(lse[:2])) and np.all(np.isfinite(lse[2:]))
    # a bad block is as if its tokens were not there
    t = np.array([[2, 7]], dtype=np.int32)
    a = okv.attention(q[:1], c, [0, 1], [30], t, 1.0)
    b = okv.attention(q[:1], c, [0, 1], [16], t, 1.0)
    assert np.array_equal(a[0], b[0])
    # one visible token: its value
    one = okv.attention(q[:1], c, [0, 1], [1], t, 1.0)[0]
    assert np.array_equal(one[0], c.token(1, 2, 0)) and e4m3.decode(np.uint8([0x7E]))[0] == 448
