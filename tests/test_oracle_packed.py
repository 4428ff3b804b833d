"""Pins of the oracle of rotation on several axes and of packed attention (CPU only)."""
import numpy as np
import pytest
import torch

from oracle import kv as okv, packed as op


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


@pytest.mark.parametrize("interleaved", [False, True])
def test_equal_positions_are_the_rotation_of_one_axis(interleaved):
    r = rng(1)
    x = r.standard_normal((5, 4 * 16))
    pos = np.array([3, 0, 9, -1, 7])
    ang = r.standard_normal((10, 6))
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    w = r.standard_normal((2, 16))
    one, _ = okv.norm_rope(x, 3, 1, 16, pos, table, w[0], w[1], interleaved=interleaved)
    many, _ = op.norm_rope_axes(x, 3, 1, 16, np.stack([pos] * 3), table, [0, 1, 2, 0, 1, 2], w[0], w[1],
                                interleaved=interleaved)
    assert np.allclose(one, many, rtol=1e-14, atol=1e-14, equal_nan=True)
    assert np.isnan(many[3]).all()


def test_an_axis_turns_its_own_pairs():
    x = rng(2).standard_normal((1, 8))
    ang = np.arange(4)[:, None] * np.array([1.0, 0.5])
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    y, _ = op.norm_rope_axes(x, 1, 0, 8, np.array([[0], [2]]), table, [0, 1])
    assert np.allclose(y[0, 0, [0, 2, 4, 5, 6, 7]], x[0, [0, 2, 4, 5, 6, 7]])
    a, b = x[0, 1], x[0, 3]
    assert np.allclose(y[0, 0, [1, 3]], [a * np.cos(1) - b * np.sin(1), b * np.cos(1) + a * np.sin(1)])


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 3)])
def test_attention_is_the_softmax_of_each_prompt(causal, window):
    r = rng(3)
    cu = np.array([0, 4, 4, 11])
    q, k, v = r.standard_normal((13, 4, 8)), r.standard_normal((13, 2, 8)), r.standard_normal((13, 2, 8))
    out, lse, _, _ = op.attention(q, k, v, cu, 0.4, causal, window)
    for a, b in zip(cu[:-1], cu[1:]):
        tq, tk, tv = (torch.from_numpy(t[a:b]).transpose(0, 1) for t in (q, k, v))
        s = tq @ tk.repeat_interleave(2, 0).transpose(1, 2) * 0.4
        n = b - a
        i = torch.arange(n)
        hide = torch.zeros(n, n, dtype=torch.bool)
        if causal:
            hide = i > i[:, None]
            if window:
                hide |= i <= i[:, None] - window
        s = s.masked_fill(hide, -np.inf)
        want = torch.softmax(s, -1) @ tv.repeat_interleave(2, 0)
        assert np.allclose(out[a:b], want.transpose(0, 1).numpy())
        assert np.allclose(lse[a:b], torch.logsumexp(s, -1).T.numpy())
    assert np.isnan(out[11:]).all()


def test_values_that_a_row_does_not_see_do_not_reach_it():
    r = rng(4)
    q, k, v = (r.standard_normal((6, 1, 4)) for _ in range(3))
    clean = op.attention(q, k, v, [0, 6], 1.0)[0]
    v[4, 0, 2] = np.nan
    v[5, 0, 1] = np.inf
    out = op.attention(q, k, v, [0, 6], 1.0)[0]
    assert np.allclose(out[:4], clean[:4]) and np.isnan(out[4:, 0, 2]).all() and np.isinf(out[5, 0, 1])
    assert np.allclose(out[4:, 0, [0, 3]], clean[4:, 0, [0, 3]])
