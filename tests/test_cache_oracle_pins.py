"""Pins of the cache and beam oracle (CPU): library routines, closed forms and
invariants that share nothing with it."""

import math

import numpy as np
import pytest
import torch

from oracle import cache_oracle as co

RNG = np.random.default_rng(0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    x, freq = RNG.standard_normal((3, 20)), co.rope_frequencies(16)
    y = co.rotate(x, 1234, freq, interleaved, 1.5)
    pairs = x[:, :16].reshape(3, 8, 2) if interleaved else np.stack([x[:, :8], x[:, 8:16]], -1)
    z = (pairs[..., 0] + 1j * pairs[..., 1]) * 1.5 * np.exp(1j * 1234 * freq)
    got = y[:, :16].reshape(3, 8, 2) if interleaved else np.stack([y[:, :8], y[:, 8:16]], -1)
    assert np.allclose(got[..., 0] + 1j * got[..., 1], z, atol=1e-12) and np.array_equal(y[:, 16:], x[:, 16:])


def test_rotated_products_depend_on_the_distance_alone():
    q, k, freq = RNG.standard_normal((1, 32)), RNG.standard_normal((1, 32)), co.rope_frequencies(32, base=500.0)
    dots = [float((co.rotate(q, p + 7, freq, False, 1.0) * co.rotate(k, p, freq, False, 1.0)).sum()) for p in (0, 5, 900)]
    assert np.allclose(dots, dots[0], atol=1e-10)


def test_scaled_frequencies():
    f = co.rope_frequencies(64)
    assert f[0] == 1.0 and np.allclose(f[1:] / f[:-1], 10000.0 ** (-1 / 32))
    assert np.allclose(co.rope_frequencies(64, factor=8.0), f / 8)          # all alike
    s = co.rope_frequencies(64, factor=8.0, original_len=4096, low=1.0, high=4.0)
    turns = 4096 * f / (2 * math.pi)
    assert np.allclose(s[turns >= 4], f[turns >= 4]) and np.allclose(s[turns <= 1], f[turns <= 1] / 8)
    between = (turns > 1) & (turns < 4)
    assert between.any() and np.all(s[between] < f[between]) and np.all(s[between] > f[between] / 8)


def test_append_writes_only_its_positions():
    q, k, v = RNG.standard_normal((5, 2, 8)), RNG.standard_normal((5, 1, 8)), RNG.standard_normal((5, 1, 8))
    kp, vp = RNG.standard_normal((4, 3, 1, 8)), RNG.standard_normal((4, 3, 1, 8))
    table = np.array([[1, 2], [3, 0]])
    out, k2, v2 = co.rope_append(q, k, v, np.zeros(4), np.array([4, 5]), table, kp, vp, cu_seqlens=np.array([0, 2, 4]))
    assert np.array_equal(out[:4], q[:4]) and np.all(out[4] == 0)           # zero frequencies rotate nothing; row 4 is padding
    assert np.array_equal(k2[1, 2], k[0]) and np.array_equal(k2[2, 0], k[1])  # positions 2 and 3 of sequence 0
    changed = (v2 != vp).any(axis=(2, 3))
    assert changed.sum() == 2 and changed[1, 2] and changed[2, 0]            # sequence 1's positions 3, 4: a null page


@pytest.mark.parametrize("window", [0, 3])
def test_attention_is_the_library_softmax(window):
    N, Hq, Hkv, D, page = 3, 6, 2, 16, 4
    q = RNG.standard_normal((N, Hq, D))
    kp, vp = RNG.standard_normal((9, page, Hkv, D)), RNG.standard_normal((9, page, Hkv, D))
    table, lens = np.array([[1, 2, 3], [4, 0, 5], [0, 0, 0]]), np.array([10, 12, 5])
    out, lse = co.paged_attention(q, kp, vp, table, lens, window=window)
    for n in range(N):
        at = [t for t in range(lens[n]) if table[n, t // page] > 0 and (window == 0 or t >= lens[n] - window)]
        if not at:
            assert np.all(out[n] == 0) and np.all(lse[n] == -np.inf)
            continue
        K = torch.tensor(np.stack([kp[table[n, t // page], t % page] for t in at])).transpose(0, 1)
        V = torch.tensor(np.stack([vp[table[n, t // page], t % page] for t in at])).transpose(0, 1)
        K, V = (x.repeat_interleave(Hq // Hkv, 0) for x in (K, V))
        ref = torch.nn.functional.scaled_dot_product_attention(torch.tensor(q[n])[:, None], K, V)[:, 0]
        assert np.allclose(out[n], ref.numpy(), atol=1e-12)
        sums = torch.logsumexp((torch.tensor(q[n])[:, None] @ K.transpose(1, 2))[:, 0] / 4.0, -1)
        assert np.allclose(lse[n], sums.numpy(), atol=1e-12)


def test_beam_values_are_the_library_log_softmax():
    x, s = RNG.standard_normal((2, 3, 50)), RNG.standard_normal((2, 3))
    c = co.beam_candidates(x, s)
    assert np.allclose(c, torch.log_softmax(torch.tensor(x), -1).numpy() + s[..., None], atol=1e-12)
    scores, parents, tokens = co.beam_select(x, s, 7)
    top = torch.topk(torch.tensor(c).view(2, -1), 7)
    assert np.allclose(scores, top.values.numpy()) and np.array_equal(parents * 50 + tokens, top.indices.numpy())


def test_beam_ties_dead_and_finished_beams():
    x = np.zeros((1, 3, 4))
    s = np.array([[0.0, 0.0, -np.inf]])
    scores, parents, tokens = co.beam_select(x, s, 8)
    assert parents[0].tolist() == [0] * 4 + [1] * 4 and tokens[0].tolist() == [0, 1, 2, 3] * 2
    scores, parents, tokens = co.beam_select(x, s, 8, finished=np.array([[0, 1, 1]]), eos_token=3)
    assert parents[0].tolist() == [1, 0, 0, 0, 0, -1, -1, -1] and tokens[0, 0] == 3 and scores[0, 0] == 0.0
    x[0, 0, 1] = np.inf
    assert co.beam_select(x, s, 1)[1][0, 0] == 1


def test_moves_are_simultaneous():
    pool = np.arange(12.0).reshape(6, 2)
    got = co.pool_move([pool], np.array([[1, 2, 3]]), np.array([[1, 2, 3]]), np.array([[1, 2, 0]]))[0]
    assert np.array_equal(got, pool[[0, 2, 3, 1, 4, 5]])
    got = co.pool_move([pool], np.array([[1], [0], [9]]), np.array([[4], [5], [0]]))[0]
    assert np.array_equal(got[4], pool[1]) and np.all(got[5] == 0) and np.array_equal(got[:4], pool[:4])
    assert np.array_equal(co.pool_move([pool], np.array([[1, 2]]), np.array([[1, 2]]), np.array([[-1, 2]]))[0], pool)
