"""CPU pins of the oracle's serving operators: the int8 block of a paged
cache against a worked example and its error bound, row attention against a
causal full computation, filtered sampling against a literal walk and the
distribution it stands for."""
import math

import numpy as np
import pytest

from oracle import qg_oracle as O


def test_kv_block_append_worked_example():
    codes = np.zeros((16, 2), dtype=np.int64)
    codes, s = O.kv_block_append(codes, 99.0, 0, [[1.27, -0.635]])     # o = 0: the old scale goes
    assert s == pytest.approx(0.01) and codes[0].tolist() == [127, -64]  # -63.5 rounds to even
    codes, s = O.kv_block_append(codes, s, 1, [[2.54, 0.02]])          # twice the scale
    assert s == pytest.approx(0.02)
    assert codes[:2].tolist() == [[64, -32], [127, 1]]                 # 63.5 -> 64, -32
    codes, s2 = O.kv_block_append(codes, s, 2, [[0.0, 0.5], [0.04, 0.0]])
    assert s2 == s and codes[:4].tolist() == [[64, -32], [127, 1], [0, 25], [2, 0]]


def test_kv_block_append_error_bound():
    """Each value is within half a step at its writing and half a step of
    every later, larger scale."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((16, 64)) * np.exp(rng.standard_normal((16, 1)))
    codes, s, bound = np.zeros((16, 64), dtype=np.int64), 0.0, np.zeros(16)
    for t in range(16):
        was = s
        codes, s = O.kv_block_append(codes, s, t, x[t:t + 1])
        if s != was:
            bound[:t] += s / 2
        bound[t] = s / 2
        assert np.all(np.abs(codes[:t + 1] * s - x[:t + 1]) <= bound[:t + 1, None] * (1 + 1e-12))


def test_kv_block_append_zero_and_not_finite():
    z, s = O.kv_block_append(np.full((16, 4), 5), 1.0, 0, np.zeros((3, 4)))
    assert s == 0 and not z[:3].any() and (z[3:] == 5).all()
    assert math.isnan(O.kv_block_append(z, 0.0, 3, [[1, np.inf, 0, 0]])[1])
    assert math.isnan(O.kv_block_append(z, math.nan, 3, [[1, 1, 0, 0]])[1])
    assert O.kv_block_append(z, math.nan, 0, [[1, 1, 0, 0]])[1] == pytest.approx(1 / 127)


def test_rows_attention_is_the_causal_softmax():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((3, 4 * 8)), rng.standard_normal((2, 7, 8)), rng.standard_normal((2, 7, 8))
    got = O.rows_attention(q, k, v, 4, 2, 8)
    full = O.mha_rows(q, k.transpose(1, 0, 2).reshape(7, 16), v.transpose(1, 0, 2).reshape(7, 16),
                      4, causal=True, kv_heads=2)
    np.testing.assert_allclose(got, full, rtol=1e-12, atol=1e-12)


def _walk(l, u, temperature, top_k, top_p, min_p):
    """The definition, one candidate after another."""
    cand = sorted((i for i in range(len(l)) if l[i] > -math.inf), key=lambda i: (-l[i], i))
    if temperature <= 0:
        return cand[0], 1
    w = [math.exp((l[i] - l[cand[0]]) / temperature) for i in cand]
    if top_k > 0:
        cand, w = cand[:top_k], w[:top_k]
    if top_p < 1:
        total, acc, m = sum(w), 0.0, 0
        while m < len(w) and (m == 0 or acc < top_p * total):
            acc += w[m]
            m += 1
        cand, w = cand[:m], w[:m]
    m = len([x for x in w if x >= min_p])
    cand, w = cand[:m], w[:m]
    acc = 0.0
    for i, x in zip(cand, w):
        acc += x
        if acc >= u * sum(w):
            return i, m
    return cand[-1], m


@pytest.mark.parametrize("seed", range(12))
def test_sample_filtered_against_a_walk(seed):
    rng = np.random.default_rng(seed)
    l = np.round(rng.standard_normal(57) * 2, 1 if seed % 2 else 6)  # ties at odd seeds
    l[rng.integers(0, 57, 5)] = -np.inf
    for _ in range(20):
        args = (float(rng.random()), float(rng.choice([0.0, 0.5, 1.0, 2.0])),
                int(rng.choice([0, 1, 5, 57, 100])), float(rng.choice([0.0, 0.3, 0.9, 1.0])),
                float(rng.choice([0.0, 0.05, 0.5, 1.0])))
        token, kept, _ = O.sample_filtered(l, *args)
        assert (token, kept) == _walk(l.tolist(), *args)


def test_sample_filtered_draws_its_distribution():
    l = np.log([0.1, 0.4, 0.2, 0.25, 0.05])
    u = (np.arange(20000) + 0.5) / 20000
    got = np.bincount([O.sample_filtered(l, x, top_p=0.8)[0] for x in u], minlength=5) / 20000
    np.testing.assert_allclose(got, np.array([0, 0.4, 0.2, 0.25, 0]) / 0.85, atol=1e-4)
    assert O.sample_filtered(l, 0.0)[0] == 1 and O.sample_filtered(l, 0.0)[1] == 5
    assert O.sample_filtered(l, 0.3)[2] == pytest.approx(math.log(0.4))


def test_sample_filtered_odd_rows():
    nan, inf = math.nan, math.inf
    assert O.sample_filtered([nan, -inf, nan], 0.5)[:2] == (0, 0)
    assert O.sample_filtered([nan, 1.0, -inf, 1.0], 0.9)[:2] == (3, 2)
    assert O.sample_filtered([0.0, inf, 5.0, inf], 0.9, top_p=0.5)[:2] == (1, 1)
    assert O.sample_filtered([0.0, inf, 5.0, inf], 0.9)[0] == 3
    assert O.sample_filtered([2.0, 2.0, 1.0], 0.5, temperature=0.0) == (0, 1, 0.0)
