"""Pins of the batched serving oracle: closed forms, brute force, statistics."""
import numpy as np
import pytest

from oracle import batch as ob
from oracle.bf16 import round_bf16
from oracle.model import attention


def test_quantise_grid_rows_are_exact():
    x = np.arange(-127, 128, 2, dtype=np.float32)[None] * np.float32(2.0 ** -5)   # ends on 127 steps
    c, s = ob.kv8_quantise(x)
    assert s[0] == np.float32(2.0 ** -5) and np.array_equal(c[0], np.arange(1, 256, 2))
    assert np.array_equal(ob.kv8_values(c, s), x)


def test_quantise_error_is_at_most_half_a_step():
    x = round_bf16(np.random.default_rng(0).standard_normal((64, 128)).astype(np.float32))
    c, s = ob.kv8_quantise(x)
    err = np.abs(ob.kv8_values(c, s).astype(np.float64) - x)
    # half a step, and three roundings of 2^-24 of a value up to 127 steps
    assert np.all(err <= s[:, None] * (0.5 + 3 * 127 * 2.0 ** -24))
    assert c.min() >= 1 and c.max() <= 255


def test_quantise_special_rows():
    x = np.zeros((5, 64), np.float32)
    x[1, 3] = 2.0 ** -101
    x[2, 3] = 2.0 ** -99
    x[3, 5], x[3, 6] = np.inf, 1
    x[4, 5] = np.nan
    c, s = ob.kv8_quantise(x)
    assert s[0] == 1 and s[1] == 1 and np.all(c[:2] == 128)
    assert c[2, 3] == 255 and c[2, 0] == 128
    assert np.isnan(s[3]) and np.isnan(s[4]) and np.all(c[3:] == 128)


@pytest.mark.parametrize("pos,n", [(0, 5), (7, 1), (12, 4)])
def test_chunk_attention_is_causal_attention(pos, n):
    rng = np.random.default_rng(pos)
    q = rng.standard_normal((n, 4, 16)).astype(np.float32)
    k, v = (rng.standard_normal((pos + n, 2, 16)).astype(np.float32) for _ in range(2))
    mask = np.arange(pos + n)[None] <= pos + np.arange(n)[:, None]
    o, w = ob.chunk_attention(q, k, v, pos)
    np.testing.assert_allclose(o, attention(q, k, v, mask, 2).reshape(o.shape), rtol=1e-6, atol=1e-6)
    assert np.all(w >= np.abs(o) - 1e-12)


def test_chunk_attention_without_keys_is_zero():
    q, k = np.ones((2, 1, 4)), np.ones((3, 1, 4))
    o, _ = ob.chunk_attention(q, k, k, -1)      # row 0 stands at -1, row 1 at 0
    assert np.all(o[0] == 0) and np.all(o[1] == 1)
    o, _ = ob.chunk_attention(q, k, k, 1, have=np.zeros(3, bool))
    assert np.all(o == 0)


def test_probs():
    p = ob.probs(np.array([[0.0, np.log(3.0)], [-np.inf, 5.0], [-np.inf, -np.inf]]), 1.0)
    np.testing.assert_allclose(p, [[0.25, 0.75], [0, 1], [0, 0]], atol=1e-15)


def test_verify_by_hand():
    p = np.array([[0.5, 0.5, 0.0], [0.25, 0.25, 0.5], [1.0, 0.0, 0.0]], np.float32)
    q = np.array([[0.25, 0.25, 0.5], [0.75, 0.25, 0.0]], np.float32)
    # both accepted (p >= q; 0.3 * 0.75 < 0.25), then p[2]
    assert ob.verify_sample(p, q, [1, 0], [0.9, 0.3, 0.99])[0].tolist() == [1, 0, 0]
    # token 1 refused: the rest of p[1] - q[1] is all on token 2
    assert ob.verify_sample(p, q, [1, 0], [0.9, 0.4, 0.0])[0].tolist() == [1, 2, -1]
    # p(2) = 0 is never accepted, even at u = 0
    assert ob.verify_sample(p, q, [2, 0], [0.0, 0.4, 0.6])[0].tolist() == [1, -1, -1]
    # the draft ends: a sample of p[1]
    assert ob.verify_sample(p, q, [1, -1], [0.9, 0.4, 0.25])[0].tolist() == [1, 1, -1]
    # certain drafts: accepted with p, the rest without them
    assert ob.verify_sample(p, None, [0, 0], [0.6, 0.0, 0.0])[0].tolist() == [1, -1, -1]
    # equal rows, refused all the same (u = 1 is no number of [0, 1)): sample p
    assert ob.verify_sample(p[:2], p[:1], [0], [1.0, 0.75])[0].tolist() == [1, -1]
    assert ob.verify_sample(np.zeros((1, 3)), None, [], [0.5])[0].tolist() == [0]


@pytest.mark.parametrize("soft", [True, False])
def test_emitted_tokens_are_distributed_as_the_target(soft):
    """Chi-square of the first emitted token against p, whatever the draft."""
    rng = np.random.default_rng(3)
    v, runs = 6, 6000
    p = rng.dirichlet(np.ones(v), 2).astype(np.float32)
    q = rng.dirichlet(np.ones(v), 1).astype(np.float32)
    count = np.zeros(v)
    for _ in range(runs):
        x = rng.choice(v, p=q[0].astype(np.float64) / q[0].sum(dtype=np.float64)) if soft else 2
        t, _ = ob.verify_sample(p, q if soft else None, [x], rng.random(2).astype(np.float32))
        count[t[0]] += 1
    chi = ((count - runs * p[0]) ** 2 / (runs * p[0])).sum()
    assert chi < 25      # 5 degrees of freedom: 0.0001 above it
