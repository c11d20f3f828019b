"""Pins of the oracle of batched trees: closed forms and brute force."""
import itertools

import numpy as np
import pytest

from oracle import batch as ob
from oracle import model
from oracle import tree_batch as ot


def test_rotation_is_the_decoders():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 64))
    at = np.array([0, 1, 7, 100, 3])
    freqs = 1e4 ** (-2.0 * np.arange(32) / 64)
    y = ot.rotate(x, at, freqs)
    assert np.array_equal(y[0], x[0])
    z = (x[..., :32] + 1j * x[..., 32:]) * np.exp(1j * at[:, None, None] * freqs)
    assert np.allclose(y, np.concatenate([z.real, z.imag], -1), atol=1e-13)
    # turned alike, two rows' product depends on the difference of their positions alone
    a, b = ot.rotate(x[:1], [11], freqs), ot.rotate(x[1:2], [4], freqs)
    c, d = ot.rotate(x[:1], [1007], freqs), ot.rotate(x[1:2], [1000], freqs)
    assert np.allclose((a * b).sum(-1), (c * d).sum(-1), atol=1e-10)
    assert np.allclose(model.rope(x.astype(np.float32), at, 1e4), y, atol=1e-4)


def test_masks_hold_the_paths():
    parents = [-1, 0, 0, 1, 2, 3, 3] + list(range(6, 70))
    m = ot.path_masks(parents, 3).view(np.uint32)
    for s in range(len(parents)):
        path, p = set(), s
        while p >= 0:
            path.add(p)
            p = parents[p]
        assert path == {t for t in range(96) if m[s, t // 32] >> (t % 32) & 1}


def test_masked_attention_is_causal_attention_of_each_path():
    rng = np.random.default_rng(1)
    parents = [-1, 0, 0, 2, 1, 3]
    n, base = len(parents), 9
    q = rng.standard_normal((n, 4, 8))
    k, v = rng.standard_normal((base + n, 2, 8)), rng.standard_normal((base + n, 2, 8))
    see = ot.sees(n, base + n, base, base, ot.path_masks(parents, 1))
    o, w = ot.masked_attention(q, k, v, see, 0.3)
    for s in range(n):
        path, p = [], s
        while p >= 0:
            path.append(p)
            p = parents[p]
        at = list(range(base)) + [base + t for t in path[::-1]]
        ref, rw = ob.chunk_attention(q[s:s + 1], k[at], v[at], len(at) - 1, scale=0.3)
        assert np.allclose(o[s], ref[0], atol=1e-12) and np.allclose(w[s], rw[0], atol=1e-12)
    # a chain's mask is the causal one; past its words a mask reads nothing
    chain = ot.path_masks([-1] + list(range(n - 1)), 1)
    assert np.array_equal(ot.sees(n, base + n, base, base, chain), np.tri(n, base + n, base, dtype=bool))
    assert not ot.sees(2, 40, 39, 5, np.full((2, 1), -1, np.int32))[:, 37:].any()


@pytest.mark.parametrize("first", [False, True])
def test_beams_against_all_continuations(first):
    rng = np.random.default_rng(2)
    z = np.round(rng.standard_normal((3, 11)) * 2).astype(np.float32)      # many ties
    z[1, 4] = -np.inf
    s = np.array([-1.0, -0.5, -2.0])
    if first:
        s[1:] = -np.inf
    everything = []
    for j, x in itertools.product(range(3), range(11)):
        t = z[j].astype(np.float64) / 0.5
        everything.append((s[j] + t[x] - np.log(np.exp(t).sum()), j, x))
    everything = [e for e in everything if e[0] > -np.inf]
    everything.sort(key=lambda e: (-round(e[0], 9), e[1], e[2]))
    for k in (1, 4, 40):
        slot = 3 if k < 30 else -1
        token, parent, score, state, _ = ot.beam_select(z, s, k, 0.5, np.array([[1], [2], [4]], np.int32), slot)
        m = min(k, len(everything))
        assert list(zip(parent[:m], token[:m])) == [e[1:] for e in everything[:m]]
        assert np.allclose(score[:m], [e[0] for e in everything[:m]], atol=1e-9)
        assert (token[m:] == -1).all() and (parent[m:] == -1).all() and np.isneginf(score[m:]).all()
        if k < 30:
            want = [(1 << parent[r]) | (1 << (3 + r)) for r in range(m)]
            assert state[:m, 0].tolist() == want and not state[m:].any()


def test_moves_read_before_they_write():
    x = np.arange(10)
    assert ot.moved(x, 2, [5, 2, 3]).tolist() == [0, 1, 5, 2, 3, 5, 6, 7, 8, 9]
