"""The sums behind the scores of beams where every term is rounded alike."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("shape", [(1, 1, 1 << 20), (1, 2, (1 << 20) - 3), (8, 8, 152064), (1, 1, 152064), (4, 3, 5000)])
@pytest.mark.parametrize("temp", [0.3, 1.0, 1.7])
def test_one_large_logit_and_all_others_equal(shape, temp):
    """The others' exponent is common to all: a difference of logits, its product by log2(e) / T
    (2^-24 of it each) and an exponential (2^-22), before 2^20 at most of them are counted as whole
    numbers.  At 2^-21 of the largest and above that is below 2^-19 + 2^-22 of the sum; a CTA then
    adds its parts in 16 steps at most (2^-24 each): 2^-18 together."""
    import substitute_speculative_decoding_gb300 as sub
    b, n, v = shape
    t = float(np.float32(temp))
    for e in (1.0, math.log2(v) - 2, math.log2(v) - 0.7, math.log2(v), 16.37, 17.9, 19.99, 20.6):
        z = torch.full(shape, -3.1, device=DEV)
        at = torch.arange(b * n, device=DEV).view(b, n) * 77 % v
        z.scatter_(2, at[..., None], -3.1 + e * t * math.log(2))
        score = -torch.arange(b * n, dtype=torch.float32, device=DEV).view(b, n)
        token, parent, out = sub.beam_select(z, score, 2 * n if 2 * n <= 64 else n, temp)
        x = z.double() / t
        lse = x.logsumexp(-1)
        for i in range(b):
            j, s = parent[i].long(), token[i].long()
            assert (j >= 0).all()
            want = score[i, j].double() + x[i, j, s] - lse[i, j]
            assert ((out[i].double() - want).abs() <= 2.0 ** -18 + 2.0 ** -24 * want.abs()).all(), (e, i)
            assert (want.diff() <= 2.0 ** -17).all()
            assert (s[0] == at[i, j[0]]).all()
