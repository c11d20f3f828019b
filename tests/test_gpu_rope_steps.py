"""Rows turned by any frequencies to any positions, against angles reduced in rational arithmetic."""
import random

import numpy as np
import pytest
import torch

from test_gpu_batch import Case, np32
from test_gpu_tree_batch import rope_slack
from test_rope_steps import exact_step

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits_", [16, 8])
@pytest.mark.parametrize("top", [1.0, 100.0, 1e6])
def test_far_positions_of_any_frequency(d, bits_, top):
    import substitute_speculative_decoding_gb300 as sub
    rng = random.Random(int(top))
    freqs = [top, top * 0.9999997] + [top * 10.0 ** rng.uniform(-8, 0) for _ in range(d // 2 - 2)]
    c = Case(sub, [(3, 9), (40, 4)], 6, 2, d, bits=bits_)
    n = c.batch.n_rows
    at = [2 ** 31 - 1, -2 ** 31, 100000, 100003, 0, 1, -1, 2 ** 24 + 1, 2 ** 30 + 12345] + \
        [rng.randrange(-2 ** 31, 2 ** 31) for _ in range(n - 9)]
    x = torch.randn(n, 6, d, generator=torch.Generator().manual_seed(d)).to(BF)
    k = torch.randn(n, 2, d, generator=torch.Generator().manual_seed(1)).to(BF)
    q = sub.kv_append_rope(x.to(DEV), k.to(DEV), k.to(DEV), c.kv, c.layer, c.batch, sub.rope(d, freqs=freqs),
                           at=torch.tensor(at, dtype=torch.int32, device=DEV))
    # a position's angle in turns, whole ones dropped: exact_step is in units of 2^-64
    steps = [exact_step(f) for f in freqs]
    angle = np.array([[float(p * s / 2 ** 64 % 1) for s in steps] for p in at])[:, None] * 2 * np.pi

    def turned(y):
        a, b = np32(y).astype(np.float64)[..., :d // 2], np32(y).astype(np.float64)[..., d // 2:]
        return np.concatenate([a * np.cos(angle) - b * np.sin(angle), b * np.cos(angle) + a * np.sin(angle)], -1)
    # rope_slack: an angle known to 2^-33 of a turn; here to 2^-33 + 2^-34, far below its 2^-20
    ref = turned(x)
    assert np.all(np.abs(np32(q) - ref) <= 2.0 ** -8 * np.abs(ref) + rope_slack(np32(x), at, freqs))
    ref, slack = turned(k), rope_slack(np32(k), at, freqs)
    for b, (p, m) in enumerate(c.seqs):
        rows = slice(int(c.start[b]), int(c.start[b]) + m)
        t = torch.arange(p, p + m)
        pg, pl = c.table[b, t // c.page].long(), t % c.page
        got = c.pools[0][c.layer].cpu()[pg, :, pl]
        if bits_ == 16:
            assert np.all(np.abs(np32(got) - ref[rows]) <= 2.0 ** -8 * np.abs(ref[rows]) + slack[rows])
            continue
        s = c.scales[0][c.layer].cpu()[pg, :, pl].numpy()[..., None]
        a = np.abs(ref[rows]).max(-1, keepdims=True)
        err = np.abs((got.numpy().astype(np.float64) - 128) * s - ref[rows])
        # half a step, the row's own error, and the product's rounding before the code's
        assert np.all(err <= s * (0.5 + 2.0 ** -15) + slack[rows] + 2.0 ** -20 * a)
