"""Trees over an 8-bit cache with scales that are not finite, at keys that rows read, by each kernel."""
import numpy as np
import pytest
import torch

from test_gpu_batch import np32
from test_gpu_tree_batch import DEV, WIDTHS, TreeCase

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [2, 5, 8, 33, 260])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("committed", [False, True])
@pytest.mark.parametrize("width", WIDTHS)
def test_scales_of_keys_that_are_read(n, bad, side, committed, width):
    """A head whose row reads a key with a scale of V that is not finite is not finite; one with a scale
    of K that is not, unless the score is -infinity (that key's weight is 0).  All others stay as they were."""
    import substitute_speculative_decoding_gb300 as sub
    base, first = 300, 40
    c = TreeCase(sub, [(base, first, n), (20, 0, 2)], 8, 2, 128, bits=8, seed=3, width=width)
    clean = c.run().clone()
    hurt = [5, 17, 38, first + n - 2]
    keys = [base + s for s in hurt] + ([130] if committed else [])
    codes = [c.pools[0][c.layer, int(c.table[0, t // 16]), :, t % 16].cpu().numpy().astype(np.float64) - 128 for t in keys]
    for t in keys:
        c.scales[side][c.layer, int(c.table[0, t // 16]), :, t % 16] = bad
    o = c.run()
    see, q = c.see(0), np32(c.q[:n]).astype(np.float64)
    have = torch.isfinite(o[:n]).cpu().numpy()
    reads = see[:, keys].any(1)
    assert reads.any() and (committed or not reads.all())
    free = torch.from_numpy(~reads).to(DEV)
    assert torch.isfinite(o[n:]).all() and have[~reads].all()
    assert not (~reads).any() or (o[:n][free].float() - clean[:n][free].float()).abs().max() < 0.05
    assert (o[n:].float() - clean[n:].float()).abs().max() < 0.05
    for t, code in zip(keys, codes):
        for i in np.flatnonzero(see[:, t]):
            for h in range(8):
                dot = q[i, h] @ code[h // 4]
                # (a product of sums that all but cancel may have either sign: 2^-11 of each term)
                unsure = abs(dot) <= 2.0 ** -11 * (np.abs(q[i, h]) @ np.abs(code[h // 4]))
                if side == 0 and not np.isnan(bad) and (unsure or dot * bad < 0):
                    continue
                assert not have[i, h].any(), (i, h, t)
