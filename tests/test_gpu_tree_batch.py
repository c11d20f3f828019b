"""Batched trees on the GPU against the oracle: rotated rows, attention by masks, the
best continuations of beams, moved rows."""
import numpy as np
import pytest
import torch

from oracle import batch as ob
from oracle import tree_batch as ot
from test_gpu_batch import Case, np32

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def sub():
    import substitute_speculative_decoding_gb300 as s
    return s


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def bits(t):
    return t.contiguous().view(torch.uint8)


# ------------------------------------------------------------ rotated rows --
ROWS = [dict(seqs=[(5, 1)], hq=4, hkv=2, d=64),
        dict(seqs=[(0, 3), (17, 0), (30, 40), (15, 2)], hq=4, hkv=2, d=64, pad=3, before=2),
        dict(seqs=[(100, 1)] * 9, hq=40, hkv=8, d=128, page=64),
        dict(seqs=[(0, 70), (1, 1)], hq=7, hkv=1, d=128, page=48, pad=1),
        dict(seqs=[(3, 5), (0, 9)], hq=33, hkv=11, d=64, page=32),
        dict(seqs=[(70000, 6)], hq=2, hkv=2, d=128, page=128)]


def rope_slack(x, at, freqs):
    """Error of a turned pair beside its rounding: the angle in half turns is rounded to
    fp32 (2^-25, times pi) and known to 2^-33 of a turn, sincospi is off by 2 ulp (2^-22), and
    two products and a sum are rounded (2^-24 each): below 2^-20 of |x1| + |x2| together."""
    a = np.abs(np.asarray(x, np.float64))
    half = a.shape[-1] // 2
    s = a[..., :half] + a[..., half:]
    return 2.0 ** -20 * np.concatenate([s, s], -1)


@pytest.mark.parametrize("kw", ROWS)
@pytest.mark.parametrize("bits_", [16, 8])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("given", [False, True])
def test_rows_are_turned_on_their_way(sub, kw, bits_, fused, given):
    c = Case(sub, bits=bits_, **kw)
    n, d = c.batch.n_rows, c.d
    g = torch.Generator().manual_seed(7)
    qkv = torch.randn(n, c.hq + 2 * c.hkv, d, generator=g).to(BF)
    qkv[0, c.hq] = 0
    qkv[n // 2, -1] *= 2.0 ** -104
    qkv[n - 1, c.hq] *= 2.0 ** 100
    qkv = qkv.to(DEV)
    parts = [qkv[:, :c.hq], qkv[:, c.hq:c.hq + c.hkv], qkv[:, c.hq + c.hkv:]]
    q, k, v = parts if fused else [t.contiguous() for t in parts]
    theta = 1e4 if d == 64 else 5e5
    freqs = theta ** (-2.0 * np.arange(d // 2) / d)
    rope = sub.rope(d, theta)
    at = None
    if given:
        at = torch.randint(-2 ** 31, 2 ** 31, (n,), generator=g).to(torch.int32)
        at[0], at[n - 1] = 2 ** 31 - 1, 0
    pools = [t.clone() for t in c.pools]
    scales = [t.clone() for t in c.scales] if bits_ == 8 else []
    out = torch.full((n, c.hq, d), 7.0, dtype=BF, device=DEV)
    got = sub.kv_append_rope(q, k, v, c.kv, c.layer, c.batch, rope, q_out=out,
                             at=None if at is None else at.to(DEV))
    assert got is out
    lo, hi = int(c.start[0]), int(c.start[-1])
    assert torch.all(out[:lo] == 7) and torch.all(out[hi:] == 7)
    touched = torch.zeros(c.pools[0].shape[:4], dtype=torch.bool)
    for b, (p, m) in enumerate(c.seqs):
        if m == 0:
            continue
        rows = slice(int(c.start[b]), int(c.start[b]) + m)
        t = torch.arange(p, p + m)
        turn = t.numpy() if at is None else at[rows].numpy()
        pg, pl = c.table[b, t // c.page].long(), t % c.page
        touched[c.layer, pg, :, pl] = True
        x = np32(q[rows])
        ref = ot.rotate(x, turn, freqs)
        assert np.all(np.abs(np32(out[rows]) - ref) <= 2.0 ** -8 * np.abs(ref) + rope_slack(x, turn, freqs))
        kr, slack = ot.rotate(np32(k[rows]), turn, freqs), rope_slack(np32(k[rows]), turn, freqs)
        kc, vc = (pool[c.layer].cpu()[pg, :, pl] for pool in c.pools)
        if bits_ == 16:
            assert np.all(np.abs(np32(kc) - kr) <= 2.0 ** -8 * np.abs(kr) + slack)
            assert torch.equal(bits(vc), bits(v[rows].cpu()))
            continue
        ks, vs = (x[c.layer].cpu()[pg, :, pl].numpy() for x in c.scales)
        wc, ws = ob.kv8_quantise(np32(v[rows]))
        assert np.array_equal(vc.numpy(), wc) and np.array_equal(vs, ws)
        a = np.abs(kr).max(-1)
        none = a < 2.0 ** -101
        assert np.array_equal(ks[none], np.ones_like(ks[none])) and (kc.numpy()[none] == 128).all()
        wide = slack.max(-1)
        assert np.all(np.abs(ks.astype(np.float64) * 127 - a)[~none] <= (wide + 2.0 ** -23 * a)[~none])
        err = np.abs((kc.numpy().astype(np.float64) - 128) * ks[..., None] - kr)
        # half a step, the row's own error, and the product's rounding before the code's
        assert np.all((err <= ks[..., None] * (0.5 + 2.0 ** -15) + slack + 2.0 ** -20 * a[..., None])[~none])
    for pool, old in list(zip(c.pools, pools)) + list(zip(c.scales, scales) if bits_ == 8 else []):
        same = ~touched if pool.dim() == 4 else ~touched[..., None].expand_as(pool.cpu())
        assert torch.equal(bits(pool.cpu()[same]), bits(old.cpu()[same]))


@pytest.mark.parametrize("bits_", [16, 8])
def test_turned_in_place_and_without_q(sub, bits_):
    c = Case(sub, [(9, 5), (3, 2)], 8, 2, 64, bits=bits_, pad=2)
    n = c.batch.n_rows
    rope = sub.rope(64, 1e4)
    wide = torch.randn(n, 14, 64, device=DEV).to(BF)
    q, k, v = wide[:, :8], wide[:, 8:10], wide[:, 10:12]
    apart = sub.kv_append_rope(q, k, v, c.kv, c.layer, c.batch, rope)
    after = [t.clone() for t in c.pools]
    kept = wide.clone()
    assert torch.all(apart[7:] == 0)
    assert sub.kv_append_rope(q, k, v, c.kv, c.layer, c.batch, rope, q_out=q) is q
    assert torch.equal(q[:7], apart[:7]) and torch.equal(q[7:], kept[7:, :8])
    assert torch.equal(wide[:, 8:], kept[:, 8:])
    for pool, x in zip(c.pools, after):
        assert torch.equal(bits(pool), bits(x))
        pool.fill_(0)
    assert sub.kv_append_rope(None, k, v, c.kv, c.layer, c.batch, rope) is None
    for b, (p, m) in enumerate(c.seqs):
        t = torch.arange(p, p + m)
        pg, pl = c.table[b, t // 16].long().to(DEV), (t % 16).to(DEV)
        for pool, x in zip(c.pools, after):
            assert torch.equal(pool[c.layer, pg, :, pl], x[c.layer, pg, :, pl])


@pytest.mark.parametrize("bits_", [16, 8])
def test_turned_rows_without_a_place(sub, bits_):
    """Positions below 0, past the capacity, on a missing page: q is turned all the same,
    nothing is written; rows that are not finite."""
    c = Case(sub, [(0, 16), (0, 32)], 4, 2, 64, bits=bits_)
    c.table_d[1, 1] = -1
    c.table_d[0, 0] = 10 ** 6
    rope = sub.rope(64, 1e4)
    freqs = 1e4 ** (-2.0 * np.arange(32) / 64)
    for pos, n_rows in ((0, 4), (-6, 6), (40, 8)):
        x = torch.randn(n_rows, 4, 64, device=DEV).to(BF)
        before = [t.clone() for t in c.pools]
        b = sub.batch(ints([0, n_rows, n_rows]), ints([pos, 0]), n_rows)
        q = sub.kv_append_rope(x, x[:, :2], x[:, 2:], c.kv, c.layer, b, rope)
        at = pos + np.arange(n_rows)
        ref = ot.rotate(np32(x), at, freqs)
        assert np.all(np.abs(np32(q) - ref) <= 2.0 ** -8 * np.abs(ref) + rope_slack(np32(x), at, freqs))
        for pool, old in zip(c.pools, before):
            assert torch.equal(bits(pool), bits(old))
    x = torch.ones(2, 2, 64, dtype=BF, device=DEV)
    x[0, 0, 3], x[1, 1, 40] = float("inf"), float("nan")
    b = sub.batch(ints([0, 0, 2]), ints([0, 3]), 2)
    sub.kv_append_rope(None, x, x, c.kv, c.layer, b, rope)
    pg = int(c.table[1, 0])
    k = c.pools[0][c.layer, pg, :, 3:5].cpu()
    if bits_ == 8:
        s = c.scales[0][c.layer, pg, :, 3:5].cpu()
        assert torch.isnan(s[0, 0]) and torch.isnan(s[1, 1]) and torch.isfinite(s[[0, 1], [1, 0]]).all()
        assert (k[0, 0] == 128).all() and (k[1, 1] == 128).all()
    else:
        bad = (~torch.isfinite(k)).nonzero().tolist()
        assert bad == [[0, 0, 3], [0, 0, 35], [1, 1, 8], [1, 1, 40]]


# -------------------------------------------------------------- attention --
class TreeCase(Case):
    """The last rows of each sequence are nodes of a tree that begins at base: seqs
    (base, slots before the new rows, new rows)."""

    def __init__(self, sub, trees, hq, hkv, d, words=0, kind="tree", seed=0, **kw):
        super().__init__(sub, [(base + first, n) for base, first, n in trees], hq, hkv, d, seed=seed, **kw)
        rng = np.random.default_rng(seed)
        slots = max(first + n for _, first, n in trees)
        words = words or -(-slots // 32)
        self.trees, self.masks = trees, []
        for base, first, n in trees:
            if kind == "tree":
                parents = [-1] + [int(rng.integers(max(0, s - 9), s)) for s in range(1, first + n)]
                m = ot.path_masks(parents, max(words, -(-(first + n) // 32)))[first:first + n, :words]
            else:
                m = rng.integers(-2 ** 31, 2 ** 31, (n, words)).astype(np.int32)
                if kind == "none":
                    m[:] = 0
            self.masks.append(m.copy())
        self.base = ints([t[0] for t in trees])
        rows = self.batch.n_rows
        mask = np.full((rows, words), -1, np.int32)      # of rows of no sequence: anything
        for b, m in enumerate(self.masks):
            mask[int(self.start[b]):int(self.start[b]) + len(m)] = m
        self.mask = torch.from_numpy(mask).to(DEV)

    def see(self, b, base=None):
        p, n = self.seqs[b]
        return ot.sees(n, max(0, p + n), p, self.trees[b][0] if base is None else base, self.masks[b])

    def run(self, **kw):
        return self.sub.chunk_tree_attn(self.q.to(DEV), self.kv, self.layer, self.batch, self.base, self.mask, **kw)

    def check_tree(self, o, scale=None, see=None, only=None):
        """The bound of Case.check, over the keys that each row reads."""
        sc = self.d ** -0.5 if scale is None else scale
        for b, (p, n) in enumerate(self.seqs):
            if n == 0 or (only is not None and b not in only):
                continue
            r0 = int(self.start[b])
            q, k, v = np32(self.q[r0:r0 + n]), self.values(0, b), self.values(1, b)
            s = self.see(b) if see is None else see[b]
            ref, w = ot.masked_attention(q, k, v, s, sc)
            top = np.zeros((n, self.hq, 1))
            if len(k):
                big = np.repeat(np.where(np.isfinite(k), np.abs(k), 0).max(0), self.hq // self.hkv, 0)
                top = (np.abs(q) * big).sum(-1, keepdims=True) * sc
            c = (2.0 ** -8 if self.bits == 16 else 2.0 ** -11) + \
                2 * (self.d / 16 + 4) * 2.0 ** -22 * top + (len(k) / 16 + 4) * 2.0 ** -22
            if self.bits == 8 and self.batch.n_rows * self.hq > 64 * self.hkv * len(self.seqs):
                c = c + 2 * 2.0 ** -11 + 2 * 2.0 ** -11 * top
            err = np.abs(np32(o[r0:r0 + n]).astype(np.float64) - ref)
            bound = 2.0 ** -8 * np.abs(ref) + c * w + 1e-30
            if self.bits == 8 and len(v):
                bound = bound + len(k) * 2.0 ** -36 * np.abs(v[np.isfinite(v)]).max()
            assert np.all(err <= bound), (b, float((err / bound).max()))


# Further columns of the page table: with room for many keys, rows go to the kernels of long sequences,
# and units are cut
WIDTHS = [0, 30000]

TREES = [dict(trees=[(0, 0, 1)], hq=4, hkv=2, d=64),
         dict(trees=[(511, 9, 8)], hq=4, hkv=2, d=64),
         dict(trees=[(31, 0, 1), (32, 1, 1), (0, 3, 1), (60, 8, 1), (1000, 40, 1)], hq=28, hkv=4, d=128, page=64),
         dict(trees=[(300, 9, 8), (5, 0, 0), (40, 0, 3), (0, 2, 20)], hq=28, hkv=4, d=128, page=48, pad=5,
              before=3),
         dict(trees=[(700, 0, 2), (3, 4, 1), (129, 33, 1)], hq=16, hkv=8, d=128, page=16),
         dict(trees=[(0, 0, 130)], hq=8, hkv=8, d=64, page=32),
         dict(trees=[(77, 0, 300), (500, 400, 1), (0, 5, 257)], hq=8, hkv=2, d=128, page=64, pad=1),
         dict(trees=[(255, 0, 129)], hq=16, hkv=1, d=64, page=128),
         dict(trees=[(2500, 17, 8)], hq=56, hkv=8, d=128, page=16),
         dict(trees=[(600, 0, 33), (0, 0, 1), (90, 1, 64)], hq=6, hkv=2, d=64, page=48),
         dict(trees=[(b * 7, b % 5, 1 + b % 3) for b in range(70)], hq=4, hkv=2, d=64, page=16),
         dict(trees=[(4096, 0, 65), (130, 0, 65)], hq=40, hkv=8, d=128, page=64)]


@pytest.mark.parametrize("kw", TREES)
@pytest.mark.parametrize("bits_", [16, 8])
@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("width", WIDTHS)
def test_tree_attn(sub, kw, bits_, kind, width):
    c = TreeCase(sub, bits=bits_, kind=kind, seed=len(kw["trees"]) + bits_, width=width, **kw)
    o = torch.full((c.batch.n_rows, c.hq, c.d), 7.0, dtype=BF, device=DEV)
    c.run(out=o)
    c.check_tree(o)
    lo, hi = int(c.start[0]), int(c.start[-1])
    assert torch.all(o[:lo] == 7) and torch.all(o[hi:] == 7)
    again = c.run()
    assert torch.equal(again[lo:hi], o[lo:hi])          # the same call, the same bits
    assert torch.all(again[:lo] == 0) and torch.all(again[hi:] == 0)


@pytest.mark.parametrize("bits_", [16, 8])
@pytest.mark.parametrize("n", [1, 8, 40, 300])
@pytest.mark.parametrize("width", WIDTHS)
def test_many_ctas_and_wide_masks(sub, bits_, n, width):
    """Many CTAs on one sequence's keys beside short ones, masks of 64 words, and masks that
    end before the new rows' own slots."""
    c = TreeCase(sub, [(9000, 1700, n), (64, 0, n), (0, 31, n)], 4, 1, 128, page=64, bits=bits_, seed=n, words=64,
                 width=width)
    c.check_tree(c.run())
    c = TreeCase(sub, [(900, 60, n), (64, 0, n), (0, 0, n)], 4, 1, 128, page=64, bits=bits_, seed=n, words=1,
                 width=width)
    c.check_tree(c.run(scale=0.3), scale=0.3)


@pytest.mark.parametrize("bits_", [16, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 48, 64, 128])
@pytest.mark.parametrize("trees", [[(900, 9, 8), (0, 0, 8), (33, 1, 8)], [(129, 17, 7), (1500, 0, 9), (5, 0, 2)],
                                   [(700, 3, 16)], [(260, 0, 31), (90, 40, 20), (0, 0, 45)]])
def test_a_few_dozen_rows(sub, bits_, d, page, trees):
    """Rows of one tile or two of the kernel with the keys on the lanes (which wants room
    for more than 1024 of them), in boxes of all sizes."""
    c = TreeCase(sub, trees, 8, 2, d, page=page, bits=bits_, kind="any", seed=page + d, width=70)
    c.table_d[0, 2] = -1
    see = [c.see(b) for b in range(len(trees))]
    see[0][:, 2 * page:3 * page] = False
    c.check_tree(c.run(), see=see)


@pytest.mark.parametrize("bits_", [16, 8])
@pytest.mark.parametrize("n", [2, 8, 60])
@pytest.mark.parametrize("width", WIDTHS)
def test_a_path_of_all_is_chunk_attention(sub, bits_, n, width):
    """Masks with all bits, and a base behind all keys."""
    c = TreeCase(sub, [(300, 5, n), (40, 0, n), (0, 0, n)], 8, 2, 128, page=48, bits=bits_, seed=4,
                 width=width)
    c.check(sub.chunk_attn(c.q.to(DEV), c.kv, c.layer, c.batch))
    c.mask.fill_(-1)
    c.check(c.run())
    c.mask.zero_()
    for far in (2 ** 31 - 1, 300 + 5 + n):
        c.base.fill_(far)
        c.check(c.run())


@pytest.mark.parametrize("bits_", [16, 8])
@pytest.mark.parametrize("n", [1, 4, 8, 150])
@pytest.mark.parametrize("width", WIDTHS)
def test_rows_that_read_nothing(sub, bits_, n, width):
    c = TreeCase(sub, [(0, 3, n), (50, 0, n), (0, 0, n)], 8, 2, 128, bits=bits_, kind="none", width=width)
    o = c.run()
    c.check_tree(o)
    assert torch.all(o[:n] == 0) and torch.all(o[2 * n:] == 0) and torch.isfinite(o).all()
    # far below any slot: every key lies behind the mask's words
    c.mask.fill_(-1)
    for low in (-2 ** 31, -4096, -64 * 32):
        c.base.fill_(low)
        assert torch.all(c.run() == 0)
    c.base.fill_(-5)
    see = []
    for b, (p, m) in enumerate(c.seqs):
        c.masks[b] = np.full_like(c.masks[b], -1)
        see.append(c.see(b, base=-5))
    c.check_tree(c.run(), see=see)


@pytest.mark.parametrize("bits_", [16, 8])
@pytest.mark.parametrize("n", [3, 8, 150])
@pytest.mark.parametrize("width", WIDTHS)
def test_missing_pages_under_a_tree(sub, bits_, n, width):
    c = TreeCase(sub, [(200, 9, n), (64, 0, n)], 8, 2, 128, bits=bits_, seed=2, width=width)
    c.table_d[0, 3] = -1
    c.table_d[0, 13] = c.kv.n_pages           # slots 8 .. 23
    c.table_d[1] = -7
    see = [c.see(0), np.zeros_like(c.see(1))]
    see[0][:, 48:64] = see[0][:, 208:224] = False
    c.check_tree(c.run(), see=see)


@pytest.mark.parametrize("bits_", [16, 8])
@pytest.mark.parametrize("n", [2, 8, 33, 260])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("width", WIDTHS)
def test_slots_that_a_row_does_not_read_hold_anything(sub, bits_, n, bad, width):
    """Infinities and NaN in K, V (codes: in their scales) of slots off a row's path."""
    base, first = 45, 40
    c = TreeCase(sub, [(base, first, n), (20, 0, 2)], 8, 2, 128, bits=bits_, seed=3, width=width)
    clean = c.run().clone()
    hurt = np.zeros(first + n, bool)
    hurt[[5, 17, 38, first + n - 2]] = True
    for s in np.flatnonzero(hurt):
        t = base + s
        pg, pl = int(c.table[0, t // 16]), t % 16
        for j in range(2):
            if bits_ == 16:
                c.pools[j][c.layer, pg, :, pl, (3 * s) % 128] = bad
            else:
                c.scales[j][c.layer, pg, :, pl] = bad
    o = c.run()
    see = c.see(0)[:, base:]
    reads = (see & hurt[None]).any(1)
    assert reads.any() and not reads.all()
    free = torch.from_numpy(~reads).to(DEV)
    assert torch.isfinite(o[:n][free]).all() and torch.isfinite(o[n:]).all()
    # as before, up to the weights' rounding
    assert (o[:n][free].float() - clean[:n][free].float()).abs().max() < 0.05
    assert (o[n:].float() - clean[n:].float()).abs().max() < 0.05
    # a head that reads one is not finite, unless its score is -infinity: that key's weight is 0
    hit = torch.from_numpy(reads).to(DEV)
    if bits_ == 8:
        assert bad == bad or not torch.isfinite(o[:n][hit]).any()
        return
    have, q = torch.isfinite(o[:n]).cpu().numpy(), np32(c.q[:n])
    for s in np.flatnonzero(hurt):
        x = (3 * s) % 128
        for i in np.flatnonzero(see[:, s]):
            for h in range(8):
                if not q[i, h, x] * bad == -np.inf:
                    assert not have[i, h, x], (i, h, s)


@pytest.mark.parametrize("width", WIDTHS)
def test_strides_streams_workspaces_and_graphs(sub, width):
    """Strided queries; a call on another stream with a given workspace; a captured call
    replayed with other masks, bases and queries."""
    for bits_, n in ((16, 3), (8, 3), (16, 70), (8, 70)):
        c = TreeCase(sub, [(90, 4, n), (13, 0, n)], 8, 2, 64, page=32, bits=bits_, seed=1, width=width)
        wide = torch.randn(c.batch.n_rows, 12, 64, device=DEV).to(BF)
        wide[:, :8] = c.q.to(DEV)
        ws = torch.empty(sub.chunk_attn_workspace(8, 2, 64, 2, c.batch.n_rows), dtype=torch.uint8, device=DEV)
        o = torch.zeros(c.batch.n_rows, 8, 64, dtype=BF, device=DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        sub.chunk_tree_attn(wide[:, :8], c.kv, c.layer, c.batch, c.base, c.mask, out=o, workspace=ws, stream=side)
        side.synchronize()
        c.check_tree(o)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sub.chunk_tree_attn(wide[:, :8], c.kv, c.layer, c.batch, c.base, c.mask, out=o, workspace=ws)
        other = TreeCase(sub, [(90, 4, n), (13, 0, n)], 8, 2, 64, page=32, bits=bits_, kind="any", seed=1,
                         width=width)
        c.mask.copy_(other.mask)
        c.masks = other.masks
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        c.check_tree(o)


def test_workspaces_of_the_calls_own(sub):
    """Without a workspace: on another stream beside work of this one, and in two captured
    graphs of one memory pool, replayed in turn; chunk_attn and beam_select alike."""
    cases = [TreeCase(sub, [(3000, 4, n), (13, 0, n)], 8, 2, 64, page=32, bits=bits_, seed=n, width=width)
             for bits_, n, width in ((16, 3, 0), (8, 3, 9000), (16, 8, 0), (8, 20, 0), (16, 70, 9000), (8, 70, 9000))]
    z = torch.randn(3, 5, 4000, device=DEV)
    score = -torch.rand(3, 5, device=DEV).cumsum(1)
    want = [c.run() for c in cases]
    causal = [sub.chunk_attn(c.q.to(DEV), c.kv, c.layer, c.batch) for c in cases]
    best = sub.beam_select(z, score, 4)
    qs = [c.q.to(DEV) for c in cases]

    def all_(stream=None):
        return ([sub.chunk_tree_attn(q, c.kv, c.layer, c.batch, c.base, c.mask, stream=stream)
                 for c, q in zip(cases, qs)],
                [sub.chunk_attn(q, c.kv, c.layer, c.batch, stream=stream) for c, q in zip(cases, qs)],
                sub.beam_select(z, score, 4, stream=stream))

    def same(got):
        for x, y in zip(got[0] + got[1] + list(got[2]), want + causal + list(best)):
            assert torch.equal(x, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there, here = all_(side), all_()
    torch.cuda.synchronize()
    same(there)
    same(here)
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        a = all_()
    with torch.cuda.graph(second, pool=first.pool()):
        b = all_()
    for g, got in ((first, a), (second, b), (second, b), (first, a)):
        g.replay()
        torch.cuda.synchronize()
        same(got)


# ------------------------------------------------------------------ beams --
def beams(sub, z, score, k, temp=1.0, state=None, slot=-1, **kw):
    """Compare a call with the oracle; returns its outputs."""
    got = sub.beam_select(z, score, k, temp, state=state, slot=slot, **kw)
    for b in range(z.shape[0]):
        token, parent, out, new, gap = ot.beam_select(
            z[b].cpu().numpy(), score[b].cpu().numpy(), k, temp, None if state is None else state[b].cpu().numpy(),
            slot)
        pairs = list(zip(got[1][b].tolist(), got[0][b].tolist()))
        if gap == 0 or gap > 1e-5:
            assert pairs == list(zip(parent.tolist(), token.tolist()))
        else:
            # beams that meet within the error of their sums (below) may change places there:
            # each chosen pair still has the score of its place, and beams keep their order
            assert len(set(pairs)) == k and (token >= 0).all()
            for j in range(z.shape[1]):
                mine, ref = ([t for i, t in x if i == j] for x in (pairs, zip(parent.tolist(), token.tolist())))
                assert mine[:len(ref)] == ref[:len(mine)]
            x = z[b].double().cpu().numpy() / float(np.float32(temp))
            lse = x.max(-1) + np.log(np.exp(x - x.max(-1, keepdims=True)).sum(-1))
            have = [score[b, j].item() + x[j, t] - lse[j] for j, t in pairs]
            assert np.all(np.abs(np.array(have) - out) <= 2.0 ** -18)
        have, fine = got[2][b].cpu().numpy().astype(np.float64), np.isfinite(out)
        assert np.array_equal(np.isneginf(have), ~fine)
        # the score's own rounding; sums of exp: terms of 2^-22, sums of at most 2^13 terms in
        # fp32, two factors per merge of partial sums: below 2^-9 of a unit even if all point one way,
        # 2^-19 as they come; the fp32 logit's product by 1 / T rounded to 2^-24 of it
        big = np.abs(np.nan_to_num(z[b].cpu().numpy(), posinf=0, neginf=0)).max() / temp
        have, out = have[fine], out[fine]
        assert np.all(np.abs(have - out) <= 2.0 ** -24 * np.abs(out) + 2.0 ** -19 + 2.0 ** -22 * big)
        if state is not None:
            assert np.array_equal(got[3][b].cpu().numpy(), new)
    return got


@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 1, 7), (3, 2, 33), (2, 5, 128), (2, 8, 1000), (5, 3, 5001),
                                   (1, 8, 20011), (2, 64, 513), (1, 16, 65537), (3, 13, 700), (2, 31, 5000), (2, 1, 152064), (3, 3, 50003)])
@pytest.mark.parametrize("k", [1, 3, 8, 64])
@pytest.mark.parametrize("temp", [0.2, 1.0])
def test_beam_select(sub, shape, k, temp):
    b, n, v = shape
    g = torch.Generator().manual_seed(sum(shape) + k)
    z = (2.5 * torch.randn(b, n, v, generator=g)).to(DEV)
    score = (-3 * torch.rand(b, n, generator=g).cumsum(1)).to(DEV)
    state = torch.randint(-2 ** 31, 2 ** 31, (b, n, 3), generator=g).to(torch.int32).to(DEV)
    beams(sub, z, score, k, temp, state, 96 - k)
    beams(sub, z, score, k, temp)


@pytest.mark.parametrize("off", [0, 1, 2, 3])
def test_beams_at_any_address(sub, off):
    z = torch.empty(2 * 3 * 4099 + 8, device=DEV).normal_()[off:off + 2 * 3 * 4099].view(2, 3, 4099)
    z[0, 0, 0] = z[1, 2, 4098] = 9.0
    score = torch.empty(9, device=DEV).uniform_(-1, 0)[off:off + 6].view(2, 3)
    beams(sub, z, score, 5, 0.7)


def test_equal_logits_go_by_token_and_beam(sub):
    v = 6000
    g = torch.Generator().manual_seed(0)
    z = torch.randint(-3, 4, (2, 4, v), generator=g).float().to(DEV)
    z[0, 1] = z[0, 2]                       # beams alike in all
    z[1, :] = 0.0
    z[1, 0, ::2] = -0.0                     # -0 is 0
    score = torch.tensor([[-1.0, -0.5, -0.5, -2.0], [-1.0, -1.0, -3.0, -1.0]], device=DEV)
    for k in (1, 8, 64):
        beams(sub, z, score, k, 0.5)
    for run in (torch.arange(v).float(), -torch.arange(v).float()):        # rising, falling
        z[:] = run.to(DEV) / 100
        beams(sub, z, score * torch.tensor([1.0, 1.1, 1.3, 1.7], device=DEV), 64, 2.0)
    z[:] = 1.5                              # one value throughout
    beams(sub, z, score, 64, 1.0)


def test_beams_and_logits_that_are_none(sub):
    inf, nan = float("inf"), float("nan")
    z = torch.randn(6, 3, 300, device=DEV)
    score = torch.empty(6, 3, device=DEV).uniform_(-1, 0)
    score[0, 1:] = -inf                     # a first step
    score[1] = -inf                         # a sequence without beams
    z[1] = nan                              # whose logits are not looked at
    score[2, 0], score[2, 1] = nan, inf
    z[3, :, ::3] = -inf
    z[3, 1, 1::3] = nan                     # no logits
    z[4, 0] = -inf
    z[4, 1, 7] = inf
    z[5, :, 2:] = -inf                      # fewer than asked for
    state = torch.randint(0, 99, (6, 3, 2), dtype=torch.int32, device=DEV)
    for k in (1, 7, 40):
        got = beams(sub, z, score, k, 0.9, state, 0)
        assert (got[0][1] == -1).all() and (got[3][1] == 0).all()
    z = torch.full((1, 2, 5), -3.0e38, device=DEV)
    z[0, 0, 3] = 3.0e38
    got = sub.beam_select(z, torch.zeros(1, 2, device=DEV), 3, 1.0)
    assert got[0][0].tolist() == [3, 0, 1] and got[1][0].tolist() == [0, 1, 1]


def test_the_longest_rows_and_most_beams(sub):
    z = 2 * torch.randn(1, 2, 1 << 20, device=DEV)
    beams(sub, z, torch.tensor([[-0.3, -0.1]], device=DEV), 64, 1.0)
    z = torch.randn(3, 64, 999, device=DEV)
    beams(sub, z, -torch.rand(3, 64, device=DEV).cumsum(1) * 0.05, 64, 0.6)


def test_beams_on_a_stream_and_in_a_graph(sub):
    z = torch.randn(4, 6, 3000, device=DEV)
    score = -torch.rand(4, 6, device=DEV).cumsum(1)
    state = torch.zeros(4, 6, 2, dtype=torch.int32, device=DEV)
    ws = torch.empty(sub.beam_workspace(4, 6, 3000), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = sub.beam_select(z, score, 6, 0.8, state=state, slot=6, workspace=ws, stream=side)
    side.synchronize()
    for x, y in zip(out, beams(sub, z, score, 6, 0.8, state, 6)):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sub.beam_select(z, score, 6, 0.8, state=state, slot=6, out=out, workspace=ws)
    z.normal_()
    state.random_(0, 64)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(out, beams(sub, z, score, 6, 0.8, state, 6)):
        assert torch.equal(x, y)


# ------------------------------------------------------------- moved rows --
@pytest.mark.parametrize("bits_", [16, 8])
@pytest.mark.parametrize("d,hkv,most", [(64, 2, 4), (128, 4, 12), (64, 11, 33), (128, 3, 128), (64, 1, 128)])
def test_moved_rows(sub, bits_, d, hkv, most):
    """Sources and destinations overlap in any order; some rows lie on no page."""
    seqs = [(300, 0), (140, 3), (40, 0), (0, 5), (600, 1)]
    c = Case(sub, seqs, hkv, hkv, d, page=48, bits=bits_, layers=3, seed=most)
    g = torch.Generator().manual_seed(most)
    for t in c.pools:       # all layers
        t.copy_(torch.randint(0, 255, bits(t).shape, generator=g, dtype=torch.uint8).to(DEV).view(t.dtype).view(t.shape))
    for t in c.scales if bits_ == 8 else ():
        t.copy_(torch.randn(t.shape, generator=g).to(DEV))
    c.table_d[4, 2] = -1                                    # positions 96 .. 143
    to = [7, 3, -2, 1, 90]
    count = [most, most + 9, 5, -3, min(most, 60)]
    src = torch.zeros(5, most, dtype=torch.int64)
    for b, (p, n) in enumerate(seqs):
        src[b] = torch.randint(-3, max(1, p + n + 9), (most,), generator=g)
    src[0, :min(3, most)] = torch.tensor([7 + most, 8, 9])[:min(3, most)]      # a later row's place
    pools = list(c.pools) + (list(c.scales) if bits_ == 8 else [])
    want = [t.clone() for t in pools]
    table = c.table_d.cpu()
    for b in range(5):
        def place(t):
            if t < 0 or t >= c.kv.capacity:
                return None
            page = int(table[b, t // 48])
            return (page, t % 48) if 0 <= page < c.kv.n_pages else None
        for i in range(max(0, min(count[b], most))):
            x, y = place(int(src[b, i])), place(to[b] + i)
            if x and y:
                for new, old in zip(want, pools):
                    new[:, y[0], :, y[1]] = old[:, x[0], :, x[1]]
    sub.kv_move(c.kv, ints(to), src.to(torch.int32).to(DEV), ints(count))
    for got, new in zip(pools, want):
        assert torch.equal(bits(got), bits(new))


# ------------------------------------------------------ a step of them all --
@pytest.mark.parametrize("bits_", [16, 8])
def test_a_decode_step_with_trees(sub, bits_):
    """One layer's worth of a decoder for a batch of three sequences: prompts enter the cache,
    trees are drafted level by level, verified in one pass, and the accepted paths committed.
    The verified rows equal attention over each node's own path, and after the commit a next
    row reads what a cache filled token by token would hold."""
    torch.manual_seed(0)
    hq, hkv, d, page, vocab, width, depth = 8, 2, 64, 16, 500, 4, 3
    n_seqs, prompt = 3, [37, 5, 80]
    rope, freqs = sub.rope(d, 1e4), 1e4 ** (-2.0 * np.arange(32) / 64)
    emb = torch.randn(vocab, (hq + 2 * hkv) * d, device=DEV).to(BF)     # a token's q, k, v
    head = torch.randn(hq * d, vocab, device=DEV) * 0.05
    pages = torch.randperm(n_seqs * 8, device=DEV).to(torch.int32).view(n_seqs, 8)
    if bits_ == 16:
        pools = [torch.full((1, n_seqs * 8, hkv, page, d), float("nan"), dtype=BF, device=DEV) for _ in range(2)]
        kv = sub.paged_kv(*pools, pages)
    else:
        pools = [torch.zeros((1, n_seqs * 8, hkv, page, d), dtype=torch.uint8, device=DEV) for _ in range(2)]
        scales = [torch.full((1, n_seqs * 8, hkv, page), float("nan"), device=DEV) for _ in range(2)]
        kv = sub.paged_kv8(*pools, *scales, pages)

    def rows(tokens):
        x = emb[tokens.long()].view(-1, hq + 2 * hkv, d)
        return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    text = [torch.randint(0, vocab, (n,), device=DEV) for n in prompt]
    start = ints([0] + list(np.cumsum(prompt)))
    b0 = sub.batch(start, ints([0] * n_seqs), sum(prompt))
    q, k, v = rows(torch.cat(text))
    sub.kv_append_rope(q, k, v, kv, 0, b0, rope)
    base = ints(prompt)
    # ---- the trees: slot 0 is a first token, then levels of four
    root = torch.randint(0, vocab, (n_seqs, 1), device=DEV, dtype=torch.int32)
    token, parent = [root], [torch.full_like(root, -1)]
    words = 1
    state = torch.ones(n_seqs, 1, words, dtype=torch.int32, device=DEV)
    score = torch.zeros(n_seqs, 1, device=DEV)
    masks, first = [state], 0
    for level in range(depth + 1):
        n = token[-1].shape[1]
        batch = sub.batch(ints([i * n for i in range(n_seqs + 1)]), base + first, n_seqs * n)
        q, k, v = rows(token[-1].reshape(-1))
        at = (base + level).repeat_interleave(n)
        q = sub.kv_append_rope(q, k, v, kv, 0, batch, rope, at=at)
        o = sub.chunk_tree_attn(q, kv, 0, batch, base, state.reshape(n_seqs * n, words))
        if level == depth:
            break
        logits = (o.reshape(n_seqs, n, -1).float() @ head).contiguous()
        before = first
        first += n
        t, p, score, state = sub.beam_select(logits, score, width, 0.5, state=state, slot=first)
        token.append(t)
        parent.append(p + before)
        masks.append(state)
    token, parent, mask = torch.cat(token, 1), torch.cat(parent, 1).cpu().numpy(), torch.cat(masks, 1)
    slots = token.shape[1]
    for b in range(n_seqs):
        assert np.array_equal(mask[b].cpu().numpy(), ot.path_masks(parent[b], words))
    # ---- verified in one pass: all nodes written and attended together
    depth_of = np.array([[sum(1 for _ in _path(parent[b], s)) - 1 for s in range(slots)] for b in range(n_seqs)])
    batch = sub.batch(ints([i * slots for i in range(n_seqs + 1)]), base, n_seqs * slots)
    q, k, v = rows(token.reshape(-1))
    at = (base[:, None] + ints(depth_of)).reshape(-1)
    q_out = sub.kv_append_rope(q, k, v, kv, 0, batch, rope, at=at)
    o = sub.chunk_tree_attn(q_out, kv, 0, batch, base, mask.reshape(-1, words))
    for b in range(n_seqs):
        for s in range(slots):
            path = list(_path(parent[b], s))[::-1]
            seq = torch.cat([text[b], token[b][path].long()])
            q, k, v = (np32(x) for x in rows(seq))
            pos = np.arange(len(seq))
            k = ot.rotate(k, pos, freqs)
            qr = ot.rotate(q, pos, freqs)[-1:]
            ref, w = ob.chunk_attention(qr, k, v, len(seq) - 1)
            # K and q rounded once to bf16 (2^-8) or to steps of 1 / 254 of their largest value,
            # V alike: every score moves by at most that of sum |q||k|, the result by twice its
            # exponential on the weights' mean of |v|, and by the weights' and its own rounding
            step = 2.0 ** -8 if bits_ == 16 else 1 / 254
            top = (np.abs(qr[0]) * np.repeat(np.abs(k).max(0), hq // hkv, 0)).sum(-1).max() * d ** -0.5
            vmax = np.abs(v).max()
            move = 2 * np.expm1(2 * (2.0 ** -8 + step) * top)
            bound = 2.0 ** -7 * np.abs(ref) + move * w + step * vmax
            err = np.abs(np32(o[b * slots + s]) - ref[0])
            assert np.all(err <= bound[0]), (b, s, float((err / bound[0]).max()))
            assert np.sqrt((err ** 2).mean()) <= 0.02 * np.sqrt((ref ** 2).mean()) + step * vmax
    # ---- the longest paths are accepted: their rows move behind the root's
    deep = slots - 1 - np.arange(n_seqs)
    paths = [list(_path(parent[b], deep[b]))[::-1][1:] for b in range(n_seqs)]
    src = torch.zeros(n_seqs, depth + 2, dtype=torch.int32)
    for b, p in enumerate(paths):
        src[b, :len(p)] = torch.tensor(p) + prompt[b]
    sub.kv_move(kv, base + 1, src.to(DEV), ints([len(p) for p in paths]))
    base += ints([1 + len(p) for p in paths])
    nxt = torch.randint(0, vocab, (n_seqs,), device=DEV)
    batch = sub.batch(ints(list(range(n_seqs + 1))), base, n_seqs)
    q, k, v = rows(nxt)
    q = sub.kv_append_rope(q, k, v, kv, 0, batch, rope)
    o = sub.chunk_attn(q, kv, 0, batch)
    # the same text in a cache of its own, row by row in order
    for t in pools:
        t.zero_()
    texts = [torch.cat([text[b], token[b][[0] + paths[b]].long(), nxt[b:b + 1]]) for b in range(n_seqs)]
    start = ints([0] + list(np.cumsum([len(t) for t in texts])))
    b1 = sub.batch(start, ints([0] * n_seqs), int(start[-1]))
    q, k, v = rows(torch.cat(texts))
    q = sub.kv_append_rope(q, k, v, kv, 0, b1, rope)
    last = (start[1:] - 1).long()
    again = sub.chunk_attn(q[last].contiguous(), kv, 0, batch)
    assert torch.equal(o, again)


def _path(parent, s):
    while s >= 0:
        yield int(s)
        s = parent[s]


@pytest.mark.parametrize("n", [4, 90, 300])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_scales_of_later_keys_do_not_reach_earlier_rows(sub, n, bad):
    """Causal attention over codes: whatever the scales of keys behind a row hold."""
    c = Case(sub, [(45, n), (20, 2)], 8, 2, 128, bits=8, seed=3)
    clean = sub.chunk_attn(c.q.to(DEV), c.kv, c.layer, c.batch).clone()
    at = 45 + n - 2
    for x in c.scales:
        x[c.layer, int(c.table[0, at // 16]), :, at % 16] = bad
    o = sub.chunk_attn(c.q.to(DEV), c.kv, c.layer, c.batch)
    rows = torch.cat([o[:n - 2], o[n:]])
    assert torch.isfinite(rows).all()
    assert (rows.float() - torch.cat([clean[:n - 2], clean[n:]]).float()).abs().max() < 0.05
