"""Batched serving operators on the GPU against the oracle: cache rows bit for
bit, attention and probabilities within derived bounds, sampled tokens exactly."""
import numpy as np
import pytest
import torch

from oracle import batch as ob

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def sub():
    import substitute_speculative_decoding_gb300 as s
    return s


def np32(t):
    return t.detach().float().cpu().numpy()


class Case:
    """Sequences of (position of the first new row, new rows) over one pool,
    pages in random order.  Everything that no sequence owns holds NaN."""

    def __init__(self, sub, seqs, hq, hkv, d, page=16, bits=16, layers=2, layer=1, pad=0, seed=0,
                 width=0, qscale=1.5, max_keys=0, before=0):
        g = torch.Generator().manual_seed(seed)
        self.sub, self.seqs, self.layer, self.bits = sub, seqs, layer, bits
        self.hq, self.hkv, self.d, self.page = hq, hkv, d, page
        keys = [max(0, p + n) for p, n in seqs]
        need = [-(-k // page) for k in keys]
        n_pages, self.width = sum(need) + 2, max(need + [1]) + width
        order = torch.randperm(n_pages, generator=g).tolist()
        self.table = torch.full((len(seqs), self.width), -1, dtype=torch.int32)
        for b, m in enumerate(need):
            for j in range(m):
                self.table[b, j] = order.pop()
        # values by sequence, exact bf16
        def rnd(*shape):
            return torch.randn(*shape, generator=g)
        self.k = [(rnd(n, hkv, d) * torch.exp(0.5 * rnd(1, hkv, d))).to(BF) for n in keys]
        self.v = [rnd(n, hkv, d).to(BF) for n in keys]
        self.before, total = before, before + sum(n for _, n in seqs)
        self.q = (rnd(total + pad, hq, d) * qscale).to(BF)
        self.start = torch.tensor([before] + [n for _, n in seqs]).cumsum(0).to(torch.int32)
        self.pos = torch.tensor([p for p, _ in seqs], dtype=torch.int32)
        shape = (layers, n_pages, hkv, page, d)
        if bits == 16:
            self.pools = [torch.full(shape, float("nan"), dtype=BF) for _ in range(2)]
        else:
            self.pools = [torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)
                          for _ in range(2)]
            self.scales = [torch.full(shape[:4], float("nan")) for _ in range(2)]
            self.codes = [[ob.kv8_quantise(np32(x)) for x in side] for side in (self.k, self.v)]
        for b, n in enumerate(keys):
            t = torch.arange(n)
            pg, at = self.table[b, t // page].long(), t % page
            for j, side in enumerate((self.k, self.v)):
                if bits == 16:
                    self.pools[j][layer, pg, :, at] = side[b]
                else:
                    c, s = self.codes[j][b]
                    self.pools[j][layer, pg, :, at] = torch.from_numpy(c)
                    self.scales[j][layer, pg, :, at] = torch.from_numpy(s)
        self.pools = [t.to(DEV) for t in self.pools]
        self.table_d = self.table.to(DEV)
        if bits == 16:
            self.kv = sub.paged_kv(*self.pools, self.table_d)
        else:
            self.scales = [t.to(DEV) for t in self.scales]
            self.kv = sub.paged_kv8(*self.pools, *self.scales, self.table_d)
        self.batch = sub.batch(self.start.to(DEV), self.pos.to(DEV), total + pad, max_keys)

    def values(self, j, b):
        side = (self.k, self.v)[j][b]
        return np32(side) if self.bits == 16 else ob.kv8_values(*self.codes[j][b])

    def check(self, o, have=None, scale=None, only=None):
        """Bound: half a step of the bf16 result, plus the weights' errors on the
        weights' mean of |v|.  A weight is rounded once to bf16 (half a step 2^-8;
        a bf16 cache) or fp16 (2^-11; codes), its exponent carries the error of a
        score: at most D/16 + 4 roundings of 2^-22 of sum |q_d k_d| * scale (the
        tensor core truncates), twice (sum and product), and its products are
        summed with one rounding of 2^-22 per 16 keys.  The largest fp16 weight times
        scale is at least 2^11, so one that falls below fp16's normal numbers is off by at
        most half of 2^-24, 2^-36 of the largest: per key, 2^-36 of the largest |v|
        (which matters in a column where the largest weights meet codes 128).
        Tiles of many rows (more than 64 per sequence and KV head) round the values of
        codes to fp16, too (2^-11): V's scale and V's value, K in every term of a score,
        and with 2^-25 of the block's largest scale where that is below fp16's normal
        numbers."""
        sc = self.d ** -0.5 if scale is None else scale
        for b, (p, n) in enumerate(self.seqs):
            if n == 0 or (only is not None and b not in only):
                continue
            r0 = int(self.start[b])
            q = np32(self.q[r0:r0 + n])
            k, v = self.values(0, b), self.values(1, b)
            hv = None if have is None else have[b]
            ref, w = ob.chunk_attention(q, k, v, p, have=hv, scale=sc)
            top = np.zeros((n, self.hq, 1))
            if len(k):
                fine = np.where(np.isfinite(k), np.abs(k), 0)
                big = np.repeat(fine.max(0), self.hq // self.hkv, 0)
                top = (np.abs(q) * big).sum(-1, keepdims=True) * sc
            c = (2.0 ** -8 if self.bits == 16 else 2.0 ** -11) + \
                2 * (self.d / 16 + 4) * 2.0 ** -22 * top + (len(k) / 16 + 4) * 2.0 ** -22
            if self.bits == 8 and self.batch.n_rows * self.hq > 64 * self.hkv * len(self.seqs):
                c = c + 2 * 2.0 ** -11 + 2 * 2.0 ** -11 * top
            err = np.abs(np32(o[r0:r0 + n]).astype(np.float64) - ref)
            bound = 2.0 ** -8 * np.abs(ref) + c * w + 1e-30
            if self.bits == 8 and len(v):
                bound = bound + len(k) * 2.0 ** -36 * np.abs(v).max()
            assert np.all(err <= bound), (b, float((err / bound).max()))


# ------------------------------------------------------------- cache rows --
ROWS = [dict(seqs=[(5, 1)], hq=4, hkv=2, d=64),
        dict(seqs=[(0, 3), (17, 0), (30, 40), (15, 2)], hq=4, hkv=2, d=64, pad=3, before=2),
        dict(seqs=[(100, 1)] * 9, hq=40, hkv=8, d=128, page=64),
        dict(seqs=[(0, 70), (1, 1)], hq=7, hkv=1, d=128, page=48, pad=1),
        dict(seqs=[(3, 5), (0, 9)], hq=33, hkv=11, d=64, page=32)]


@pytest.mark.parametrize("kw", ROWS)
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("fused", [False, True])
def test_append(sub, kw, bits, fused):
    c = Case(sub, bits=bits, **kw)
    n = c.batch.n_rows
    g = torch.Generator().manual_seed(7)
    heads = c.hq + 2 * c.hkv
    qkv = torch.randn(n, heads, c.d, generator=g).to(BF)
    qkv[0, c.hq] = 0
    qkv[n // 2, -1] *= 2.0 ** -104
    qkv[n - 1, c.hq] *= 2.0 ** 100
    qkv = qkv.to(DEV)
    k, v = qkv[:, c.hq:c.hq + c.hkv], qkv[:, c.hq + c.hkv:]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    want = [t.clone() for t in c.pools]
    wants = [t.clone() for t in c.scales] if bits == 8 else []
    for b, (p, m) in enumerate(c.seqs):
        t = torch.arange(p, p + m)
        pg, at = c.table[b, t // c.page].long().to(DEV), (t % c.page).to(DEV)
        for j, x in enumerate((k, v)):
            x = x[int(c.start[b]):int(c.start[b]) + m]
            if bits == 16:
                want[j][c.layer, pg, :, at] = x
            else:
                codes, s = ob.kv8_quantise(np32(x))
                want[j][c.layer, pg, :, at] = torch.from_numpy(codes).to(DEV)
                wants[j][c.layer, pg, :, at] = torch.from_numpy(s).to(DEV)
    (sub.kv8_append if bits == 8 else sub.kv_append)(k, v, c.kv, c.layer, c.batch)
    for got, ref in zip(c.pools, want):     # bits: the pools hold NaN elsewhere
        assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8))
    if bits == 8:
        for got, ref in zip(c.scales, wants):
            assert torch.equal(got.view(torch.int32), ref.view(torch.int32))
        back = [torch.full((n, c.hkv, c.d), 7.0, dtype=BF, device=DEV) for _ in range(2)]
        sub.kv8_read(c.kv, c.layer, c.batch, out=tuple(back))
        lo, hi = int(c.start[0]), int(c.start[-1])
        for x, y in zip((k, v), back):
            ref = torch.from_numpy(ob.kv8_values(*ob.kv8_quantise(np32(x)))).to(BF)
            assert torch.equal(y[lo:hi].cpu(), ref[lo:hi])
            assert torch.all(y[:lo] == 7) and torch.all(y[hi:] == 7)


@pytest.mark.parametrize("bits", [16, 8])
def test_append_skips_what_has_no_place(sub, bits):
    """Positions below 0, past the capacity, on a missing page; rows that are not finite."""
    c = Case(sub, [(0, 16), (0, 32)], 4, 2, 64, bits=bits)
    c.table_d[1, 1] = -1
    c.table_d[0, 0] = 10 ** 6
    b = sub.batch(torch.tensor([0, 4, 12], dtype=torch.int32, device=DEV),
                  torch.tensor([0, 14], dtype=torch.int32, device=DEV), 12)
    x = torch.ones(12, 2, 64, dtype=BF, device=DEV)
    x[4, 0, 3], x[5, 1, 0] = float("inf"), float("nan")
    before = [t.clone() for t in c.pools]
    fn = sub.kv8_append if bits == 8 else sub.kv_append
    fn(x, x, c.kv, c.layer, b)
    first = int(c.table[1, 0])
    for got, ref in zip(c.pools, before):
        ref[c.layer, first, :, 14:16] = x[4:6].transpose(0, 1) if bits == 16 else 255
        if bits == 8:
            ref[c.layer, first, 0, 14] = ref[c.layer, first, 1, 15] = 128
        assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8))
    if bits == 8:
        s = c.scales[0][c.layer, first, :, 14:16].cpu()
        assert torch.isnan(s[0, 0]) and torch.isnan(s[1, 1])
        assert float(s[1, 0]) == float(s[0, 1]) == float(np.float32(1) / np.float32(127))
        k, v = sub.kv8_read(c.kv, c.layer, b)
        assert torch.all(k[:4] == 0) and torch.all(v[6:] == 0)      # no page
        assert torch.isnan(k[4, 0]).all() and not torch.isnan(k[4, 1]).any()
    b = sub.batch(torch.tensor([0, 6, 12], dtype=torch.int32, device=DEV),
                  torch.tensor([-6, 32], dtype=torch.int32, device=DEV), 12)
    before = [t.clone() for t in c.pools]
    fn(x, x, c.kv, c.layer, b)
    for got, ref in zip(c.pools, before):
        assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8))


# -------------------------------------------------------------- attention --
ATTN = [dict(seqs=[(0, 1)], hq=4, hkv=2, d=64),
        dict(seqs=[(511, 1)], hq=4, hkv=2, d=64),
        dict(seqs=[(31, 1), (32, 1), (0, 1), (63, 1), (1000, 1)], hq=28, hkv=4, d=128, page=64),
        dict(seqs=[(300, 8), (5, 0), (40, 3), (0, 20)], hq=28, hkv=4, d=128, page=48, pad=5, before=3),
        dict(seqs=[(700, 1), (3, 1), (129, 1)], hq=40, hkv=8, d=128, page=16),
        dict(seqs=[(0, 130)], hq=8, hkv=8, d=64, page=32),
        dict(seqs=[(77, 300), (500, 1), (0, 257)], hq=8, hkv=2, d=128, page=64, pad=1),
        dict(seqs=[(255, 129)], hq=16, hkv=1, d=64, page=128),
        dict(seqs=[(2500, 4)], hq=64, hkv=1, d=128, page=16),
        dict(seqs=[(600, 33), (0, 1), (90, 64)], hq=6, hkv=2, d=64, page=48),
        dict(seqs=[(b * 7, 1 + b % 3) for b in range(70)], hq=4, hkv=2, d=64, page=16)]


@pytest.mark.parametrize("kw", ATTN)
@pytest.mark.parametrize("bits", [16, 8])
def test_chunk_attn(sub, kw, bits):
    c = Case(sub, bits=bits, seed=len(kw["seqs"]) + bits, **kw)
    o = torch.full((c.batch.n_rows, c.hq, c.d), 7.0, dtype=BF, device=DEV)
    sub.chunk_attn(c.q.to(DEV), c.kv, c.layer, c.batch, out=o)
    c.check(o)
    lo, hi = int(c.start[0]), int(c.start[-1])
    assert torch.all(o[:lo] == 7) and torch.all(o[hi:] == 7)
    again = sub.chunk_attn(c.q.to(DEV), c.kv, c.layer, c.batch)
    assert torch.equal(again[lo:hi], o[lo:hi])          # the same call, the same bits
    assert torch.all(again[:lo] == 0) and torch.all(again[hi:] == 0)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("n", [1, 40, 300])
def test_chunk_attn_long(sub, bits, n):
    """Many CTAs on one sequence's keys, beside short ones."""
    c = Case(sub, [(9000, n), (64, n), (0, n)], 4, 1, 128, page=64, bits=bits, seed=n)
    c.check(sub.chunk_attn(c.q.to(DEV), c.kv, c.layer, c.batch))


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("n", [2, 200])
def test_strided_queries_and_scale(sub, bits, n):
    c = Case(sub, [(90, n), (13, n)], 8, 2, 64, page=32, bits=bits, seed=1)
    wide = torch.randn(c.batch.n_rows, 12, 64, device=DEV).to(BF)
    wide[:, :8] = c.q.to(DEV)
    for scale in (0.0, 0.05, 0.6):
        c.check(sub.chunk_attn(wide[:, :8], c.kv, c.layer, c.batch, scale=scale), scale=scale)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("n", [4, 150])
def test_rows_without_keys_and_missing_pages(sub, bits, n):
    """Rows at negative positions and sequences whose pages are all missing give
    zeros; a missing page's keys count for nobody; past the capacity a row reads
    what the table covers."""
    c = Case(sub, [(200, n), (64, n), (-2, n), (170, n)], 8, 2, 128, bits=bits, seed=2)
    c.table_d[0, 3] = -1
    c.table_d[0, 5] = c.kv.n_pages
    c.table_d[1] = -7
    have = [np.ones(max(0, p + m), bool) for p, m in c.seqs]
    have[0][48:64] = have[0][80:96] = False
    have[1][:] = False
    c.check(sub.chunk_attn(c.q.to(DEV), c.kv, c.layer, c.batch), have=have)
    # rows placed beyond the table's width read all of it, its last page's
    # garbage too, until that holds something: keys and values of zero
    cap = c.kv.capacity
    b = sub.batch(c.start.to(DEV), torch.tensor([cap + 50, 0, 0, cap - 1], dtype=torch.int32,
                                                device=DEV), c.batch.n_rows)
    assert torch.isnan(sub.chunk_attn(c.q.to(DEV), c.kv, c.layer, b)[:n]).all()
    keys = 200 + n
    end = -(-keys // 16) * 16
    last = int(c.table[0, keys // 16])
    for pool in c.pools:
        pool[c.layer, last, :, keys % 16:] = 0 if bits == 16 else 128
    for pool in c.scales if bits == 8 else ():
        pool[c.layer, last, :, keys % 16:] = 1
    o = sub.chunk_attn(c.q.to(DEV), c.kv, c.layer, b)
    k, v = (np.concatenate([c.values(j, 0), np.zeros((end - keys, 2, 128), np.float32)])
            for j in range(2))
    hv = np.concatenate([have[0], np.ones(end - keys, bool)])
    ref, w = ob.chunk_attention(np32(c.q[:2]), k, v, cap, have=hv)
    assert np.all(np.abs(np32(o[:2]) - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 1e-4) * w)


@pytest.mark.parametrize("n", [3, 40, 260])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_later_keys_do_not_reach_earlier_rows(sub, n, bad):
    """Infinities and NaN in a chunk's own later rows: rows before them are as
    without, the row itself and those after it are not finite where it is not."""
    c = Case(sub, [(45, n), (20, 2)], 8, 2, 128, seed=3)
    at = 45 + n - 2
    clean = sub.chunk_attn(c.q.to(DEV), c.kv, c.layer, c.batch).clone()
    pg, pl = int(c.table[0, at // 16]), at % 16
    c.pools[1][c.layer, pg, 1, pl, 5] = bad
    o = sub.chunk_attn(c.q.to(DEV), c.kv, c.layer, c.batch)
    early = slice(0, n - 2)
    c_rows = torch.cat([o[early], o[n:]])
    assert torch.isfinite(c_rows).all()
    assert (c_rows - torch.cat([clean[early], clean[n:]])).abs().max() < 0.05
    late = o[n - 2:n]
    assert not torch.isfinite(late[:, 4:, 5]).any()       # KV head 1: query heads 4..7
    assert torch.isfinite(late[:, :4]).all()
    c.pools[0][c.layer, pg, 0, pl, 7] = bad               # and in K
    o = sub.chunk_attn(c.q.to(DEV), c.kv, c.layer, c.batch)
    assert torch.isfinite(torch.cat([o[early], o[n:]])).all()


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("n", [1, 4, 40])
def test_operators_right_after_each_other(sub, bits, n):
    """Each call sees all that the one just before it wrote, with no pause between:
    rows, then attention; logits' probabilities, then verification."""
    c = Case(sub, [(100, n), (37, n), (1500, n)], 8, 2, 128, bits=bits, seed=10)
    q, g = c.q.to(DEV), torch.Generator(device=DEV).manual_seed(1)
    append = sub.kv_append if bits == 16 else sub.kv8_append
    rows = [torch.randn(3 * n, 2, 128, device=DEV, generator=g).to(BF) for _ in range(8)]
    z = torch.randn(3, 3, 5000, device=DEV, generator=g)
    draft = torch.randint(0, 5000, (3, 2), device=DEV, generator=g, dtype=torch.int32)
    u = torch.rand(3, 3, device=DEV, generator=g)
    p = torch.empty_like(z)
    o = torch.empty_like(q)
    for i in range(24):
        append(rows[i % 8], rows[(3 * i + 1) % 8], c.kv, c.layer, c.batch)
        sub.chunk_attn(q, c.kv, c.layer, c.batch, out=o)
        sub.probs(z[i % 3], 0.3 + 0.1 * i, out=p[i % 3])
        tokens, _ = sub.verify_sample(p[i % 3][None], None, draft[:1], u[:1])
        torch.cuda.synchronize()
        assert torch.equal(o, sub.chunk_attn(q, c.kv, c.layer, c.batch)), i
        assert torch.equal(tokens, sub.verify_sample(p[i % 3][None], None, draft[:1], u[:1])[0])


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("n", [2, 12, 40])
def test_positions_at_the_end_of_int32(sub, bits, n):
    """Rows beyond the capacity read all of it, however far beyond."""
    c = Case(sub, [(64 - n, n)], 8, 2, 64, bits=bits, seed=9)
    q = c.q.to(DEV)
    o = [sub.chunk_attn(q, c.kv, c.layer,
                        sub.batch(c.start.to(DEV), torch.tensor([pos], dtype=torch.int32, device=DEV), n))
         for pos in (c.kv.capacity, 2 ** 31 - 2)]
    assert torch.isfinite(o[0]).all() and o[0].abs().min(-1).values.max() > 0
    assert torch.equal(o[0], o[1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_later_keys_do_not_reach_earlier_rows_in_small_tiles(sub, d, bad):
    """The same for at most 8 rows per sequence and KV head."""
    c = Case(sub, [(45, 4), (20, 1), (33, 1)], 4, 2, d, seed=8)
    clean = sub.chunk_attn(c.q.to(DEV), c.kv, c.layer, c.batch).clone()
    pg, pl = int(c.table[0, 47 // 16]), 47 % 16
    c.pools[1][c.layer, pg, 1, pl, 5] = bad
    c.pools[0][c.layer, pg, 0, pl, 7] = bad
    o = sub.chunk_attn(c.q.to(DEV), c.kv, c.layer, c.batch)
    assert torch.equal(torch.cat([o[:2], o[4:]]), torch.cat([clean[:2], clean[4:]]))
    assert not torch.isfinite(o[2:4, 2:, 5]).any()
    other = [x for x in range(d) if x != 5]
    assert (o[2:4, 2:, other] - clean[2:4, 2:, other]).abs().max() < 0.05
    assert not torch.isfinite(o[2:4, :2]).all()


@pytest.mark.parametrize("bits,d", [(16, 128), (16, 64), (8, 128), (8, 64)])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_a_key_that_is_not_a_number_is_not_lost(sub, bits, d, n):
    """A NaN in K that rows read, alone in its block for the first of them."""
    c = Case(sub, [(128, n), (20, 1)], 8, 2, d, bits=bits, seed=6)
    pg, pl = int(c.table[0, 128 // 16]), 128 % 16
    where = c.pools[0] if bits == 16 else c.scales[0]
    where[c.layer, pg, 0, pl] = float("nan")
    o = sub.chunk_attn(c.q.to(DEV), c.kv, c.layer, c.batch)
    assert torch.isnan(o[:n, :4]).all()
    assert torch.isfinite(o[:n, 4:]).all() and torch.isfinite(o[n:]).all()


def test_scales_and_queries_of_any_size_in_an_8_bit_cache(sub):
    """Scales over 2^-60 .. 2^60 and queries of 2^-90 .. 2^60: sums stay in range."""
    for n in (1, 140):
        c = Case(sub, [(100, n), (60, n)], 4, 2, 64, bits=8, seed=4)
        rng = np.random.default_rng(5)
        for b in range(2):
            keys = 100 + n if b == 0 else 60 + n
            f = np.float32(2.0) ** rng.integers(-60, 60, (keys, 2)).astype(np.float32)
            t = torch.arange(keys)
            pg, at = c.table[b, t // 16].long(), t % 16
            codes, s = c.codes[1][b]
            c.codes[1][b] = codes, s * f
            c.scales[1][c.layer, pg.to(DEV), :, at.to(DEV)] = torch.from_numpy(s * f).to(DEV)
        c.q[0] *= 2.0 ** -90
        o = sub.chunk_attn(c.q.to(DEV), c.kv, c.layer, c.batch)
        assert torch.isfinite(o).all()
        c.check(o)
        c.q[0] *= 2.0 ** 90
        c.check(sub.chunk_attn((c.q.to(DEV) * 2.0 ** 60), c.kv, c.layer, c.batch,
                               scale=0.125 * 2.0 ** -60), scale=0.125)


def test_pools_past_32_bits(sub):
    """Pages whose elements lie beyond 2^32 bytes and 2^31 elements."""
    n_pages = 2 ** 31 // (8 * 64 * 128) + 40
    k = torch.empty(1, n_pages, 8, 64, 128, dtype=BF, device=DEV)
    v = torch.empty_like(k)
    pages = [n_pages - 1, 3, n_pages - 20]
    q, kk, vv = (torch.randn(150, h, 128, device=DEV).to(BF) for h in (16, 8, 8))
    table = torch.tensor([pages], dtype=torch.int32, device=DEV)
    kv = sub.paged_kv(k, v, table)
    all_rows = sub.batch(torch.tensor([0, 150], dtype=torch.int32, device=DEV),
                         torch.tensor([0], dtype=torch.int32, device=DEV), 150)
    sub.kv_append(kk, vv, kv, 0, all_rows)
    assert torch.equal(k[0, pages[0]], kk[:64].transpose(0, 1))
    o = sub.chunk_attn(q, kv, 0, all_rows)
    last = sub.batch(torch.tensor([0, 1], dtype=torch.int32, device=DEV),
                     torch.tensor([149], dtype=torch.int32, device=DEV), 1)
    one = sub.chunk_attn(q[149:], kv, 0, last)
    ref, w = ob.chunk_attention(np32(q[100:]), np32(kk), np32(vv), 100)
    for got, rf, ww in ((o[100:], ref, w), (one, ref[49:], w[49:])):
        assert np.all(np.abs(np32(got) - rf) <= 2.0 ** -8 * np.abs(rf) + (2.0 ** -8 + 1e-4) * ww)
    del k, v, kv


def test_workspaces_streams_and_graphs(sub):
    c = Case(sub, [(3000, 1), (20, 1)], 8, 2, 128, bits=8, seed=6)
    q = c.q.to(DEV)
    ref = sub.chunk_attn(q, c.kv, c.layer, c.batch)
    need = sub.chunk_attn_workspace(8, 2, 128, 2, 2)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(sub.chunk_attn(q, c.kv, c.layer, c.batch, workspace=ws), ref)
    with pytest.raises(sub.SubError):
        sub.chunk_attn(q, c.kv, c.layer, c.batch, workspace=ws[:need - 16])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = sub.chunk_attn(q, c.kv, c.layer, c.batch, stream=side)
    b = sub.chunk_attn(q, c.kv, c.layer, c.batch)       # two at once
    side.synchronize()
    assert torch.equal(a, ref) and torch.equal(b, ref)
    # a captured step replays with the lengths of that moment
    outs, graphs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        o = torch.zeros_like(ref)
        with torch.cuda.graph(g):
            sub.chunk_attn(q, c.kv, c.layer, c.batch, out=o)
        graphs.append(g)
        outs.append(o)
    c.batch.keep[1].copy_(torch.tensor([1500, 7], dtype=torch.int32))
    want = sub.chunk_attn(q, c.kv, c.layer, c.batch)
    assert not torch.equal(want, ref)
    for g in graphs:
        g.replay()
    for o in outs:
        assert torch.equal(o, want)


# ----------------------------------------------------------- probabilities --
@pytest.mark.parametrize("rows,v", [(1, 1), (3, 2), (5, 1023), (200, 1024), (2, 2049), (1, 5000), (7, 5001),
                                    (160, 20001), (1, 152064), (3, 128255), (2, 400003),
                                    (1, 1 << 20)])
@pytest.mark.parametrize("t", [0.2, 1.0, 3.0])
def test_probs(sub, rows, v, t):
    """Relative error: 2 ulp of the base-2 exponential, one rounding of its
    argument and of the difference to the maximum (each 2^-24 of an exponent of at most
    |z - max| log2(e) / T, times ln 2), the factor's exponential, the sum's
    roundings (at most 2^-24 * 400 along one path) and three products."""
    g = torch.Generator().manual_seed(rows + v)
    z = 2.5 * torch.randn(rows, v, generator=g)
    ref = ob.probs(z.numpy(), t)
    span = (z.max(1, keepdim=True).values - z).numpy().astype(np.float64) / t
    zd = z.to(DEV)
    p = sub.probs(zd, t)
    rel = 2.0 ** -24 * (2.5 * span + 2.5 * span.max() + 400 + 12)
    err = np.abs(p.cpu().numpy().astype(np.float64) - ref)
    assert np.all(err <= rel * ref + 2.0 ** -126), float((err / (rel * ref + 2.0 ** -126)).max())
    assert sub.probs(zd, t, out=zd) is zd and torch.equal(zd, p)


def test_probs_of_masked_rows(sub):
    for v in (7, 5000, 152064):
        z = torch.full((4, v), float("-inf"))
        z[1, v - 1] = -3e38
        z[2, :2] = torch.tensor([1.0, 1.0])
        z[3] = torch.arange(v) % 3 * 1.0
        z[3, 1] = float("nan")
        p = sub.probs(z.to(DEV), 0.7).cpu()
        assert torch.all(p[0] == 0) and p[1, v - 1] == 1 and p[1].sum() == 1
        assert torch.equal(p[2, :2], torch.tensor([0.5, 0.5])) and torch.all(p[2, 2:] == 0)
        assert torch.isnan(p[3]).all()


# ------------------------------------------------------------ verification --
def _draws(b, n, v, soft, seed, t=0.6):
    g = torch.Generator().manual_seed(seed)
    z = 2.5 * torch.randn(b, n + 1, v, generator=g)
    p = torch.softmax(z / t, -1)
    zq = z[:, :n] + 0.4 * torch.randn(b, n, v, generator=g)
    q = torch.softmax(zq / t, -1) if soft else None
    if n and soft:
        draft = torch.multinomial(q.reshape(b * n, v), 1, generator=g).reshape(b, n)
    else:
        draft = zq.argmax(-1).reshape(b, n)
    return p, q, draft.to(torch.int32), torch.rand(b, n + 1, generator=g)


def _check_tokens(sub, p, q, draft, u):
    tok, acc = sub.verify_sample(p.to(DEV), None if q is None else q.to(DEV), draft.to(DEV), u.to(DEV))
    for b in range(p.shape[0]):
        want, a = ob.verify_sample(p[b].numpy(), None if q is None else q[b].numpy(),
                                   draft[b].tolist(), u[b].tolist())
        assert int(acc[b]) == a and tok[b].cpu().tolist() == want.tolist(), b
    return acc


@pytest.mark.parametrize("b,n,v", [(1, 0, 1), (4, 0, 1000), (3, 1, 5), (40, 4, 1024), (9, 7, 5003),
                                   (2, 33, 3001), (5, 70, 130), (3, 3, 8192), (3, 3, 8193), (2, 4, 152064),
                                   (3, 2, 128257), (1, 1, 1 << 20)])
@pytest.mark.parametrize("soft", [True, False])
def test_verify_sample(sub, b, n, v, soft):
    acc = _check_tokens(sub, *_draws(b, n, v, soft, seed=b + n + v))
    assert 0 <= int(acc.min()) and int(acc.max()) <= n


@pytest.mark.parametrize("v", [6, 1024, 20000])
def test_verify_sample_borders(sub, v):
    """Numbers at both ends, equal and empty rows, drafts that end early or are
    no tokens, probabilities out of range or NaN, numbers that sit on a border."""
    p, q, draft, u = _draws(14, 3, v, True, seed=v)
    u[0] = 0
    u[1] = 1 - 2.0 ** -24
    u[2, 3] = 1.0
    u[3, 3] = -1.0
    q[4] = p[4, :3]                    # p / q = 1: everything is accepted
    q[5, 0] = p[5, 0]
    u[5, 0] = 1.0                      # refused all the same: nothing is left, sample p
    p[6] = 0                           # a row without probability: token 0
    draft[7, 1] = -1
    draft[8, 0] = v
    draft[9, 2] = 2 ** 31 - 1
    p[10, 0, :3] = torch.tensor([2.0, float("nan"), -1.0])
    draft[10, 0] = 0
    draft[11, 0] = 1
    p[11, 0, 1] = float("nan")
    p[12] = 0
    p[12, :, [1, v - 1]] = 0.5
    u[12, 3] = 0.5                     # the running sum has to exceed it: the last token
    p[13] = 0
    p[13, :, v - 1] = 1e-30            # below half of 2^-43
    _check_tokens(sub, p, q, draft, u)
    _check_tokens(sub, p, None, draft, u)


def test_verify_sample_on_given_buffers_and_none(sub):
    p, _, _, u = _draws(6, 0, 2000, False, seed=1)
    out = (torch.full((6, 1), 5, dtype=torch.int32, device=DEV),
           torch.full((6,), 5, dtype=torch.int32, device=DEV))
    t, a = sub.verify_sample(p.to(DEV), None, None, u.to(DEV), out=out)
    assert t is out[0] and torch.all(a == 0)
    want = [ob.verify_sample(p[b].numpy(), None, [], u[b].tolist())[0][0] for b in range(6)]
    assert t[:, 0].tolist() == want


# ---------------------------------------------------------------- together --
@pytest.mark.parametrize("bits", [16, 8])
def test_a_speculative_step_of_a_batch(sub, bits):
    """Rows enter the cache, the new rows attend, a head makes logits, the draft
    is verified; the same step token by token on the cache gives the same
    attention (within rounding) and a graph replays the whole of it."""
    hq, hkv, d, v, n = 8, 2, 64, 1000, 4
    seqs = [(37, n), (5, n), (130, n)]
    c = Case(sub, seqs, hq, hkv, d, bits=bits, seed=8)
    append = sub.kv8_append if bits == 8 else sub.kv_append
    rows = c.batch.n_rows
    k = torch.cat([c.k[b][p:p + m] for b, (p, m) in enumerate(seqs)]).to(DEV)
    w = torch.cat([c.v[b][p:p + m] for b, (p, m) in enumerate(seqs)]).to(DEV)
    head = (torch.randn(v, hq * d, generator=torch.Generator().manual_seed(1)) * 0.2).to(BF).to(DEV)
    q = c.q.to(DEV)
    z = torch.zeros(rows, v, device=DEV)
    _, _, draft, u = (None if t is None else t.to(DEV) for t in _draws(3, n - 1, v, False, 2))
    tok, acc = sub.verify_sample(torch.ones(3, n, v, device=DEV), None, draft, u)   # buffers
    p, o = torch.zeros(rows, v, device=DEV), torch.zeros(rows, hq, d, dtype=BF, device=DEV)

    def step():
        append(k, w, c.kv, c.layer, c.batch)
        sub.chunk_attn(q, c.kv, c.layer, c.batch, out=o)
        z.copy_(sub.bf16_gemm(o.view(rows, hq * d), head).float())
        sub.probs(z, 0.8, out=p)
        sub.verify_sample(p.view(3, n, v), None, draft, u, out=(tok, acc))

    step()
    c.check(o)
    for b in range(3):
        want, a = ob.verify_sample(p.view(3, n, v)[b].cpu().numpy(), None, draft[b].tolist(),
                                   u[b].tolist())
        assert tok[b].tolist() == want.tolist() and int(acc[b]) == a
    for i in range(n):      # one token at a time
        b1 = sub.batch(torch.arange(4, dtype=torch.int32, device=DEV),
                       c.pos.to(DEV) + i, 3)
        one = sub.chunk_attn(q[i::n].contiguous(), c.kv, c.layer, b1)
        assert (one.float() - o[i::n].float()).abs().max() < 0.04
    first = [t.clone() for t in (o, p, tok, acc)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for t in (o, p, tok, acc):
        t.zero_()
    g.replay()
    assert all(torch.equal(x, y) for x, y in zip(first, (o, p, tok, acc)))
