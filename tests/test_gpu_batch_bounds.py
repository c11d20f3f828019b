"""Serving batches where a result depends on what lies beside it: scales of keys
that a row does not read, weights' second halves, probabilities below the
normal numbers, tensors at any address, caches of one sequence, batches of unlike
and of very many sequences."""
import numpy as np
import pytest
import torch

from oracle import batch as ob
from test_gpu_batch import BF, DEV, Case, np32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sub():
    import substitute_speculative_decoding_gb300 as s
    return s


# ------------------------------------------------- scales of unread keys --
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [4, 20, 40, 300])
@pytest.mark.parametrize("side", [0, 1])
def test_scales_of_later_keys_leave_earlier_rows_as_they_are(sub, d, n, side):
    """The largest finite scales in an 8-bit cache, of keys that only the last two rows
    read: the rows before them keep their bits, whichever tiles the batch gets."""
    c = Case(sub, [(45, n), (20, 2)], 8, 2, d, bits=8, seed=3)
    q = c.q.to(DEV)
    at = 45 + n - 2
    pg, pl = int(c.table[0, at // 16]), at % 16
    clean = sub.chunk_attn(q, c.kv, c.layer, c.batch)
    c.check(clean)
    one = c.scales[side][c.layer, pg, :, pl].clone()
    for f in (2.0 ** 16, 2.0 ** 24, 2.0 ** 30, 2.0 ** 100):
        c.scales[side][c.layer, pg, :, pl] = one * f
        o = sub.chunk_attn(q, c.kv, c.layer, c.batch)
        assert torch.equal(o[:n - 2], clean[:n - 2]) and torch.equal(o[n:], clean[n:]), f
        assert not torch.equal(o[n - 2:n], clean[n - 2:n])


# ------------------------------------------ infinities, tile after tile --
def test_infinite_values_of_neighbouring_tiles_are_all_kept(sub):
    """Tiles whose second half is empty between tiles where both halves read an infinite
    value, several to a CTA: every row from the second on of each long sequence has it."""
    rows = [50, 25, 50, 25, 25, 40] * 100          # times 4 heads: 200, 100, .. of 256 rows
    seqs = [(3 + b % 5, n) for b, n in enumerate(rows)]
    c = Case(sub, seqs, 8, 2, 64, page=64, seed=21)
    q = c.q.to(DEV)
    clean = sub.chunk_attn(q, c.kv, c.layer, c.batch)
    assert torch.isfinite(clean).all()
    want = torch.ones(clean.shape, dtype=torch.bool)
    for b, (p, n) in enumerate(seqs):
        if n > 30:
            at = p + 1                             # the second row's own key
            c.pools[1][c.layer, int(c.table[b, 0]), 1, at, 5] = float("inf")
            want[int(c.start[b]) + 1:int(c.start[b]) + n, 4:, 5] = False
    for _ in range(5):
        o = sub.chunk_attn(q, c.kv, c.layer, c.batch)
        assert torch.equal(torch.isfinite(o).cpu(), want)
        assert torch.equal(o.cpu()[want], clean.cpu()[want])


# --------------------------------------------------------- both halves --
def _check_tight(c, o):
    """As Case.check for a bf16 cache, with the weights in two bf16 halves: the second
    half's rounding is half a step of half a step, 2^-16 of the weight.  The result's own
    rounding counts as what it is, half the distance of bf16 numbers there."""
    for b, (p, n) in enumerate(c.seqs):
        r0 = int(c.start[b])
        q, k, v = np32(c.q[r0:r0 + n]), c.values(0, b), c.values(1, b)
        ref, w = ob.chunk_attention(q, k, v, p)
        top = (np.abs(q) * np.repeat(np.abs(k).max(0), c.hq // c.hkv, 0)).sum(-1, keepdims=True)
        e = 2.0 ** -16 + 2 * (c.d / 16 + 4) * 2.0 ** -22 * top * c.d ** -0.5 + \
            (len(k) / 16 + 4) * 2.0 ** -22
        mag = np.abs(ref) + e * w
        half = 2.0 ** (np.floor(np.log2(np.maximum(mag, 1e-30))) - 8)
        err = np.abs(np32(o[r0:r0 + n]).astype(np.float64) - ref)
        assert np.all(err <= half + e * w), (b, float((err / (half + e * w)).max()))


@pytest.mark.parametrize("kw", [dict(seqs=[(300, 1), (17, 2)], hq=8, hkv=2, d=128),
                                dict(seqs=[(300, 4), (17, 3)], hq=8, hkv=2, d=64),
                                dict(seqs=[(700, 9), (90, 12)], hq=28, hkv=4, d=128, page=48),
                                dict(seqs=[(77, 300), (500, 1)], hq=8, hkv=2, d=128, page=64),
                                dict(seqs=[(0, 130)], hq=8, hkv=8, d=64, page=32)])
def test_weights_over_a_bf16_cache_keep_two_halves(sub, kw):
    """In every tile: a token's row comes out alike whatever else the batch holds."""
    c = Case(sub, seed=17, **kw)
    _check_tight(c, sub.chunk_attn(c.q.to(DEV), c.kv, c.layer, c.batch))


# -------------------------------------------------------- probabilities --
@pytest.mark.parametrize("v", [9, 5000, 152064])
@pytest.mark.parametrize("t", [0.5, 1.0])
def test_probabilities_below_the_normal_numbers(sub, v, t):
    """They are kept down to fp32's smallest step: two roundings to it (the
    exponential, the product with 1 / sum), each off by a step at most."""
    g = torch.Generator().manual_seed(v)
    z = -(85 + 25 * torch.rand(2, v, generator=g)) * t
    z[:, 0] = 0
    z[1, v - 1] = 0
    p = sub.probs(z.to(DEV), t).cpu().numpy().astype(np.float64)
    ref = ob.probs(z.numpy(), t)
    tiny = (ref > 2.0 ** -148) & (ref < 2.0 ** -126)
    assert tiny.sum() >= 2 and np.all(p[ref > 2.0 ** -146] > 0)
    rel = 2.0 ** -24 * (2.5 * 110 + 2.5 * 110 + 400 + 12)
    assert np.all(np.abs(p - ref) <= rel * ref + 2.0 ** -148)


# ------------------------------------------------------------ addresses --
def _at(t, off):
    """The same values, `off` values past a 16-byte boundary."""
    flat = torch.zeros(t.numel() + 8, dtype=t.dtype, device=t.device)
    view = flat[off:off + t.numel()].view(t.shape)
    return view.copy_(t)


@pytest.mark.parametrize("v", [7, 5001, 128255])
def test_probs_at_any_address(sub, v):
    """Where the logits lie decides which four values are summed first, so their address
    moves a result within test_probs' bound (span / T at most 40 here); where the
    probabilities go moves nothing."""
    z = 2.5 * torch.randn(3, v, device=DEV, generator=torch.Generator(device=DEV).manual_seed(v))
    ref = ob.probs(z.cpu().numpy(), 0.7)
    assert float(z.max() - z.min()) / 0.7 < 40
    bound = 2.0 ** -24 * (2.5 * 40 + 2.5 * 40 + 400 + 12) * ref + 2.0 ** -126
    want = sub.probs(z, 0.7)
    assert torch.equal(sub.probs(z[1:2], 0.7), want[1:2])
    for i in range(4):
        want = sub.probs(_at(z, i), 0.7)
        assert np.all(np.abs(want.cpu().numpy().astype(np.float64) - ref) <= bound)
        for j in range(4):
            flat = torch.full((3 * v + 16,), 5.0, device=DEV)
            out = flat[8 + j:8 + j + 3 * v].view(3, v)
            assert sub.probs(_at(z, i), 0.7, out=out) is out and torch.equal(out, want)
            assert torch.all(flat[:8 + j] == 5) and torch.all(flat[8 + j + 3 * v:] == 5)
        own = _at(z, i)
        assert torch.equal(sub.probs(own, 0.7, out=own), want)


@pytest.mark.parametrize("v", [7, 5001, 128255])
def test_verify_sample_at_any_address(sub, v):
    g = torch.Generator(device=DEV).manual_seed(v)
    p = torch.softmax(2.5 * torch.randn(4, 3, v, device=DEV, generator=g), -1)
    q = torch.softmax(p.log()[:, :2] + 0.4 * torch.randn(4, 2, v, device=DEV, generator=g), -1)
    draft = q.argmax(-1).to(torch.int32)
    u = torch.rand(4, 3, device=DEV, generator=g)
    tok, acc = sub.verify_sample(p, q, draft, u)
    t1, a1 = sub.verify_sample(p[1:2], q[1:2], draft[1:2], u[1:2])
    assert torch.equal(t1, tok[1:2]) and torch.equal(a1, acc[1:2])
    for i in range(4):
        for j in range(4):
            t, a = sub.verify_sample(_at(p, i), _at(q, j), draft, u)
            assert torch.equal(t, tok) and torch.equal(a, acc)


# ------------------------------------------- caches of one sequence --
def test_a_cache_of_one_sequence_takes_batches(sub):
    """make_kv's cache: the same rows and results as a paged_kv of its tensors."""
    kv, (k, v, pt) = sub.make_kv(2, 2, 64, 100, page_size=16, shuffle_seed=1)
    g = torch.Generator(device=DEV).manual_seed(0)
    rows = [torch.randn(90, 2, 64, device=DEV, generator=g).to(BF) for _ in range(2)]
    q = torch.randn(90, 8, 64, device=DEV, generator=g).to(BF)
    b = sub.batch(torch.tensor([0, 90], dtype=torch.int32, device=DEV),
                  torch.tensor([0], dtype=torch.int32, device=DEV), 90)
    sub.kv_append(*rows, kv, 1, b)
    o = sub.chunk_attn(q, kv, 1, b)
    k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
    other = sub.paged_kv(k2, v2, pt[None])
    sub.kv_append(*rows, other, 1, b)
    assert torch.equal(k, k2) and torch.equal(v, v2) and k.any()
    assert torch.equal(o, sub.chunk_attn(q, other, 1, b))
    two = sub.batch(torch.tensor([0, 45, 90], dtype=torch.int32, device=DEV),
                    torch.tensor([0, 0], dtype=torch.int32, device=DEV), 90)
    with pytest.raises(sub.SubError):
        sub.chunk_attn(q, kv, 1, two)


def test_a_model_s_cache_takes_batches(sub):
    import synthetic
    cfg = synthetic.CONFIGS["tiny"]
    m = sub.Model(cfg, synthetic.make_model(cfg, norm_gain_std=0.1), max_seq=128, max_depth=4,
                  max_width=2, max_prompt=32)
    m.generate(synthetic.make_prompt(cfg), 4, depth=2, width=2)
    kv = m.kv()
    g = torch.Generator(device=DEV).manual_seed(0)
    n, h, d = 6, kv.n_heads_kv, kv.head_dim
    rows = [torch.randn(n, h, d, device=DEV, generator=g).to(BF) for _ in range(2)]
    q = torch.randn(n, 2 * h, d, device=DEV, generator=g).to(BF)
    b = sub.batch(torch.tensor([0, n], dtype=torch.int32, device=DEV),
                  torch.tensor([0], dtype=torch.int32, device=DEV), n)
    sub.kv_append(*rows, kv, 0, b)
    o = sub.chunk_attn(q, kv, 0, b)
    ref, w = ob.chunk_attention(np32(q), np32(rows[0]), np32(rows[1]), 0)
    assert np.all(np.abs(np32(o) - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 1e-4) * w)
    m.close()


# ------------------------------------------------------ unlike sequences --
@pytest.mark.parametrize("bits", [16, 8])
def test_one_prompt_among_single_rows(sub, bits):
    """The batch's average picks another kernel than its longest sequence would, and
    the other way round."""
    many = [(100 + 9 * b, 1) for b in range(40)]
    for seqs in (many + [(30, 90)], many[:3] + [(64, 200)], [(5, 300)] + many[:1]):
        c = Case(sub, seqs, 8, 2, 64, bits=bits, seed=12)
        o = sub.chunk_attn(c.q.to(DEV), c.kv, c.layer, c.batch)
        c.check(o)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("n_seqs", [33, 1023, 1024])
def test_as_many_sequences_as_a_batch_takes(sub, bits, n_seqs):
    """Rows find their sequence and the work its place with every entry of start used;
    some sequences are empty."""
    seqs = [(b % 13, (b * 5) % 3) for b in range(n_seqs - 1)] + [(7, 2)]
    c = Case(sub, seqs, 2, 1, 64, bits=bits, layers=1, layer=0, seed=13, pad=2)
    lo, hi = int(c.start[0]), int(c.start[-1])
    if bits == 16:
        for t in c.pools:
            t.nan_to_num_(nan=3.0)
    want = [t.clone() for t in c.pools]
    rows = [torch.zeros(c.batch.n_rows, 1, 64, dtype=BF) for _ in range(2)]
    for b, (p, n) in enumerate(seqs):
        for new, side in zip(rows, (c.k, c.v)):
            new[int(c.start[b]):int(c.start[b]) + n] = side[b][p:]
        for t in c.pools if n else ():        # cleared, to be written again
            t[0, int(c.table[b, 0]), :, p] = 1
    append = sub.kv_append if bits == 16 else sub.kv8_append
    append(rows[0].to(DEV), rows[1].to(DEV), c.kv, 0, c.batch)
    assert all(torch.equal(got, ref) for got, ref in zip(c.pools, want))
    o = torch.full((c.batch.n_rows, 2, 64), 7.0, dtype=BF, device=DEV)
    sub.chunk_attn(c.q.to(DEV), c.kv, 0, c.batch, out=o)
    c.check(o)
    assert torch.all(o[:lo] == 7) and torch.all(o[hi:] == 7)


@pytest.mark.parametrize("bits", [16, 8])
def test_a_thousand_prompts(sub, bits):
    """The same for the tiles of many rows, on one page that all sequences share."""
    n_seqs, n = 1024, 33
    c = Case(sub, [(5, n)], 4, 1, 64, page=48, bits=bits, layers=1, layer=0, seed=14)
    table = c.table_d[:, :1].expand(n_seqs, 1).contiguous()
    kv = sub.paged_kv(*c.pools, table) if bits == 16 else sub.paged_kv8(*c.pools, *c.scales, table)
    start = torch.arange(n_seqs + 1, dtype=torch.int32, device=DEV) * n
    b = sub.batch(start, torch.full((n_seqs,), 5, dtype=torch.int32, device=DEV), n_seqs * n)
    o = sub.chunk_attn(c.q.to(DEV).repeat(n_seqs, 1, 1), kv, 0, b).view(n_seqs, n, 4, 64)
    c.check(o[0])
    assert torch.equal(o, o[:1].expand_as(o))
