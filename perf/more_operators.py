"""Cases of drafted trees in serving batches: new rows rotated to their positions
on their way into a paged cache (bf16, or 8-bit codes with a scale per row),
attention of tree nodes over such a cache, the choice of a tree's next nodes over
beams and vocabulary with their states, and accepted rows moved into place.

``own`` false: the plain form in elementary torch operations.  ``own`` true:
the calls a user makes of the library.
"""
import math

import torch

own = False

# (query heads, KV heads, head size, base of the rotation) of the repository's decoder shapes
TINY, QWEN7 = (4, 2, 64, 1e4), (28, 4, 128, 1e6)
LLAMA8, QWEN32 = (32, 8, 128, 5e5), (40, 8, 128, 1e6)
SHAPES = (TINY, QWEN7, LLAMA8, QWEN32)
VOCABS = (1024, 5000, 128256, 152064)
PAGES = (16, 32, 48, 64, 128)
TINY_AMAX = 2.0 ** -100     # rows whose largest value is below it are stored as zeros


def _shape(kind, heads, n_seqs, ctx, page, bits):
    return {"kind": kind, "hq": heads[0], "hkv": heads[1], "d": heads[2], "theta": heads[3],
            "n_seqs": n_seqs, "ctx": ctx, "page": page, "bits": bits}


def _rope(heads, n_seqs, n_new, ctx, page, bits, at="chain", pad=0, fused=False, scaled=False):
    """at: "chain": row i stands at position pos + i; "tree": eight rows each depth."""
    return _shape("rope", heads, n_seqs, ctx, page, bits) | {
        "n_new": n_new, "at": at, "pad": pad, "fused": fused, "scaled": scaled}


def _tree(heads, n_seqs, width, levels, whole, ctx, page, bits, pad=0, fused=False):
    """Trees of 1 + width * levels nodes at most; rows: all of them, or the last level's."""
    return _shape("tree", heads, n_seqs, ctx, page, bits) | {
        "width": width, "levels": levels, "whole": whole, "pad": pad, "fused": fused}


def _beam(n_seqs, n_beams, n_best, vocab, temp, words, first=False, coarse=False):
    return {"kind": "beam", "n_seqs": n_seqs, "n_beams": n_beams, "n_best": n_best, "vocab": vocab,
            "temp": temp, "words": words, "first": first, "coarse": coarse}


def _move(heads, n_seqs, n_max, layers, ctx, page, bits):
    return _shape("move", heads, n_seqs, ctx, page, bits) | {"n_max": n_max, "layers": layers}


def listed():
    cases = {
        # the next token of one short conversation
        "rope16 1x1": _rope(TINY, 1, 1, 511, 16, 16),
        # a tree level of eight nodes for each sequence of a full batch, out of
        # the fused q/k/v product
        "rope8 tree 64x8": _rope(QWEN7, 64, 8, 4096, 64, 8, at="tree", fused=True),
        # prompts of three requests far into their documents, frequencies scaled for
        # long contexts, the last rows are padding
        "rope16 prompts": _rope(LLAMA8, 3, 4096, 100000, 64, 16, pad=5, scaled=True),
        # one short conversation's second tree level
        "tree16 1x8 short": _tree(TINY, 1, 8, 2, False, 511, 16, 16),
        # a draft step of a batch: the nodes of one level
        "tree16 draft 32x8": _tree(QWEN7, 32, 8, 6, False, 8192, 64, 16, fused=True),
        # the target's pass over the whole of four deep trees
        "tree16 verify 4x385": _tree(QWEN7, 4, 8, 48, True, 8192, 64, 16),
        # a draft step over an 8-bit cache of long documents
        "tree8 draft 16x8": _tree(LLAMA8, 16, 8, 4, False, 16384, 64, 8),
        # small trees of a batch verified over an 8-bit cache, the last rows are padding
        "tree8 verify 8x65": _tree(QWEN32, 8, 4, 16, True, 4000, 48, 8, pad=9),
        # one sequence's tree: the next eight nodes of eight, sharpened
        "beam 1x8": _beam(1, 8, 8, 152064, 0.2, 13),
        # a batch's trees; bf16 logits, so that values repeat
        "beam 64x8": _beam(64, 8, 8, 128256, 0.2, 13, coarse=True),
        # one accepted path in a small cache
        "move16 1": _move(TINY, 1, 4, 2, 511, 16, 16),
        # a batch's accepted paths through all layers
        "move8 32": _move(QWEN7, 32, 12, 28, 200, 64, 8),
    }
    return [{"name": n} | c for n, c in cases.items()]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["rope", "rope", "tree", "tree", "tree", "tree", "beam", "beam", "move"])
    heads, page, bits = rng.choice(SHAPES), rng.choice(PAGES), rng.choice([8, 16])
    pad, fused = rng.choice([0, 0, 1, 13]), rng.random() < 0.5
    while True:
        n_seqs = _log(rng, 1, 64)
        if kind == "rope":
            n_new, ctx = _log(rng, 1, 4096), _log(rng, 1, 100000)
            if n_seqs * n_new <= 12288 and n_seqs * (ctx + n_new) <= 310000:
                return _rope(heads, n_seqs, n_new, ctx, page, bits, rng.choice(["chain", "tree"]),
                             pad, fused, rng.random() < 0.5)
        elif kind == "tree":
            c = _tree(heads, n_seqs, rng.choice([1, 2, 4, 5, 8, 11, 16]), rng.randint(0, 48),
                      rng.random() < 0.5, _log(rng, 1, 65536), page, bits, pad, fused)
            slots = 1 + c["width"] * c["levels"]
            rows = slots if c["whole"] else c["width"]
            keys = n_seqs * (c["ctx"] + slots)
            if keys <= 300000 and heads[0] * rows * keys <= 3.0e8 and slots <= 640:
                return c
        elif kind == "beam":
            beams, best = rng.choice([1, 2, 4, 5, 8, 16, 31]), rng.choice([1, 2, 3, 8, 12, 16, 40, 64])
            vocab = rng.choice(VOCABS + (_log(rng, 100, 150000),))
            if n_seqs * beams * vocab <= 512 * 128256:
                return _beam(n_seqs, beams, best, vocab, rng.choice([0.2, 0.6, 1.0, 1.7]),
                             rng.choice([0, 2, 4, 13, 64]), rng.random() < 0.2, rng.random() < 0.5)
        else:
            n_max, layers, ctx = rng.choice([1, 2, 4, 9, 16, 33, 64]), _log(rng, 1, 28), _log(rng, 1, 2000)
            room = n_seqs * (ctx + 3 * n_max + page) * layers * heads[1] * heads[2]
            if room <= 1.2e8:
                return _move(heads, n_seqs, n_max, layers, ctx, page, bits)


def _spread(top, b, step):
    """Sequence b's share of a size: between a quarter and the whole of it."""
    return int(top * (1 - 0.75 * ((b * step) % 1.0)))


def _lengths(c):
    """Each sequence's committed tokens, its tree slots before the new rows, its new rows."""
    base, before, new = [], [], []
    for b in range(c["n_seqs"]):
        base.append(_spread(c["ctx"], b, 0.6180339887))
        if c["kind"] == "rope":
            before.append(0)
            new.append(max(1, round(c["n_new"] * (1 - 0.75 * ((b * 0.7548776662) % 1.0)))))
        else:
            levels = c["levels"] - int(c["levels"] * 0.75 * ((b * 0.7548776662) % 1.0))
            whole = c["whole"] or levels == 0
            before.append(0 if whole else 1 + c["width"] * (levels - 1))
            new.append(1 + c["width"] * levels if whole else c["width"])
    return base, before, new


def _slot(c):
    """First slot of the chosen nodes: the last level that the states have room for."""
    return 32 * c["words"] - c["n_best"]


def _moved(c):
    return [1 + (3 * b) % c["n_max"] for b in range(c["n_seqs"])]


def work(c):
    if c["kind"] == "beam":
        rows = c["n_seqs"] * (1 if c["first"] else c["n_beams"])
        picked = c["n_seqs"] * c["n_best"]
        return {"bytes": 4 * rows * c["vocab"] + picked * (12 + 8 * c["words"]),
                "flops": 4 * rows * c["vocab"]}
    width = c["hkv"] * c["d"]
    stored = width * 2 if c["bits"] == 16 else width + 4 * c["hkv"]   # a row of K or of V
    if c["kind"] == "move":
        return {"bytes": 4 * sum(_moved(c)) * c["layers"] * stored, "flops": 0}
    base, before, new = _lengths(c)
    n = sum(new)
    if c["kind"] == "rope":
        back = 2 * n * (stored + 2 * width) if c["bits"] == 8 else 0   # read back as bf16
        return {"bytes": 2 * n * (2 * width + stored) + 4 * n * c["hq"] * c["d"] + back,
                "flops": 3 * n * (c["hq"] + c["hkv"]) * c["d"]}
    keys = sum(p + s + m for p, s, m in zip(base, before, new))
    # a node reads the committed keys and its path, half the tree's depth on average
    path = [1 + (s + m) // c["width"] / (2 if c["whole"] else 1) for s, m in zip(before, new)]
    pairs = sum(m * (p + t) for p, m, t in zip(base, new, path))
    words = -(-(1 + c["width"] * c["levels"]) // 32)
    return {"bytes": 2 * keys * stored + 4 * n * c["hq"] * c["d"] + 4 * n * words,
            "flops": int(4 * c["d"] * c["hq"] * pairs)}


# ------------------------------------------------------------------ inputs --
def _quantise(x):
    """A row's largest value to 127: codes 1..255 around 128, fp32 scale."""
    x = x.float()
    a = x.abs().amax(-1, keepdim=True)
    none = a < TINY_AMAX
    s = torch.where(none, torch.ones_like(a), a / 127.0)
    t = torch.where(none, torch.zeros_like(a), 127.0 / a)
    return (torch.round(x * t) + 128.0).to(torch.uint8), s.squeeze(-1)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cache(c, keys, layers, dev):
    """Pools whose pages lie in random order, and the table of them; entries past
    a sequence's own pages hold none."""
    need = [-(-k // c["page"]) for k in keys]
    n_pages = sum(need)
    owner = torch.randperm(n_pages, **dev).to(torch.int32)
    have = torch.tensor(need, device="cuda")[:, None]
    col = torch.arange(max(need), device="cuda")[None]
    idx = have.cumsum(0) - have + col
    shape = (layers, n_pages, c["hkv"], c["page"], c["d"])
    # keys have channels of unlike size, as trained ones do
    chan = torch.exp(0.5 * torch.randn(c["hkv"], 1, c["d"], **dev))
    s = {"c": c, "chan": chan,
         "table": torch.where(col < have, owner[idx.clamp(max=n_pages - 1)], -1).to(torch.int32)}
    pools = (torch.randn(shape, **dev) * chan).to(torch.bfloat16), torch.randn(shape, **dev).to(torch.bfloat16)
    if c["bits"] == 8:
        s["pool_k"], s["scale_k"] = _quantise(pools[0])
        s["pool_v"], s["scale_v"] = _quantise(pools[1])
    else:
        s["pool_k"], s["pool_v"] = pools
    return s


def _paths(c, dev):
    """Of every slot of every sequence's tree: its path from the root, itself
    included, as truth values [n_seqs, slots, slots]."""
    slots, width = 1 + c["width"] * c["levels"], c["width"]
    path = torch.eye(slots, dtype=torch.bool, device="cuda").repeat(c["n_seqs"], 1, 1)
    path[:, :, 0] = True
    seqs = torch.arange(c["n_seqs"], device="cuda")[:, None]
    for level in range(2, c["levels"] + 1):     # parents: any of the level before
        first = 1 + (level - 1) * width
        parent = first - width + torch.randint(0, width, (c["n_seqs"], width), **dev)
        path[:, first:first + width] |= path[seqs, parent]
    return path


def _prepare_rows(c, dev):
    base, before, new = _lengths(c)
    total = sum(new) + c["pad"]
    s = _cache(c, [p + t + n for p, t, n in zip(base, before, new)], 1, dev)
    s["new_max"], s["keys_max"] = max(new), max(p + t + n for p, t, n in zip(base, before, new))
    s["start"] = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
    s["base"], s["pos"] = _ints(base), _ints([p + t for p, t in zip(base, before)])
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    qkv = torch.randn(total, (hq + 2 * hkv) * d, **dev)
    qkv[:, :hq * d] *= 1.5
    qkv[:, hq * d:(hq + hkv) * d] *= s["chan"].reshape(1, -1)
    qkv = qkv.to(torch.bfloat16).reshape(total, hq + 2 * hkv, d)
    parts = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    s["q"], s["k"], s["v"] = parts if c["fused"] else [t.contiguous() for t in parts]
    s["o"] = torch.zeros(total, hq, d, dtype=torch.bfloat16, device="cuda")
    seq = torch.repeat_interleave(torch.arange(c["n_seqs"], device="cuda"),
                                  torch.tensor(new, device="cuda"))
    i = torch.arange(len(seq), device="cuda") - s["start"][seq]
    if c["kind"] == "rope":
        s["back"] = torch.zeros(2, total, hkv, d, dtype=torch.bfloat16, device="cuda")
        s["at"] = None
        if c["at"] == "tree":
            s["at"] = torch.zeros(total, dtype=torch.int32, device="cuda")
            s["at"][:len(seq)] = (s["pos"][seq] + (i + 7) // 8).to(torch.int32)
        freqs = [c["theta"] ** (-2.0 * j / d) for j in range(d // 2)]
        if c["scaled"]:     # slow turns slower by 8, what turns often as it is, in between a blend
            turns = [8192.0 * f / (2.0 * math.pi) for f in freqs]
            keep = [min(1.0, max(0.0, (t - 1.0) / 3.0)) for t in turns]
            freqs = [f * (k + (1.0 - k) / 8.0) for f, k in zip(freqs, keep)]
        s["freqs"] = freqs
        return s
    path = _paths(c, dev)[seq, torch.tensor(before, device="cuda")[seq] + i]
    words = -(-path.shape[1] // 32)
    bits = torch.zeros(len(seq), words * 32, dtype=torch.long, device="cuda")
    bits[:, :path.shape[1]] = path
    packed = (bits.reshape(len(seq), words, 32) << torch.arange(32, device="cuda")).sum(-1)
    s["mask"] = torch.zeros(total, words, dtype=torch.int32, device="cuda")
    s["mask"][:len(seq)] = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).to(torch.int32)
    return s


def _prepare_move(c, dev):
    count = _moved(c)
    base = [_spread(c["ctx"], b, 0.6180339887) for b in range(c["n_seqs"])]
    s = _cache(c, [p + 1 + 3 * c["n_max"] for p in base], c["layers"], dev)
    s["count"], s["to"] = _ints(count), _ints([p + 1 for p in base])
    # level by level further into the tree, behind all places that are written
    skip = torch.randint(0, 2, (c["n_seqs"], c["n_max"]), **dev).cumsum(1)
    s["src"] = (s["to"][:, None] + c["n_max"] + torch.arange(c["n_max"], device="cuda")[None] + skip
                - skip[:, :1]).to(torch.int32)
    return s


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = {"device": "cuda", "generator": g}
    if c["kind"] in ("rope", "tree"):
        return _prepare_rows(c, dev)
    if c["kind"] == "move":
        return _prepare_move(c, dev)
    b, n, v = c["n_seqs"], c["n_beams"], c["vocab"]
    z = 2.5 * torch.randn(b, n, v, **dev)
    if c["coarse"]:
        z = z.to(torch.bfloat16).float()
    score = -3.0 * torch.rand(b, n, **dev).cumsum(1)
    if c["first"]:      # a tree's root: one beam, the others are not there yet
        score[:, 1:] = -torch.inf
    state = None
    if c["words"]:
        state = torch.randint(-2 ** 31, 2 ** 31, (b, n, c["words"]), **dev).to(torch.int32)
    return {"c": c, "logits": z, "score": score, "state": state}


# --------------------------------------------------------------- plain form --
def _row_places(s):
    """Of every row of the sequences: sequence, its number there, position, page, place in it."""
    n = s["start"][1:] - s["start"][:-1]
    total = s["q"].shape[0] - s["c"]["pad"]
    seq = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n, output_size=total)
    i = torch.arange(total, device="cuda") - s["start"][seq]
    p = s["pos"][seq] + i
    page = s["table"][seq, p // s["c"]["page"]].long()
    return seq, i, p, page, p % s["c"]["page"]


def _rotate(s, x, at):
    """Pairs (i, i + d / 2) of each head turned by the position's angles."""
    f = torch.tensor(s["freqs"], dtype=torch.float64, device="cuda")
    angle = at.double()[:, None] * f[None]      # far positions: 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x1, x2 = x.float().chunk(2, -1)
    return torch.cat((x1 * cos - x2 * sin, x2 * cos + x1 * sin), -1)


def _append_rope(s):
    c = s["c"]
    _, _, p, page, place = _row_places(s)
    total = len(page)
    at = p if s["at"] is None else s["at"][:total]
    s["o"][:total] = _rotate(s, s["q"][:total], at).to(torch.bfloat16)
    head = torch.arange(c["hkv"], device="cuda")[None]
    where = (0, page[:, None], head, place[:, None])
    k, v = _rotate(s, s["k"][:total], at), s["v"][:total]
    if c["bits"] == 16:
        s["pool_k"][where], s["pool_v"][where] = k.to(torch.bfloat16), v
        return s["o"], s["pool_k"], s["pool_v"]
    s["pool_k"][where], s["scale_k"][where] = _quantise(k)
    s["pool_v"][where], s["scale_v"][where] = _quantise(v)
    s["back"][0, :total] = ((s["pool_k"][where].float() - 128.0) * s["scale_k"][where][..., None]).to(torch.bfloat16)
    s["back"][1, :total] = ((s["pool_v"][where].float() - 128.0) * s["scale_v"][where][..., None]).to(torch.bfloat16)
    return s["o"], s["back"], s["scale_k"], s["scale_v"]


def _dense(s, name):
    """[sequence, key, head, d] in fp32, as far as the longest sequence."""
    c = s["c"]
    pages = s["table"].clamp(min=0).long()
    x = s["pool_" + name][0][pages].float()                  # [seq, page, head, place, d]
    if c["bits"] == 8:
        x = (x - 128.0) * s["scale_" + name][0][pages][..., None]
    return x.transpose(2, 3).reshape(c["n_seqs"], -1, c["hkv"], c["d"])[:, :s["keys_max"]]


def _tree_attn(s):
    c = s["c"]
    seq, i, p, _, _ = _row_places(s)
    n, g, b, total = s["new_max"], c["hq"] // c["hkv"], c["n_seqs"], len(seq)
    q = torch.zeros(b, n, c["hq"], c["d"], device="cuda")
    q[seq, i] = s["q"][:total].float()
    q = q.reshape(b, n, c["hkv"], g, c["d"]).permute(0, 2, 1, 3, 4).reshape(b, c["hkv"], n * g, -1)
    k, v = _dense(s, "k").transpose(1, 2), _dense(s, "v").transpose(1, 2)
    key = torch.arange(k.shape[2], device="cuda")[None]
    slot = key - s["base"][seq][:, None]                                    # [row, key]
    words = s["mask"].shape[1]
    word = s["mask"][:total].gather(1, (slot // 32).clamp(0, words - 1))
    bit = ((word >> (slot % 32)) & 1).bool() & (slot < 32 * words)
    row_sees = (key <= p[:, None]) & ((slot < 0) | bit)
    sees = torch.zeros(b, n, k.shape[2], dtype=torch.bool, device="cuda")
    sees[seq, i] = row_sees
    sees = sees[:, None].repeat_interleave(g, 2)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(c["d"] ** -0.5).masked_fill_(~sees, -torch.inf)
    x = torch.exp(x.sub_(x.amax(-1, keepdim=True).clamp(min=-3.0e38)))
    o = torch.matmul(x, v) / x.sum(-1, keepdim=True)
    o = o.reshape(b, c["hkv"], n, g, c["d"]).permute(0, 2, 1, 3, 4).reshape(b, n, c["hq"], c["d"])
    s["o"][:total] = o[seq, i].to(torch.bfloat16)
    return s["o"]


def _beam_select(s):
    c, z = s["c"], s["logits"]
    b, n, v = z.shape
    # candidates of a beam: its largest logits, equal ones by token.  A beam's order and the
    # places where beams meet have to be right: whole numbers, and sums in 64 bits
    bits = (z + 0.0).view(torch.int32).long()
    key = torch.where(bits >= 0, bits, bits ^ 0x7fffffff) * 2 ** 20 + (2 ** 20 - 1 - torch.arange(v, device="cuda"))
    token = 2 ** 20 - 1 - torch.topk(key, min(c["n_best"], v), -1)[0] % 2 ** 20
    zt = z.double() / c["temp"]
    top = zt.amax(-1, keepdim=True)
    lse = top + torch.log(torch.exp(zt - top).sum(-1, keepdim=True))
    score = (s["score"].double()[..., None] + zt.gather(2, token) - lse).reshape(b, -1)
    token = token.reshape(b, -1)
    if score.shape[1] < c["n_best"]:
        more = c["n_best"] - score.shape[1]
        score = torch.cat((score, score.new_full((b, more), -torch.inf)), 1)
        token = torch.cat((token, token.new_zeros(b, more)), 1)
    score, order = torch.sort(score, dim=1, descending=True, stable=True)
    score, order = score[:, :c["n_best"]], order[:, :c["n_best"]]
    none = score == -torch.inf
    parent = (order // min(c["n_best"], v)).clamp(max=n - 1)
    token = torch.where(none, -1, token.gather(1, order)).to(torch.int32)
    out = [token, torch.where(none, -1, parent).to(torch.int32), score.float()]
    if s["state"] is None:
        return tuple(out)
    state = s["state"].gather(1, parent[..., None].expand(-1, -1, c["words"]))
    state = torch.where(none[..., None], 0, state)
    new = _slot(c) + torch.arange(c["n_best"], device="cuda")      # the new nodes' slots
    one = (torch.arange(c["words"], device="cuda")[None] == (new // 32)[:, None])
    bit = torch.where(one, (1 << (new % 32))[:, None], 0)
    bit = torch.where(bit >= 2 ** 31, bit - 2 ** 32, bit).to(torch.int32)[None]
    return (*out, torch.where(none[..., None], state, state | bit))


def _move_rows(s):
    c = s["c"]
    col = torch.arange(c["n_max"], device="cuda")[None]
    real = col < s["count"][:, None]
    seq = torch.arange(c["n_seqs"], device="cuda")[:, None].expand_as(real)[real]
    src, to = s["src"][real], (s["to"][:, None] + col)[real]
    fp, tp = s["table"][seq, src // c["page"]].long(), s["table"][seq, to // c["page"]].long()
    fr, tr = src % c["page"], to % c["page"]
    names = ("pool_k", "pool_v") if c["bits"] == 16 else ("pool_k", "pool_v", "scale_k", "scale_v")
    for name in names:
        s[name][:, tp, :, tr] = s[name][:, fp, :, fr]
    return tuple(s[name] for name in names)


# --------------------------------------------------------- the library's calls --
def _run_own(s):
    import substitute_speculative_decoding_gb300 as sub
    c = s["c"]
    if c["kind"] == "beam":
        if s["state"] is None:
            return sub.beam_select(s["logits"], s["score"], c["n_best"], c["temp"])
        return sub.beam_select(s["logits"], s["score"], c["n_best"], c["temp"], state=s["state"],
                               slot=_slot(c))
    if "kv" not in s:      # the cache's handle: a program makes it once
        s["kv"] = (sub.paged_kv8(s["pool_k"], s["pool_v"], s["scale_k"], s["scale_v"], s["table"])
                   if c["bits"] == 8 else sub.paged_kv(s["pool_k"], s["pool_v"], s["table"]))
        if c["kind"] == "rope":
            s["rope"] = sub.rope(c["d"], freqs=s["freqs"])
    kv = s["kv"]
    if c["kind"] == "move":
        sub.kv_move(kv, s["to"], s["src"], s["count"])
        pools = s["pool_k"], s["pool_v"]
        return pools if c["bits"] == 16 else (*pools, s["scale_k"], s["scale_v"])
    batch = sub.batch(s["start"], s["pos"], s["q"].shape[0], max_keys=s["keys_max"])
    if c["kind"] == "tree":
        return sub.chunk_tree_attn(s["q"], kv, 0, batch, s["base"], s["mask"], out=s["o"])
    sub.kv_append_rope(s["q"], s["k"], s["v"], kv, 0, batch, s["rope"], at=s["at"], q_out=s["o"])
    if c["bits"] == 16:
        return s["o"], s["pool_k"], s["pool_v"]
    sub.kv8_read(kv, 0, batch, out=(s["back"][0], s["back"][1]))
    return s["o"], s["back"], s["scale_k"], s["scale_v"]


def run(s):
    if own:
        return _run_own(s)
    return {"rope": _append_rope, "tree": _tree_attn, "beam": _beam_select,
            "move": _move_rows}[s["c"]["kind"]](s)


# ------------------------------------------------- the definitions in 64 bits --
def _exact_rope(c, s):
    base, _, new = _lengths(c)
    start, page, half = s["start"].tolist(), c["page"], c["d"] // 2
    f = torch.tensor(s["freqs"], dtype=torch.float64, device="cuda")
    out = s["o"].double()
    pools = [s["pool_k"].double(), s["pool_v"].double()]
    back = s["back"].double()
    scales = [s["scale_k"].double(), s["scale_v"].double()] if c["bits"] == 8 else []
    for b, n in enumerate(new):
        rows = slice(start[b], start[b] + n)
        p = torch.arange(base[b], base[b] + n, device="cuda")
        at = p if s["at"] is None else s["at"][rows]
        angle = at.double()[:, None] * f
        turn = torch.polar(torch.ones_like(angle), angle)

        def rotated(x):
            z = torch.complex(x[..., :half].double(), x[..., half:].double()) * turn[:, None]
            return torch.cat((z.real, z.imag), -1)
        out[rows] = rotated(s["q"][rows])
        pg, pl = s["table"][b][p // page].long(), p % page
        for j, x in enumerate((rotated(s["k"][rows]), s["v"][rows].double())):
            if c["bits"] == 16:
                pools[j][0, pg, :, pl] = x
                continue
            step = x.abs().amax(-1) / 127.0
            step = torch.where(step * 127.0 < TINY_AMAX, 1.0, step)
            scales[j][0, pg, :, pl] = step
            back[j, rows] = torch.round(x / step[..., None]) * step[..., None]
    return (out, *pools) if c["bits"] == 16 else (out, back, *scales)


def _exact_tree(c, s):
    base, before, new = _lengths(c)
    start, page, group = s["start"].tolist(), c["page"], c["hq"] // c["hkv"]
    out = s["o"].double()
    for b, n in enumerate(new):
        first = base[b] + before[b]
        keys = first + n
        rows = slice(start[b], start[b] + n)
        pages = s["table"][b, :-(-keys // page)].long()
        bits = (s["mask"][rows].long()[..., None] >> torch.arange(32, device="cuda")) & 1
        own_slots = bits.reshape(n, -1)[:, :keys - base[b]].bool()
        late = torch.arange(keys, device="cuda") > torch.arange(first, keys, device="cuda")[:, None]
        late[:, base[b]:] |= ~own_slots
        for h in range(c["hkv"]):
            k, v = s["pool_k"][0, pages, h].double(), s["pool_v"][0, pages, h].double()
            if c["bits"] == 8:
                k = (k - 128.0) * s["scale_k"][0, pages, h].double()[..., None]
                v = (v - 128.0) * s["scale_v"][0, pages, h].double()[..., None]
            k, v = k.reshape(-1, c["d"])[:keys], v.reshape(-1, c["d"])[:keys]
            for j in range(h * group, (h + 1) * group):
                z = s["q"][rows, j].double() @ k.T / c["d"] ** 0.5
                out[rows, j] = torch.softmax(z.masked_fill(late, -torch.inf), -1) @ v
    return out


def _exact_beam(c, s):
    """Sequence by sequence: all scores, sorted with equal ones in order."""
    tokens, parents, scores, states = [], [], [], []
    v, k = c["vocab"], c["n_best"]
    for b in range(c["n_seqs"]):
        z = s["logits"][b].double() / c["temp"]
        all_ = (s["score"][b].double()[:, None] + torch.log_softmax(z, -1)).reshape(-1)
        top, order = torch.sort(all_, descending=True, stable=True)
        top, order = top[:k], order[:k]
        if len(top) < k:
            top = torch.cat((top, top.new_full((k - len(top),), -torch.inf)))
            order = torch.cat((order, order.new_zeros(k - len(order))))
        none = top == -torch.inf
        token, parent = order % v, order // v
        tokens.append(torch.where(none, -1, token))
        parents.append(torch.where(none, -1, parent))
        scores.append(top)
        if s["state"] is not None:
            state = s["state"][b][parent].clone()
            for r in range(k):
                slot = _slot(c) + r
                bit = 1 << (slot % 32)
                state[r, slot // 32] |= bit - 2 ** 32 if bit >= 2 ** 31 else bit
            state[none] = 0
            states.append(state)
    out = [torch.stack(tokens).to(torch.int32), torch.stack(parents).to(torch.int32), torch.stack(scores)]
    return (*out, torch.stack(states)) if states else tuple(out)


def _exact_move(c, s):
    names = ("pool_k", "pool_v") if c["bits"] == 16 else ("pool_k", "pool_v", "scale_k", "scale_v")
    out = [s[name].clone() for name in names]
    page = c["page"]
    for b, (n, to) in enumerate(zip(s["count"].tolist(), s["to"].tolist())):
        for i, src in enumerate(s["src"][b, :n].tolist()):
            fp, tp = (int(s["table"][b, t // page]) for t in (src, to + i))
            for x, name in zip(out, names):
                x[:, tp, :, (to + i) % page] = s[name][:, fp, :, src % page]
    return tuple(x.double() if x.is_floating_point() else x for x in out)


def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] == "beam":
        return _exact_beam(c, s)
    return {"rope": _exact_rope, "tree": _exact_tree, "move": _exact_move}[c["kind"]](c, s)
