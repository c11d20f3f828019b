"""Cases of the batched serving operators: rows written into a paged cache
(bf16, or 8-bit codes with a scale per row) and read back, attention of new
tokens over such a cache, probabilities from logits, and the verification of
drafted tokens against probabilities from given random numbers.

``own`` false: the plain form in elementary torch operations.  ``own`` true:
the calls a user makes of the library.
"""
import torch

own = False

# (query heads, KV heads, head size) of the repository's decoder shapes
TINY, QWEN7, LLAMA8, QWEN32 = (4, 2, 64), (28, 4, 128), (32, 8, 128), (40, 8, 128)
SHAPES = (TINY, QWEN7, LLAMA8, QWEN32)
VOCABS = (1024, 5000, 128256, 152064)
PAGES = (16, 32, 48, 64, 128)
TINY_AMAX = 2.0 ** -100     # rows whose largest value is below it are stored as zeros


def _rows(kind, name, heads, n_seqs, n_new, ctx, page, bits, pad=0, fused=False):
    return {"kind": kind, "name": name, "hq": heads[0], "hkv": heads[1], "d": heads[2],
            "n_seqs": n_seqs, "n_new": n_new, "ctx": ctx, "page": page, "bits": bits, "pad": pad,
            "fused": fused}


def listed():
    return [
        # one decode step of a full batch writes one row per sequence, straight
        # out of the fused q/k/v product
        _rows("append", "append8 64x1", QWEN32, 64, 1, 4096, 64, 8, fused=True),
        # prompts of three requests enter the cache, the last rows are padding
        _rows("append", "append8 prompts", LLAMA8, 3, 4096, 1000, 64, 8, pad=5),
        # the smallest call: the next token of one short conversation
        _rows("attn", "attn16 1x1 short", TINY, 1, 1, 511, 16, 16),
        # a decode step of a batch of conversations of many lengths
        _rows("attn", "attn16 32x1", QWEN32, 32, 1, 16384, 64, 16),
        # the target's pass over eight tokens (seven drafted) of eight sequences
        _rows("attn", "attn16 verify 8x8", QWEN7, 8, 8, 4096, 64, 16, fused=True),
        # a chunk of a long prompt behind what is cached of it
        _rows("attn", "attn16 chunk 2048", LLAMA8, 1, 2048, 14336, 64, 16),
        # two long documents, the next token of each, 8-bit cache
        _rows("attn", "attn8 2x1 long", LLAMA8, 2, 1, 65001, 64, 8),
        # prompts of three requests behind shared history, 8-bit cache
        _rows("attn", "attn8 prompts", QWEN7, 3, 1537, 2600, 48, 8, pad=9),
        # one row of draft logits, sharpened
        {"kind": "probs", "name": "probs 1", "rows": 1, "vocab": 152064, "temp": 0.2},
        # target logits of 64 sequences with eight drafted tokens each
        {"kind": "probs", "name": "probs 576", "rows": 576, "vocab": 128256, "temp": 0.6},
        # one sequence's four drafted tokens
        {"kind": "verify", "name": "verify 1x4", "n_seqs": 1, "n_draft": 4, "vocab": 152064,
         "temp": 0.6, "soft": True},
        # a batch's eight drafted tokens each
        {"kind": "verify", "name": "verify 64x8", "n_seqs": 64, "n_draft": 8, "vocab": 128256,
         "temp": 0.6, "soft": True},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["append", "attn", "attn", "attn", "probs", "verify"])
    if kind in ("append", "attn"):
        heads, page, bits = rng.choice(SHAPES), rng.choice(PAGES), rng.choice([8, 16])
        pad = rng.choice([0, 0, 1, 13])
        while True:
            if kind == "append":
                n_seqs, n_new, ctx = _log(rng, 1, 64), _log(rng, 1, 4096), _log(rng, 1, 8192)
                ok = n_seqs * n_new <= 12288 and n_seqs * (ctx + n_new) <= 300000
            else:
                n_seqs, ctx = _log(rng, 1, 64), _log(rng, 1, 65536)
                n_new = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 16, 2048)])
                keys = n_seqs * (ctx + n_new)
                ok = (keys <= 400000 and heads[0] * n_new * keys <= 1.0e9 and
                      4.0 * heads[2] * heads[0] * n_new * keys <= 4.5e11)
            if ok:
                break
        c = _rows(kind, "", heads, n_seqs, n_new, ctx, page, bits, pad, rng.random() < 0.5)
        del c["name"]
        return c
    vocab = rng.choice(VOCABS + (_log(rng, 100, 150000),))
    if kind == "probs":
        return {"kind": kind, "rows": _log(rng, 1, 448), "vocab": vocab,
                "temp": rng.choice([0.2, 0.6, 1.0, 1.7])}
    n_draft = rng.choice([0, 1, 2, 4, 7, 12, 48])
    return {"kind": kind, "n_seqs": _log(rng, 1, max(1, 448 // (n_draft + 1))), "n_draft": n_draft,
            "vocab": vocab, "temp": rng.choice([0.6, 1.0]), "soft": rng.random() < 0.75}


def _lengths(c):
    """Each sequence's new rows and the position of the first: spread between
    a quarter and the whole of the case's sizes."""
    new, pos = [], []
    for b in range(c["n_seqs"]):
        new.append(max(1, round(c["n_new"] * (1 - 0.75 * ((b * 0.7548776662) % 1.0)))))
        pos.append(int(c["ctx"] * (1 - 0.75 * ((b * 0.6180339887) % 1.0))))
    return new, pos


def work(c):
    if c["kind"] == "probs":
        n = c["rows"] * c["vocab"]
        return {"bytes": 8 * n, "flops": 4 * n}
    if c["kind"] == "verify":   # one row of p and (soft drafts) one of q per sequence
        n = c["n_seqs"] * c["vocab"]
        small = c["n_seqs"] * (c["n_draft"] + 1) * 16
        return {"bytes": (8 if c["soft"] and c["n_draft"] else 4) * n + small, "flops": 3 * n}
    new, pos = _lengths(c)
    width = c["hkv"] * c["d"]
    stored = width * 2 if c["bits"] == 16 else width + 4 * c["hkv"]   # a row of K or of V
    if c["kind"] == "append":
        n = sum(new)
        back = 2 * n * (stored + 2 * width) if c["bits"] == 8 else 0  # read back as bf16
        return {"bytes": 2 * n * (2 * width + stored) + back, "flops": 6 * n * width}
    keys = sum(p + n for p, n in zip(pos, new))
    pairs = sum(n * p + n * (n + 1) // 2 for p, n in zip(pos, new))
    return {"bytes": 2 * keys * stored + 4 * sum(new) * c["hq"] * c["d"],
            "flops": 4 * c["d"] * c["hq"] * pairs}


# ------------------------------------------------------------------ inputs --
def _quantise(x):
    """A row's largest value to 127: codes 1..255 around 128, fp32 scale."""
    x = x.float()
    a = x.abs().amax(-1, keepdim=True)
    none = a < TINY_AMAX
    s = torch.where(none, torch.ones_like(a), a / 127.0)
    t = torch.where(none, torch.zeros_like(a), 127.0 / a)
    return (torch.round(x * t) + 128.0).to(torch.uint8), s.squeeze(-1)


def _prepare_rows(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = {"device": "cuda", "generator": g}
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    new, pos = _lengths(c)
    total = sum(new) + c["pad"]
    need = [-(-(p + n) // page) for p, n in zip(pos, new)]
    n_pages, row = sum(need), max(need)
    # pages in random order; entries past a sequence's own pages hold none
    owner = torch.randperm(n_pages, **dev).to(torch.int32)
    ends = torch.tensor(need, device="cuda").cumsum(0)
    col = torch.arange(row, device="cuda")[None]
    have = torch.tensor(need, device="cuda")[:, None]
    idx = ends[:, None] - have + col
    table = torch.where(col < have, owner[idx.clamp(max=n_pages - 1)], -1).to(torch.int32)
    # keys have channels of unlike size, as trained ones do
    chan = torch.exp(0.5 * torch.randn(hkv, 1, d, **dev))
    pool_k = (torch.randn(1, n_pages, hkv, page, d, **dev) * chan).to(torch.bfloat16)
    pool_v = torch.randn(1, n_pages, hkv, page, d, **dev).to(torch.bfloat16)
    s = {"c": c, "table": table, "new_max": max(new),
         "keys_max": max(p + n for p, n in zip(pos, new)),
         "start": torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32),
         "pos": torch.tensor(pos, dtype=torch.int32, device="cuda")}
    width = (hq + 2 * hkv) * d
    qkv = torch.randn(total, width, **dev)
    qkv[:, :hq * d] *= 1.5
    qkv[:, hq * d:(hq + hkv) * d] *= chan.reshape(1, -1)
    qkv = qkv.to(torch.bfloat16).reshape(total, hq + 2 * hkv, d)
    parts = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    s["q"], s["k"], s["v"] = parts if c["fused"] else [t.contiguous() for t in parts]
    if c["bits"] == 8:
        s["pool_k"], s["scale_k"] = _quantise(pool_k)
        s["pool_v"], s["scale_v"] = _quantise(pool_v)
    else:
        s["pool_k"], s["pool_v"] = pool_k, pool_v
    s["o"] = torch.zeros(total, hq, d, dtype=torch.bfloat16, device="cuda")
    s["back"] = torch.zeros(2, total, hkv, d, dtype=torch.bfloat16, device="cuda")
    return s


def prepare(c, seed):
    if c["kind"] in ("append", "attn"):
        return _prepare_rows(c, seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = {"device": "cuda", "generator": g}
    if c["kind"] == "probs":
        return {"c": c, "logits": 2.5 * torch.randn(c["rows"], c["vocab"], **dev),
                "out": torch.empty(c["rows"], c["vocab"], device="cuda")}
    b, n, v = c["n_seqs"], c["n_draft"], c["vocab"]
    z = 2.5 * torch.randn(b, n + 1, v, **dev)
    p = torch.softmax(z / c["temp"], -1)
    zq = z[:, :n] + 0.4 * torch.randn(b, n, v, **dev)   # a draft that mostly agrees
    q = torch.softmax(zq / c["temp"], -1)
    if c["soft"] and n:
        draft = torch.multinomial(q.reshape(b * n, v), 1, generator=g).reshape(b, n)
    else:
        draft, q = zq.argmax(-1).reshape(b, n), None
    # a batch's drafts end at different lengths: every fifth is two tokens short
    short = (torch.arange(b, device="cuda") % 5 == 4)[:, None]
    draft = torch.where(short & (torch.arange(n, device="cuda")[None] >= n - 2), -1, draft)
    return {"c": c, "p": p, "q": q, "draft": draft.to(torch.int32),
            "u": torch.rand(b, n + 1, **dev)}


# --------------------------------------------------------------- plain form --
def _row_places(s):
    """Of every row of the sequences: sequence, position, page, place in it."""
    n = s["start"][1:] - s["start"][:-1]
    total = s["q"].shape[0] - s["c"]["pad"]
    seq = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n, output_size=total)
    i = torch.arange(total, device="cuda") - s["start"][seq]
    p = s["pos"][seq] + i
    page = s["table"][seq, p // s["c"]["page"]].long()
    return seq, i, p, page, p % s["c"]["page"]


def _append(s):
    c = s["c"]
    _, _, _, page, at = _row_places(s)
    total = len(page)
    head = torch.arange(c["hkv"], device="cuda")[None]
    where = (0, page[:, None], head, at[:, None])
    for x, name in ((s["k"], "k"), (s["v"], "v")):
        if c["bits"] == 16:
            s["pool_" + name][where] = x[:total]
        else:
            s["pool_" + name][where], s["scale_" + name][where] = _quantise(x[:total])
    if c["bits"] == 16:
        return s["pool_k"], s["pool_v"]
    for j, name in ((0, "k"), (1, "v")):
        codes, scale = s["pool_" + name][where], s["scale_" + name][where]
        s["back"][j, :total] = ((codes.float() - 128.0) * scale[..., None]).to(torch.bfloat16)
    return s["back"], s["scale_k"], s["scale_v"]


def _dense(s, name):
    """[sequence, key, head, d] in fp32, as far as the longest sequence."""
    c = s["c"]
    pages = s["table"].clamp(min=0).long()
    x = s["pool_" + name][0][pages].float()                  # [seq, page, head, place, d]
    if c["bits"] == 8:
        x = (x - 128.0) * s["scale_" + name][0][pages][..., None]
    return x.transpose(2, 3).reshape(c["n_seqs"], -1, c["hkv"], c["d"])[:, :s["keys_max"]]


def _attn(s):
    c = s["c"]
    seq, i, p, _, _ = _row_places(s)
    n, g, b = s["new_max"], c["hq"] // c["hkv"], c["n_seqs"]
    q = torch.zeros(b, n, c["hq"], c["d"], device="cuda")
    q[seq, i] = s["q"][:len(seq)].float()
    q = q.reshape(b, n, c["hkv"], g, c["d"]).permute(0, 2, 1, 3, 4).reshape(b, c["hkv"], n * g, -1)
    k, v = _dense(s, "k").transpose(1, 2), _dense(s, "v").transpose(1, 2)
    at = s["pos"][:, None].long() + torch.arange(n, device="cuda")[None]
    sees = torch.arange(k.shape[2], device="cuda")[None, None] <= at[..., None]   # [seq, row, key]
    sees = sees[:, None].repeat_interleave(g, 2)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(c["d"] ** -0.5).masked_fill_(~sees, -torch.inf)
    x = torch.exp(x.sub_(x.amax(-1, keepdim=True)))
    o = torch.matmul(x, v) / x.sum(-1, keepdim=True)
    o = o.reshape(b, c["hkv"], n, g, c["d"]).permute(0, 2, 1, 3, 4).reshape(b, n, c["hq"], c["d"])
    s["o"][:len(seq)] = o[seq, i].to(torch.bfloat16)
    return s["o"]


def _probs(s):
    z = s["logits"] / s["c"]["temp"]
    e = torch.exp(z - z.amax(-1, keepdim=True))
    torch.div(e, e.sum(-1, keepdim=True), out=s["out"])
    return s["out"]


def _verify(s):
    p, q, draft, u = s["p"], s["q"], s["draft"].long(), s["u"]
    b, n, v = p.shape[0], draft.shape[1], p.shape[2]
    seqs = torch.arange(b, device="cuda")
    real = (draft >= 0) & (draft < v)
    x = draft.clamp(0, v - 1)[..., None]
    px = p[:, :n].gather(2, x).squeeze(2).double()
    qx = q.gather(2, x).squeeze(2).double() if q is not None else torch.ones_like(px)
    taken = (real & (u[:, :n].double() * qx < px)).long().cumprod(1)
    a = taken.sum(1)                                                   # accepted tokens
    row = p[seqs, a]
    rest = row
    if n:
        at = a.clamp(max=n - 1)
        refused = (a < n) & real[seqs, at]
        qr = (q[seqs, at] if q is not None else
              torch.zeros_like(row).scatter_(1, x[seqs, at], 1.0))
        rest = torch.where(refused[:, None], row - qr, row)
    # whole numbers of 2^-43: their sums are exact in any order
    w = torch.round(rest.clamp(0.0, 1.0).double() * 2.0 ** 43).long()
    wp = torch.round(row.clamp(0.0, 1.0).double() * 2.0 ** 43).long()
    w = torch.where(w.sum(1, keepdim=True) > 0, w, wp)
    below = w.cumsum(1)
    t = torch.floor(below[:, -1:].double() * u[:, n:].double()).long()
    new = (below <= t).sum(1).clamp(max=v - 1)
    col = torch.arange(n + 1, device="cuda")[None]
    tokens = torch.full((b, n + 1), -1, dtype=torch.int32, device="cuda")
    tokens[:, :n] = torch.where(taken > 0, s["draft"], -1)
    tokens = torch.where(col == a[:, None], new[:, None].to(torch.int32), tokens)
    return tokens, a.to(torch.int32)


# --------------------------------------------------------- the library's calls --
def _run_own(s):
    import substitute_speculative_decoding_gb300 as sub
    c = s["c"]
    if c["kind"] == "probs":
        return sub.probs(s["logits"], c["temp"], out=s["out"])
    if c["kind"] == "verify":
        return sub.verify_sample(s["p"], s["q"], s["draft"], s["u"])
    if "kv" not in s:      # the cache's handle: a program makes it once
        s["kv"] = (sub.paged_kv8(s["pool_k"], s["pool_v"], s["scale_k"], s["scale_v"], s["table"])
                   if c["bits"] == 8 else sub.paged_kv(s["pool_k"], s["pool_v"], s["table"]))
    kv = s["kv"]
    batch = sub.batch(s["start"], s["pos"], s["q"].shape[0], max_keys=s["keys_max"])
    if c["kind"] == "attn":
        return sub.chunk_attn(s["q"], kv, 0, batch, out=s["o"])
    if c["bits"] == 16:
        sub.kv_append(s["k"], s["v"], kv, 0, batch)
        return s["pool_k"], s["pool_v"]
    sub.kv8_append(s["k"], s["v"], kv, 0, batch)
    sub.kv8_read(kv, 0, batch, out=(s["back"][0], s["back"][1]))
    return s["back"], s["scale_k"], s["scale_v"]


def run(s):
    if own:
        return _run_own(s)
    return {"append": _append, "attn": _attn, "probs": _probs, "verify": _verify}[s["c"]["kind"]](s)


# ------------------------------------------------- the definitions in 64 bits --
def _exact_verify(s):
    """Token by token, with running sums of the probabilities themselves."""
    n, v = s["draft"].shape[1], s["p"].shape[2]
    tokens, counts = [], []
    for b, (x, u) in enumerate(zip(s["draft"].tolist(), s["u"].tolist())):
        a, rest = 0, None
        while a < n and 0 <= x[a] < v:
            p = s["p"][b, a].double()
            q = (torch.zeros_like(p).index_fill_(0, torch.tensor(x[a], device="cuda"), 1.0)
                 if s["q"] is None else s["q"][b, a].double())
            if not u[a] * q[x[a]].item() < p[x[a]].item():
                rest = (p - q).clamp(min=0)
                break
            a += 1
        rest = s["p"][b, a].double() if rest is None else rest
        new = int((rest.cumsum(0) <= u[n] * rest.sum()).sum().clamp(max=v - 1))
        tokens.append(x[:a] + [new] + [-1] * (n - a))
        counts.append(a)
    ints = {"dtype": torch.int32, "device": "cuda"}
    return torch.tensor(tokens, **ints), torch.tensor(counts, **ints)


def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] == "probs":
        return torch.log_softmax(s["logits"].double() / c["temp"], -1).exp()
    if c["kind"] == "verify":
        return _exact_verify(s)
    new, pos = _lengths(c)
    start, page = s["start"].tolist(), c["page"]
    if c["kind"] == "append" and c["bits"] == 16:
        pools = s["pool_k"].double(), s["pool_v"].double()
        for b, n in enumerate(new):
            at = torch.arange(pos[b], pos[b] + n, device="cuda")
            for x, pool in zip((s["k"], s["v"]), pools):
                pool[0, s["table"][b][at // page].long(), :, at % page] = \
                    x[start[b]:start[b] + n].double()
        return pools
    if c["kind"] == "append":
        back = s["back"].double()
        scales = s["scale_k"].double(), s["scale_v"].double()
        for b, n in enumerate(new):
            at = torch.arange(pos[b], pos[b] + n, device="cuda")
            pg, pl = s["table"][b][at // page].long(), at % page
            for j, x in enumerate((s["k"], s["v"])):
                x = x[start[b]:start[b] + n].double()
                step = x.abs().amax(-1) / 127.0
                step = torch.where(step * 127.0 < TINY_AMAX, 1.0, step)
                scales[j][0, pg, :, pl] = step
                back[j, start[b]:start[b] + n] = torch.round(x / step[..., None]) * step[..., None]
        return back, scales[0], scales[1]
    out = s["o"].double()
    group = c["hq"] // c["hkv"]
    for b, n in enumerate(new):
        keys = pos[b] + n
        pages = s["table"][b, :-(-keys // page)].long()
        late = torch.arange(keys, device="cuda")[None] > torch.arange(pos[b], keys, device="cuda")[:, None]
        for h in range(c["hkv"]):
            k, v = s["pool_k"][0, pages, h].double(), s["pool_v"][0, pages, h].double()
            if c["bits"] == 8:
                k = (k - 128.0) * s["scale_k"][0, pages, h].double()[..., None]
                v = (v - 128.0) * s["scale_v"][0, pages, h].double()[..., None]
            k, v = k.reshape(-1, c["d"])[:keys], v.reshape(-1, c["d"])[:keys]
            for j in range(h * group, (h + 1) * group):
                z = s["q"][start[b]:start[b] + n, j].double() @ k.T / c["d"] ** 0.5
                out[start[b]:start[b] + n, j] = torch.softmax(z.masked_fill(late, -torch.inf), -1) @ v
    return out
