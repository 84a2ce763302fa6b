"""The serving and training operators next to the routed attention, as cases to measure.

Three families, each in a plain form (elementary torch operations) and as the package's calls:

* rotary positions: `rope` on its own (and its transpose, the gradient) and
  `paged_rope_append`, which rotates new queries and keys and writes keys and values into
  the pages of a cache;
* `paged_gqa_attn_decode`: attention of one new token per sequence over a paged cache: the
  whole prefix, a window with the first tokens, or routed positions;
* `window_gqa_attn_fwd` / `window_gqa_attn_bwd`: attention of packed documents over a
  sliding window and the documents' first tokens, and its gradients.
"""
import math
import random

import torch

own = False

TWO_PI = 2.0 * math.pi


def _dev():
    return torch.device("cuda", torch.cuda.current_device()) if torch.cuda.is_available() else torch.device("cpu")


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def listed():
    return [
        # one decoding step of a batch: every sequence's new token is rotated and appended; latency counts
        dict(name="append step 64", kind="append", B=64, new_lo=1, new_hi=1, len_hi=8192, Hq=32, Hkv=8, Dqk=128, Dv=128,
             rope=128, start=0, layout="half", factor=1.0, page=64),
        # ragged prompts with a part of each head rotated, pairs interleaved, positions far behind the trained length
        dict(name="append prompts scaled", kind="append", B=9, new_lo=300, new_hi=2500, len_hi=900000, Hq=64, Hkv=4,
             Dqk=192, Dv=128, rope=64, start=128, layout="interleaved", factor=16.0, page=16),
        # the gradient of the queries' rotation in a training step
        dict(name="rope gradient", kind="rope", T=16384, H=64, D=128, rope=128, start=0, layout="half", factor=1.0,
             len_hi=16384, transpose=True),
        # one user's step over a medium cache: too few (sequence, head) pairs to fill the GPU without a split
        dict(name="decode one", kind="decode", B=1, len_lo=4099, len_hi=4099, Hq=32, Hkv=8, Dqk=128, Dv=128, page=64,
             window=0, sinks=0, W=0),
        # a full serving batch of ragged lengths; the cache's offsets pass 32 bits
        dict(name="decode ragged 64", kind="decode", B=64, len_lo=20000, len_hi=50000, Hq=64, Hkv=8, Dqk=128, Dv=128, page=64,
             window=0, sinks=0, W=0),
        # two long contexts, small pages, key rows wider than value rows
        dict(name="decode long 2", kind="decode", B=2, len_lo=150001, len_hi=300007, Hq=64, Hkv=4, Dqk=192, Dv=128, page=16,
             window=0, sinks=0, W=0),
        # a windowed layer's step: the last 512 tokens and the first four
        dict(name="decode window sinks", kind="decode", B=128, len_lo=33, len_hi=9000, Hq=64, Hkv=4, Dqk=192, Dv=128,
             page=16, window=512, sinks=4, W=0),
        # a routed layer's step: the positions that an indexer kept (budget 2048, blocks of 4)
        dict(name="decode routed", kind="decode", B=96, len_lo=2500, len_hi=16000, Hq=32, Hkv=8, Dqk=128, Dv=128, page=64,
             window=0, sinks=0, W=2051),
        # a short ragged prompt: latency counts
        dict(name="window small", kind="window", T=333, docs=3, Hq=8, Hkv=2, Dqk=128, Dv=128, window=100, sinks=4,
             train=False),
        # a prompt batch of windowed layers at the workload's head shape
        dict(name="window prompt", kind="window", T=65536, docs=7, Hq=64, Hkv=4, Dqk=192, Dv=128, window=512, sinks=4,
             train=False),
        # a training step's attention, one sequence, no first tokens
        dict(name="window train mid", kind="window", T=8192, docs=1, Hq=32, Hkv=8, Dqk=128, Dv=128, window=1024, sinks=0,
             train=True),
        # a training step's attention over packed documents with first tokens
        dict(name="window train packed", kind="window", T=32768, docs=11, Hq=64, Hkv=4, Dqk=192, Dv=128, window=512,
             sinks=4, train=True),
    ]


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["append", "rope", "decode", "decode", "window", "window"])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8, 16])
    Hq = min(Hq, 64 // Hkv * Hkv)
    Dqk, Dv = rng.choice([(64, 64), (128, 128), (192, 128), (128, 64)])
    if kind == "rope":
        rope = rng.choice([d for d in (16, 32, 64, 128, 192) if d <= Dqk])
        return dict(kind="rope", T=_between(rng, 1, 16384), H=Hq, D=Dqk, rope=rope, start=rng.choice([0, Dqk - rope]),
                    layout=rng.choice(["half", "interleaved"]), factor=rng.choice([1.0, 4.0, 32.0]),
                    len_hi=_between(rng, 2048, 2000000), transpose=rng.choice([False, True]))
    if kind == "append":
        rope = rng.choice([d for d in (16, 32, 64, 128, 192) if d <= Dqk])
        B = _between(rng, 1, 128)
        hi = _between(rng, 1, max(1, 12000 // B))
        return dict(kind="append", B=B, new_lo=rng.randint(1, hi), new_hi=hi, len_hi=_between(rng, 100, 1000000), Hq=Hq,
                    Hkv=Hkv, Dqk=Dqk, Dv=Dv, rope=rope, start=rng.choice([0, Dqk - rope]),
                    layout=rng.choice(["half", "interleaved"]), factor=rng.choice([1.0, 8.0]),
                    page=rng.choice([1, 16, 48, 64, 128]))
    if kind == "decode":
        B = _between(rng, 1, 128)
        hi = _between(rng, 20, max(20, min(200000, 600000 // B)))
        lo = rng.randint(1, hi)
        mode = rng.choice(["all", "window", "routes", "both"])
        return dict(kind="decode", B=B, len_lo=lo, len_hi=hi, Hq=Hq, Hkv=Hkv, Dqk=Dqk, Dv=Dv,
                    page=rng.choice([1, 16, 48, 64, 128]), window=rng.randint(1, 2000) if mode in ("window", "both") else 0,
                    sinks=rng.choice([0, 1, 4, 30]) if mode in ("window", "both") else 0,
                    W=rng.randint(1, 3000) if mode in ("routes", "both") else 0)
    train = rng.choice([False, True])
    T = _between(rng, 48 if train else 1, 16384)
    return dict(kind="window", T=T, docs=min(-(-T // 3), rng.choice([1, 1, 2, 5, 17])), Hq=Hq, Hkv=Hkv, Dqk=Dqk, Dv=Dv,
                window=_between(rng, 4, 1500), sinks=rng.choice([0, 0, 1, 4, 16]), train=train)


def _spread(n, lo, hi, salt):
    """n ragged lengths of [lo, hi], both ends among them where n allows: the case's own, not the seed's."""
    rng = random.Random(n * 1000003 + lo * 1009 + hi * 31 + salt)
    got = [hi, lo] + [_between(rng, lo, hi) if hi > 16 * lo else rng.randint(lo, hi) for _ in range(n)]
    return got[:n]


def _documents(c):
    """Document lengths: `docs` of them that add up to T, ragged."""
    T, n = c["T"], c["docs"]
    rng = random.Random(T * 7919 + n)
    cuts = sorted(rng.sample(range(1, T), n - 1)) if n > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [T])]


def _new_counts(c):
    return _spread(c["B"], c["new_lo"], c["new_hi"], 1)


def _lengths(c):
    return _spread(c["B"], c["len_lo"], c["len_hi"], 2)


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _inv_freq(c, device):
    """Radians per token of each rotated pair, in 64 bits, and the rotation's amplitude: base 10000; a factor over 1
    stretches the pairs that turn less than once (none of those that turn 32 times) over the trained length, 8192."""
    n = c["rope"] // 2
    f = 10000.0 ** (-torch.arange(n, dtype=torch.float64, device=device) / n)
    if c["factor"] == 1.0:
        return f, 1.0
    turns = 8192.0 * f / TWO_PI
    keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
    return f * (keep + (1.0 - keep) / c["factor"]), 0.1 * math.log(c["factor"]) + 1.0


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=g.device, dtype=torch.float32).to(torch.bfloat16)


def _cache(g, pages, page, H, D):
    t = torch.empty(pages, page, H, D, dtype=torch.bfloat16, device=g.device)
    return t.normal_(generator=g)


def prepare(case, seed):
    c, dev = case, _dev()
    g = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": c}
    if c["kind"] == "rope":
        s["inv_freq"], s["amplitude"] = _inv_freq(c, dev)
        s["x"] = _normal(g, c["T"], c["H"], c["D"])
        s["positions"] = torch.randint(0, c["len_hi"], (c["T"],), generator=g, device=dev, dtype=torch.int32)
    elif c["kind"] == "append":
        s["inv_freq"], s["amplitude"] = _inv_freq(c, dev)
        new = _new_counts(c)
        T, page = sum(new), c["page"]
        before = [int(x) for x in torch.randint(0, c["len_hi"], (c["B"],), generator=g, device=dev).tolist()]
        s["q"], s["k"], s["v"] = (_normal(g, T, h, d) for h, d in ((c["Hq"], c["Dqk"]), (c["Hkv"], c["Dqk"]), (c["Hkv"], c["Dv"])))
        # the pool holds the pages that the new tokens fall in; the older pages of each sequence are not this call's
        need = [((a + n - 1) // page) - a // page + 1 for a, n in zip(before, new)]
        pool = sum((n + page - 2) // page + 1 for n in new)
        order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
        table = torch.full((c["B"], (c["len_hi"] + c["new_hi"] - 2) // page + 1), -1, dtype=torch.int32, device=dev)
        at = 0
        for b, (a, n) in enumerate(zip(before, need)):
            table[b, a // page: a // page + n] = order[at: at + n]
            at += n
        s["page_table"] = table
        s["k_cache"] = _cache(g, pool, page, c["Hkv"], c["Dqk"])
        s["v_cache"] = _cache(g, pool, page, c["Hkv"], c["Dv"])
        s["cache_lens"] = torch.tensor(before, dtype=torch.int32, device=dev)
        s["cu_new"] = torch.tensor([0] + new, dtype=torch.int32, device=dev).cumsum(0).to(torch.int32)
    elif c["kind"] == "decode":
        lens, page = _lengths(c), c["page"]
        need = [(n + page - 1) // page for n in lens]
        order = torch.randperm(sum(need) + 3, generator=g, device=dev).to(torch.int32)
        table = torch.zeros(c["B"], max(need), dtype=torch.int32, device=dev)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at: at + n]
            at += n
        s["page_table"] = table
        s["cache_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["q"] = _normal(g, c["B"], c["Hq"], c["Dqk"])
        s["k_cache"] = _cache(g, sum(need) + 3, page, c["Hkv"], c["Dqk"])
        s["v_cache"] = _cache(g, sum(need) + 3, page, c["Hkv"], c["Dv"])
        s["route_ids"] = None
        if c["W"]:
            # distinct positions in ascending order: one of each stretch of the sequence; what is left over is -1
            n = s["cache_lens"][:, None].double()
            j = torch.arange(c["W"], device=dev)[None].double()
            kept = torch.clamp(n, max=float(c["W"]))
            lo, hi = torch.floor(j * n / kept), torch.floor((j + 1) * n / kept)
            r = lo + torch.floor(torch.rand(c["B"], c["W"], generator=g, device=dev, dtype=torch.float64) * (hi - lo))
            s["route_ids"] = torch.where(j < kept, torch.minimum(r, n - 1), -torch.ones_like(r)).to(torch.int32)
    else:
        T = c["T"]
        s["q"], s["k"], s["v"] = (_normal(g, T, h, d) for h, d in ((c["Hq"], c["Dqk"]), (c["Hkv"], c["Dqk"]), (c["Hkv"], c["Dv"])))
        s["cu_seqlens"] = torch.tensor([0] + _documents(c), dtype=torch.int32, device=dev).cumsum(0).to(torch.int32)
        if c["train"]:
            s["dout"] = _normal(g, T, c["Hq"], c["Dv"])
    return s


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------
def run(state):
    c = state["case"]
    if own:
        return _framework(state)
    return {"rope": _rope_plain, "append": _append_plain, "decode": _decode_plain, "window": _window_plain}[c["kind"]](state)


def _framework(s):
    import indexer_routed_sparse_gb300 as irs

    c = s["case"]
    if c["kind"] == "rope":
        return {"out": irs.rope(s["x"], s["positions"], s["inv_freq"], layout=c["layout"], start=c["start"],
                                amplitude=s["amplitude"], transpose=c["transpose"])}
    if c["kind"] == "append":
        q = irs.paged_rope_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["cache_lens"],
                                  s["inv_freq"], cu_new=s["cu_new"], layout=c["layout"], start=c["start"],
                                  amplitude=s["amplitude"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if c["kind"] == "decode":
        out, lse = irs.paged_gqa_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["cache_lens"],
                                             window=c["window"], sinks=c["sinks"], route_ids=s["route_ids"])
        return {"out": out, "lse": lse}
    out, lse = irs.window_gqa_attn_fwd(s["q"], s["k"], s["v"], s["cu_seqlens"], c["window"], sinks=c["sinks"])
    if not c["train"]:
        return {"out": out, "lse": lse}
    dq, dk, dv = irs.window_gqa_attn_bwd(s["q"], s["k"], s["v"], s["cu_seqlens"], c["window"], out, lse, s["dout"],
                                         sinks=c["sinks"])
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _rotate_plain(x, positions, inv_freq, c, amplitude, transpose=False):
    """x [T, H, D] rotated: the angles in 64 bits, the products in 32."""
    angle = positions.double()[:, None] * inv_freq[None]
    cos = (torch.cos(angle) * amplitude).float()[:, None]
    sin = (torch.sin(angle) * (-amplitude if transpose else amplitude)).float()[:, None]
    a, n = c["start"], c["rope"]
    y = x.float()
    z = y[..., a: a + n]
    if c["layout"] == "half":
        u, w = z[..., : n // 2], z[..., n // 2:]
        z = torch.cat((u * cos - w * sin, w * cos + u * sin), dim=-1)
    else:
        u, w = z[..., 0::2], z[..., 1::2]
        z = torch.stack((u * cos - w * sin, w * cos + u * sin), dim=-1).flatten(-2)
    return torch.cat((y[..., :a], z, y[..., a + n:]), dim=-1).to(x.dtype)


def _rope_plain(s):
    return {"out": _rotate_plain(s["x"], s["positions"], s["inv_freq"], s["case"], s["amplitude"], s["case"]["transpose"])}


def _append_plain(s):
    c = s["case"]
    T = s["q"].shape[0]
    i = torch.arange(T, device=s["q"].device)
    b = torch.searchsorted(s["cu_new"][1:].long(), i, right=True)
    pos = s["cache_lens"].long()[b] + i - s["cu_new"].long()[b]
    page, off = s["page_table"].long()[b, pos // c["page"]], pos % c["page"]
    q = _rotate_plain(s["q"], pos, s["inv_freq"], c, s["amplitude"])
    s["k_cache"][page, off] = _rotate_plain(s["k"], pos, s["inv_freq"], c, s["amplitude"])
    s["v_cache"][page, off] = s["v"]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _positions_plain(s):
    """Positions that each sequence's new token attends, [B, n], and which of them count."""
    c, L = s["case"], s["cache_lens"].long()[:, None]
    dev = L.device
    n = s["page_table"].shape[1] * c["page"]
    if not c["window"] and not c["W"]:
        at = torch.arange(n, device=dev)[None].expand(L.shape[0], -1)
        return at, at < L
    first = (L - c["window"]).clamp(min=0) if c["window"] else L
    recent = first + torch.arange(c["window"], device=dev)[None]
    early = torch.arange(c["sinks"], device=dev)[None].expand(L.shape[0], -1)
    at, ok = [early, recent], [early < first, recent < L]
    if c["W"]:
        r = s["route_ids"].long()
        at.append(r)
        ok.append((r >= c["sinks"]) & (r < first))
    return torch.cat(at, 1), torch.cat(ok, 1)


def _decode_plain(s):
    c = s["case"]
    B, Hq, Hkv = c["B"], c["Hq"], c["Hkv"]
    at, ok = _positions_plain(s)
    at = torch.where(ok, at, torch.zeros_like(at))
    row = s["page_table"].long().gather(1, at // c["page"]) * c["page"] + at % c["page"]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, c["Dqk"])
    k = s["k_cache"].flatten(0, 1)[row].permute(0, 2, 3, 1).float()
    x = torch.matmul(q, k) * (1.0 / math.sqrt(c["Dqk"]))
    del k
    x = torch.where(ok[:, None, None], x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    v = s["v_cache"].flatten(0, 1)[row].permute(0, 2, 1, 3).float()
    out = torch.matmul(e, v) / z
    return {"out": out.reshape(B, Hq, c["Dv"]).to(torch.bfloat16), "lse": (m + torch.log(z)).reshape(B, Hq)}


def _window_plain(s):
    """Blocks of `window` queries against their own and the previous block's keys, and every query against the first
    tokens of its document that lie before its window."""
    c = s["case"]
    T, Hq, Hkv, w, ns = c["T"], c["Hq"], c["Hkv"], c["window"], c["sinks"]
    G, scale, dev = Hq // Hkv, 1.0 / math.sqrt(c["Dqk"]), s["q"].device
    blk = min(w, T)
    n = -(-T // blk)
    cu = s["cu_seqlens"].long()
    t = torch.arange(n * blk, device=dev)
    doc = torch.searchsorted(cu[1:], t, right=True)
    start = cu[doc.clamp(max=cu.numel() - 2)]

    def blocks(x):  # [n, H, blk, D]
        x = torch.cat((x.float(), torch.zeros(n * blk - T, *x.shape[1:], device=dev)))
        return x.view(n, blk, *x.shape[1:]).transpose(1, 2)

    def queries(x):  # [n, Hkv, G * blk, D]
        return blocks(x).reshape(n, Hkv, G * blk, x.shape[-1])

    def pairs(x):  # [n, H, 2 * blk, D]: the previous block, then the own one
        x = blocks(x)
        return torch.cat((torch.cat((torch.zeros_like(x[:1]), x[:-1])), x), dim=2)

    tq = t.view(n, blk, 1)
    tk = torch.cat((tq - blk, tq), dim=1).transpose(1, 2)
    seen = ((tk <= tq) & (tk > tq - w) & (tk >= start.view(n, blk, 1)) & (tq < T)) | ((tq >= T) & (tk == tq))
    seen = seen[:, None, None]  # [n, 1, 1, blk, 2 * blk]
    q, k, v = queries(s["q"]), pairs(s["k"]), pairs(s["v"])
    x = (torch.matmul(q, k.transpose(2, 3)) * scale).view(n, Hkv, G, blk, 2 * blk)
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    first = start[:, None] + torch.arange(ns, device=dev)[None]
    early = (first < (t - w + 1)[:, None]) & (t < T)[:, None]
    first = torch.where(early, first, torch.zeros_like(first))
    early = early.view(n, 1, 1, blk, ns)
    # [n, Hkv, G, blk, D] queries against [n, Hkv, 1, blk, ns, D] first tokens
    ks, vs = (y[first].float().view(n, blk, ns, Hkv, y.shape[-1]).permute(0, 3, 1, 2, 4)[:, :, None] for y in (s["k"], s["v"]))
    qe = q.view(n, Hkv, G, blk, -1)
    y = torch.matmul(ks, qe[..., None])[..., 0] * scale
    y = torch.where(early, y, torch.full_like(y, -math.inf))
    m = x.amax(-1, keepdim=True)
    m = torch.maximum(m, y.amax(-1, keepdim=True)) if ns else m
    p, e = torch.exp(x - m), torch.exp(y - m)
    del x, y
    z = p.sum(-1, keepdim=True) + e.sum(-1, keepdim=True)
    p, e = p.div_(z), e.div_(z)
    flat = (n, Hkv, G * blk, 2 * blk)
    out = torch.matmul(p.view(flat), v).view(n, Hkv, G, blk, -1) + torch.matmul(e[..., None, :], vs)[..., 0, :]

    def tokens(a):  # [n, Hkv, G, blk, D] -> [T, Hq, D]
        return a.permute(0, 3, 1, 2, 4).reshape(n * blk, Hq, -1)[:T]

    got = {"out": tokens(out).to(torch.bfloat16), "lse": tokens(m + torch.log(z))[..., 0].contiguous()}
    if not c["train"]:
        return got
    do = queries(s["dout"])
    de = do.view(n, Hkv, G, blk, -1)
    dp = torch.matmul(do, v.transpose(2, 3)).view(p.shape)
    dy = torch.matmul(vs, de[..., None])[..., 0]
    mean = (p * dp).sum(-1, keepdim=True) + (e * dy).sum(-1, keepdim=True)
    ds, dy = dp.sub_(mean).mul_(p).mul_(scale), e * (dy - mean) * scale
    dq = torch.matmul(ds.view(flat), k).view(n, Hkv, G, blk, -1) + torch.matmul(dy[..., None, :], ks)[..., 0, :]

    def keys(a, late):  # gradients of the pairs [n, Hkv, 2 * blk, D] and of the first tokens [n, Hkv, blk, ns, D]
        a = a[:, :, blk:] + torch.cat((a[1:, :, :blk], torch.zeros_like(a[:1, :, :blk])))
        a = a.transpose(1, 2).reshape(n * blk, Hkv, -1)[:T]
        if not ns:
            return a
        late = late.permute(0, 2, 3, 1, 4).reshape(n * blk, -1)
        own_doc = (doc[None] == torch.arange(cu.numel() - 1, device=dev)[:, None]).float()
        late = torch.matmul(own_doc, late).view(cu.numel() - 1, ns, Hkv, -1)
        at = cu[:-1, None] + torch.arange(ns, device=dev)[None]
        inside = at < cu[1:, None]
        return a.index_put((at[inside],), late[inside], accumulate=True)

    dk = keys(torch.matmul(ds.view(flat).transpose(2, 3), q), torch.matmul(dy.permute(0, 1, 3, 4, 2), qe.transpose(2, 3)) if ns else None)
    dv = keys(torch.matmul(p.view(flat).transpose(2, 3), do), torch.matmul(e.permute(0, 1, 3, 4, 2), de.transpose(2, 3)) if ns else None)
    got.update(dq=tokens(dq).to(torch.bfloat16), dk=dk.to(torch.bfloat16), dv=dv.to(torch.bfloat16))
    return got


# ---------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------
def _attended(c):
    """Keys that each sequence's new token attends (a routed position inside the window or the first tokens counts once)."""
    total = 0
    for n in _lengths(c):
        if not c["window"] and not c["W"]:
            total += n
            continue
        first = max(0, n - c["window"]) if c["window"] else n
        early = min(c["sinks"], first)
        between = first - early
        total += n - first + early + (min(c["W"], n) * between // n if c["W"] else 0)
    return total


def _window_pairs(c):
    """(query, key) pairs of the documents, each with its window and the first tokens before it."""
    total, w = 0, c["window"]
    for n in _documents(c):
        full = max(0, n - w)
        m = n - full
        total += m * (m + 1) // 2 + full * w
        # query i >= w sees min(sinks, i - w + 1) first tokens before its window
        k = min(c["sinks"], full)
        total += k * (k + 1) // 2 + (full - k) * k if k else 0
    return total


def work(case):
    c = case
    if c["kind"] == "rope":
        return {"bytes": 4 * c["T"] * c["H"] * c["D"] + 4 * c["T"], "flops": 3 * c["T"] * c["H"] * c["rope"]}
    if c["kind"] == "append":
        T = sum(_new_counts(c))
        return {"bytes": 4 * T * (c["Hq"] * c["Dqk"] + c["Hkv"] * (c["Dqk"] + c["Dv"])),
                "flops": 3 * T * (c["Hq"] + c["Hkv"]) * c["rope"]}
    if c["kind"] == "decode":
        n = _attended(c)
        return {"bytes": 2 * n * c["Hkv"] * (c["Dqk"] + c["Dv"]) + 4 * n // c["page"] + 4 * c["B"] * c["W"]
                + 2 * c["B"] * c["Hq"] * (c["Dqk"] + c["Dv"] + 2),
                "flops": 2 * n * c["Hq"] * (c["Dqk"] + c["Dv"])}
    n, d = _window_pairs(c), c["Dqk"] + c["Dv"]
    moved = 2 * c["T"] * (c["Hq"] + c["Hkv"]) * d + 4 * c["T"] * c["Hq"]
    if not c["train"]:
        return {"bytes": moved, "flops": 2 * n * c["Hq"] * d}
    return {"bytes": 2 * moved, "flops": 6 * n * c["Hq"] * d}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _rope_exact, "append": _append_exact, "decode": _decode_exact, "window": _window_exact}[case["kind"]](s)


def _turn(x, pos, s, transpose=False):
    """Rotation as a product of complex numbers."""
    c = s["case"]
    y = x.double().clone()
    a, n = c["start"], c["rope"]
    if c["layout"] == "half":
        i = torch.arange(a, a + n // 2, device=x.device)
        j = i + n // 2
    else:
        i = torch.arange(a, a + n, 2, device=x.device)
        j = i + 1
    angle = (pos.double()[:, None] * s["inv_freq"])[:, None]
    turn = torch.polar(torch.full_like(angle, s["amplitude"]), -angle if transpose else angle)
    z = torch.complex(y[..., i], y[..., j]) * turn
    y[..., i], y[..., j] = z.real, z.imag
    return y


def _rope_exact(s):
    return {"out": _turn(s["x"], s["positions"], s, s["case"]["transpose"])}


def _append_exact(s):
    c = s["case"]
    new = _new_counts(c)
    before = s["cache_lens"].tolist()
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    pos = torch.cat([torch.arange(a, a + n, device=kc.device) for a, n in zip(before, new)])
    seq = torch.cat([torch.full((n,), b, device=kc.device) for b, n in enumerate(new)])
    slot = s["page_table"][seq, pos // c["page"]].long() * c["page"] + pos % c["page"]
    kc.flatten(0, 1)[slot] = _turn(s["k"], pos, s)
    vc.flatten(0, 1)[slot] = s["v"].double()
    return {"q": _turn(s["q"], pos, s), "k_cache": kc, "v_cache": vc}


def _decode_exact(s):
    c = s["case"]
    G, dev = c["Hq"] // c["Hkv"], s["q"].device
    out = torch.empty(c["B"], c["Hq"], c["Dv"], dtype=torch.float64, device=dev)
    lse = torch.empty(c["B"], c["Hq"], dtype=torch.float64, device=dev)
    routes = None if s["route_ids"] is None else s["route_ids"].tolist()
    for b, n in enumerate(_lengths(c)):
        seen = set() if c["window"] or c["W"] else None
        if seen is None:
            at = torch.arange(n, device=dev)
        else:
            if c["window"]:
                seen |= set(range(max(0, n - c["window"]), n))
            seen |= set(range(min(c["sinks"], n)))
            if c["W"]:
                seen |= {r for r in routes[b] if 0 <= r < n}
            at = torch.tensor(sorted(seen), device=dev)
        page = s["page_table"][b].long()[at // c["page"]]
        k, v = (x[page, at % c["page"]].double() for x in (s["k_cache"], s["v_cache"]))
        q = s["q"][b].double().view(c["Hkv"], G, c["Dqk"])
        x = torch.einsum("hgd,khd->hgk", q, k) / math.sqrt(c["Dqk"])
        out[b] = torch.einsum("hgk,khd->hgd", torch.softmax(x, -1), v).reshape(c["Hq"], c["Dv"])
        lse[b] = torch.logsumexp(x, -1).reshape(-1)
    return {"out": out, "lse": lse}


def _window_exact(s):
    """Document by document, a stretch of queries at a time, over the keys that the stretch can see."""
    c = s["case"]
    if c["T"] * c["Hq"] > 1 << 21 and not c["train"]:
        rows = 1024
    else:
        rows = 256
    G, scale, dev, w, ns = c["Hq"] // c["Hkv"], 1.0 / math.sqrt(c["Dqk"]), s["q"].device, c["window"], c["sinks"]
    zeros = lambda x: torch.zeros(x.shape, dtype=torch.float64, device=dev)  # noqa: E731
    out = torch.zeros(c["T"], c["Hq"], c["Dv"], dtype=torch.float64, device=dev)
    lse = torch.zeros(c["T"], c["Hq"], dtype=torch.float64, device=dev)
    dq, dk, dv = zeros(s["q"]), zeros(s["k"]), zeros(s["v"])
    a = 0
    for n in _documents(c):
        for i in range(0, n, rows):
            i1 = min(n, i + rows)
            lo = max(0, i - w + 1)
            at = torch.cat((torch.arange(min(ns, lo), device=dev), torch.arange(lo, i1, device=dev)))
            t = torch.arange(i, i1, device=dev)[:, None]
            seen = (at[None] <= t) & ((at[None] > t - w) | (at[None] < ns))
            q = s["q"][a + i: a + i1].double().view(i1 - i, c["Hkv"], G, -1).permute(1, 2, 0, 3)
            k, v = (x[a + at].double().transpose(0, 1)[:, None] for x in (s["k"], s["v"]))
            x = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, -math.inf)
            lse[a + i: a + i1] = torch.logsumexp(x, -1).permute(2, 0, 1).reshape(i1 - i, -1)
            p = torch.softmax(x, -1)
            o = torch.matmul(p, v)
            out[a + i: a + i1] = o.permute(2, 0, 1, 3).reshape(i1 - i, c["Hq"], -1)
            if c["train"]:
                do = s["dout"][a + i: a + i1].double().view(i1 - i, c["Hkv"], G, -1).permute(1, 2, 0, 3)
                g = (torch.matmul(do, v.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
                dq[a + i: a + i1] = torch.matmul(g, k).permute(2, 0, 1, 3).reshape(i1 - i, c["Hq"], -1)
                dk[a + at] += torch.matmul(g.transpose(-1, -2), q).sum(1).transpose(0, 1)
                dv[a + at] += torch.matmul(p.transpose(-1, -2), do).sum(1).transpose(0, 1)
        a += n
    got = {"out": out, "lse": lse}
    if c["train"]:
        got.update(dq=dq, dk=dk, dv=dv)
    return got
