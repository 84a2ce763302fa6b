"""Serving requests that share a long prefix, over the paged cache, as cases to measure.

Three operators, each in a plain form (elementary torch operations) and as the package's calls:

* `paged_plan`: a step's page tables, token positions and slots in the pool, from the
  requests' lengths and a list of free pages;
* `shared_prefix_gqa_attn_fwd`: prompt tokens of many requests over the prefix that their
  group shares, joined with the attention over their own tokens;
* `shared_prefix_gqa_attn_decode`: one new token per sequence over its group's prefix and its
  own positions; the prefix is read once a group.
"""
import math
import random

import torch

own = False


def _dev():
    return torch.device("cuda", torch.cuda.current_device()) if torch.cuda.is_available() else torch.device("cpu")


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def listed():
    return [
        # one decoding step of a batch of unrelated requests: now and then one needs a page; latency counts
        dict(name="plan step 64", kind="plan", B=64, new_lo=1, new_hi=1, len_lo=1, len_hi=8192, page=64, groups=0,
             prefix=0, pad=0),
        # samples of a few prompts, admitted in one step: their tables take the prompts' pages; the batch is padded
        dict(name="plan shared 480", kind="plan", B=480, new_lo=1, new_hi=40, len_lo=1, len_hi=3000, page=16, groups=7,
             prefix=20000, pad=61),
        # a step that takes in whole documents, a page a token
        dict(name="plan prompts", kind="plan", B=48, new_lo=2000, new_hi=60000, len_lo=1, len_hi=4000, page=1, groups=0,
             prefix=0, pad=1000),
        # two short questions behind a cached prompt: latency counts
        dict(name="prompt short", kind="fwd", rows="77", prefix="4099", Hq=8, Hkv=2, Dqk=128, Dv=128, page=64,
             heads_first=False, joined=True, pad=0),
        # a prefill step: questions to three documents of ragged lengths
        dict(name="prompts of three", kind="fwd", rows="1500, 333, 2267", prefix="8000, 2051, 5003", Hq=32, Hkv=8,
             Dqk=128, Dv=128, page=64, heads_first=False, joined=True, pad=0),
        # a prefill step of many requests behind one long prompt, key rows wider than value rows; pages by heads
        dict(name="prompts long", kind="fwd", rows="8192", prefix="16384", Hq=64, Hkv=4, Dqk=192, Dv=128, page=16,
             heads_first=True, joined=True, pad=0),
        # the prefix part alone, from a cache that is kept by tokens
        dict(name="prompts by tokens", kind="fwd", rows="900, 0, 451", prefix="7001, 500, 12001", Hq=32, Hkv=8,
             Dqk=128, Dv=128, page=1, heads_first=False, joined=False, pad=13),
        # a few samples of one prompt: latency counts
        dict(name="decode samples 8", kind="decode", rows="8", prefix="2000", own_lo=1, own_hi=300, Hq=32, Hkv=8,
             Dqk=128, Dv=128, page=16, heads_first=False, idle=0),
        # a serving batch behind one system prompt
        dict(name="decode shared 128", kind="decode", rows="128", prefix="8192", own_lo=100, own_hi=4000, Hq=32, Hkv=8,
             Dqk=128, Dv=128, page=16, heads_first=False, idle=0),
        # groups of ragged sizes and prefixes, one of them a single sequence, idle slots among them
        dict(name="decode groups", kind="decode", rows="20, 1, 33, 8, 34", prefix="30000, 9001, 16007, 2501, 6000",
             own_lo=1, own_hi=900, Hq=64, Hkv=4, Dqk=192, Dv=128, page=64, heads_first=True, idle=5),
        # a long document under many questions
        dict(name="decode long 32", kind="decode", rows="32", prefix="120011", own_lo=30, own_hi=600, Hq=64, Hkv=8,
             Dqk=128, Dv=128, page=64, heads_first=False, idle=0),
        # many samples of one prompt, narrow heads, a cache that is kept by tokens
        dict(name="decode by tokens", kind="decode", rows="256", prefix="5001", own_lo=1, own_hi=2000, Hq=16, Hkv=2,
             Dqk=64, Dv=64, page=1, heads_first=False, idle=0),
    ]


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _text(numbers):
    return ", ".join(str(n) for n in numbers)


def _numbers(text):
    return [int(n) for n in text.split(",")]


def draw(rng):
    kind = rng.choice(["plan", "fwd", "fwd", "decode", "decode"])
    page = rng.choice([1, 16, 48, 64, 128])
    if kind == "plan":
        B = _between(rng, 1, 512)
        hi = _between(rng, 1, max(1, 600000 // B))
        return dict(kind="plan", B=B, new_lo=rng.randint(0, hi), new_hi=hi, len_lo=1, len_hi=_between(rng, 1, 8000),
                    page=page, groups=rng.choice([0, 1, min(B, 5)]),
                    prefix=_between(rng, 1, min(20000, 1000000 * page // B)), pad=rng.choice([0, rng.randint(1, 500)]))
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = min(Hkv * rng.choice([1, 2, 3, 4, 8, 16]), 64 // Hkv * Hkv)
    Dqk, Dv = rng.choice([(64, 64), (128, 128), (192, 128), (128, 64)])
    heads = dict(Hq=Hq, Hkv=Hkv, Dqk=Dqk, Dv=Dv, page=page, heads_first=rng.choice([False, True]))
    groups = rng.choice([1, 1, 2, 3, 7])
    if kind == "fwd":
        rows = [rng.choice([0, _between(rng, 1, 8192 // groups), _between(rng, 1, 8192 // groups)]) for _ in range(groups)]
        rows[rng.randrange(groups)] = _between(rng, 1, 8192 // groups)
        most = max(64, 16384 * 8192 // max(1, 2 * sum(rows)))
        return dict(kind="fwd", rows=_text(rows), prefix=_text(_between(rng, 1, min(40000, most)) for _ in rows),
                    joined=rng.choice([True, True, False]), pad=rng.choice([0, 0, 9]), **heads)
    rows = [_between(rng, 1, 192 // groups) for _ in range(groups)]
    hi = _between(rng, 1, max(1, 300000 // sum(rows)))
    return dict(kind="decode", rows=_text(rows), prefix=_text(_between(rng, 1, 100000 // groups) for _ in rows),
                own_lo=rng.randint(1, hi), own_hi=hi, idle=rng.choice([0, 0, sum(rows) // 8]), **heads)


def _spread(n, lo, hi, salt):
    """n ragged numbers of [lo, hi], both ends among them where n allows: the case's own, not the seed's."""
    rng = random.Random(n * 1000003 + lo * 1009 + hi * 31 + salt)
    got = [hi, lo] + [_between(rng, lo, hi) if lo > 0 and hi > 16 * lo else rng.randint(lo, hi) for _ in range(n)]
    return got[:n]


def _cumulated(n):
    got = [0]
    for x in n:
        got.append(got[-1] + x)
    return got


def _plan_sizes(c):
    """(lengths before, new tokens, group borders, prefix lengths) of a plan case. A group's first sequence holds its
    prefix; the others come with it cached and own what follows its last whole page."""
    before, new = _spread(c["B"], c["len_lo"], c["len_hi"], 1), _spread(c["B"], c["new_lo"], c["new_hi"], 2)
    random.Random(c["B"]).shuffle(new)
    if not c["groups"]:
        return before, new, None, None
    rng = random.Random(c["B"] * 31 + c["groups"])
    cuts = [0] + sorted(rng.randint(0, c["B"]) for _ in range(c["groups"] - 1)) + [c["B"]]
    prefix = _spread(c["groups"], 1, c["prefix"], 3)
    for g, n in enumerate(prefix):
        for b in range(cuts[g], cuts[g + 1]):
            before[b] += n
    return before, new, cuts, prefix


def _own_lengths(c):
    """Own positions of each sequence of a decode case (None: an idle slot)."""
    own_n = _spread(sum(_numbers(c["rows"])), c["own_lo"], c["own_hi"], 4)
    random.Random(len(own_n)).shuffle(own_n)
    for i in range(c["idle"]):
        own_n[(i * 7 + 3) % len(own_n)] = None
    first = 0
    for n in _numbers(c["rows"]):   # a group's first sequence, whose table the prefix is read by, is not idle
        if n and own_n[first] is None:
            own_n[first] = 1
        first += n
    return own_n


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=g.device, dtype=torch.float32).to(torch.bfloat16)


def _cache(g, c, pages, D):
    """A pool [pages, page, Hkv, D]; heads_first: a view of one that is laid out [pages, Hkv, page, D]."""
    p, h = c["page"], c["Hkv"]
    t = torch.empty((pages, h, p, D) if c["heads_first"] else (pages, p, h, D), dtype=torch.bfloat16, device=g.device)
    t.normal_(generator=g)
    return t.transpose(1, 2) if c["heads_first"] else t


def _ints(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _pages(n, page):
    return -(-n // page)


def prepare(case, seed):
    c, dev = case, _dev()
    g = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": c}
    page = c["page"]
    if c["kind"] == "plan":
        before, new, cuts, prefix = _plan_sizes(c)
        held = [_pages(n, page) for n in before]
        need = [_pages(n + m, page) - h for n, m, h in zip(before, new, held)]
        shared = [0] * c["B"]
        if cuts:
            for i, n in enumerate(prefix):
                for b in range(cuts[i] + 1, cuts[i + 1]):
                    shared[b] = n // page
        total = sum(held) - sum(shared) + sum(need) + 5
        order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
        width = max(h + m for h, m in zip(held, need)) + 1
        table = torch.full((c["B"], width), -1, dtype=torch.int32, device=dev)
        at = 0
        for b in range(c["B"]):   # the pages that sequences hold themselves
            n = held[b] - shared[b]
            table[b, shared[b]: held[b]] = order[at: at + n]
            at += n
        s["page_table"], s["free_pages"] = table, order[at:].contiguous()
        s["free_count"] = _ints([total - at], dev)
        s["cache_lens"], s["new_lens"] = _ints(before, dev), _ints(new, dev)
        s["cu_groups"] = None if cuts is None else _ints(cuts, dev)
        s["prefix_lens"] = None if cuts is None else _ints(prefix, dev)
        s["tokens"] = sum(new) + c["pad"]
        return s
    if c["kind"] == "fwd":
        T = sum(_numbers(c["rows"])) + c["pad"]
        s["q"] = _normal(g, T, c["Hq"], c["Dqk"])
        s["cu_rows"] = _ints(_cumulated(_numbers(c["rows"])), dev)
        need = [_pages(n, page) for n in _numbers(c["prefix"])]
        s["own_out"] = s["own_lse"] = None
        if c["joined"]:   # the attention over a token's own prompt: a mean of a few to a few thousand values
            s["own_lse"] = torch.rand(T, c["Hq"], generator=g, device=dev) * 9.0
            s["own_out"] = (torch.randn(T, c["Hq"], c["Dv"], generator=g, device=dev)
                            * torch.exp(-0.5 * s["own_lse"])[..., None]).to(torch.bfloat16)
        s["out"] = torch.zeros(T, c["Hq"], c["Dv"], dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.zeros(T, c["Hq"], dtype=torch.float32, device=dev)
    else:
        own_n = _own_lengths(c)
        B = len(own_n)
        s["q"] = _normal(g, B, c["Hq"], c["Dqk"])
        s["cu_groups"] = _ints(_cumulated(_numbers(c["rows"])), dev)
        prefix = [n for n, m in zip(_numbers(c["prefix"]), _numbers(c["rows"])) for _ in range(m)]
        lens = [0 if m is None else n + m for n, m in zip(prefix, own_n)]
        s["cache_lens"] = _ints(lens, dev)
        need = [_pages(n, page) for n in lens]
    s["prefix_lens"] = _ints(_numbers(c["prefix"]), dev)
    first, lead = 0, [0] * len(need)
    if c["kind"] == "decode":   # a group's first sequence holds all its pages, the others none of the prefix's whole ones
        lead = [min(n, m // page) for n, m in zip(need, prefix)]
        for b in _cumulated(_numbers(c["rows"]))[:-1]:
            lead[b] = 0
    total = sum(need) - sum(lead)
    order = torch.randperm(total + 3, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(len(need), max(need), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        if lead[b] == 0 and n:
            first = b if c["kind"] == "fwd" or b in _cumulated(_numbers(c["rows"])) else first
        table[b, : lead[b]] = table[first, : lead[b]]
        table[b, lead[b]: n] = order[at: at + n - lead[b]]
        at += n - lead[b]
    s["page_table"] = table
    s["k_cache"], s["v_cache"] = _cache(g, c, total + 3, c["Dqk"]), _cache(g, c, total + 3, c["Dv"])
    if c["kind"] == "decode":   # the page that a prefix fills in part: each sequence has its copy
        cu = _cumulated(_numbers(c["rows"]))
        for a, z, n in zip(cu, cu[1:], _numbers(c["prefix"])):
            rest, mine = n % page, [b for b in range(a + 1, z) if lens[b]]
            if rest and mine:
                for x in (s["k_cache"], s["v_cache"]):
                    x[table[mine, n // page].long(), :rest] = x[int(table[a, n // page]), :rest]
    return s


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------
def run(state):
    if own:
        return _framework(state)
    return {"plan": _plan_plain, "fwd": _fwd_plain, "decode": _decode_plain}[state["case"]["kind"]](state)


def _framework(s):
    import indexer_routed_sparse_gb300 as irs

    c = s["case"]
    if c["kind"] == "plan":
        p = irs.paged_plan(s["cache_lens"], s["new_lens"], s["page_table"], s["free_pages"], s["free_count"], c["page"],
                           s["tokens"], cu_groups=s["cu_groups"], prefix_lens=s["prefix_lens"])
        return {"page_table": s["page_table"], "cu_new": p.cu_new, "positions": p.positions, "slots": p.slots,
                "lens": p.cache_lens, "free": p.free_count}
    if c["kind"] == "fwd":
        joined = None if s["own_out"] is None else (s["own_out"], s["own_lse"])
        out, lse = irs.shared_prefix_gqa_attn_fwd(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["cu_rows"],
                                                  s["prefix_lens"], own=joined, out=s["out"], lse=s["lse"])
        return {"out": out, "lse": lse}
    out, lse = irs.shared_prefix_gqa_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["cache_lens"],
                                                 s["cu_groups"], s["prefix_lens"])
    return {"out": out, "lse": lse}


def _plan_plain(s):
    c = s["case"]
    page, table, T = c["page"], s["page_table"], s["tokens"]
    n, m = s["cache_lens"].long(), s["new_lens"].long()
    B, width, dev = n.numel(), table.shape[1], n.device
    held = (n + page - 1) // page
    need = (n + m + page - 1) // page - held
    upto = need.cumsum(0)
    j = torch.arange(width, device=dev)[None]
    taken = s["free_count"].long() - 1 - (upto - need)[:, None] - (j - held[:, None])
    fresh = (j >= held[:, None]) & (j < (held + need)[:, None])
    got = torch.where(fresh, s["free_pages"][taken.clamp(0, s["free_pages"].numel() - 1)], table)
    if s["cu_groups"] is not None:
        cu = s["cu_groups"].long()
        b = torch.arange(B, device=dev)
        g = torch.searchsorted(cu[1:], b, right=True)
        shared = torch.where(b > cu[g], s["prefix_lens"].long()[g] // page, torch.zeros_like(b))
        got = torch.where(j < shared[:, None], got[cu[g]], got)
    table.copy_(got)
    cu_new = torch.cat((torch.zeros_like(m[:1]), m.cumsum(0)))
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(cu_new[1:], t, right=True)
    live = b < B
    b = b.clamp(max=B - 1)
    pos = n[b] + t - cu_new[b]
    slot = table[b, (pos // page).clamp(max=width - 1)].long() * page + pos % page
    gone = torch.full_like(pos, -1)
    return {"page_table": table, "cu_new": cu_new.to(torch.int32), "positions": torch.where(live, pos, gone).to(torch.int32),
            "slots": torch.where(live, slot, gone), "lens": (n + m).to(torch.int32),
            "free": (s["free_count"].long() - upto[-1:]).to(torch.int32)}


def _prefix_plain(s, q, row, n):
    """Rows q [R, Hq, Dqk] over the first n positions of a page table's row: (out, lse) in 32 bits, rows in pieces so that
    the scores stay below 4 GB."""
    c = s["case"]
    Hq, Hkv, page = c["Hq"], c["Hkv"], c["page"]
    G = Hq // Hkv
    at = torch.arange(n, device=q.device)
    pg = row.long()[at // page]
    k, v = (x[pg, at % page].float().transpose(0, 1) for x in (s["k_cache"], s["v_cache"]))   # [Hkv, n, D]
    piece = max(1, (1 << 30) // (Hq * n))
    outs, lses = [], []
    for i in range(0, q.shape[0], piece):
        x = q[i: i + piece].float()
        r = x.shape[0]
        x = x.view(r, Hkv, G, -1).transpose(0, 1).reshape(Hkv, r * G, -1)
        x = torch.matmul(x, k.transpose(1, 2)) * (1.0 / math.sqrt(c["Dqk"]))
        m = x.amax(-1, keepdim=True)
        e = torch.exp_(x.sub_(m))
        z = e.sum(-1, keepdim=True)
        o = torch.matmul(e, v) / z
        outs.append(o.view(Hkv, r, G, -1).transpose(0, 1).reshape(r, Hq, -1))
        lses.append((m + torch.log(z)).view(Hkv, r, G).transpose(0, 1).reshape(r, Hq))
    return torch.cat(outs), torch.cat(lses)


def _join_plain(a, la, b, lb):
    m = torch.maximum(la, lb)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x, y = torch.exp(la - m), torch.exp(lb - m)
    z = x + y
    out = (a * x[..., None] + b * y[..., None]) / torch.where(z == 0, torch.ones_like(z), z)[..., None]
    return out, m + torch.log(z)


def _fwd_plain(s):
    c = s["case"]
    cu = _cumulated(_numbers(c["rows"]))
    for g, n in enumerate(_numbers(c["prefix"])):
        a, b = cu[g], cu[g + 1]
        if a == b:
            continue
        o, l = _prefix_plain(s, s["q"][a:b], s["page_table"][g], n)
        if c["joined"]:
            o, l = _join_plain(o, l, s["own_out"][a:b].float(), s["own_lse"][a:b])
        s["out"][a:b] = o.to(torch.bfloat16)
        s["lse"][a:b] = l
    return {"out": s["out"], "lse": s["lse"]}


def _decode_plain(s):
    """The prefixes group by group; then every sequence's own positions, padded to the longest."""
    c = s["case"]
    B, Hq, Hkv, page = sum(_numbers(c["rows"])), c["Hq"], c["Hkv"], c["page"]
    cu = _cumulated(_numbers(c["rows"]))
    parts = [_prefix_plain(s, s["q"][a:b], s["page_table"][a], n) for a, b, n in zip(cu, cu[1:], _numbers(c["prefix"]))]
    o, l = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
    L = s["cache_lens"].long()
    first = torch.repeat_interleave(s["prefix_lens"].long(), s["cu_groups"].long().diff(), output_size=B)
    idle = (L == 0)[:, None]
    o, l = torch.where(idle[..., None], torch.zeros_like(o), o), torch.where(idle, torch.full_like(l, -math.inf), l)
    at = first[:, None] + torch.arange(c["own_hi"], device=L.device)[None]
    ok = at < L[:, None]
    at = torch.where(ok, at, torch.zeros_like(at))
    row = s["page_table"].long().gather(1, at // page)
    q = s["q"].float().view(B, Hkv, Hq // Hkv, c["Dqk"])
    k = s["k_cache"][row, at % page].permute(0, 2, 3, 1).float()
    x = torch.matmul(q, k) * (1.0 / math.sqrt(c["Dqk"]))
    del k
    x = torch.where(ok[:, None, None], x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    v = s["v_cache"][row, at % page].permute(0, 2, 1, 3).float()
    mine = torch.matmul(e, v) / torch.where(z == 0, torch.ones_like(z), z)
    o, l = _join_plain(o, l, mine.reshape(B, Hq, -1), (m + torch.log(z)).reshape(B, Hq))
    return {"out": o.to(torch.bfloat16), "lse": l}


# ---------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["kind"] == "plan":
        before, new, cuts, prefix = _plan_sizes(c)
        need = sum(_pages(n + m, c["page"]) - _pages(n, c["page"]) for n, m in zip(before, new))
        T, B = sum(new), c["B"]
        shared = 0 if cuts is None else sum(max(0, b - a - 1) * (n // c["page"]) for a, b, n in zip(cuts, cuts[1:], prefix))
        return {"bytes": 16 * B + 8 * need + 4 * shared + 12 * (T + c["pad"]), "flops": B + T}
    d = c["Dqk"] + c["Dv"]
    T = sum(_numbers(c["rows"]))
    pairs = sum(r * n for r, n in zip(_numbers(c["rows"]), _numbers(c["prefix"])))
    held = sum(n for r, n in zip(_numbers(c["rows"]), _numbers(c["prefix"])) if r)
    moved = 2 * T * c["Hq"] * (d + 2)
    if c["kind"] == "fwd":
        moved += 2 * T * c["Hq"] * (c["Dv"] + 2) if c["joined"] else 0
    else:
        own_n = sum(n or 0 for n in _own_lengths(c))
        pairs, held = pairs + own_n, held + own_n
    return {"bytes": 2 * held * c["Hkv"] * d + 4 * held // c["page"] + moved, "flops": 2 * pairs * c["Hq"] * d}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _plan_exact, "fwd": _fwd_exact, "decode": _decode_exact}[case["kind"]](s)


def _plan_exact(s):
    """Request after request, as an allocator on the host would."""
    c = s["case"]
    page, dev = c["page"], s["cache_lens"].device
    before, new, cuts, prefix = _plan_sizes(c)
    free = s["free_pages"].tolist()
    table = s["page_table"].tolist()
    positions, slots, cu = [], [], [0]
    for b, (n, m) in enumerate(zip(before, new)):
        for j in range(_pages(n, page), _pages(n + m, page)):
            table[b][j] = free.pop()
        positions += range(n, n + m)
        cu.append(cu[-1] + m)
    if cuts:
        for a, z, n in zip(cuts, cuts[1:], prefix):
            for b in range(a + 1, z):
                table[b][: n // page] = table[a][: n // page]
    for row, n, m in zip(table, before, new):
        slots += [row[i // page] * page + i % page for i in range(n, n + m)]
    behind = [-1] * (s["tokens"] - len(slots))
    return {"page_table": _ints(table, dev), "cu_new": _ints(cu, dev), "positions": _ints(positions + behind, dev),
            "slots": torch.tensor(slots + behind, dtype=torch.int64, device=dev),
            "lens": _ints([n + m for n, m in zip(before, new)], dev), "free": _ints([len(free)], dev)}


def _rows_exact(s, q, tables, n, more=None):
    """softmax(q k) v of rows q [R, Hq, D] over n positions of a table's row, and `more` = (k, v) [Hkv, m, D] behind them."""
    c = s["case"]
    Hkv, G = c["Hkv"], c["Hq"] // c["Hkv"]
    at = torch.arange(n, device=q.device)
    k, v = (torch.stack([x[tables.long()[at // c["page"]], at % c["page"], h].double() for h in range(Hkv)])
            for x in (s["k_cache"], s["v_cache"]))
    if more is not None:
        k, v = torch.cat((k, more[0]), 1), torch.cat((v, more[1]), 1)
    out = torch.zeros(q.shape[0], c["Hq"], c["Dv"], dtype=torch.float64, device=q.device)
    lse = torch.zeros(q.shape[0], c["Hq"], dtype=torch.float64, device=q.device)
    piece = max(1, (1 << 28) // (G * k.shape[1]))
    for h in range(Hkv):
        for i in range(0, q.shape[0], piece):
            x = torch.einsum("rgd,kd->rgk", q[i: i + piece, h * G: (h + 1) * G].double(), k[h]) / math.sqrt(c["Dqk"])
            lse[i: i + piece, h * G: (h + 1) * G] = torch.logsumexp(x, -1)
            out[i: i + piece, h * G: (h + 1) * G] = torch.einsum("rgk,kd->rgd", torch.softmax(x, -1), v[h])
    return out, lse


def _fwd_exact(s):
    c = s["case"]
    out, lse = s["out"].double(), s["lse"].double()
    a = 0
    for g, r in enumerate(_numbers(c["rows"])):
        if r:
            o, l = _rows_exact(s, s["q"][a: a + r], s["page_table"][g], _numbers(c["prefix"])[g])
            if c["joined"]:
                both = torch.logaddexp(l, s["own_lse"][a: a + r].double())
                o = o * torch.exp(l - both)[..., None]
                o = o + s["own_out"][a: a + r].double() * torch.exp(s["own_lse"][a: a + r].double() - both)[..., None]
                l = both
            out[a: a + r], lse[a: a + r] = o, l
        a += r
    return {"out": out, "lse": lse}


def _decode_exact(s):
    """Every sequence over its own table, position after position, as if nothing were shared."""
    c = s["case"]
    dev = s["q"].device
    B, G = sum(_numbers(c["rows"])), c["Hq"] // c["Hkv"]
    out = torch.zeros(B, c["Hq"], c["Dv"], dtype=torch.float64, device=dev)
    lse = torch.full((B, c["Hq"]), -math.inf, dtype=torch.float64, device=dev)
    for b, n in enumerate(s["cache_lens"].tolist()):
        if n == 0:
            continue
        at = torch.arange(n, device=dev)
        pg = s["page_table"][b].long()[at // c["page"]]
        k, v = (x[pg, at % c["page"]].double() for x in (s["k_cache"], s["v_cache"]))
        x = torch.einsum("hgd,khd->hgk", s["q"][b].double().view(c["Hkv"], G, -1), k) / math.sqrt(c["Dqk"])
        out[b] = torch.einsum("hgk,khd->hgd", torch.softmax(x, -1), v).reshape(c["Hq"], -1)
        lse[b] = torch.logsumexp(x, -1).reshape(-1)
    return {"out": out, "lse": lse}
