"""64-bit definitions of the page plan and of shared-prefix attention, written from the formulas, with
element-wise error bounds from the arithmetic the kernels may use.

Roundings counted, as in serving_ref: a value stored in bf16 is off by at most 2^-8 of itself, a softmax
weight rounded to bf16 as a product operand by 2^-8, an FP32 sum of n products by n 2^-24 of the sum of their
magnitudes, an approximate exponential by 2^-21. Tensors may lie on any device.
"""
import math

import torch

U16 = 2.0 ** -8
U32 = 2.0 ** -24


def plan(lens, new, table, free, count, page, tokens, groups=None, prefix=None):
    """(table, cu_new, positions, slots, lens, free left, whether anything was refused): an allocator on the host."""
    table = [list(r) for r in table]
    B, width = len(lens), len(table[0])
    new = [0 if n < 0 or m < 0 or n + m > width * page else m for n, m in zip(lens, new)]
    bad = [n < 0 or n > width * page for n in lens]
    count = min(max(count, 0), len(free))
    held = [0 if x else -(-n // page) for n, x in zip(lens, bad)]
    need = [0 if x else -(-(n + m) // page) - h for n, m, h, x in zip(lens, new, held, bad)]
    cu, positions, slots, after, left, asked, ok = [0], [], [], [], count, 0, []
    for b in range(B):
        asked += need[b]
        ok.append(need[b] == 0 or asked <= count)
        for i in range(need[b]):
            table[b][held[b] + i] = free[count - 1 - (asked - need[b]) - i] if ok[b] else -1
        if ok[b]:
            left = left if need[b] == 0 else count - asked
        after.append(lens[b] + new[b] if ok[b] else lens[b])
        cu.append(cu[-1] + new[b])
    if groups:
        for a, z, n in zip(groups, groups[1:], prefix):
            for b in range(a + 1, z):
                if 0 < n <= lens[b] and not bad[b]:
                    for j in range(min(n // page, held[a] + need[a])):
                        table[b][j] = table[a][j]
    for b in range(B):
        for p in range(lens[b], lens[b] + new[b]):
            pg = table[b][p // page]
            positions.append(p)
            slots.append(pg * page + p % page if ok[b] and pg >= 0 else -1)
    pad = [-1] * max(0, tokens - len(positions))
    return table, cu, (positions + pad)[:tokens], (slots + pad)[:tokens], after, left


def rows(cache, row, at):
    """Rows [n, H, D] of the positions `at` through a page table's row, in 64 bits."""
    page = cache.shape[1]
    return cache[row[at // page].long(), at % page].double()


def attend(q, k, v, scale):
    """Rows q [r, Hq, D] over k [n, Hkv, D], v [n, Hkv, Dv]: (out, lse, bounds)."""
    r, Hq, D = q.shape
    n, Hkv, Dv = v.shape
    if n == 0:
        z = torch.zeros(r, Hq, Dv, dtype=torch.float64, device=q.device)
        l = torch.full((r, Hq), -math.inf, dtype=torch.float64, device=q.device)
        return z, l, z.clone(), torch.zeros_like(l)
    qd = q.double().view(r, Hkv, Hq // Hkv, D)
    x = torch.einsum("rhgd,nhd->rhgn", qd, k) * scale
    mag = torch.einsum("rhgd,nhd->rhgn", qd.abs(), k.abs()).amax(-1) * scale
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[..., None])
    out = torch.einsum("rhgn,nhd->rhgd", p, v)
    spread = torch.einsum("rhgn,nhd->rhgd", p, v.abs())
    dx = (D + 4) * U32 * mag
    rel = 2 * dx + 2.0 ** -21 + U16 + (n + 4) * U32
    el = dx + 2.0 ** -21 * (1 + lse.abs()) + (n + 8) * U32
    return (out.reshape(r, Hq, Dv), lse.reshape(r, Hq), (U16 * out.abs() + rel[..., None] * spread).reshape(r, Hq, Dv),
            el.reshape(r, Hq))


def join(a, b):
    """Two parts (out, lse, bound, bound) of the same rows as one. A part's weight is off by its lse's error and by
    two approximate exponentials and a quotient: under 2^-20 (1 + |lse|) more; the result is rounded to bf16."""
    oa, la, ea, fa = a
    ob, lb, eb, fb = b
    lse = torch.logaddexp(la, lb)
    none = torch.isinf(lse) & (lse < 0)
    wa = torch.where(torch.isinf(la) & (la < 0), 0.0, torch.exp(la - lse))[..., None]
    wb = torch.where(torch.isinf(lb) & (lb < 0), 0.0, torch.exp(lb - lse))[..., None]
    oa, ob = torch.where(wa == 0, 0.0, oa), torch.where(wb == 0, 0.0, ob)
    out = torch.where(none[..., None], 0.0, wa * oa + wb * ob)
    big = torch.where(torch.isinf(la), 0.0, la.abs()) + torch.where(torch.isinf(lb), 0.0, lb.abs())
    f = fa + fb + 2.0 ** -20 * (1 + big)
    bound = U16 * out.abs() + wa * ea + wb * eb + 2 * f[..., None] * (wa * oa.abs() + wb * ob.abs())
    return out, lse, bound, f


def fwd(q, kc, vc, table, cu, prefix, scale, own=None):
    """(out, lse, bounds) of the rows of all groups, [cu[-1], ...]."""
    got = []
    for g, n in enumerate(prefix):
        x = q[cu[g]: cu[g + 1]]
        at = torch.arange(n, device=q.device)
        part = attend(x, rows(kc, table[g], at), rows(vc, table[g], at), scale)
        if own is not None:
            o, l = (y[cu[g]: cu[g + 1]].double() for y in own)
            part = join(part, (o, l, torch.zeros_like(o), torch.zeros_like(l)))
        got.append(part)
    return tuple(torch.cat([p[i] for p in got]) for i in range(4))


def decode(q, kc, vc, table, lens, cu, prefix, scale):
    """(out, lse, bounds): every sequence over its group's prefix and its own positions."""
    shared = [None] * q.shape[0]
    for g, n in enumerate(prefix):
        for b in range(cu[g], cu[g + 1]):
            shared[b] = (cu[g], n)
    got = []
    for b, L in enumerate(lens):
        first, n = shared[b] or (b, 0)
        L = 0 if L < n or L > table.shape[1] * kc.shape[1] else L
        n = min(n, L)
        at = torch.arange(L, device=q.device)
        k, v = (torch.cat((rows(c, table[first], at[:n]), rows(c, table[b], at[n:]))) for c in (kc, vc))
        o, l, eo, el = attend(q[b: b + 1], k, v, scale)
        # joined from parts: their weights are off by 2^-20 (1 + |lse|) at most
        more = 2.0 ** -20 * (1 + torch.where(torch.isinf(l), 0.0, l.abs()))
        spread = torch.zeros_like(o) if L == 0 else v.abs().amax(0).repeat_interleave(q.shape[1] // v.shape[1], 0)[None]
        got.append((o, l, eo + 2 * more[..., None] * spread, el + more))
    return tuple(torch.cat([p[i] for p in got]) for i in range(4))


def check(got, ref, bound, what):
    got = got.detach().to(ref.device).double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    over = ((got - ref).abs() - bound)[~inf]
    if over.numel():
        assert not torch.isnan(over).any(), f"{what}: NaN"
        assert over.max() <= 0, f"{what}: an element is {over.max():.3e} past its bound"
