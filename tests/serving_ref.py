"""64-bit definitions of the rotary, paged-cache and window operators, written from the
formulas, with element-wise error bounds from the arithmetic the kernels may use.

Roundings counted: a value stored in bf16 is off by at most 2^-8 of itself; a softmax weight
or score gradient rounded to bf16 as a product operand by 2^-8 of itself; an FP32 sum of n
products by n 2^-24 of the sum of their magnitudes.
"""
import math

import torch

U16 = 2.0 ** -8     # half a bf16 step, relative
U32 = 2.0 ** -24    # half an fp32 step, relative


def rotate(x, pos, inv_freq, layout, start, amplitude, transpose=False):
    """(rotated x in 64 bits, bound on a bf16 result's error); x [T, H, D]."""
    y = x.double().clone()
    mag = y.abs()
    n = inv_freq.numel()
    a = pos.double()[:, None] * inv_freq.double()[None]
    c, s = torch.cos(a)[:, None] * amplitude, torch.sin(a)[:, None] * (-amplitude if transpose else amplitude)
    i = torch.arange(n)
    i1, i2 = (start + i, start + n + i) if layout == "half" else (start + 2 * i, start + 2 * i + 1)
    u, w = x.double()[..., i1], x.double()[..., i2]
    y[..., i1], y[..., i2] = u * c - w * s, w * c + u * s
    mag[..., i1] = mag[..., i2] = (u.abs() + w.abs()) * abs(amplitude)
    # cosine and sine in FP32 (an argument rounded at 2^-25 half turns, a few steps of the
    # function, one each for amplitude, products and sum): within 8 steps of 2^-24
    return y, U16 * y.abs() + 16 * U32 * mag


def cache_rows(cache, page_table, b, n):
    """The first n rows [n, H, D] of sequence b (64-bit)."""
    page = cache.shape[1]
    at = torch.arange(n)
    return cache[page_table[b, at // page].long(), at % page].double()


def _attend(q, k, v, scale):
    """One query [Hkv, G, Dq] over rows k [n, Hkv, Dq], v [n, Hkv, Dv]:
    out, lse and their bounds."""
    x = torch.einsum("hgd,nhd->hgn", q, k) * scale
    mag = torch.einsum("hgd,nhd->hgn", q.abs(), k.abs()).amax(-1) * scale
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[..., None])
    out = torch.einsum("hgn,nhd->hgd", p, v)
    dx = (q.shape[-1] + 4) * U32 * mag                      # error of a score
    spread = torch.einsum("hgn,nhd->hgd", p, v.abs())
    # an exponential is off by its argument's error and 2^-21; the weight by 2^-8 more as an operand
    rel = 2 * dx + 2.0 ** -21 + U16 + (k.shape[0] + 4) * U32
    return out, lse, U16 * out.abs() + rel[..., None] * spread, dx + 2.0 ** -21 * (1 + lse.abs()) + (k.shape[0] + 8) * U32


def decode(q, k_cache, v_cache, page_table, lens, scale, window=0, sinks=0, routes=None):
    """(out, lse, bound of out, bound of lse) of one new token per sequence; CPU tensors."""
    B, Hq, Dq = q.shape
    Hkv, Dv = k_cache.shape[2], v_cache.shape[3]
    out, bo = torch.zeros(B, Hq, Dv, dtype=torch.float64), torch.zeros(B, Hq, Dv, dtype=torch.float64)
    lse, bl = torch.full((B, Hq), -math.inf, dtype=torch.float64), torch.zeros(B, Hq, dtype=torch.float64)
    page = k_cache.shape[1]
    for b in range(B):
        n = int(lens[b])
        if window == 0 and routes is None:
            at = list(range(n))
        else:
            seen = set(range(min(sinks, n)))
            if window:
                seen |= set(range(max(0, n - window), n))
            if routes is not None:
                seen |= {int(r) for r in routes[b] if 0 <= r < n}
            at = sorted(seen)
        at = [p for p in at if 0 <= int(page_table[b, p // page]) < k_cache.shape[0]]
        if not at:
            continue
        i = torch.tensor(at)
        pg = page_table[b, i // page].long()
        o, l, eo, el = _attend(q[b].double().view(Hkv, Hq // Hkv, Dq), k_cache[pg, i % page].double(),
                               v_cache[pg, i % page].double(), scale)
        out[b], lse[b], bo[b], bl[b] = o.reshape(Hq, Dv), l.reshape(Hq), eo.reshape(Hq, Dv), el.reshape(Hq)
    return out, lse, bo, bl


def window_mask(cu, T, window, sinks):
    """[T, T] truth values: query t sees key s."""
    t = torch.arange(T)
    doc = torch.bucketize(t, cu[1:].long(), right=True)
    start = cu.long()[doc]
    s = t[None]
    q = t[:, None]
    return (doc[:, None] == doc[None]) & (s <= q) & ((s > q - window) | (s < (start + sinks)[:, None]))


def window_fwd(q, k, v, cu, window, sinks, scale):
    """(out, lse, bound of out, bound of lse); masked rows may hold anything."""
    T, Hq, Dq = q.shape
    Hkv, Dv = k.shape[1], v.shape[2]
    G = Hq // Hkv
    seen = window_mask(cu, T, window, sinks)
    out, bo = torch.zeros(T, Hq, Dv, dtype=torch.float64), torch.zeros(T, Hq, Dv, dtype=torch.float64)
    lse, bl = torch.zeros(T, Hq, dtype=torch.float64), torch.zeros(T, Hq, dtype=torch.float64)
    for t in range(T):
        at = seen[t].nonzero()[:, 0]
        o, l, eo, el = _attend(q[t].double().view(Hkv, G, Dq), k[at].double(), v[at].double(), scale)
        out[t], lse[t], bo[t], bl[t] = o.reshape(Hq, Dv), l.reshape(Hq), eo.reshape(Hq, Dv), el.reshape(Hq)
    return out, lse, bo, bl


def window_bwd(q, k, v, cu, window, sinks, scale, out, lse, dout):
    """(dq, dk, dv) from the forward's (rounded) out and lse as given, and a bound of each."""
    T, Hq, Dq = q.shape
    Hkv, Dv = k.shape[1], v.shape[2]
    G = Hq // Hkv
    seen = window_mask(cu, T, window, sinks)
    f = lambda x: x.double().view(T, Hkv, -1, x.shape[-1])  # noqa: E731
    qd, dd, od = f(q), f(dout), f(out)
    kd, vd = k.double(), v.double()
    x = torch.einsum("thgd,shd->hgts", qd, kd) * scale
    mag = torch.einsum("thgd,shd->hgts", qd.abs(), kd.abs()) * scale
    p = torch.where(seen, torch.exp(x - lse.double().view(T, Hkv, G).permute(1, 2, 0)[..., None]), 0.0)
    D = (dd * od).sum(-1).permute(1, 2, 0)[..., None]
    y = torch.einsum("thgd,shd->hgts", dd, vd) - D
    ymag = torch.einsum("thgd,shd->hgts", dd.abs(), vd.abs()) + (dd.abs() * od.abs()).sum(-1).permute(1, 2, 0)[..., None]
    ds = p * y
    # a weight: its score's error (and the given lse's last bits) in the exponent, 2^-21 of the exponential
    ep = p * ((Dq + 4) * U32 * mag + 2.0 ** -21 + 4 * U32 * lse.abs().double().view(T, Hkv, G).permute(1, 2, 0)[..., None])
    eds = ep * y.abs() + p * (Dv + 4) * U32 * ymag + U16 * ds.abs()
    ep = ep + U16 * p
    got = {}
    for name, w, e, a, eq, n in (("dq", ds * scale, eds * scale, kd, "hgts,shd->thgd", T),
                                 ("dk", ds * scale, eds * scale, qd, "hgts,thgd->shd", T * G),
                                 ("dv", p, ep, dd, "hgts,thgd->shd", T * G)):
        r = torch.einsum(eq, w, a)
        e = torch.einsum(eq, e + 64 * U32 * w.abs(), a.abs())   # FP32 sums by blocks: far below 64 steps a term
        shape = (T, Hq, Dq) if name == "dq" else r.shape
        got[name] = (r.reshape(shape), (U16 * r.abs() + e).reshape(shape) + 1e-30)
    return got


def window_loss_grads(q, k, v, cu, window, sinks, scale, dout):
    """(loss sum(out * dout), its gradients) by autograd in 64 bits; all float64 inputs."""
    q, k, v = (a.detach().clone().requires_grad_(True) for a in (q, k, v))
    T, Hq, _ = q.shape
    G = Hq // k.shape[1]
    x = torch.einsum("thd,shd->hts", q, k.repeat_interleave(G, 1)) * scale
    x = x.masked_fill(~window_mask(cu, T, window, sinks), -math.inf)
    out = torch.einsum("hts,shd->thd", torch.softmax(x, -1), v.repeat_interleave(G, 1))
    loss = (out * dout).sum()
    return loss.detach(), torch.autograd.grad(loss, (q, k, v))


def check(got, ref, bound, what):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    over = ((got - ref).abs() - bound)[~inf]
    if over.numel():
        assert not torch.isnan(over).any(), f"{what}: NaN"
        assert over.max() <= 0, f"{what}: an element is {over.max():.3e} past its bound"
