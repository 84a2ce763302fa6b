"""Attention over a sliding window and the documents' first tokens, forward and backward, on
the GPU (through the C ABI), against the 64-bit definition."""
import math

import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module")
def irs():
    import indexer_routed_sparse_gb300 as m

    m.lib()
    return m


def _inputs(T, Hq, Hkv, Dqk, Dv, docs, seed=0):
    g = torch.Generator().manual_seed(seed + T + Hq)
    n = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    cu = torch.tensor([0] + docs).cumsum(0).to(torch.int32)
    assert int(cu[-1]) == T
    return n(T, Hq, Dqk), n(T, Hkv, Dqk), n(T, Hkv, Dv), n(T, Hq, Dv), cu


def _case(irs, q, k, v, do, cu, window, sinks, scale=None, gpu=None):
    scale = 1 / math.sqrt(q.shape[2]) if scale is None else scale
    ref = R.window_fwd(q, k, v, cu, window, sinks, scale)
    qd, kd, vd = gpu if gpu is not None else (q.to(DEV), k.to(DEV), v.to(DEV))
    cd, dd = cu.to(DEV), do.to(DEV)
    out, lse = irs.window_gqa_attn_fwd(qd, kd, vd, cd, window, scale, sinks=sinks)
    irs.check_device_errors(DEV)
    R.check(out, ref[0], ref[2], "out")
    R.check(lse, ref[1], ref[3], "lse")
    got = irs.window_gqa_attn_bwd(qd, kd, vd, cd, window, out, lse, dd, scale, sinks=sinks)
    irs.check_device_errors(DEV)
    want = R.window_bwd(q, k, v, cu, window, sinks, scale, out.cpu(), lse.cpu(), do)
    for name, t in zip(("dq", "dk", "dv"), got):
        R.check(t, *want[name], name)
    again = irs.window_gqa_attn_fwd(qd, kd, vd, cd, window, scale, sinks=sinks)
    grads = irs.window_gqa_attn_bwd(qd, kd, vd, cd, window, out, lse, dd, scale, sinks=sinks)
    assert all(torch.equal(a, b) for a, b in zip((out, lse) + tuple(got), tuple(again) + tuple(grads)))
    return out, lse, got


@pytest.mark.parametrize("Hq,Hkv,Dqk,Dv", [(1, 1, 64, 64), (8, 2, 128, 128), (6, 2, 192, 128), (3, 3, 128, 64),
                                           (16, 1, 192, 128), (5, 1, 64, 128), (32, 2, 192, 64), (40, 1, 128, 128)])
def test_head_shapes(irs, Hq, Hkv, Dqk, Dv):
    _case(irs, *_inputs(203, Hq, Hkv, Dqk, Dv, [90, 1, 112]), window=37, sinks=3)


@pytest.mark.parametrize("docs", [[1], [2], [63], [64], [65], [127, 1], [128, 129], [1] * 40, [500], [3, 400, 7, 90]])
def test_document_lengths(irs, docs):
    _case(irs, *_inputs(sum(docs), 4, 2, 128, 128, docs), window=50, sinks=4)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 128), (16, 0), (64, 5), (100, 64), (128, 0), (200, 128),
                                          (299, 1), (300, 4), (5000, 4), (1 << 30, 0)])
def test_windows_and_first_tokens(irs, window, sinks):
    _case(irs, *_inputs(420, 4, 2, 128, 128, [120, 300]), window=window, sinks=sinks)


@pytest.mark.parametrize("Dqk,Dv", [(64, 64), (64, 128), (128, 64), (192, 64), (192, 128)])
@pytest.mark.parametrize("window,sinks", [(3, 128), (40, 97), (250, 33)])
def test_many_first_tokens(irs, Dqk, Dv, window, sinks):
    """More first tokens than one block of keys holds, at every pair of head dims."""
    _case(irs, *_inputs(420, 6, 2, Dqk, Dv, [110, 10, 300]), window=window, sinks=sinks)


def test_long_document_with_first_tokens(irs):
    """First tokens seen by thousands of queries: their gradients are sums over all of them."""
    _case(irs, *_inputs(1500, 8, 1, 64, 64, [1490, 10]), window=64, sinks=4)


def test_strides_and_broadcast_heads(irs):
    q, k, v, do, cu = _inputs(150, 8, 2, 128, 128, [100, 50])
    big = torch.zeros(150, 14, 256, dtype=torch.bfloat16, device=DEV)   # one packed tensor of all heads
    big[:, :8, :128], big[:, 8:10, 64:192], big[:, 11:13, 128:] = q.to(DEV), k.to(DEV), v.to(DEV)
    _case(irs, q, k, v, do, cu, 40, 2, gpu=(big[:, :8, :128], big[:, 8:10, 64:192], big[:, 11:13, 128:]))
    hm = tuple(t.to(DEV).transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v))   # head-major rows
    _case(irs, q, k, v, do, cu, 40, 2, gpu=hm)
    one_k, one_v = k[:, :1].expand(150, 2, 128), v[:, :1].expand(150, 2, 128)   # stride 0 over the heads
    _case(irs, q, one_k, one_v, do, cu, 40, 2, gpu=(q.to(DEV), k.to(DEV)[:, :1].expand(150, 2, 128),
                                                    v.to(DEV)[:, :1].expand(150, 2, 128)))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_masked_rows_may_hold_anything(irs, bad):
    """A key, value or output gradient reaches only the rows that see it: all others are within
    their bounds of the definition on clean inputs."""
    T, docs, window, sinks = 330, [130, 90, 110], 30, 2
    q, k, v, do, cu = _inputs(T, 4, 2, 128, 128, docs)
    dev = lambda *a: [t.to(DEV) for t in a]  # noqa: E731
    qd, kd, vd, dd, cd = dev(q, k, v, do, cu)
    scale = 1 / math.sqrt(128)
    out, lse = irs.window_gqa_attn_fwd(qd, kd, vd, cd, window, sinks=sinks)
    ref = R.window_fwd(q, k, v, cu, window, sinks, scale)
    want = R.window_bwd(q, k, v, cu, window, sinks, scale, out.cpu(), lse.cpu(), do)
    seen = R.window_mask(cu, T, window, sinks)

    def same(t, r, e, rows, what):
        R.check(t.cpu()[rows], r[rows], e[rows], what)

    for at in (60, 135, 329):                                # mid-document, near a document's start, the last row
        for which in ("k", "v"):
            kb, vb = k.clone(), v.clone()
            (kb if which == "k" else vb)[at] = bad
            kb, vb = dev(kb, vb)
            o, l = irs.window_gqa_attn_fwd(qd, kb, vb, cd, window, sinks=sinks)
            clean = ~seen[:, at]                             # queries that do not see the row
            same(o, ref[0], ref[2], clean, (at, which, "out"))
            same(l, ref[1], ref[3], clean, (at, which, "lse"))
            g = irs.window_gqa_attn_bwd(qd, kb, vb, cd, window, out, lse, dd, sinks=sinks)
            same(g[0], *want["dq"], clean, (at, which, "dq"))
            hit = seen[~clean].any(0)                        # keys that share a query with the row
            same(g[1], *want["dk"], ~hit, (at, which, "dk"))
            same(g[2], *want["dv"], ~hit, (at, which, "dv"))
        dob = do.clone()
        dob[at] = bad
        g = irs.window_gqa_attn_bwd(qd, kd, vd, cd, window, out, lse, dob.to(DEV), sinks=sinks)
        same(g[0], *want["dq"], torch.arange(T) != at, (at, "dout", "dq"))
        same(g[1], *want["dk"], ~seen[at], (at, "dout", "dk"))
        same(g[2], *want["dv"], ~seen[at], (at, "dout", "dv"))


def test_large_scores(irs):
    q, k, v, do, cu = _inputs(200, 4, 2, 128, 128, [200])
    _case(irs, q * 20, k, v * 50, do, cu, 70, 4, scale=1.0)


def test_malformed_documents_are_reported(irs):
    q, k, v, do, _ = _inputs(40, 2, 1, 64, 64, [40])
    dev = [t.to(DEV) for t in (q, k, v)]
    for cu in ([0, 20, 20, 40], [0, 41], [1, 40], [0, 30, 20, 40], [0, 39]):
        irs.read_device_errors(DEV)
        irs.window_gqa_attn_fwd(*dev, torch.tensor(cu, dtype=torch.int32, device=DEV), 8, sinks=2)
        assert irs.read_device_errors(DEV) & irs.DEVERR_CU_SEQLENS, cu


def test_given_outputs_no_lse_and_no_tokens(irs):
    q, k, v, do, cu = _inputs(100, 4, 2, 64, 64, [60, 40])
    dev = [t.to(DEV) for t in (q, k, v, cu)]
    out, lse = irs.window_gqa_attn_fwd(*dev, 20)
    mine = torch.empty_like(out)
    o, l = irs.window_gqa_attn_fwd(*dev, 20, out=mine, want_lse=False)
    assert o is mine and l is None and torch.equal(mine, out)
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    o, l = irs.window_gqa_attn_fwd(e, e[:, :2], e[:, :2], torch.zeros(1, dtype=torch.int32, device=DEV), 5)
    assert o.shape == (0, 4, 64) and l.shape == (0, 4)


def test_training_step_captured(irs):
    """Rotation, attention, its gradients and the rotation's gradient in one graph, replayed on
    new inputs, equal the same calls made eagerly."""
    q, k, v, do, cu = _inputs(300, 8, 2, 128, 128, [170, 130])
    qd, kd, vd, dd, cd = (t.to(DEV) for t in (q, k, v, do, cu))
    f = irs.rope_frequencies(128)[0].to(DEV)
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in (170, 130)]).to(DEV)

    def step():
        qr, kr = irs.rope(qd, pos, f), irs.rope(kd, pos, f)
        out, lse = irs.window_gqa_attn_fwd(qr, kr, vd, cd, 50, sinks=4)
        dq, dk, dv = irs.window_gqa_attn_bwd(qr, kr, vd, cd, 50, out, lse, dd, sinks=4)
        return out, irs.rope(dq, pos, f, transpose=True), irs.rope(dk, pos, f, transpose=True), dv

    eager = step()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = step()
    gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, eager))
    for t in (qd, kd, vd, dd):
        t.copy_(t.flip(0))
    gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))
    irs.check_device_errors(DEV)


@pytest.mark.parametrize("Hq,Hkv,Dqk,Dv", [(100, 1, 64, 64), (130, 2, 128, 64), (24, 2, 64, 128)])
def test_groups_that_do_not_fill_tiles(irs, Hq, Hkv, Dqk, Dv):
    """More query heads a KV head than a block of columns holds, and numbers that do not divide it."""
    _case(irs, *_inputs(160, Hq, Hkv, Dqk, Dv, [100, 60]), window=33, sinks=3)


@pytest.mark.parametrize("Hq,Hkv,Dqk,Dv,window,sinks,longest", [
    (4, 4, 64, 64, 20, 3, 90), (6, 3, 192, 128, 100, 4, 700), (16, 2, 128, 128, 64, 0, 300), (5, 5, 128, 128, 300, 40, 900)])
def test_many_tiles_a_block(irs, Hq, Hkv, Dqk, Dv, window, sinks, longest):
    """Tokens enough that every block of the kernels works through several tiles, over documents of
    mixed lengths; a sample of the documents, the first and the last among them, is checked."""
    g = torch.Generator().manual_seed(longest)
    docs = []
    while sum(docs) < 24000:
        docs.append(int(torch.randint(1, longest + 1, (1,), generator=g)))
    T = sum(docs)
    q, k, v, do, cu = _inputs(T, Hq, Hkv, Dqk, Dv, docs)
    dev = [t.to(DEV) for t in (q, k, v, cu, do)]
    qd, kd, vd, cd, dd = dev
    out, lse = irs.window_gqa_attn_fwd(qd, kd, vd, cd, window, sinks=sinks)
    got = irs.window_gqa_attn_bwd(qd, kd, vd, cd, window, out, lse, dd, sinks=sinks)
    irs.check_device_errors(DEV)
    oc, lc, gc = out.cpu(), lse.cpu(), [t.cpu() for t in got]
    scale = 1 / math.sqrt(Dqk)
    picks = {0, len(docs) - 1} | {int(i) for i in torch.randint(0, len(docs), (18,), generator=g)}
    for d in sorted(picks):
        a, b = int(cu[d]), int(cu[d + 1])
        one = torch.tensor([0, b - a], dtype=torch.int32)
        x = (q[a:b], k[a:b], v[a:b], one, window, sinks, scale)
        ref = R.window_fwd(*x)
        R.check(oc[a:b], ref[0], ref[2], (d, "out"))
        R.check(lc[a:b], ref[1], ref[3], (d, "lse"))
        want = R.window_bwd(*x, oc[a:b], lc[a:b], do[a:b])
        for name, t in zip(("dq", "dk", "dv"), gc):
            R.check(t[a:b], *want[name], (d, name))
    for _ in range(3):   # and every run gives the same bits
        again = irs.window_gqa_attn_fwd(qd, kd, vd, cd, window, sinks=sinks)
        grads = irs.window_gqa_attn_bwd(qd, kd, vd, cd, window, out, lse, dd, sinks=sinks)
        assert all(torch.equal(a, b) for a, b in zip((out, lse) + tuple(got), tuple(again) + tuple(grads)))


def test_calls_on_two_streams_at_once(irs):
    q, k, v, do, cu = _inputs(2000, 8, 2, 128, 128, [900, 1100])
    qd, kd, vd, cd, dd = (t.to(DEV) for t in (q, k, v, cu, do))

    def step(x):
        out, lse = irs.window_gqa_attn_fwd(x, kd, vd, cd, 200, sinks=4)
        return (out, lse) + tuple(irs.window_gqa_attn_bwd(x, kd, vd, cd, 200, out, lse, dd, sinks=4))

    xs = [qd, qd.flip(0).contiguous()]
    alone = [step(x) for x in xs]
    streams = [torch.cuda.Stream(DEV) for _ in xs]
    torch.cuda.synchronize()
    runs = []
    for _ in range(4):
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                runs.append(step(x))
    torch.cuda.synchronize()
    for i, r in enumerate(runs):
        assert all(torch.equal(a, b) for a, b in zip(r, alone[i % 2]))
    irs.check_device_errors(DEV)


def test_columns_of_a_wider_tensor_and_one_head_of_many(irs):
    """Rows of one token, and of one head, whose other strides are any number."""
    q, k, v, do, cu = _inputs(1, 2, 1, 64, 64, [1])
    wide = lambda t: torch.zeros(t.shape[0], t.shape[1], 200, dtype=t.dtype, device=DEV)  # noqa: E731
    gpu = []
    for t in (q, k, v):
        w = wide(t)
        w[:, :, 8:72] = t.to(DEV)
        gpu.append(w[:, :, 8:72])
    _case(irs, q, k, v, do, cu, 5, 1, gpu=tuple(gpu))


@pytest.mark.parametrize("Hq,Hkv,Dqk,Dv", [(8, 8, 64, 64), (32, 2, 192, 128)])
def test_short_items_follow_one_another(irs, Hq, Hkv, Dqk, Dv):
    """Window 1: a tile has hardly any work between its row sums and the next tile's first maxima, which the
    same threads exchange, many times a block. A row's output is its own value, its lse its own score."""
    T = 30000
    g = torch.Generator(device=DEV).manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    q, k, v = n(T, Hq, Dqk), n(T, Hkv, Dqk), n(T, Hkv, Dv)
    cu = torch.tensor([0, 7, T], dtype=torch.int32, device=DEV)
    x = q.double() * k.double().repeat_interleave(Hq // Hkv, 1)
    bound = (Dqk + 8) * R.U32 * x.abs().sum(-1) / 8 + 2.0 ** -21   # an FP32 sum of products, then a rounded scale and sum
    for _ in range(20):
        out, lse = irs.window_gqa_attn_fwd(q, k, v, cu, 1, 0.125)
        assert torch.equal(out, v.repeat_interleave(Hq // Hkv, 1))
        assert ((lse.double() - x.sum(-1) / 8).abs() <= bound).all()
    irs.check_device_errors(DEV)


def _rows(cu, rows, window, sinks):
    """(row, the keys it sees) of some rows."""
    for t in rows:
        start = int(cu[torch.searchsorted(cu, t, right=True) - 1])
        lo = max(start, t - window + 1)
        yield t, torch.cat((torch.arange(start, max(start, min(start + sinks, lo))), torch.arange(lo, t + 1)))


def _same(got, ref, bound, what):
    """NaN where the definition has NaN, within its bound elsewhere."""
    got, nan = got.cpu().double(), torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), (what, "NaN in other places")
    R.check(got.masked_fill(nan, 0.0), ref.masked_fill(nan, 0.0), bound.masked_fill(nan, 1.0), what)


def _check_fwd_rows(q, k, v, cu, window, sinks, out, lse, rows):
    Hkv = k.shape[1]
    for t, at in _rows(cu, rows, window, sinks):
        o, l, eo, el = R._attend(q[t].double().view(Hkv, -1, q.shape[2]), k[at].double(), v[at].double(), 1 / math.sqrt(q.shape[2]))
        _same(out[t].view(o.shape), o, eo, (t, "out"))
        _same(lse[t].view(l.shape), l, el, (t, "lse"))


def test_forward_rows_that_see_nan_and_their_neighbours(irs):
    """Long windows, several tiles a block: rows that see a NaN or an infinity hold what the definition does, also in
    the columns that it does not reach, and the rows that share their tiles stay within their bounds."""
    window, sinks = 6000, 2
    q, k, v, _, cu = _inputs(16400, 16, 1, 64, 64, [9000, 7400])
    v[50, 0, 3], v[9100, 0, 5], k[9500], q[4000, 2] = math.nan, math.inf, math.nan, math.nan
    out, lse = irs.window_gqa_attn_fwd(*(t.to(DEV) for t in (q, k, v, cu)), window, sinks=sinks)
    irs.check_device_errors(DEV)
    _check_fwd_rows(q, k, v, cu, window, sinks, out, lse, [
        0, 40, 49, 50, 51, 60, 3999, 4000, 4001, 6049, 6050, 6051, 6070, 8999, 9000, 9096, 9099, 9100, 9101, 9490, 9499,
        9500, 9501, 15098, 15099, 15100, 15101, 15499, 15500, 15501, 16399])


def test_forward_repairs_do_not_hold_up_the_pipeline(irs):
    """A NaN in a long document's last value row meets the rows before it in that tile with weight 0. Each of them has
    450,000 keys: computed again while the block's next tiles wait, they outlast the limit of those waits (2 s by the
    time of a key, some 0.5 us a warp, and 32 rows a warp)."""
    A, T = 450_000, 470_000
    g = torch.Generator(device=DEV).manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    q, k, v = n(T, 16, 64), n(T, 1, 64), n(T, 1, 64)
    v[A - 1] = math.nan
    cu = torch.tensor([0, A, T], dtype=torch.int32)
    out, lse = irs.window_gqa_attn_fwd(q, k, v, cu.to(DEV), T)
    irs.check_device_errors(DEV)
    nan = torch.isnan(out).flatten(1).sum(1).nonzero()[:, 0].tolist()
    assert nan == [A - 1] and torch.isnan(out[A - 1]).all() and not torch.isnan(lse).any()
    _check_fwd_rows(*(t.cpu() for t in (q, k, v)), cu, T, 0, out, lse,
                    [0, 1000, A - 17, A - 16, A - 9, A - 2, A - 1, A, A + 9, T - 3000, T - 1])


def _check_dq_rows(q, k, v, cu, window, sinks, out, lse, do, dq, rows):
    """Some rows of dq against the formula, with the roundings that serving_ref.window_bwd counts."""
    Hkv, Dq, Dv = k.shape[1], q.shape[2], v.shape[2]
    scale, G = 1 / math.sqrt(Dq), q.shape[1] // k.shape[1]
    for t, at in _rows(cu, rows, window, sinks):
        qt, dt, ot = (x[t].double().view(Hkv, G, -1) for x in (q, do, out))
        l = lse[t].double().view(Hkv, G, 1)
        kt, vt = k[at].double(), v[at].double()
        x = torch.einsum("hgd,shd->hgs", qt, kt) * scale
        p = torch.exp(x - l)
        D = (dt * ot).sum(-1, keepdim=True)
        y = torch.einsum("hgd,shd->hgs", dt, vt) - D
        ymag = torch.einsum("hgd,shd->hgs", dt.abs(), vt.abs()) + (dt.abs() * ot.abs()).sum(-1, keepdim=True)
        ds = p * y
        ep = p * ((Dq + 4) * R.U32 * torch.einsum("hgd,shd->hgs", qt.abs(), kt.abs()) * scale + 2.0 ** -21 + 4 * R.U32 * l.abs())
        e = ep * y.abs() + p * (Dv + 4) * R.U32 * ymag + (R.U16 + 64 * R.U32) * ds.abs()
        r = torch.einsum("hgs,shd->hgd", ds, kt) * scale
        bound = R.U16 * r.abs() + torch.einsum("hgs,shd->hgd", e, kt.abs()) * scale + 1e-30
        _same(dq[t].view(r.shape), r, bound, (t, "dq"))


def test_dq_rows_that_see_nan_and_their_neighbours(irs):
    window, sinks = 6000, 2
    q, k, v, do, cu = _inputs(16400, 16, 1, 64, 64, [9000, 7400])
    dev = [t.to(DEV) for t in (q, k, v, cu)]
    out, lse = irs.window_gqa_attn_fwd(*dev, window, sinks=sinks)
    kb, vb = k.clone(), v.clone()
    kb[8990], vb[9100, 0, 5], vb[16390, 0, 3] = math.nan, math.inf, math.nan
    dq = irs.window_gqa_attn_bwd(dev[0], kb.to(DEV), vb.to(DEV), dev[3], window, out, lse, do.to(DEV), sinks=sinks)[0]
    irs.check_device_errors(DEV)
    _check_dq_rows(q, kb, vb, cu, window, sinks, out.cpu(), lse.cpu(), do, dq, [
        0, 1, 4000, 8983, 8984, 8988, 8989, 8990, 8991, 8999, 9000, 9001, 9099, 9100, 9101, 15099, 15100, 15101, 15110,
        16384, 16389, 16390, 16391, 16399])


def test_dq_repairs_do_not_hold_up_the_pipeline(irs):
    """As for the forward: rows of 250,000 keys beside one that sees a NaN, and tiles behind them."""
    A, T = 250_000, 270_000
    g = torch.Generator(device=DEV).manual_seed(4)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    q, k, v, do = n(T, 16, 64), n(T, 1, 64), n(T, 1, 64), n(T, 16, 64)
    cu = torch.tensor([0, A, T], dtype=torch.int32)
    out, lse = irs.window_gqa_attn_fwd(q, k, v, cu.to(DEV), T)
    k[A - 1] = math.nan
    dq, dk, dv = irs.window_gqa_attn_bwd(q, k, v, cu.to(DEV), T, out, lse, do)
    irs.check_device_errors(DEV)
    for t in (dq, dk, dv):
        assert torch.isnan(t).flatten(1).sum(1).nonzero()[:, 0].tolist() == [A - 1]
    _check_dq_rows(*(t.cpu() for t in (q, k, v)), cu, T, 0, out.cpu(), lse.cpu(), do.cpu(), dq,
                   [0, 1000, A - 17, A - 9, A - 8, A - 2, A - 1, A, A + 9, T - 3000, T - 1])


def _check_key_rows(q, k, v, cu, window, sinks, out, lse, do, dk, dv, keys):
    """Some rows of dk and dv (one KV head) against the formula in 64 bits on the GPU, with the roundings that
    serving_ref.window_bwd counts."""
    Dq, Dv, G = q.shape[2], v.shape[2], q.shape[1]
    scale = 1 / math.sqrt(Dq)
    for s in keys:
        b = int(torch.searchsorted(cu, s, right=True)) - 1
        start, end = int(cu[b]), int(cu[b + 1])
        end = end if s - start < sinks else min(end, s + window)
        qs, ds_, os_ = (x[s:end].double().flatten(0, 1) for x in (q, do, out))
        l, kt, vt = lse[s:end].double().flatten(), k[s, 0].double(), v[s, 0].double()
        p = torch.exp(qs @ kt * scale - l)
        y = ds_ @ vt - (ds_ * os_).sum(-1)
        ymag = ds_.abs() @ vt.abs() + (ds_ * os_).abs().sum(-1)
        ep = p * ((Dq + 4) * R.U32 * (qs.abs() @ kt.abs()) * scale + 2.0 ** -21 + 4 * R.U32 * l.abs())
        w = p * y * scale
        ew = (ep * y.abs() + p * (Dv + 4) * R.U32 * ymag) * scale + R.U16 * w.abs()
        for got, x, e, a, what in ((dk, w, ew, qs, "dk"), (dv, p, ep + R.U16 * p, ds_, "dv")):
            r = x @ a
            bound = R.U16 * r.abs() + (e + 64 * R.U32 * x.abs()) @ a.abs() + 1e-30
            _same(got[s, 0], r.cpu(), bound.cpu(), (s, what))


@pytest.mark.parametrize("window,sinks", [(40_000, 0), (300, 3), (5000, 64)])
@pytest.mark.parametrize("which", ["q", "dout", "lse"])
def test_keys_repaired_outside_the_pipeline(irs, window, sinks, which):
    """A NaN in one head of a query reaches every key of the tiles that load it. Those that do not see it are computed
    again; with a window of 40,000 and 16 heads a key that is done by one warp while its tile's block waits takes longer
    than the waits last (32 keys of 640,000 rows of some 0.3 us). First tokens that see it and first tokens that do not
    are summed over stretches."""
    A, T = 40_000, 60_000
    g = torch.Generator(device=DEV).manual_seed(window)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    q, k, v, do = n(T, 16, 64), n(T, 1, 64), n(T, 1, 64), n(T, 16, 64)
    cu = torch.tensor([0, A, T], dtype=torch.int32)
    out, lse = irs.window_gqa_attn_fwd(q, k, v, cu.to(DEV), window, sinks=sinks)
    for t in (10, 29_000):
        {"q": q, "dout": do, "lse": lse}[which][t, 2] = math.nan
    dq, dk, dv = irs.window_gqa_attn_bwd(q, k, v, cu.to(DEV), window, out, lse, do, sinks=sinks)
    irs.check_device_errors(DEV)
    seen = {s for t in (10, 29_000) for s in (*range(min(sinks, t + 1)), *range(max(0, t - window + 1), t + 1))}
    for t in (dk, dv):
        assert set(torch.isnan(t).flatten(1).any(1).nonzero()[:, 0].tolist()) == seen
    _check_key_rows(q, k, v, cu, window, sinks, out, lse, do, dk, dv,
                    [0, 1, 2, 3, 10, 11, 12, 63, 64, 127, 128, 130, 28_000, 28_672, 28_701, 28_999, 29_000, 29_001, 29_055,
                     29_100, 39_999, A, A + 1, A + 70, T - 1])
    again = irs.window_gqa_attn_bwd(q, k, v, cu.to(DEV), window, out, lse, do, sinks=sinks)
    for a, b in zip((dq, dk, dv), again):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))   # NaN as well


def test_everything_nan_and_the_next_call(irs):
    """A step that has diverged gives NaN everywhere, and the same workspace then serves a clean one."""
    q, k, v, do, cu = (t.to(DEV) for t in _inputs(3000, 8, 2, 128, 128, [1700, 1, 1299]))
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)
    out, lse = irs.window_gqa_attn_fwd(q, k, v, cu, 500, sinks=4)
    want = irs.window_gqa_attn_bwd(q, k, v, cu, 500, out, lse, do, sinks=4, workspace=ws)
    bad = torch.full_like(q, math.nan)
    o, l = irs.window_gqa_attn_fwd(bad, k, v, cu, 500, sinks=4)
    got = irs.window_gqa_attn_bwd(bad, k, v, cu, 500, o, l, do, sinks=4, workspace=ws)
    assert all(torch.isnan(t).all() for t in (o, l) + tuple(got))
    again = irs.window_gqa_attn_bwd(q, k, v, cu, 500, out, lse, do, sinks=4, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    irs.check_device_errors(DEV)


@pytest.mark.parametrize("docs,window,sinks", [
    ([21, 22, 100, 275, 276, 277, 278, 300, 700], 20, 5), ([31, 349, 350, 351, 352, 40, 700], 30, 40),
    ([600, 1, 1030, 1156, 1157], 130, 128), ([17] * 60 + [9, 8, 300], 8, 64), ([5, 520, 519, 515, 3], 259, 3)])
def test_first_tokens_just_past_the_window(irs, docs, window, sinks):
    """Documents with as many queries beyond the window as their first tokens' tile takes, one fewer and one more, and
    first tokens in two tiles."""
    _case(irs, *_inputs(sum(docs), 4, 2, 64, 64, docs), window=window, sinks=sinks)


def test_tensors_side_by_side_in_one_buffer(irs):
    """Inputs and outputs that touch but do not overlap."""
    q, k, v, do, cu = _inputs(70, 4, 2, 128, 64, [30, 40])
    dev = [t.to(DEV) for t in (q, k, v, cu)]
    out, lse = irs.window_gqa_attn_fwd(*dev, 20, sinks=2)
    want = irs.window_gqa_attn_bwd(*dev, 20, out, lse, do.to(DEV), sinks=2)
    buf = torch.zeros(2 * sum(t.numel() for t in (q, k, v, do)), dtype=torch.bfloat16, device=DEV)
    at, mine = 0, []
    for t in (out, q, v, do, want[1], k, want[0], want[2]):
        mine.append(buf[at:at + t.numel()].view(t.shape))
        at += t.numel()
    for d, t in zip(mine, (None, q, v, do, None, k)):
        if t is not None:
            d.copy_(t)
    o, qm, vm, dm, dk, km, dq, dv = mine
    _, l = irs.window_gqa_attn_fwd(qm, km, vm, dev[3], 20, sinks=2, out=o)
    irs.window_gqa_attn_bwd(qm, km, vm, dev[3], 20, o, l, dm, sinks=2, dq=dq, dk=dk, dv=dv)
    assert torch.equal(o, out) and all(torch.equal(a, b) for a, b in zip((dq, dk, dv), want))
    with pytest.raises(ValueError, match="overlap"):
        irs.window_gqa_attn_bwd(qm, km, vm, dev[3], 20, o, l, dm, sinks=2, dq=qm)
    with pytest.raises(ValueError, match="overlap"):
        irs.window_gqa_attn_fwd(qm, km, vm, dev[3], 20, out=buf[64:64 + o.numel()].view(o.shape))
    irs.check_device_errors(DEV)


@pytest.mark.parametrize("shared", [True, False])
def test_scores_of_minus_infinity(irs, shared):
    """A visible key with a score of -inf has weight 0, also as the first that a row sees; a row that sees no other key
    is NaN, as the formula's 0 / 0. On the path for shared key rows, and where a NaN in a masked value row makes the
    rows be computed again."""
    q, k, v, _, cu = _inputs(90, 4, 2, 64, 64, [40, 50])
    q[:, :, 0] = 1.0
    k[40, :, 0], v[39] = -math.inf, math.nan                 # the second document's first key; the first one's last value
    if shared:
        k, v = (t[:, :1].expand(90, 2, 64) for t in (k, v))
    dev = [t.to(DEV) for t in (q, cu)]
    kd, vd = ((t[:, :1].to(DEV).expand(90, 2, 64) if shared else t.to(DEV)) for t in (k, v))
    out, lse = irs.window_gqa_attn_fwd(dev[0], kd, vd, dev[1], 30, sinks=2)
    irs.check_device_errors(DEV)
    assert torch.isnan(out[40]).all() and torch.isnan(lse[40]).all() and torch.isnan(out[39]).all()
    for t, at in _rows(cu, [0, 30, 38, *range(41, 90)], 30, 2):
        at = at[at != 40]
        o, l, eo, el = R._attend(q[t].double().view(2, 2, 64), k[at].double(), v[at].double(), 0.125)
        _same(out[t].view(o.shape), o, eo, (t, "out"))
        _same(lse[t].view(l.shape), l, el, (t, "lse"))


@pytest.mark.parametrize("window,sinks", [(60, 3), (2000, 0)])
def test_gradients_over_the_output(irs, window, sinks):
    """dq in out's place, and dk and dv over out: it is not read again, also where rows are computed again."""
    q, k, v, do, cu = (t.to(DEV) for t in _inputs(3000, 8, 2, 64, 64, [1400, 1600]))
    out, lse = irs.window_gqa_attn_fwd(q, k, v, cu, window, sinks=sinks)
    k[700, 0], do[2500, 3] = math.nan, math.nan
    want = irs.window_gqa_attn_bwd(q, k, v, cu, window, out, lse, do, sinks=sinks)
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))  # noqa: E731
    o = out.clone()
    got = irs.window_gqa_attn_bwd(q, k, v, cu, window, o, lse, do, sinks=sinks, dq=o)
    assert got[0] is o and all(same(a, b) for a, b in zip(got, want))
    o = out.clone()
    n = k.numel()
    dk, dv = o.view(-1)[64:64 + n].view(k.shape), o.view(-1)[64 + n:64 + 2 * n].view(v.shape)
    got = irs.window_gqa_attn_bwd(q, k, v, cu, window, o, lse, do, sinks=sinks, dk=dk, dv=dv)
    assert all(same(a, b) for a, b in zip(got, want))
    irs.check_device_errors(DEV)


def test_first_call_of_a_process_captured(irs):
    """The device's error word is made outside the graph: it is clear before the first replay, and a replay does not
    clear what another call reported."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch
import indexer_routed_sparse_gb300 as irs
q = torch.ones(40, 2, 64, dtype=torch.bfloat16, device="cuda")
cu = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out, lse = irs.window_gqa_attn_fwd(q, q, q, cu, 8)
assert irs.read_device_errors() == 0
g.replay()
torch.cuda.synchronize()
assert (out == 1).all()
irs.window_gqa_attn_fwd(q, q, q, torch.tensor([0, 41], dtype=torch.int32, device="cuda"), 8)
g.replay()
assert irs.read_device_errors() == irs.DEVERR_CU_SEQLENS
g.replay()
assert irs.read_device_errors() == 0
"""
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=root)
    assert done.returncode == 0, done.stderr[-2000:]
