"""Rotary positions, the paged cache's writer and the attention of one new token over it, on
the GPU (through the C ABI), against their 64-bit definitions."""
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


def _normal(g, *shape):
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


def _pool(g, lens, page, Hkv, Dqk, Dv, spare=2, heads_first=False):
    """(k_cache, v_cache, page_table) with shuffled pages; CPU tensors [pages, page, H, D]."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    shape = (pages, Hkv, page) if heads_first else (pages, page, Hkv)
    k, v = _normal(g, *shape, Dqk), _normal(g, *shape, Dv)
    return (k.transpose(1, 2), v.transpose(1, 2), table) if heads_first else (k, v, table)


def _gpu(t):
    """To the GPU with its strides kept (a transposed pool stays transposed)."""
    if t.dim() == 4 and not t.is_contiguous():
        return t.transpose(1, 2).to(DEV).transpose(1, 2)
    return t.to(DEV)


# ---------------------------------------------------------------------------------------
# rope
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("T,H,D,n,start,layout", [
    (1, 1, 64, 64, 0, "half"), (7, 3, 128, 128, 0, "interleaved"), (130, 5, 192, 64, 128, "half"),
    (33, 2, 192, 64, 128, "interleaved"), (5, 4, 72, 16, 8, "half"), (64, 64, 128, 32, 48, "interleaved"),
    (3, 128, 576, 64, 512, "interleaved"), (5000, 3, 128, 128, 0, "half"), (40000, 2, 64, 48, 8, "interleaved"),
])
@pytest.mark.parametrize("transpose", [False, True])
def test_rope(irs, T, H, D, n, start, layout, transpose):
    g = torch.Generator().manual_seed(T + D)
    x = _normal(g, T, H, D)
    pos = torch.randint(-5, 3_000_000, (T,), generator=g, dtype=torch.int32)
    f, amp = irs.rope_frequencies(n, scaling="by_parts", factor=8.0, trained_len=4096)
    ref, bound = R.rotate(x, pos, f, layout, start, amp, transpose)
    xd = x.to(DEV)
    out = irs.rope(xd, pos.to(DEV), f.to(DEV), layout=layout, start=start, amplitude=amp, transpose=transpose)
    R.check(out, ref, bound, "rope")
    assert torch.equal(xd.cpu(), x)
    again = irs.rope(xd, pos.to(DEV), f.to(DEV), layout=layout, start=start, amplitude=amp, transpose=transpose, out=xd)
    assert again is xd and torch.equal(again, out)          # in place


def test_rope_strided_rows_and_outputs(irs):
    g = torch.Generator().manual_seed(1)
    big = _normal(g, 50, 6, 160).to(DEV)
    x = big[3:40, 1:4, 16:144]                              # odd rows and heads of a larger tensor
    pos = torch.arange(37, dtype=torch.int32)
    f, _ = irs.rope_frequencies(64)
    out = torch.zeros(37, 5, 128, dtype=torch.bfloat16, device=DEV)
    before = big.clone()
    irs.rope(x, pos.to(DEV), f.to(DEV), out=out[:, 1:4])
    ref, bound = R.rotate(x.cpu(), pos, f, "half", 0, 1.0)
    R.check(out[:, 1:4], ref, bound, "strided rope")
    assert torch.equal(big, before) and not out[:, 0].any() and not out[:, 4].any()
    wide = x[:, :1].expand(37, 4, 128)                      # one head read for four
    R.check(irs.rope(wide, pos.to(DEV), f.to(DEV)), *(r[:, :1].expand(37, 4, 128) for r in (ref, bound)), "expanded rope")


def test_rope_far_positions_turn_exactly(irs):
    """Position 2^31 - 1 and frequency 1: the angle is right to 2^-20 (an FP32 product is off by over 60 radians)."""
    pos = torch.tensor([2**31 - 1, -2**31, 2**24 + 1, 0], dtype=torch.int32)
    f = torch.ones(8, dtype=torch.float64)
    x = torch.zeros(4, 1, 16, dtype=torch.bfloat16)
    x[..., :8] = 1
    out = irs.rope(x.to(DEV), pos.to(DEV), f.to(DEV))
    ref, bound = R.rotate(x, pos, f, "half", 0, 1.0)
    R.check(out, ref, bound + 2.0 ** -20, "far rope")


def test_rope_transpose_is_the_gradient(irs):
    """<rope(x), y> = <x, rope^T(y)> within the roundings of the two results."""
    g = torch.Generator().manual_seed(9)
    x, y = _normal(g, 200, 4, 128).to(DEV), _normal(g, 200, 4, 128).to(DEV)
    pos = torch.randint(0, 100000, (200,), generator=g, dtype=torch.int32).to(DEV)
    f = irs.rope_frequencies(128)[0].to(DEV)
    a = irs.rope(x, pos, f, amplitude=1.25)
    b = irs.rope(y, pos, f, amplitude=1.25, transpose=True)
    left, right = (a.double() * y.double()).sum(), (x.double() * b.double()).sum()
    slack = (R.U16 + 16 * R.U32) * 2 * ((a.double().abs() * y.double().abs()).sum() + (x.double().abs() * b.double().abs()).sum())
    assert abs(left - right) <= slack


# ---------------------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("new,before,page,heads_first", [
    ([1], [0], 1, False), ([1, 1, 1], [15, 16, 17], 16, False), ([3, 0, 40, 1], [0, 9, 30, 4095], 16, True),
    ([100, 1, 0], [7, 0, 3], 48, False), ([0, 2], [5, 63], 64, True), ([1000, 513], [1, 1023], 64, False),
])
@pytest.mark.parametrize("rotate", [True, False])
def test_append(irs, new, before, page, heads_first, rotate):
    Hq, Hkv, Dqk, Dv = 6, 2, 192, 128
    g = torch.Generator().manual_seed(sum(new) + page)
    kc, vc, table = _pool(g, [a + n for a, n in zip(before, new)], page, Hkv, Dqk, Dv, heads_first=heads_first)
    T = sum(new) + 3                                         # three rows behind the last sequence
    q, k, v = _normal(g, T, Hq, Dqk), _normal(g, T, Hkv, Dqk), _normal(g, T, Hkv, Dv)
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    f, amp = irs.rope_frequencies(64, scaling="linear", factor=4.0)
    kd, vd = _gpu(kc), _gpu(vc)
    q_out = torch.full((T, Hq, Dqk), 7.0, dtype=torch.bfloat16, device=DEV)
    k_out = torch.full((T, Hkv, Dqk), 7.0, dtype=torch.bfloat16, device=DEV)
    got = irs.paged_rope_append(q.to(DEV), k.to(DEV), v.to(DEV), kd, vd, table.to(DEV),
                                torch.tensor(before, dtype=torch.int32, device=DEV), f.to(DEV) if rotate else None,
                                cu_new=cu.to(DEV), layout="interleaved", start=128, amplitude=amp, q_out=q_out, k_out=k_out)
    irs.check_device_errors(DEV)
    assert got is q_out
    n = sum(new)
    pos = torch.cat([torch.arange(a, a + m) for a, m in zip(before, new)])
    seq = torch.cat([torch.full((m,), b) for b, m in enumerate(new)])
    slots = (table[seq, pos // page].long(), pos % page)
    rot = (lambda x: R.rotate(x, pos, f, "interleaved", 128, amp)) if rotate else (lambda x: (x.double(), torch.zeros(x.shape)))
    R.check(q_out[:n], *rot(q[:n]), "queries")
    ref, bound = rot(k[:n])
    R.check(k_out[:n], ref, bound, "keys")
    assert (q_out[n:] == 7).all() and (k_out[n:] == 7).all()
    kn, vn = kd.cpu(), vd.cpu()
    assert torch.equal(kn[slots], k_out[:n].cpu()) and torch.equal(vn[slots], v[:n])
    kn[slots], vn[slots] = kc[slots], vc[slots]              # nothing else changed
    assert torch.equal(kn, kc) and torch.equal(vn, vc)


def test_append_one_token_each_without_queries(irs):
    g = torch.Generator().manual_seed(3)
    kc, vc, table = _pool(g, [5, 17, 1], 16, 1, 64, 64)
    k, v = _normal(g, 3, 1, 64), _normal(g, 3, 1, 64)
    kd, vd = kc.to(DEV), vc.to(DEV)
    f = irs.rope_frequencies(32)[0]
    before = torch.tensor([4, 16, 0], dtype=torch.int32)
    assert irs.paged_rope_append(None, k.to(DEV), v.to(DEV), kd, vd, table.to(DEV), before.to(DEV), f.to(DEV)) is None
    irs.check_device_errors(DEV)
    for b in range(3):
        p = int(before[b])
        ref, bound = R.rotate(k[b:b + 1], before[b:b + 1], f, "half", 0, 1.0)
        row = kd[int(table[b, p // 16]), p % 16]
        R.check(row[None], ref, bound, "key")
        assert torch.equal(vd[int(table[b, p // 16]), p % 16].cpu(), v[b])


def test_append_reports_pages_outside_the_pool(irs):
    g = torch.Generator().manual_seed(4)
    kc, vc, table = _pool(g, [20, 20, 20, 20], 16, 2, 64, 64)
    table[1, 1] = kc.shape[0]                                # a page past the pool
    k, v = _normal(g, 4, 2, 64), _normal(g, 4, 2, 64)
    kd, vd = kc.to(DEV), vc.to(DEV)
    before = torch.tensor([32, 19, -1, 7], dtype=torch.int32)   # past the table, bad page, negative, fine
    irs.read_device_errors(DEV)
    irs.paged_rope_append(None, k.to(DEV), v.to(DEV), kd, vd, table.to(DEV), before.to(DEV))
    assert irs.read_device_errors(DEV) == irs.DEVERR_PAGE
    kc[int(table[3, 0]), 7], vc[int(table[3, 0]), 7] = k[3], v[3]
    assert torch.equal(kd.cpu(), kc) and torch.equal(vd.cpu(), vc)


def test_append_reports_malformed_cu_new(irs):
    g = torch.Generator().manual_seed(5)
    kc, vc, table = _pool(g, [20, 20], 16, 1, 64, 64)
    k, v = _normal(g, 4, 1, 64).to(DEV), _normal(g, 4, 1, 64).to(DEV)
    lens = torch.zeros(2, dtype=torch.int32, device=DEV)
    for cu in ([0, 3, 2], [1, 2, 4], [0, 2, 5]):
        irs.read_device_errors(DEV)
        irs.paged_rope_append(None, k, v, kc.to(DEV), vc.to(DEV), table.to(DEV), lens,
                              cu_new=torch.tensor(cu, dtype=torch.int32, device=DEV))
        assert irs.read_device_errors(DEV) & irs.DEVERR_CU_SEQLENS, cu


# ---------------------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------------------
def _decode_case(irs, lens, Hq, Hkv, Dqk, Dv, page, window=0, sinks=0, W=0, seed=0, heads_first=False, routes=None):
    g = torch.Generator().manual_seed(seed + sum(lens) + Dqk)
    kc, vc, table = _pool(g, lens, page, Hkv, Dqk, Dv, heads_first=heads_first)
    q = _normal(g, len(lens), Hq, Dqk)
    if W:
        routes = torch.full((len(lens), W), -1, dtype=torch.int32)
        for b, n in enumerate(lens):
            m = min(n, max(0, W - b % 3))
            routes[b, :m] = torch.randperm(n, generator=g)[:m].to(torch.int32)
    ln = torch.tensor(lens, dtype=torch.int32)
    scale = 1 / math.sqrt(Dqk)
    ref = R.decode(q, kc, vc, table, ln, scale, window, sinks, routes)
    args = [q.to(DEV), _gpu(kc), _gpu(vc), table.to(DEV), ln.to(DEV)]
    kw = dict(window=window, sinks=sinks, route_ids=None if routes is None else routes.to(DEV))
    out, lse = irs.paged_gqa_attn_decode(*args, **kw)
    irs.check_device_errors(DEV)
    R.check(out, ref[0], ref[2], "out")
    R.check(lse, ref[1], ref[3], "lse")
    o2, l2 = irs.paged_gqa_attn_decode(*args, **kw)
    assert torch.equal(out, o2) and torch.equal(lse, l2)     # the same in every run
    return args, kw, ref


@pytest.mark.parametrize("Hq,Hkv,Dqk,Dv", [(1, 1, 64, 64), (8, 8, 128, 128), (6, 2, 192, 128), (16, 1, 128, 64),
                                           (64, 4, 192, 128), (20, 1, 64, 128), (40, 2, 256, 256), (3, 1, 64, 256),
                                           (12, 12, 64, 64), (3, 3, 192, 128), (48, 16, 128, 128), (90, 5, 256, 64)])
@pytest.mark.parametrize("page", [1, 16, 48])
def test_decode_head_shapes_and_lengths(irs, Hq, Hkv, Dqk, Dv, page):
    _decode_case(irs, [1, 0, 15, 16, 17, 64, 333, 700], Hq, Hkv, Dqk, Dv, page, heads_first=page == 16)


@pytest.mark.parametrize("lens", [[1], [2], [5000], [63, 65], [1] * 300, [0, 0, 0], list(range(0, 130, 3)), [9000, 1, 40]])
def test_decode_ragged(irs, lens):
    _decode_case(irs, lens, 8, 2, 128, 128, 64)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (100, 0), (64, 30), (512, 4), (100000, 3)])
def test_decode_window_and_first_tokens(irs, window, sinks):
    _decode_case(irs, [0, 1, 2, 5, 8, 64, 99, 100, 101, 104, 130, 700, 1500], 6, 2, 64, 64, 16, window, sinks)


@pytest.mark.parametrize("window,sinks,W", [(0, 0, 1), (0, 0, 130), (0, 5, 77), (33, 0, 64), (33, 4, 2051)])
def test_decode_routes(irs, window, sinks, W):
    _decode_case(irs, [0, 1, 3, 34, 40, 200, 900, 3000], 8, 4, 128, 128, 16, window, sinks, W)


def test_decode_rows_with_no_position(irs):
    routes = torch.full((3, 9), -1, dtype=torch.int32)
    routes[1, 4] = 2
    _, _, ref = _decode_case(irs, [5, 5, 0], 4, 2, 64, 64, 16, routes=routes)
    assert torch.isinf(ref[1][0]).all() and torch.isinf(ref[1][2]).all() and not torch.isinf(ref[1][1]).any()


def test_decode_reads_only_attended_rows(irs):
    """NaN and infinities in every other row of the pool (the rest of a page, spare pages, masked positions)."""
    for window, sinks, W in ((0, 0, 0), (20, 3, 0), (0, 0, 40), (9, 2, 40)):
        g = torch.Generator().manual_seed(W + window)
        lens = [37, 100, 5, 0]
        kc, vc, table = _pool(g, lens, 16, 2, 64, 64)
        q = _normal(g, 4, 4, 64)
        routes = None
        if W:
            routes = torch.full((4, W), -1, dtype=torch.int32)
            for b, n in enumerate(lens):
                m = min(n // 2, W)
                routes[b, :m] = torch.randperm(max(n, 1), generator=g)[:m].to(torch.int32)
        keep = torch.zeros(kc.shape[:2], dtype=torch.bool)
        for b, n in enumerate(lens):
            seen = set(range(n)) if not window and not W else set(range(min(sinks, n))) | (
                set(range(max(0, n - window), n)) if window else set()) | (
                {int(r) for r in routes[b] if r >= 0} if W else set())
            for p in seen:
                keep[int(table[b, p // 16]), p % 16] = True
        ln = torch.tensor(lens, dtype=torch.int32)
        ref = R.decode(q, kc, vc, table, ln, 0.125, window, sinks, routes)
        kb, vb = kc.clone(), vc.clone()
        kb[~keep], vb[~keep] = math.nan, math.inf
        out, lse = irs.paged_gqa_attn_decode(q.to(DEV), kb.to(DEV), vb.to(DEV), table.to(DEV), ln.to(DEV), 0.125,
                                             window=window, sinks=sinks, route_ids=None if routes is None else routes.to(DEV))
        irs.check_device_errors(DEV)
        R.check(out, ref[0], ref[2], "out")
        R.check(lse, ref[1], ref[3], "lse")


def test_decode_large_scores_and_values(irs):
    """Scores of several hundred: one position dominates; the running maximum has to carry the rest."""
    g = torch.Generator().manual_seed(21)
    lens = [500, 70]
    kc, vc, table = _pool(g, lens, 16, 2, 128, 128)
    q = _normal(g, 2, 8, 128) * 30
    ln = torch.tensor(lens, dtype=torch.int32)
    ref = R.decode(q, kc, vc * 100, table, ln, 1.0)
    out, lse = irs.paged_gqa_attn_decode(q.to(DEV), kc.to(DEV), (vc * 100).to(DEV), table.to(DEV), ln.to(DEV), 1.0)
    R.check(out, ref[0], ref[2], "out")
    R.check(lse, ref[1], ref[3], "lse")


def test_decode_strided_queries_shared_pages_and_given_outputs(irs):
    g = torch.Generator().manual_seed(8)
    lens = [40, 40, 33]
    kc, vc, table = _pool(g, lens, 16, 2, 128, 128)
    table[1, :2] = table[0, :2]                              # a forked prefix
    table[2] = table[0]
    big = _normal(g, 3, 12, 160)
    q = big[:, 2:10, 16:144]
    ln = torch.tensor(lens, dtype=torch.int32)
    ref = R.decode(q, kc, vc, table, ln, 0.1)
    out = torch.empty(3, 8, 128, dtype=torch.bfloat16, device=DEV)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)   # scratch holds anything
    o, l = irs.paged_gqa_attn_decode(big.to(DEV)[:, 2:10, 16:144], kc.to(DEV), vc.to(DEV), table.to(DEV), ln.to(DEV), 0.1,
                                     out=out, workspace=ws, want_lse=False)
    assert o is out and l is None
    R.check(out, ref[0], ref[2], "out")


def test_decode_reports_bad_routes_pages_and_lengths(irs):
    g = torch.Generator().manual_seed(6)
    lens = [40, 40, 40]
    kc, vc, table = _pool(g, lens, 16, 2, 64, 64)
    q = _normal(g, 3, 4, 64)
    ln = torch.tensor(lens, dtype=torch.int32)
    dev = [t.to(DEV) for t in (q, kc, vc)]
    irs.read_device_errors(DEV)
    routes = torch.tensor([[1, 5, 40, -1], [2, -7, 3, 4], [9, 39, 0, 2**31 - 1]], dtype=torch.int32)
    out, lse = irs.paged_gqa_attn_decode(*dev, table.to(DEV), ln.to(DEV), 0.125, route_ids=routes.to(DEV))
    assert irs.read_device_errors(DEV) == irs.DEVERR_ROUTE_ID
    ref = R.decode(q, kc, vc, table, ln, 0.125, routes=routes)
    R.check(out, ref[0], ref[2], "out")
    bad = table.clone()
    bad[0, 1], bad[1, 0] = -1, kc.shape[0]                   # positions on these pages are skipped
    out, lse = irs.paged_gqa_attn_decode(*dev, bad.to(DEV), ln.to(DEV), 0.125)
    assert irs.read_device_errors(DEV) == irs.DEVERR_PAGE
    ref = R.decode(q, kc, vc, bad, ln, 0.125)
    R.check(out, ref[0], ref[2], "out")
    R.check(lse, ref[1], ref[3], "lse")
    far = torch.tensor([40, -1, 49], dtype=torch.int32)      # the table reaches 48
    out, lse = irs.paged_gqa_attn_decode(*dev, table.to(DEV), far.to(DEV), 0.125)
    assert irs.read_device_errors(DEV) == irs.DEVERR_PAGE
    assert not out[1:].any() and torch.isinf(lse[1:]).all() and not torch.isinf(lse[0]).any()


def test_decode_offsets_past_32_bits(irs):
    """A pool of over 2^31 elements: the last pages are read where they are."""
    page, Hkv, D = 256, 8, 128
    pages = (1 << 31) // (page * Hkv * D) + 40
    kc = torch.zeros(pages, page, Hkv, D, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros(pages, page, Hkv, D, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(2)
    table = torch.tensor([[pages - 1, pages - 3, 0], [pages - 2, 1, pages - 5]], dtype=torch.int32)
    for p in table.flatten().tolist():
        kc[p], vc[p] = _normal(g, page, Hkv, D).to(DEV), _normal(g, page, Hkv, D).to(DEV)
    q = _normal(g, 2, 16, D)
    ln = torch.tensor([600, 768], dtype=torch.int32)
    used = sorted(set(table.flatten().tolist()))
    small = torch.tensor([[used.index(int(p)) for p in r] for r in table], dtype=torch.int32)
    ref = R.decode(q, kc[used].cpu(), vc[used].cpu(), small, ln, 0.1)
    out, lse = irs.paged_gqa_attn_decode(q.to(DEV), kc, vc, table.to(DEV), ln.to(DEV), 0.1)
    irs.check_device_errors(DEV)
    R.check(out, ref[0], ref[2], "out")
    R.check(lse, ref[1], ref[3], "lse")
    k = _normal(g, 2, Hkv, D).to(DEV)
    irs.paged_rope_append(None, k, k, kc, vc, table.to(DEV), torch.tensor([511, 0], dtype=torch.int32, device=DEV))
    assert torch.equal(kc[pages - 3, 255], k[0]) and torch.equal(vc[pages - 2, 0], k[1])


def test_decode_captured_and_on_another_stream(irs):
    """A captured step replays on new lengths, queries and caches; two graphs with a workspace
    each do not disturb one another; a side stream gives the same result."""
    g = torch.Generator().manual_seed(12)
    kc, vc, table = _pool(g, [600, 600, 600], 16, 2, 128, 128)
    args = [_normal(g, 3, 8, 128).to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV),
            torch.tensor([600, 1, 77], dtype=torch.int32, device=DEV)]
    want = [irs.paged_gqa_attn_decode(*args), irs.paged_gqa_attn_decode(*args, window=50, sinks=2)]
    torch.cuda.synchronize()
    graphs, got = [], []
    for kw in (dict(), dict(window=50, sinks=2)):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            got.append(irs.paged_gqa_attn_decode(*args, **kw))
        graphs.append(gr)
    for _ in range(2):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(got, want):
        assert torch.equal(o, wo) and torch.equal(l, wl)
    args[4].copy_(torch.tensor([3, 599, 0], dtype=torch.int32))
    args[0].mul_(0.5)
    for gr in graphs:
        gr.replay()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fresh = [irs.paged_gqa_attn_decode(*args), irs.paged_gqa_attn_decode(*args, window=50, sinks=2)]
    s.synchronize()
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(got, fresh):
        assert torch.equal(o, wo) and torch.equal(l, wl)


def test_prompt_then_steps_together(irs):
    """As a served model runs them: a ragged prompt is rotated and appended, attended with its
    window and first tokens; then steps of one token, whose attention over the cache equals
    the attention of the longer prompt's last row; and a routed step equals the routed
    attention over the same keys."""
    Hq, Hkv, Dqk, Dv, page, window, sinks = 8, 2, 128, 128, 16, 48, 4
    g = torch.Generator().manual_seed(33)
    total, steps = [70, 21, 150], 3
    T = sum(total)
    x = {n: _normal(g, T, h, d) for n, h, d in (("q", Hq, Dqk), ("k", Hkv, Dqk), ("v", Hkv, Dv))}
    cu = torch.tensor([0] + total).cumsum(0).to(torch.int32)
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in total])
    f = irs.rope_frequencies(Dqk)[0].to(DEV)
    full = {n: t.to(DEV) for n, t in x.items()}
    qr, kr = irs.rope(full["q"], pos.to(DEV), f), irs.rope(full["k"], pos.to(DEV), f)
    want, want_l = irs.window_gqa_attn_fwd(qr, kr, full["v"], cu.to(DEV), window, sinks=sinks)

    kc, vc, table = _pool(g, total, page, Hkv, Dqk, Dv)
    kc, vc, table = kc.to(DEV), vc.to(DEV), table.to(DEV)
    first = [n - steps for n in total]
    rows = torch.cat([torch.arange(int(cu[b]), int(cu[b]) + n) for b, n in enumerate(first)])
    cun = torch.tensor([0] + first).cumsum(0).to(torch.int32).to(DEV)
    part = {n: t[rows].to(DEV) for n, t in x.items()}
    k_out = torch.empty_like(part["k"])
    lens = torch.zeros(3, dtype=torch.int32, device=DEV)
    q0 = irs.paged_rope_append(part["q"], part["k"], part["v"], kc, vc, table, lens, f, cu_new=cun, k_out=k_out)
    assert torch.equal(q0, qr[rows.to(DEV)]) and torch.equal(k_out, kr[rows.to(DEV)])
    lens += torch.tensor(first, dtype=torch.int32, device=DEV)
    for i in range(steps):
        at = torch.tensor([int(cu[b]) + first[b] + i for b in range(3)])
        new = {n: t[at].to(DEV) for n, t in x.items()}
        qn = irs.paged_rope_append(new["q"], new["k"], new["v"], kc, vc, table, lens, f)
        lens += 1
        out, lse = irs.paged_gqa_attn_decode(qn, kc, vc, table, lens, window=window, sinks=sinks)
        ref = R.decode(qr[at.to(DEV)].cpu(), kc.cpu(), vc.cpu(), table.cpu(), lens.cpu(), 1 / math.sqrt(Dqk), window, sinks)
        R.check(out, ref[0], ref[2], f"step {i}")
        R.check(lse, ref[1], ref[3], f"step {i} lse")
        # both within their bounds of the same definition
        assert ((out.cpu().double() - want[at.to(DEV)].cpu().double()).abs() <= 2 * ref[2]).all()
    irs.check_device_errors(DEV)
    # a routed step: the indexer's routes of each document's last token, as positions of its sequence
    c, budget, Hi, Di = 4, 16, 4, 64
    qI, kI = _normal(g, T, Hi, Di).to(DEV), _normal(g, T, Di).to(DEV)
    w = torch.rand(T, Hi, generator=g).to(DEV)
    routes = irs.sparse_index_score_topk(qI, kI, w, cu.to(DEV), c, budget)
    last = (cu[1:] - 1).long().to(DEV)
    local = torch.where(routes[last] >= 0, routes[last] - cu[:-1, None].to(DEV), routes[last]).to(torch.int32)
    out, lse = irs.paged_gqa_attn_decode(qr[last], kc, vc, table, lens, route_ids=local)
    dense, dense_l = irs.sparse_gqa_attn_fwd(qr[last], kr, full["v"], routes[last])
    irs.check_device_errors(DEV)
    ref = R.decode(qr[last].cpu(), kc.cpu(), vc.cpu(), table.cpu(), lens.cpu(), 1 / math.sqrt(Dqk), routes=local.cpu())
    R.check(out, ref[0], ref[2], "routed step")
    assert ((out.cpu().double() - dense.cpu().double()).abs() <= 2 * ref[2]).all()
    assert (lse - dense_l).abs().max() <= 1e-4


@pytest.mark.parametrize("Dqk,Dv,n,start,layout", [(64, 256, 32, 16, "half"), (8, 24, 0, 0, "half"), (200, 8, 16, 8, "interleaved"),
                                                   (16, 1000, 16, 0, "half"), (256, 64, 256, 0, "interleaved")])
@pytest.mark.parametrize("new", [[1, 1, 1], [30, 1, 9]])
def test_append_values_of_other_widths(irs, Dqk, Dv, n, start, layout, new):
    """Value rows wider and narrower than key rows, odd numbers of 16-byte pieces."""
    g = torch.Generator().manual_seed(Dqk + Dv)
    before, page, Hq, Hkv = [0, 17, 31], 16, 3, 2
    kc, vc, table = _pool(g, [a + m for a, m in zip(before, new)], page, Hkv, Dqk, Dv)
    T = sum(new)
    q, k, v = _normal(g, T, Hq, Dqk), _normal(g, T, Hkv, Dqk), _normal(g, T, Hkv, Dv)
    kd, vd = kc.to(DEV), vc.to(DEV)
    f = irs.rope_frequencies(n)[0] if n else None
    cu = None if T == 3 else torch.tensor([0] + new).cumsum(0).to(torch.int32).to(DEV)
    q_out = irs.paged_rope_append(q.to(DEV), k.to(DEV), v.to(DEV), kd, vd, table.to(DEV),
                                  torch.tensor(before, dtype=torch.int32, device=DEV), f.to(DEV) if n else None,
                                  cu_new=cu, layout=layout, start=start)
    irs.check_device_errors(DEV)
    pos = torch.cat([torch.arange(a, a + m) for a, m in zip(before, new)])
    seq = torch.cat([torch.full((m,), b) for b, m in enumerate(new)])
    slots = (table[seq, pos // page].long(), pos % page)
    rot = (lambda x: R.rotate(x, pos, f, layout, start, 1.0)) if n else (lambda x: (x.double(), torch.zeros(x.shape)))
    R.check(q_out, *rot(q), "queries")
    R.check(kd.cpu()[slots], *rot(k), "keys")
    assert torch.equal(vd.cpu()[slots], v)
    kn, vn = kd.cpu(), vd.cpu()
    kn[slots], vn[slots] = kc[slots], vc[slots]              # nothing else changed
    assert torch.equal(kn, kc) and torch.equal(vn, vc)


def test_append_more_sequences_than_shared_memory_holds(irs):
    """The sequence of a token is then searched in global memory; some sequences have no new token."""
    g = torch.Generator().manual_seed(8)
    B = 5000
    new = (torch.arange(B) % 3).tolist()
    T = sum(new)
    table = torch.randperm(B, generator=g).to(torch.int32)[:, None]
    kc = torch.zeros(B, 8, 1, 64, dtype=torch.bfloat16)
    k, v = _normal(g, T, 1, 64), _normal(g, T, 1, 64)
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    before = torch.arange(B, dtype=torch.int32) % 6
    kd, vd = kc.to(DEV), kc.to(DEV)
    irs.paged_rope_append(None, k.to(DEV), v.to(DEV), kd, vd, table.to(DEV), before.to(DEV), cu_new=cu.to(DEV))
    irs.check_device_errors(DEV)
    seq = torch.repeat_interleave(torch.arange(B), torch.tensor(new))
    pos = before[seq].long() + torch.arange(T) - cu[seq].long()
    want_k, want_v = kc.clone(), kc.clone()
    want_k[table[seq, 0].long(), pos], want_v[table[seq, 0].long(), pos] = k, v
    assert torch.equal(kd.cpu(), want_k) and torch.equal(vd.cpu(), want_v)


def test_decode_more_sequences_than_threads(irs):
    """Many short sequences: each thread of a block counts the tiles of several, with empty ones among them."""
    g = torch.Generator().manual_seed(21)
    lens = torch.randint(0, 40, (1500,), generator=g).tolist()
    _decode_case(irs, lens, 4, 2, 64, 64, 16)


def test_decode_on_two_streams_at_once(irs):
    g = torch.Generator().manual_seed(14)
    lens = [3000, 1, 900, 0, 64]
    kc, vc, table = _pool(g, lens, 16, 2, 128, 128)
    args = [kc.to(DEV), vc.to(DEV), table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)]
    qs = [_normal(g, 5, 8, 128).to(DEV) for _ in range(2)]
    alone = [irs.paged_gqa_attn_decode(q, *args) for q in qs]
    streams = [torch.cuda.Stream(DEV) for _ in qs]
    torch.cuda.synchronize()
    runs = []
    for _ in range(6):
        for s, q in zip(streams, qs):
            with torch.cuda.stream(s):
                runs.append(irs.paged_gqa_attn_decode(q, *args))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(runs):
        assert torch.equal(o, alone[i % 2][0]) and torch.equal(l, alone[i % 2][1])
    irs.check_device_errors(DEV)


def test_decode_one_workspace_for_calls_in_order(irs):
    """Calls of one stream may share a workspace, whatever their sizes; a short one is replaced."""
    g = torch.Generator().manual_seed(15)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    for lens in ([2000, 5], [1] * 50, [700] * 9):
        kc, vc, table = _pool(g, lens, 16, 2, 64, 64)
        args = [_normal(g, len(lens), 4, 64).to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV),
                torch.tensor(lens, dtype=torch.int32, device=DEV)]
        want = irs.paged_gqa_attn_decode(*args)
        ws.fill_(255)                                        # NaN, were it read
        for w in (ws, ws[:64]):
            got = irs.paged_gqa_attn_decode(*args, workspace=w)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_decode_attended_infinities(irs):
    """An infinite value under a positive weight gives that infinity, two of opposite sign NaN, and the other columns and
    heads are as ever: in sequences that one run holds and in ones that are cut, with the largest weight exactly 1."""
    g = torch.Generator().manual_seed(31)
    lens = [1, 9, 40, 3000, 700, 17]
    kc, vc, table = _pool(g, lens, 16, 2, 128, 128)
    q = _normal(g, 6, 8, 128)
    at = lambda b, p: (int(table[b, p // 16]), p % 16)  # noqa: E731
    vc[at(0, 0)][0, 3] = math.inf                            # the only position
    vc[at(1, 8)][1, 7] = -math.inf
    for p, x in ((2, math.inf), (30, -math.inf)):            # opposite signs in one column
        vc[at(2, p)][0, 60] = x
    for p in (5, 1400, 2999):
        vc[at(3, p)][0, 100] = math.inf
    vc[at(4, 699)][1, 0] = -math.inf
    vc[at(5, 16)][0, 127] = math.nan
    ln = torch.tensor(lens, dtype=torch.int32)
    ref = R.decode(q, kc, vc, table, ln, 0.1)
    out, lse = irs.paged_gqa_attn_decode(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), ln.to(DEV), 0.1)
    irs.check_device_errors(DEV)
    nan = torch.isnan(ref[0])
    assert torch.isinf(ref[0]).any() and nan.any()
    assert torch.equal(torch.isnan(out.cpu()), nan)
    R.check(out.cpu().masked_fill(nan, 0), ref[0].masked_fill(nan, 0), ref[2].masked_fill(nan, 1), "out")
    R.check(lse, ref[1], ref[3], "lse")


@pytest.mark.parametrize("cu", [[2, 4, 6], [3, 3, 6], [-2, 3, 6], [-(2**31), 3, 6]])
def test_append_leaves_rows_before_the_first_sequence(irs, cu):
    """A cu_new that does not start at 0 is reported; rows that belong to no sequence are written nowhere, least of all
    over the sequence's older keys."""
    g = torch.Generator().manual_seed(41)
    lens = [20, 33]
    kc, vc, table = _pool(g, [48, 48], 16, 1, 64, 64)
    k, v, q = _normal(g, 6, 1, 64), _normal(g, 6, 1, 64), _normal(g, 6, 2, 64)
    kd, vd = kc.to(DEV), vc.to(DEV)
    q_out = torch.full((6, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    k_out = torch.full((6, 1, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    irs.read_device_errors(DEV)
    irs.paged_rope_append(q.to(DEV), k.to(DEV), v.to(DEV), kd, vd, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                          cu_new=torch.tensor(cu, dtype=torch.int32, device=DEV), q_out=q_out, k_out=k_out)
    assert irs.read_device_errors(DEV) == irs.DEVERR_CU_SEQLENS
    for b in range(2):
        for i in range(max(cu[b], 0) if cu[b] >= 0 else cu[b + 1], cu[b + 1]):
            p = lens[b] + i - cu[b]
            kc[int(table[b, p // 16]), p % 16], vc[int(table[b, p // 16]), p % 16] = k[i], v[i]
    assert torch.equal(kd.cpu(), kc) and torch.equal(vd.cpu(), vc)
    none = cu[0] if cu[0] >= 0 else cu[1]
    assert (q_out[:none] == 7).all() and (k_out[:none] == 7).all() and torch.equal(q_out[none:].cpu(), q[none:])


def test_decode_scores_of_minus_infinity(irs):
    """Positions whose score is -inf have weight 0; a sequence whose positions all have it is NaN, as the formula's
    0 / 0, in one run or cut into parts, while one with no position stays 0."""
    g = torch.Generator().manual_seed(51)
    lens = [1, 40, 3000, 3000, 0, 500, 17]
    kc, vc, table = _pool(g, lens, 16, 2, 64, 64)
    q = _normal(g, 7, 4, 64)
    q[:, :, 0] = 1.0
    gone = [range(1), range(40), range(1000, 3000), range(3000), (), range(200), [16]]
    clean = kc.clone()
    for b, ps in enumerate(gone):
        for p in ps:
            kc[int(table[b, p // 16]), p % 16, :, 0] = -math.inf
    routes = torch.full((7, 3000), -1, dtype=torch.int32)    # the definition without those positions
    for b, n in enumerate(lens):
        at = [p for p in range(n) if p not in set(gone[b])]
        routes[b, :len(at)] = torch.tensor(at, dtype=torch.int32)
    ln = torch.tensor(lens, dtype=torch.int32)
    ref = R.decode(q, clean, vc, table, ln, 0.125, routes=routes)
    out, lse = irs.paged_gqa_attn_decode(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), ln.to(DEV), 0.125)
    irs.check_device_errors(DEV)
    for b in (0, 1, 3):
        assert torch.isnan(out[b]).all() and torch.isnan(lse[b]).all(), b
    rest = [2, 4, 5, 6]
    R.check(out[rest], ref[0][rest], ref[2][rest], "out")
    R.check(lse[rest], ref[1][rest], ref[3][rest], "lse")
