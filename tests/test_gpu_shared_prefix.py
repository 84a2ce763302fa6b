"""Page plans and attention over shared prefixes, on the GPU (through the C ABI), against their
64-bit definitions."""
import math

import pytest
import torch

import prefix_ref as R

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module")
def irs():
    import indexer_routed_sparse_gb300 as m

    m.lib()
    return m


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)


def _cache(g, pages, page, H, D, heads_first):
    t = _normal(g, *((pages, H, page, D) if heads_first else (pages, page, H, D)))
    return t.transpose(1, 2) if heads_first else t


def _sums(n):
    got = [0]
    for x in n:
        got.append(got[-1] + x)
    return got


# ---------------------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------------------
def _plan(irs, lens, new, page, width, spare=2, pad=0, groups=None, prefix=None, short=0, tokens=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    held = [-(-max(n, 0) // page) for n in lens]
    need = sum(max(0, -(-(n + m) // page) - h) for n, m, h in zip(lens, new, held) if m > 0 and n >= 0)
    order = torch.randperm(sum(held) + need + spare, generator=g).tolist()
    table = [[-7] * width for _ in lens]
    at = 0
    for row, h in zip(table, held):
        row[:min(h, width)] = order[at: at + min(h, width)]
        at += h
    free = order[at:]
    count = max(0, len(free) - spare - short) if short else len(free)
    tokens = sum(max(m, 0) for m in new) + pad if tokens is None else tokens
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    dt = _i32(table)
    ins = [_i32(lens), _i32(new), _i32(free), _i32([count])]
    gr = {} if groups is None else dict(cu_groups=_i32(groups), prefix_lens=_i32(prefix))
    ref = R.plan(lens, new, table, free, count, page, tokens, groups, prefix)
    for _ in range(2):   # the inputs are unchanged: a second call gives the same again
        got = irs.paged_plan(ins[0], ins[1], dt, ins[2], ins[3], page, tokens, err=err, **gr)
        assert dt.tolist() == ref[0]
        assert got.cu_new.tolist() == ref[1] and got.positions.tolist() == ref[2] and got.slots.tolist() == ref[3]
        assert got.cache_lens.tolist() == ref[4] and got.free_count.tolist() == [ref[5]]
        assert got.slots.dtype == torch.int64
    assert [x.tolist() for x in ins] == [lens, new, free, [count]]
    return int(err)


@pytest.mark.parametrize("lens,new,page,pad", [
    ([0], [1], 1, 0), ([0], [0], 16, 3), ([15, 16, 17], [1, 1, 1], 16, 0), ([0, 5, 63, 64], [64, 0, 2, 130], 64, 5),
    ([7], [300], 48, 1), ([0, 0, 0], [0, 0, 0], 16, 0), ([1000, 3], [1, 1000], 1, 0), ([3, 100], [0, 1], 128, 0),
])
def test_plan(irs, lens, new, page, pad):
    width = max(-(-(n + m) // page) for n, m in zip(lens, new)) + 1
    assert _plan(irs, lens, new, page, width, pad=pad) == 0


@pytest.mark.parametrize("B,hi,page", [(255, 1, 16), (256, 3, 1), (257, 40, 16), (1500, 9, 48), (5000, 1, 64)])
def test_plan_many_sequences(irs, B, hi, page):
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 100, (B,), generator=g).tolist()
    new = torch.randint(0, hi + 1, (B,), generator=g).tolist()
    assert _plan(irs, lens, new, page, (100 + hi) // page + 2, pad=7, spare=100) == 0


@pytest.mark.parametrize("page,prefix", [(16, [40, 16, 0, 15]), (1, [40, 3, 9, 1]), (64, [64, 200, 5, 128])])
def test_plan_shared_prefixes(irs, page, prefix):
    """Groups of 3, 0, 1 and 4 sequences and two sequences behind the last; a first sequence that takes its prompt in
    the same call; a sequence that does not hold its prefix."""
    groups = [0, 3, 3, 4, 8]
    lens = [0, prefix[0], prefix[0] + 5, prefix[2], prefix[3], prefix[3], prefix[3] + 70, 0, 9, 0]
    new = [prefix[0] + 2, 1, 1, 3, 0, 2, 1, 4, 1, 30]
    width = max(-(-(n + m) // page) for n, m in zip(lens, new))
    assert _plan(irs, lens, new, page, width, groups=groups, prefix=prefix, pad=2) == 0


def test_plan_long_prompts(irs):
    g = torch.Generator().manual_seed(3)
    new = torch.randint(1, 30000, (9,), generator=g).tolist()
    assert _plan(irs, [5] * 9, new, 16, 2000, pad=11) == 0


def test_plan_reports_what_it_refuses(irs):
    page = irs.DEVERR_PAGE
    # two pages too few: the second sequence gets none, the third's need is covered by none either, the fourth needs none
    assert _plan(irs, [0, 16, 3, 4], [16, 32, 30, 1], 16, 5, short=2) == page
    assert _plan(irs, [0, 16], [1, 1], 16, 5, short=2) == page
    assert _plan(irs, [-1, 3, 5, 2 ** 30], [4, -2, 1, 7], 16, 4, tokens=9) == page
    assert _plan(irs, [0, 30, 31], [33, 2, 2], 16, 2, tokens=40) == page          # 32 positions at most
    assert _plan(irs, [0, 3], [5, 5], 16, 2, tokens=7) == irs.DEVERR_CU_SEQLENS   # more tokens than rows


def test_plan_reports_bad_counts_and_groups(irs):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = _i32([[0, -1], [1, -1]])
    args = (_i32([3, 3]), _i32([1, 1]), table, _i32([5, 6]))
    for count in (-1, 3):
        err.zero_()
        got = irs.paged_plan(*args, _i32([count]), 16, 2, err=err)
        assert int(err) == irs.DEVERR_PAGE and got.free_count.tolist() == [max(0, min(count, 2))]
    for cu, lens, bits in (([0, 2, 1], [4, 4], irs.DEVERR_CU_SEQLENS), ([1, 2, 2], [1, 1], irs.DEVERR_CU_SEQLENS),
                           ([0, 1, 9], [1, 1], irs.DEVERR_CU_SEQLENS), ([0, 1, 2], [-5, 1], irs.DEVERR_PAGE)):
        err.zero_()
        irs.paged_plan(*args, _i32([2]), 16, 2, cu_groups=_i32(cu), prefix_lens=_i32(lens), err=err)
        assert int(err) == bits


def test_plan_captured_with_given_outputs(irs):
    """A captured plan replays on new lengths; its results are written into the tensors it was given."""
    lens, new, free, count = _i32([15, 0, 40]), _i32([1, 1, 1]), _i32(list(range(50, 90))), _i32([40])
    table = torch.full((3, 8), -1, dtype=torch.int32, device=DEV)
    table[:, :3] = _i32([[0, 1, 2], [3, 4, 5], [6, 7, 8]])
    out = irs.paged_plan(lens, new, table, free, count, 16, 5)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            irs.paged_plan(lens, new, table, free, count, 16, 5, out=out)
    lens.copy_(_i32([16, 3, 47]))
    new.copy_(_i32([1, 0, 2]))
    before = table.clone()
    gr.replay()
    torch.cuda.synchronize()
    ref = R.plan([16, 3, 47], [1, 0, 2], before.tolist(), list(range(50, 90)), 40, 16, 5)
    assert (table.tolist(), out.cu_new.tolist(), out.positions.tolist(), out.slots.tolist(), out.cache_lens.tolist(),
            out.free_count.tolist()) == (ref[0], ref[1], ref[2], ref[3], ref[4], [ref[5]])


# ---------------------------------------------------------------------------------------
# prompts
# ---------------------------------------------------------------------------------------
def _prompts(irs, rows, prefix, Hq, Hkv, Dqk, Dv, page, heads_first=False, joined=True, pad=0, seed=0, scale=None):
    g = _gen(seed)
    need = [-(-n // page) for n in prefix]
    order = torch.randperm(sum(need) + 2, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(rows), max(need + [1])), -1, dtype=torch.int32, device=DEV)
    for i, (n, a) in enumerate(zip(need, _sums(need))):
        table[i, :n] = order[a: a + n]
    kc, vc = (_cache(g, sum(need) + 2, page, Hkv, d, heads_first) for d in (Dqk, Dv))
    T, cu = sum(rows) + pad, _sums(rows)
    q = _normal(g, T, Hq, Dqk)
    own = None
    if joined:
        own = (_normal(g, T, Hq, Dv), torch.randn(T, Hq, generator=g, device=DEV) * 4)
        own[1][::3] = -math.inf
        own[0][::3] = math.nan          # a part that attended nothing does not count
    s = scale or 1.0 / math.sqrt(Dqk)
    out = torch.full((T, Hq, Dv), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, Hq), 7.0, dtype=torch.float32, device=DEV)
    ins = [x.clone() for x in (q, kc, vc, table)]
    irs.shared_prefix_gqa_attn_fwd(q, kc, vc, table, _i32(cu), _i32(prefix), scale, own=own, out=out, lse=lse)
    irs.check_device_errors(DEV)
    ref = R.fwd(q, kc, vc, table, cu, prefix, s, own)
    n = cu[-1]
    R.check(out[:n], ref[0], ref[2], "out")
    R.check(lse[:n], ref[1], ref[3], "lse")
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()
    assert all(torch.equal(a, b) for a, b in zip(ins, (q, kc, vc, table)))
    again, lse2 = irs.shared_prefix_gqa_attn_fwd(q, kc, vc, table, _i32(cu), _i32(prefix), scale, own=own)
    assert torch.equal(again[:n], out[:n]) and torch.equal(lse2[:n], lse[:n])   # the same in every run
    return q, kc, vc, table, cu, own, out, lse


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 63, 64, 65, 95, 96, 97, 127, 128, 129, 200, 257, 1000])
def test_prompts_prefix_lengths(irs, n):
    _prompts(irs, [5], [n], 8, 2, 128, 128, 16, seed=n)


@pytest.mark.parametrize("Dqk,Dv", [(64, 64), (64, 128), (128, 64), (128, 128), (192, 64), (192, 128)])
@pytest.mark.parametrize("page,heads_first", [(16, False), (1, True), (64, True), (48, False), (8, False), (100, False)])
def test_prompts_head_dims_and_pages(irs, Dqk, Dv, page, heads_first):
    _prompts(irs, [9, 70], [333, 190], 6, 2, Dqk, Dv, page, heads_first, seed=Dqk + page)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (3, 1), (10, 2), (16, 1), (64, 4), (40, 1), (128, 1), (130, 2), (256, 2)])
def test_prompts_head_groups(irs, Hq, Hkv):
    _prompts(irs, [1, 37], [150, 260], Hq, Hkv, 128, 128, 64, seed=Hq)


@pytest.mark.parametrize("rows,prefix,pad", [
    ([0, 3, 0], [50, 60, 70], 4), ([1] * 20, [10 * i for i in range(20)], 0), ([300, 1, 130], [700, 2000, 5], 1),
    ([0], [40], 3), ([64, 65, 63], [128, 256, 384], 0),
])
def test_prompts_groups(irs, rows, prefix, pad):
    _prompts(irs, rows, prefix, 8, 4, 64, 64, 16, pad=pad, seed=len(rows))
    _prompts(irs, rows, prefix, 8, 4, 64, 64, 16, pad=pad, joined=False, seed=len(rows))


def test_prompts_many_blocks_and_rows(irs):
    _prompts(irs, [700, 900], [3001, 2500], 16, 2, 128, 128, 64, seed=1)
    _prompts(irs, [900], [2500], 32, 2, 192, 128, 16, heads_first=True, seed=2)
    _prompts(irs, [150], [9001], 8, 1, 128, 128, 1, seed=3)


def test_prompts_many_groups(irs):
    g = torch.Generator().manual_seed(5)
    rows = torch.randint(0, 4, (1400,), generator=g).tolist()
    prefix = torch.randint(0, 40, (1400,), generator=g).tolist()
    _prompts(irs, rows, prefix, 4, 2, 64, 64, 16, seed=6)


def test_prompts_large_scores(irs):
    """Scores of hundreds: the running maximum rises late and often."""
    _prompts(irs, [40], [900], 8, 2, 128, 128, 16, scale=3.0, seed=8)


def test_prompts_in_place_strided_and_broadcast(irs):
    q, kc, vc, table, cu, own, out, lse = _prompts(irs, [33, 20], [150, 80], 8, 2, 128, 128, 16)
    n, pl = cu[-1], _i32([150, 80])
    a, b = own[0].clone(), own[1].clone()
    got, l = irs.shared_prefix_gqa_attn_fwd(q, kc, vc, table, _i32(cu), pl, own=(a, b), out=a, lse=b)
    assert got is a and torch.equal(a, out) and torch.equal(b, lse)
    wide = torch.zeros(n, 11, 160, dtype=torch.bfloat16, device=DEV)
    wide[:, 2:10, 16:144] = q
    got, l = irs.shared_prefix_gqa_attn_fwd(wide[:, 2:10, 16:144], kc, vc, table, _i32(cu), pl, own=own)
    assert torch.equal(got, out) and torch.equal(l, lse)
    got, none = irs.shared_prefix_gqa_attn_fwd(q, kc, vc, table, _i32(cu), pl, own=own, want_lse=False)
    assert none is None and torch.equal(got, out)
    # one query row for every token, one head for all
    for x in (q[:1].expand(n, -1, -1), q[:, :1].expand(-1, 8, -1)):
        got, l = irs.shared_prefix_gqa_attn_fwd(x, kc, vc, table, _i32(cu), pl)
        ref = R.fwd(x, kc, vc, table, cu, [150, 80], 1 / math.sqrt(128))
        R.check(got, ref[0], ref[2], "expanded out")
        R.check(l, ref[1], ref[3], "expanded lse")


@pytest.mark.parametrize("page", [1, 16, 64])
def test_prompts_read_only_their_prefix(irs, page):
    """NaN behind a prefix's end, in its last page too, and in every page that is none of its."""
    g = _gen(4)
    n, rows = 199, 40
    need = -(-n // page)
    for Dqk, Dv in ((128, 128), (192, 64)):
        kc, vc = _cache(g, need + 3, page, 2, Dqk, False), _cache(g, need + 3, page, 2, Dv, False)
        table = (torch.arange(need + 1, device=DEV, dtype=torch.int32) + 1)[None]
        for c in (kc, vc):
            flat = c[1: need + 1].flatten(0, 1)
            flat[n:] = math.nan
            c[1: need + 1] = flat.view(need, page, *c.shape[2:])
            c[0], c[need + 1:] = math.nan, math.nan
        q = _normal(g, rows, 8, Dqk)
        out, lse = irs.shared_prefix_gqa_attn_fwd(q, kc, vc, table, _i32([0, rows]), _i32([n]))
        ref = R.fwd(q, kc, vc, table, [0, rows], [n], 1 / math.sqrt(Dqk))
        R.check(out, ref[0], ref[2], "out")
        R.check(lse, ref[1], ref[3], "lse")


def test_prompts_attended_infinities(irs):
    """An infinite value reaches its column of every row; a row with a NaN query is NaN alone; a key of which every
    score is -inf does not count, and a prefix of such keys alone gives 0 / 0."""
    g = _gen(5)
    n, rows = 150, 20
    kc, vc = _cache(g, 11, 16, 1, 128, False), _cache(g, 11, 16, 1, 128, False)
    table = torch.arange(11, device=DEV, dtype=torch.int32)[None]
    vc[2, 3, 0, 5], vc[4, 1, 0, 9] = math.inf, -math.inf
    q = _normal(g, rows, 4, 128).abs()
    q[7, 2, 0] = math.nan
    kc[3, 0] = 0
    kc[3, 0, 0, 0] = -math.inf
    out, lse = irs.shared_prefix_gqa_attn_fwd(q, kc, vc, table, _i32([0, rows]), _i32([n]))
    at = torch.arange(n, device=DEV)
    k, v = R.rows(kc, table[0], at), R.rows(vc, table[0], at)
    v[34 + 1, 0, 5] = v[64 + 1, 0, 9] = 0
    k[48, 0, 0], v[48] = 0, 0
    keep = at != 48
    ref = R.attend(q, k[keep], v[keep], 1 / math.sqrt(128))
    fine = torch.ones(rows, 4, dtype=torch.bool, device=DEV)
    fine[7, 2] = False
    assert (out[..., 5][fine] == math.inf).all() and (out[..., 9][fine] == -math.inf).all()
    assert out[7, 2].isnan().all() and lse[7, 2].isnan()
    cols = [i for i in range(128) if i not in (5, 9)]
    R.check(lse[fine], ref[1][fine], ref[3][fine], "lse")
    R.check(out[fine][:, cols], ref[0][fine][:, cols], ref[2][fine][:, cols], "out")
    kc[:] = 0
    kc[..., 0] = -math.inf
    q[7, 2, 0] = 1
    out, lse = irs.shared_prefix_gqa_attn_fwd(q, kc, vc, table, _i32([0, rows]), _i32([n]))
    assert out.isnan().all() and lse.isnan().all()


def test_prompts_report_bad_prefixes(irs):
    g = _gen(6)
    kc, vc = _cache(g, 8, 16, 2, 64, False), _cache(g, 8, 16, 2, 64, False)
    table = _i32([[0, 1, 2, 3], [4, 99, 6, 7], [4, 5, 6, 7]])
    q = _normal(g, 12, 4, 64)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for prefix, live in (([40, 20, 33], [0, 2]), ([40, 10, 33], [0, 1, 2]), ([-3, 1, 33], [1, 2]), ([65, 1, 64], [1, 2])):
        err.zero_()
        cu = [0, 4, 7, 12]
        out, lse = irs.shared_prefix_gqa_attn_fwd(q, kc, vc, table, _i32(cu), _i32(prefix), err=err)
        assert int(err) == (0 if prefix[1] == 10 else irs.DEVERR_PAGE)
        ref = R.fwd(q, kc, vc, table.clamp(max=7), cu, [0 if n < 0 or n > 64 else n for n in prefix], 0.125)
        for i in live:
            a, b = cu[i], cu[i + 1]
            R.check(out[a:b], ref[0][a:b], ref[2][a:b], "out")
            R.check(lse[a:b], ref[1][a:b], ref[3][a:b], "lse")
    for cu in ([0, 4, 3, 12], [1, 4, 7, 12], [0, 4, 7, 13]):
        err.zero_()
        irs.shared_prefix_gqa_attn_fwd(q, kc, vc, table, _i32(cu), _i32([40, 10, 33]), err=err)
        assert int(err) == irs.DEVERR_CU_SEQLENS


# ---------------------------------------------------------------------------------------
# decoding
# ---------------------------------------------------------------------------------------
def _steps(g, rows, prefix, own, Hq, Hkv, Dqk, Dv, page, heads_first=False, behind=()):
    """own: positions of each sequence behind its prefix, None for an idle slot; behind: lengths of sequences of no
    group. A page that a prefix fills in part is each sequence's own."""
    cu = _sums(rows)
    n = [p for p, r in zip(prefix, rows) for _ in range(r)]
    lens = [0 if o is None else a + o for a, o in zip(n, own)] + list(behind)
    n += [0] * len(behind)
    firsts = {b: (cu[g_], prefix[g_]) for g_ in range(len(rows)) for b in range(cu[g_], cu[g_ + 1])}
    need = [max(-(-L // page), -(-n[b] // page) if firsts.get(b, (None,))[0] == b else 0) for b, L in enumerate(lens)]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32, device=DEV)
    kc, vc = (_cache(g, pages, page, Hkv, d, heads_first) for d in (Dqk, Dv))
    for b, (m, a) in enumerate(zip(need, _sums(need))):
        table[b, :m] = order[a: a + m]
    for b, (f, p) in firsts.items():
        whole = p // page
        if b != f and lens[b]:
            table[b, :whole] = table[f, :whole]
            if p % page:
                for c in (kc, vc):
                    c[int(table[b, whole]), : p % page] = c[int(table[f, whole]), : p % page]
    return _normal(g, len(lens), Hq, Dqk), kc, vc, table, lens, cu


def _decode(irs, rows, prefix, own, Hq, Hkv, Dqk, Dv, page, heads_first=False, behind=(), seed=0, scale=None):
    q, kc, vc, table, lens, cu = _steps(_gen(seed), rows, prefix, own, Hq, Hkv, Dqk, Dv, page, heads_first, behind)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = (q, kc, vc, table, _i32(lens), _i32(cu), _i32(prefix), scale)
    out, lse = irs.shared_prefix_gqa_attn_decode(*args, err=err)
    assert int(err) == 0
    s = scale or 1 / math.sqrt(Dqk)
    ref = R.decode(q, kc, vc, table, lens, cu, prefix, s)
    R.check(out, ref[0], ref[2], "out")
    R.check(lse, ref[1], ref[3], "lse")
    again, lse2 = irs.shared_prefix_gqa_attn_decode(*args)
    assert torch.equal(again, out) and torch.equal(lse2, lse)
    return args, out, lse


@pytest.mark.parametrize("n", [0, 1, 16, 33, 96, 127, 128, 129, 600])
@pytest.mark.parametrize("own", [[0, 0, 0], [1, 7, 100], [None, 3, 64], [0, None, 500]])
def test_decode_lengths(irs, n, own):
    _decode(irs, [3], [n], own, 8, 2, 128, 128, 16, seed=n)


@pytest.mark.parametrize("Dqk,Dv", [(64, 64), (64, 128), (128, 64), (128, 128), (192, 64), (192, 128)])
@pytest.mark.parametrize("page,heads_first", [(16, False), (1, False), (64, True), (48, True)])
def test_decode_head_dims_and_pages(irs, Dqk, Dv, page, heads_first):
    _decode(irs, [4, 1], [301, 77], [1, 40, 9, 130, 5], 6, 2, Dqk, Dv, page, heads_first, seed=Dqk + page)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (3, 1), (10, 2), (16, 1), (64, 4), (40, 1), (128, 1), (32, 32)])
def test_decode_head_groups(irs, Hq, Hkv):
    _decode(irs, [5, 2], [260, 140], [3, 40, 1, 17, 90, 64, 2], Hq, Hkv, 128, 128, 64, seed=Hq)


def test_decode_groups_and_sequences_behind_them(irs):
    _decode(irs, [0, 3, 0, 1, 30], [9, 50, 70, 33, 200], [1, 20, None, 300] + list(range(30)), 8, 4, 64, 64, 16,
            behind=(40, 0, 700), seed=1)
    _decode(irs, [1] * 40, [7 * i for i in range(40)], [3 * i for i in range(40)], 4, 2, 128, 64, 16, seed=2)


def test_decode_many(irs):
    g = torch.Generator().manual_seed(1)
    own = torch.randint(0, 900, (300,), generator=g).tolist()
    _decode(irs, [260, 40], [3001, 700], own, 16, 2, 128, 128, 64, seed=3)
    _decode(irs, [60], [6001], own[:60], 32, 4, 192, 128, 1, seed=4)
    _decode(irs, [1], [20001], [5], 16, 8, 128, 128, 16, heads_first=True, seed=5)


def test_decode_large_scores(irs):
    _decode(irs, [20], [700], list(range(20)), 8, 2, 128, 128, 16, scale=3.0, seed=6)


def test_decode_is_the_paged_decode(irs):
    """With nothing shared, and with everything: the same attention as `paged_gqa_attn_decode` over whole tables."""
    (q, kc, vc, table, lens, cu, pl, s), out, lse = _decode(irs, [12], [500], [1 + 30 * i for i in range(12)], 16, 4, 128,
                                                            128, 16, seed=7)
    a, la = irs.paged_gqa_attn_decode(q, kc, vc, table, lens)
    b, lb = irs.shared_prefix_gqa_attn_decode(q, kc, vc, table, lens, _i32([0, 0]), _i32([500]))
    for x, l in ((a, la), (b, lb)):
        # two results, each within a few bf16 roundings of values under 1 / sqrt(500) of their spread
        assert (x.double() - out.double()).abs().max() <= 4 * R.U16 * out.double().abs().max()
        assert (l - lse).abs().max() <= 2.0 ** -17


def test_decode_reads_only_what_is_attended(irs):
    """NaN wherever no attended position points: behind lengths, in the other sequences' copies of the prefix."""
    q, kc, vc, table, lens, cu = _steps(_gen(8), [4], [100], [30, 1, None, 77], 8, 2, 128, 128, 16)
    used = torch.zeros(kc.shape[0], 16, dtype=torch.bool, device=DEV)
    for b, L in enumerate(lens):
        at = torch.arange(100 if b == 0 else L, device=DEV)
        at = torch.arange(L, device=DEV) if b == 0 else at[100:] if L else at[:0]
        used[table[b, at // 16].long(), at % 16] = True
    kc[~used], vc[~used] = math.nan, math.nan
    out, lse = irs.shared_prefix_gqa_attn_decode(q, kc, vc, table, _i32(lens), _i32(cu), _i32([100]))
    irs.check_device_errors(DEV)
    ref = R.decode(q, kc, vc, table, lens, cu, [100], 1 / math.sqrt(128))
    R.check(out, ref[0], ref[2], "out")
    R.check(lse, ref[1], ref[3], "lse")


def test_decode_scores_of_minus_infinity(irs):
    """A prefix whose scores are all -inf leaves the own part; with nothing else it gives 0 / 0."""
    q, kc, vc, table, lens, cu = _steps(_gen(9), [3], [160], [40, 0, 1], 8, 2, 128, 128, 16)
    q.abs_()
    shared = table[0, :10].long()
    kc[shared] = 0
    kc[shared, :, :, 0] = -math.inf
    out, lse = irs.shared_prefix_gqa_attn_decode(q, kc, vc, table, _i32(lens), _i32(cu), _i32([160]))
    for b, m in ((0, 40), (2, 1)):
        at = 160 + torch.arange(m, device=DEV)
        ref = R.attend(q[b: b + 1], R.rows(kc, table[b], at), R.rows(vc, table[b], at), 1 / math.sqrt(128))
        R.check(out[b: b + 1], ref[0], ref[2], "out")
        R.check(lse[b: b + 1], ref[1], ref[3], "lse")
    assert out[1].isnan().all() and lse[1].isnan().all()


def test_decode_reports_bad_lengths_and_pages(irs):
    q, kc, vc, table, lens, cu = _steps(_gen(10), [3, 2], [50, 20], [5, 9, 1, 4, 30], 8, 2, 64, 64, 16)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for at, L in ((1, 49), (1, -1), (4, 19), (4, 10 ** 6)):
        err.zero_()
        wrong = list(lens)
        wrong[at] = L
        out, lse = irs.shared_prefix_gqa_attn_decode(q, kc, vc, table, _i32(wrong), _i32(cu), _i32([50, 20]), err=err)
        assert int(err) == irs.DEVERR_PAGE and not out[at].any() and (lse[at] == -math.inf).all()
        ref = R.decode(q, kc, vc, table, wrong, cu, [50, 20], 0.125)
        R.check(out, ref[0], ref[2], "out")
    err.zero_()
    bad = table.clone()
    bad[1, 3] = kc.shape[0]     # sequence 1's own positions 48 .. 58
    out, lse = irs.shared_prefix_gqa_attn_decode(q, kc, vc, bad, _i32(lens), _i32(cu), _i32([50, 20]), err=err)
    assert int(err) == irs.DEVERR_PAGE
    keep = [0, 2, 3, 4]
    ref = R.decode(q, kc, vc, table, lens, cu, [50, 20], 0.125)
    R.check(out[keep], ref[0][keep], ref[2][keep], "out")
    at = torch.arange(50, device=DEV)
    ref = R.attend(q[1:2], R.rows(kc, table[0], at), R.rows(vc, table[0], at), 0.125)
    R.check(out[1:2], ref[0], ref[2] + 2.0 ** -16, "out without the own positions")
    for wrong in ([0, 3, 2], [1, 3, 5], [0, 3, 6]):
        err.zero_()
        irs.shared_prefix_gqa_attn_decode(q, kc, vc, table, _i32(lens), _i32(wrong), _i32([50, 20]), err=err)
        assert int(err) & irs.DEVERR_CU_SEQLENS


def test_decode_offsets_past_32_bits(irs):
    """A pool of more than 2^32 elements, with the shared and the own pages at its end."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    page, H, D = 64, 8, 128
    pages = (1 << 32) // (page * H * D) + 40
    kc = torch.zeros(pages, page, H, D, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    g = _gen(11)
    kc[-40:], vc[-40:] = _normal(g, 40, page, H, D), _normal(g, 40, page, H, D)
    table = (pages - 1 - torch.arange(36, device=DEV, dtype=torch.int32)).view(3, 12)
    lens, prefix = [700, 650, 641], [640]
    table[1:, :10] = table[0, :10]
    q = _normal(g, 3, 16, D)
    out, lse = irs.shared_prefix_gqa_attn_decode(q, kc, vc, table, _i32(lens), _i32([0, 3]), _i32(prefix))
    ref = R.decode(q, kc, vc, table, lens, [0, 3], prefix, 1 / math.sqrt(D))
    R.check(out, ref[0], ref[2], "out")
    out, lse = irs.shared_prefix_gqa_attn_fwd(q, kc, vc, table[:1], _i32([0, 3]), _i32(prefix))
    ref = R.fwd(q, kc, vc, table, [0, 3], prefix, 1 / math.sqrt(D))
    R.check(out, ref[0], ref[2], "out")


def test_captured_and_on_other_streams(irs):
    """Captured calls replay on new lengths, queries and borders; two graphs with workspaces of their own run at once."""
    q, kc, vc, table, lens, cu = _steps(_gen(12), [5, 4], [200, 130], [1, 50, 9, 300, 7, 20, 60, 1, 2], 16, 4, 128, 128, 16)
    dl, dc, dp = _i32(lens), _i32(cu), _i32([200, 130])
    tab2 = table[[0, 5]].contiguous()
    graphs, outs = [], []
    irs.shared_prefix_gqa_attn_decode(q, kc, vc, table, dl, dc, dp)
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append((irs.shared_prefix_gqa_attn_decode(q, kc, vc, table, dl, dc, dp),
                         irs.shared_prefix_gqa_attn_fwd(q, kc, vc, tab2, dc, dp)))
        graphs.append(gr)
    q.copy_(_normal(_gen(13), *q.shape))
    dl.copy_(_i32([L - 1 if L > 200 else L for L in lens]))
    dp.copy_(_i32([190, 100]))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(3):
        for st, gr in zip(streams, graphs):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    ref = R.decode(q, kc, vc, table, dl.tolist(), cu, [190, 100], 1 / math.sqrt(128))
    ref2 = R.fwd(q, kc, vc, tab2, cu, [190, 100], 1 / math.sqrt(128))
    for (a, la), (b, lb) in outs:
        R.check(a, ref[0], ref[2], "out")
        R.check(la, ref[1], ref[3], "lse")
        R.check(b, ref2[0], ref2[2], "prompt out")
        R.check(lb, ref2[1], ref2[3], "prompt lse")


def test_one_workspace_for_calls_in_order(irs):
    args, out, lse = _decode(irs, [30], [900], list(range(30)), 16, 2, 128, 128, 16, seed=14)
    small, out2, lse2 = _decode(irs, [2], [40], [1, 2], 16, 2, 128, 128, 16, seed=15)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        assert torch.equal(irs.shared_prefix_gqa_attn_decode(*args, workspace=ws)[0], out)
        assert torch.equal(irs.shared_prefix_gqa_attn_decode(*small, workspace=ws)[0], out2)


def test_plan_append_prompts_and_steps_together(irs):
    """Requests behind one prompt, as a server runs them: plan, append, attend the prefix and the own prompt; then
    decoding steps. Checked against attention over each request's whole text."""
    g = _gen(16)
    page, Hq, Hkv, D, B = 16, 8, 2, 128, 3
    n, new = 77, [20, 1, 45]
    table = torch.full((B + 1, 12), -1, dtype=torch.int32, device=DEV)
    kc, vc = (torch.zeros(48, page, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    free, count = torch.arange(48, dtype=torch.int32, device=DEV), _i32([48])
    inv, _ = irs.rope_frequencies(64)
    inv = inv.to(DEV)
    groups, pl = _i32([0, B + 1]), _i32([n])
    text = [[] for _ in range(B + 1)]        # (rotated keys, values) of every request

    def step(lens, counts, count):
        plan = irs.paged_plan(lens, _i32(counts), table, free, count, page, sum(counts), cu_groups=groups, prefix_lens=pl)
        T = sum(counts)
        q, k, v = _normal(g, T, Hq, D), _normal(g, T, Hkv, D), _normal(g, T, Hkv, D)
        kr = irs.rope(k, plan.positions, inv)
        qr = irs.paged_rope_append(q, k, v, kc, vc, table, lens, inv, cu_new=plan.cu_new)
        assert torch.equal(qr, irs.rope(q, plan.positions, inv))
        flat = kc.view(-1, Hkv, D)
        assert torch.equal(flat[plan.slots], kr)
        cu = _sums(counts)
        for b in range(B + 1):
            text[b].append((kr[cu[b]: cu[b + 1]], v[cu[b]: cu[b + 1]]))
        return plan, qr, kr, v, cu

    # the prompt itself, in request 0
    plan, q, k, v, cu = step(_i32([0] * (B + 1)), [n] + [0] * B, count)
    lens, count = plan.cache_lens, plan.free_count
    # the others come with its whole pages cached and copy the page that it fills in part
    whole = n // page * page
    lens[1:] = whole
    for b in range(1, B + 1):
        text[b] = [(text[0][0][0][:whole], text[0][0][1][:whole])]
    pl.fill_(whole)
    plan, q, k, v, cu = step(lens, [1] + new, count)
    irs.check_device_errors(DEV)
    docs = _i32([0] + cu[1:])
    own = irs.window_gqa_attn_fwd(q, k, v, docs, max(new) + 1)
    lead = table[:1]
    out, lse = irs.shared_prefix_gqa_attn_fwd(q[1:], kc, vc, lead, _i32([0, sum(new)]), _i32([whole]),
                                              own=(own[0][1:].contiguous(), own[1][1:].contiguous()))
    for b in range(1, B + 1):
        kk, vv = (torch.cat([t[i] for t in text[b]]).double() for i in range(2))
        for i in range(new[b - 1]):
            m = whole + i + 1
            ref = R.attend(q[cu[b] + i][None], kk[:m], vv[:m], 1 / math.sqrt(D))
            # two roundings more: the own part's output was stored in bf16, its weights too
            R.check(out[cu[b] - 1 + i][None], ref[0], 2 * ref[2] + 2 * R.U16 * ref[0].abs(), "prompt out")
            R.check(lse[cu[b] - 1 + i][None], ref[1], 2 * ref[3] + 2.0 ** -19, "prompt lse")
    lens, count = plan.cache_lens, plan.free_count
    for _ in range(18):
        plan, q, k, v, cu = step(lens, [1] * (B + 1), count)
        lens, count = plan.cache_lens, plan.free_count
        out, lse = irs.shared_prefix_gqa_attn_decode(q, kc, vc, table, lens, groups, pl)
    irs.check_device_errors(DEV)
    for b in range(B + 1):
        kk, vv = (torch.cat([t[i] for t in text[b]]).double() for i in range(2))
        assert kk.shape[0] == int(lens[b])
        ref = R.attend(q[b][None], kk, vv, 1 / math.sqrt(D))
        R.check(out[b][None], ref[0], ref[2] + 2.0 ** -18, "step out")
        R.check(lse[b][None], ref[1], ref[3] + 2.0 ** -18, "step lse")
    assert int(count) == 48 - len(set(table[table >= 0].tolist()))


@pytest.mark.parametrize("decode", [False, True])
def test_broadcast_pools_and_one_head_for_all(irs, decode):
    """Pools whose heads, or whose positions, are one row: strides of 0."""
    g = _gen(17)
    kc, vc = _normal(g, 9, 16, 1, 128), _normal(g, 9, 16, 1, 64)
    table = torch.arange(9, device=DEV, dtype=torch.int32)[None].repeat(3, 1)
    q = _normal(g, 3, 8, 128)
    for k, v in ((kc.expand(-1, -1, 4, -1), vc.expand(-1, -1, 4, -1)), (kc[:, :1].expand(-1, 16, 4, -1), vc.expand(-1, -1, 4, -1))):
        if decode:
            lens = [120, 0, 77]
            out, lse = irs.shared_prefix_gqa_attn_decode(q, k, v, table, _i32(lens), _i32([0, 3]), _i32([70]))
            ref = R.decode(q, k, v, table, lens, [0, 3], [70], 1 / math.sqrt(128))
        else:
            out, lse = irs.shared_prefix_gqa_attn_fwd(q, k, v, table[:2], _i32([0, 1, 3]), _i32([131, 70]))
            ref = R.fwd(q, k, v, table, [0, 1, 3], [131, 70], 1 / math.sqrt(128))
        irs.check_device_errors(DEV)
        R.check(out, ref[0], ref[2], "out")
        R.check(lse, ref[1], ref[3], "lse")


def test_decode_every_sequence_a_group(irs):
    """Many groups of one sequence, more than a list's first looks hold."""
    g = torch.Generator().manual_seed(18)
    n = 9000
    prefix = torch.randint(0, 30, (n,), generator=g).tolist()
    own = torch.randint(0, 4, (n,), generator=g).tolist()
    q, kc, vc, table, lens, cu = _steps(_gen(18), [1] * n, prefix, own, 2, 1, 64, 64, 16)
    out, lse = irs.shared_prefix_gqa_attn_decode(q, kc, vc, table, _i32(lens), _i32(cu), _i32(prefix))
    irs.check_device_errors(DEV)
    want, l = irs.paged_gqa_attn_decode(q, kc, vc, table, _i32(lens))
    # the same attention by a kernel that is checked on its own: both within the roundings of weights and results
    assert (out.double() - want.double()).abs().max() <= 3 * R.U16 * vc.double().abs().max()
    assert torch.equal(lse == -math.inf, l == -math.inf)
    assert (lse - l)[lse > -math.inf].abs().max() <= 2.0 ** -17


def test_two_calls_at_once(irs):
    """Calls of two host threads on two streams, each with a workspace of its own."""
    import threading

    args, out, lse = _decode(irs, [30, 9], [900, 300], list(range(39)), 16, 2, 128, 128, 16, seed=19)
    got = [None, None]

    def work(i):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.default_stream())
        with torch.cuda.stream(s):
            for _ in range(20):
                got[i] = irs.shared_prefix_gqa_attn_decode(*args)
            s.synchronize()

    torch.cuda.synchronize()
    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    for o, l in got:
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_decode_idle_first_sequence(irs):
    """A group is read through its first sequence's row also where that one's own length is 0; a group without a
    sequence that is not idle gives zeros."""
    args, out, lse = _decode(irs, [3, 2, 1], [200, 64, 33], [None, 5, 40, None, None, 7], 8, 2, 128, 128, 16, seed=23)
    assert (out[[0, 3, 4]] == 0).all() and (lse[[0, 3, 4]] == -math.inf).all()
    assert torch.isfinite(lse[[1, 2, 5]]).all()


@pytest.mark.parametrize("Hq,Hkv", [(200, 200), (160, 80), (1024, 1024)])
def test_more_heads_than_run_at_once(irs, Hq, Hkv):
    """KV heads past what has a CTA each at a time: a head's list is one run, or two."""
    _prompts(irs, [3, 70], [150, 40], Hq, Hkv, 64, 64, 16, seed=Hkv)
    _decode(irs, [2, 1], [140, 33], [3, 60, 0], Hq, Hkv, 64, 64, 16, seed=Hkv)


@pytest.mark.parametrize("page,Dqk", [(128, 128), (256, 128), (512, 192), (1000, 64), (4096, 128)])
def test_large_pages(irs, page, Dqk):
    """Pages of a block and more, down to one page a sequence."""
    _prompts(irs, [9, 70], [1033, 190], 8, 2, Dqk, 128, page, seed=page)
    _decode(irs, [3, 2], [1033, 190], [1, 40, 900, 300, 0], 8, 2, Dqk, 128, page, seed=page)


def test_calls_in_one_graph_share_a_workspace(irs):
    """A step's calls in one graph, one workspace for all of them in turn, replayed with other lengths."""
    q, kc, vc, table, lens, cu = _steps(_gen(29), [6, 3], [300, 90], [10, 4, 0, 70, 9, 33, 1, 2, 3], 8, 2, 128, 128, 16)
    L, pl = _i32(lens), _i32([300, 90])
    ws = torch.empty(128 << 20, dtype=torch.uint8, device=DEV)
    firsts = table[[0, 6]].contiguous()

    def step():
        a = irs.shared_prefix_gqa_attn_decode(q, kc, vc, table, L, _i32_cu, pl, workspace=ws)
        b = irs.shared_prefix_gqa_attn_fwd(q, kc, vc, firsts, _i32_cu, pl, own=a, workspace=ws)
        c = irs.shared_prefix_gqa_attn_decode(q, kc, vc, table, L, _i32_cu, pl, workspace=ws)
        return a, b, c

    _i32_cu = _i32(cu)
    step()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = step()
    for n in ([300, 90], [17, 0], [256, 90]):
        pl.copy_(_i32(n))
        gr.replay()
        torch.cuda.synchronize()
        want = step()
        for x, y in zip(got, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
        assert torch.equal(got[0][0], got[2][0]) and torch.equal(got[0][1], got[2][1])
        ref = R.decode(q, kc, vc, table, lens, cu, n, 1 / math.sqrt(128))
        R.check(got[0][0], ref[0], ref[2], "out")
    irs.check_device_errors(DEV)
